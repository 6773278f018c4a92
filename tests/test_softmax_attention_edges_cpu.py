"""What the bindings of softmax attention, rotary positions and the chunked mixer do around the library's call: no GPU
is used, the calls are stood in for."""
import numpy as np
import pytest
import torch
from torch.autograd import forward_ad

import gated_linear_attention_local_b200 as sg
from gated_linear_attention_local_b200 import attention


@pytest.fixture
def plain(monkeypatch):
    """The entry points without the library: outputs of zeros."""
    monkeypatch.setattr(attention, "_forward", lambda q, k, v, *a, **kw: (torch.zeros_like(q), torch.zeros(q.shape[:-1])))
    monkeypatch.setattr(attention, "_rotary", lambda q, k, *a, **kw: (q * 0, None if k is None else k * 0))
    for name in ("simple_gla_fwd", "simple_gla_chunk"):
        monkeypatch.setattr(sg, name, lambda q, *a, **kw: (torch.zeros_like(q), None))


def calls():
    pos, freq = torch.zeros(1, 4, dtype=torch.int64), torch.ones(4)
    return {"softmax_attention": lambda q, k, v: sg.softmax_attention(q, k, v),
            "multi_axis_rotary": lambda q, k, v: sg.multi_axis_rotary(q, k, pos, freq)[0],
            "chunk_simple_gla": lambda q, k, v: sg.chunk_simple_gla(q, k, v)[0]}


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("name", sorted(calls()))
def test_forward_mode_tangents_are_not_dropped(plain, name, which):
    """A dual tensor requires no gradient; its tangent must not be taken for zero without a word."""
    x = [torch.randn(1, 4, 2, 8) for _ in range(3)]
    call = calls()[name]
    assert float(call(*x).abs().max()) == 0.0
    with forward_ad.dual_level():
        assert float(call(*x).abs().max()) == 0.0  # no tangent: as ever
        x[which] = forward_ad.make_dual(x[which], torch.ones_like(x[which]))
        with pytest.raises(RuntimeError):
            call(*x)
        with torch.no_grad(), pytest.raises(RuntimeError):  # which stops reverse mode only
            call(*x)


@pytest.fixture
def library(monkeypatch):
    """Stands in for the library: every call succeeds and is recorded with the address of its status word."""
    seen = []

    class Library:
        def __getattr__(self, name):
            if name.endswith("_size"):
                return lambda *a: 256
            where = {"softmax_attention_fwd": 16, "softmax_attention_bwd": 20}[name]

            def call(*a):
                seen.append((name, a[where]))
                return 0
            return call
    monkeypatch.setattr(attention, "lib", Library)
    monkeypatch.setattr(attention, "_stream", lambda: None)
    monkeypatch.setattr(torch.Tensor, "is_cuda", True, raising=False)  # argument checks run, nothing is launched
    monkeypatch.setattr(attention, "softmax_attention_bwd", sg.softmax_attention_bwd.__wrapped__)  # no device to switch to
    return seen


def test_a_differentiable_call_reports_forward_and_gradients(library):
    q, k = torch.zeros(2, 8, 4, 64), torch.zeros(2, 8, 2, 64)
    word = torch.zeros(2, dtype=torch.int32)
    sg.softmax_attention.__wrapped__(q, k, k, device_status=word)
    assert library == [("softmax_attention_fwd", word.data_ptr())]
    library.clear()
    q.requires_grad_()
    o = sg.softmax_attention.__wrapped__(q, k, k, device_status=word)
    torch.autograd.grad(o, q, torch.ones_like(o))
    assert library == [("softmax_attention_fwd", word.data_ptr()), ("softmax_attention_bwd", word.data_ptr() + 4)]
    library.clear()
    o = sg.softmax_attention.__wrapped__(q, k, k)
    torch.autograd.grad(o, q, torch.ones_like(o))
    assert library == [("softmax_attention_fwd", None), ("softmax_attention_bwd", None)]
    library.clear()
    with pytest.raises(ValueError, match="2 elements"):  # no room for the gradients' status
        sg.softmax_attention.__wrapped__(q, k, k, device_status=word[:1])
    with pytest.raises(TypeError):
        sg.softmax_attention.__wrapped__(q, k, k, device_status=word.long())
    assert not library


@pytest.mark.parametrize("make", [list, tuple, bytes, lambda x: np.array(x, dtype=np.int64), lambda x: np.array(x, np.uint8),
                                  torch.tensor, lambda x: range(len(x))])
def test_axes_of_any_sequence(monkeypatch, make):
    """What reaches the library is one byte a pair, the axis's number, whatever kind of sequence held it."""
    seen = []

    class Library:
        @staticmethod
        def multi_axis_rotary(*a):
            seen.append(a[4])
            return 0
    monkeypatch.setattr(attention, "lib", Library)
    monkeypatch.setattr(attention, "_stream", lambda: None)
    monkeypatch.setattr(torch.Tensor, "is_cuda", True, raising=False)
    rotary = sg.multi_axis_rotary.__wrapped__
    for half in (1, 2, 8):
        axes = make(list(range(half)))
        rotary(torch.zeros(3, 2, 2 * half), None, torch.zeros(3, 9, dtype=torch.int64), torch.ones(half), axes=axes)
        assert seen.pop() == bytes(range(half))
    for axes in (make([0, 1]), make([0])):  # another number of axes than pairs, however many bytes they take
        with pytest.raises(ValueError):
            rotary(torch.zeros(3, 2, 16), None, torch.zeros(3, 9, dtype=torch.int64), torch.ones(8), axes=axes)
    one = make([0, 1])[1:2]
    rotary(torch.zeros(3, 2, 2), None, torch.zeros(3, 2, dtype=torch.int64), torch.ones(1), axes=one)
    assert seen.pop() == b"\x01"


def test_axes_that_change_after_the_call(monkeypatch):
    """The gradient turns by the axes of the call, whatever became of the caller's list."""
    seen = []

    class Library:
        @staticmethod
        def multi_axis_rotary(*a):
            seen.append(a[4])
            return 0
    monkeypatch.setattr(attention, "lib", Library)
    monkeypatch.setattr(attention, "_stream", lambda: None)
    monkeypatch.setattr(torch.Tensor, "is_cuda", True, raising=False)
    monkeypatch.setattr(attention, "multi_axis_rotary_bwd", sg.multi_axis_rotary_bwd.__wrapped__)
    axes = [0, 1, 2, 3]
    q = torch.zeros(3, 2, 8, requires_grad=True)
    o, _ = sg.multi_axis_rotary.__wrapped__(q, None, torch.zeros(3, 4, dtype=torch.int64), torch.ones(4), axes=axes)
    axes.reverse()
    torch.autograd.grad(o, q, torch.ones_like(o))
    assert seen == [bytes(range(4))] * 2
