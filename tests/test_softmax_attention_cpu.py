"""Host checks of the softmax attention and rotary entry points, and the fp64 reference itself: no GPU is used."""
import ctypes

import numpy as np
import pytest
import torch

import attention_ref as ref
import gated_linear_attention_local_b200 as sg
from gated_linear_attention_local_b200 import _lib as L
from gated_linear_attention_local_b200 import build as B

INV, UNS, WS = L.SGLA_ERR_INVALID_ARGUMENT, L.SGLA_ERR_UNSUPPORTED, L.SGLA_ERR_WORKSPACE
P = 4096  # an aligned address that no call here reaches


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.lib()


def fwd(lib, q=P, k=P, v=P, o=P, lse=P, cu=None, cuk=None, N=1, Tq=8, Tk=8, H=4, Hk=2, D=64, dt=L.SGLA_BF16):
    return lib.softmax_attention_fwd(q, k, v, float("nan"), 1, o, lse, cu, cuk, N, Tq, Tk, H, Hk, D, dt, None, None)


def test_forward_refusals(lib):
    assert fwd(lib, q=None) == INV and fwd(lib, o=None) == INV and fwd(lib, k=None) == INV
    assert fwd(lib, q=P + 8) == INV and fwd(lib, lse=P + 2) == INV
    assert fwd(lib, H=5) == INV and fwd(lib, Hk=0) == INV and fwd(lib, N=-1) == INV and fwd(lib, Tk=-1) == INV
    assert fwd(lib, cu=P) == INV and fwd(lib, cuk=P) == INV and fwd(lib, cu=P, cuk=P, N=0) == INV
    assert fwd(lib, cu=P + 4, cuk=P) == INV and fwd(lib, dt=7) == INV
    assert fwd(lib, D=136) == UNS and fwd(lib, D=12) == UNS and fwd(lib, H=258, Hk=2) == UNS
    assert fwd(lib, H=65536, Hk=65536) == UNS and fwd(lib, N=1 << 20, Tq=1 << 10) == UNS
    assert fwd(lib, cu=P, cuk=P, Tk=1 << 30) == UNS
    assert fwd(lib, N=0) == 0 and fwd(lib, Tq=0, q=None, o=None) == 0  # nothing to do


def test_backward_refusals(lib):
    def bwd(ws=P, n=1 << 20, o=P, lse=P, dout=P, dq=P, dk=P, dv=P, H=4, D=64, Tq=8):
        return lib.softmax_attention_bwd(P, P, P, o, lse, dout, float("nan"), 1, dq, dk, dv, None, None, 1, Tq, 8, H, 2,
                                         D, L.SGLA_BF16, None, ws, n, None)
    assert bwd(ws=None) == WS and bwd(n=127) == WS and bwd(ws=P + 64) == INV
    for name in ("o", "lse", "dout", "dq", "dk", "dv"):
        assert bwd(**{name: None}) == INV
    assert bwd(dk=P + 8) == INV and bwd(D=4) == UNS and bwd(H=3) == INV
    assert lib.softmax_attention_bwd_workspace_size(8, 4) == 256
    assert lib.softmax_attention_bwd_workspace_size(1 << 20, 32) == (1 << 20) * 32 * 4
    assert lib.softmax_attention_bwd_workspace_size(-1, 4) == 0


def test_decode_refusals(lib):
    def dec(q=P, kc=P, vc=P, ln=P, pk=None, pv=None, o=P, N=2, S=5000, Pn=0, H=4, Hk=2, D=64, ws=P, n=1 << 30):
        return lib.softmax_attention_decode_step(q, kc, vc, ln, pk, pv, float("nan"), o, N, S, Pn, H, Hk, D,
                                                 L.SGLA_BF16, None, ws, n, None)
    assert dec(q=None) == INV and dec(kc=None) == INV and dec(ln=None) == INV and dec(o=None) == INV
    assert dec(Pn=3) == INV and dec(Pn=3, pk=P) == INV and dec(Pn=-1) == INV and dec(ln=P + 4) == INV
    assert dec(vc=P + 8) == INV and dec(H=3) == INV and dec(D=129) == UNS and dec(D=136) == UNS
    assert dec(N=1 << 20, S=1 << 10) == UNS and dec(Pn=1 << 30, pk=P, pv=P) == UNS
    for kw in (dict(Pn=500, pk=P, pv=P), dict(H=64, Hk=2)):  # parts to join: a prefix, a large group
        assert dec(ws=None, **kw) == WS and dec(n=100, **kw) == WS and dec(ws=P + 16, **kw) == INV
    assert dec(N=0) == 0
    size = lib.softmax_attention_decode_workspace_size
    assert size(2, 5000, 500, 4, 2, 64, L.SGLA_BF16) > 0 and size(2, 5000, 0, 4, 2, 64, L.SGLA_BF16) == 0
    assert size(2, 5000, 0, 64, 2, 64, L.SGLA_BF16) > 0 and size(2, 5000, 0, 4, 3, 64, L.SGLA_BF16) == 0


def test_rotary_refusals(lib):
    def rot(q=P, k=P, pos=P, f=P, ax=bytes(32), qo=P, ko=P, t=4, H=2, Hk=1, D=64, R=64, A=1, dt=L.SGLA_BF16):
        return lib.multi_axis_rotary(q, k, pos, f, ax, qo, ko, t, H, Hk, D, R, A, 0, 0, dt, None)
    assert rot(q=None) == INV and rot(ko=None) == INV and rot(pos=None) == INV and rot(f=None) == INV
    assert rot(ax=None) == INV and rot(ax=bytes([0] * 31 + [1])) == INV and rot(q=P + 4) == INV and rot(pos=P + 4) == INV
    assert rot(R=66) == INV and rot(R=63) == INV and rot(A=0) == INV and rot(t=-1) == INV and rot(dt=3) == INV
    assert rot(D=65) == UNS and rot(D=1024, R=514, ax=bytes(257)) == UNS and rot(A=256) == UNS and rot(t=1 << 31) == UNS
    assert rot(t=0) == 0 and rot(H=0, Hk=0) == 0


def test_bindings_refuse_cpu_tensors_and_bad_types():
    q = torch.zeros(1, 4, 2, 64)
    with pytest.raises(TypeError, match="CUDA"):
        sg.softmax_attention(q, q, q)
    with pytest.raises(TypeError, match="CUDA"):
        sg.softmax_attention_bwd(q, q, q, q, q[..., 0], q)
    with pytest.raises(TypeError, match="CUDA"):
        sg.softmax_attention_decode_step(q[0], q, q, torch.ones(4, dtype=torch.int64))
    with pytest.raises(TypeError, match="CUDA"):
        sg.multi_axis_rotary(q, q, torch.zeros(1, 4, dtype=torch.int64), torch.ones(32))


class FakeCuda(torch.Tensor):
    """A CPU tensor that says it is on the GPU: argument checks run, nothing is launched."""
    is_cuda = True


def fake(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(FakeCuda)


@pytest.fixture
def refuses(monkeypatch):
    from gated_linear_attention_local_b200 import attention

    def launch(*a, **k):
        raise AssertionError("a call that must be refused reached the library")
    monkeypatch.setattr(attention, "_stream", lambda: None)

    class Library:  # host checks of the library itself run, a launch fails the test
        def __getattr__(self, name):
            fn = getattr(L.lib(), name)
            if name.endswith("_size"):
                return fn

            def call(*a):
                status = fn(*a)
                return status if status != L.SGLA_OK else launch()
            return call
    monkeypatch.setattr(attention, "lib", Library)

    def check(err, fn, *args, **kw):
        with pytest.raises(err):
            fn.__wrapped__(*args, **kw)
    return check


def test_binding_refusals(refuses):
    i64 = torch.int64
    q, k = fake(2, 8, 4, 64), fake(2, 8, 2, 64)
    f, b, d, r = sg.softmax_attention_fwd, sg.softmax_attention_bwd, sg.softmax_attention_decode_step, sg.multi_axis_rotary
    refuses(ValueError, f, q, k, fake(2, 8, 2, 32))                       # v of another head dimension
    refuses(ValueError, f, q, fake(2, 8, 3, 64), fake(2, 8, 3, 64))       # 4 heads on 3
    refuses(ValueError, f, q, fake(1, 8, 2, 64), fake(1, 8, 2, 64))       # batches differ
    refuses(TypeError, f, q, k.float(), k)
    refuses(TypeError, f, q.half(), k.half(), k.half())
    refuses(ValueError, f, q.transpose(1, 2), k, k)                       # not contiguous
    refuses(ValueError, f, q, k, k, cu_seqlens=fake(3, dtype=i64))        # a batch of 2 with cu_seqlens
    refuses(TypeError, f, q[:1], k[:1], k[:1], cu_seqlens=fake(3, dtype=torch.int32))
    refuses(ValueError, f, q[:1], k[:1], k[:1], cu_seqlens=fake(1, dtype=i64))
    refuses(ValueError, f, q[:1], k[:1], k[:1], cu_seqlens=fake(3, dtype=i64), cu_seqlens_k=fake(2, dtype=i64))
    refuses(ValueError, f, q[:1], fake(1, 9, 2, 64), fake(1, 9, 2, 64), cu_seqlens=fake(3, dtype=i64))
    refuses(ValueError, f, q, k, k, cu_seqlens_k=fake(3, dtype=i64))
    lse = fake(2, 8, 4, dtype=torch.float32)
    refuses(ValueError, b, q, k, k, q[:1], lse, q)
    refuses(ValueError, b, q, k, k, q, lse[:, :4].contiguous(), q)
    refuses(TypeError, b, q, k, k, q, lse, q.float())
    refuses(ValueError, b, q, k, k, q, lse, q, workspace=fake(16, dtype=torch.uint8))
    qt, ln = fake(2, 4, 64), fake(2, dtype=i64)
    refuses(ValueError, d, qt, k[:1], k[:1], ln)
    refuses(ValueError, d, qt, k, k, fake(3, dtype=i64))
    refuses(TypeError, d, qt, k, k, fake(2, dtype=torch.int32))
    refuses(ValueError, d, qt, k, k, ln, prefix_k=fake(5, 2, 64))
    refuses(ValueError, d, qt, k, k, ln, prefix_k=fake(5, 4, 64), prefix_v=fake(5, 4, 64))
    refuses(ValueError, d, qt, k, k, ln, prefix_k=fake(5, 2, 64), prefix_v=fake(6, 2, 64))
    refuses(ValueError, d, qt, k, k, ln, out=fake(2, 4, 32))
    pos, fr = fake(2, 8, 3, dtype=i64), fake(32, dtype=torch.float32)
    refuses(ValueError, r, q, k, pos, fr, axes=[0] * 31)
    refuses(TypeError, r, q, k, pos, fr, axes=32)
    refuses(ValueError, r, q, k, pos, fr, axes=[0] * 31 + [3])
    refuses(ValueError, r, q, k, pos, fr, axes=[0] * 31 + [-1])
    refuses(ValueError, r, q, k, fake(2, 7, 3, dtype=i64), fr)
    refuses(TypeError, r, q, k, pos.int(), fr)
    refuses(ValueError, r, q, k, pos, fake(33, dtype=torch.float32))
    refuses(ValueError, r, q, fake(2, 8, 2, 32), pos, fr)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("tq,tk", [(1, 1), (5, 9), (9, 5)])
def test_reference_gradients_against_differences(tq, tk, causal):
    gen = torch.Generator().manual_seed(tq)
    q, do = (torch.randn(1, tq, 4, 8, generator=gen, dtype=torch.float64) for _ in range(2))
    k, v = (torch.randn(1, tk, 2, 8, generator=gen, dtype=torch.float64) for _ in range(2))
    got = ref.attention(q, k, v, causal, do=do)
    for i, n in enumerate(("dq", "dk", "dv")):
        step = torch.randn([q, k, v][i].shape, generator=gen, dtype=torch.float64)
        ends = []
        for sign in (1, -1):
            x = [q, k, v]
            x[i] = x[i] + sign * 1e-5 * step
            ends.append((ref.attention(*x, causal)["o"][0] * do.numpy()).sum())
        slope = (ends[0] - ends[1]) / 2e-5
        assert abs((got[n][0] * step.numpy()).sum() - slope) < 1e-7 * max(1, abs(slope))


def test_reference_rotary_keeps_length_and_undoes_itself():
    x = torch.randn(3, 2, 24, dtype=torch.float64)
    pos, f = torch.randint(0, 1000, (3, 2)), torch.rand(8)
    for inter in (False, True):
        y, _ = ref.rotary(x, pos, f, [0, 1] * 4, inter)
        assert np.allclose((y ** 2).sum(-1), (x.numpy() ** 2).sum(-1))
        z, _ = ref.rotary(torch.from_numpy(y), pos, f, [0, 1] * 4, inter, inverse=True)
        assert np.allclose(z, x.numpy())
