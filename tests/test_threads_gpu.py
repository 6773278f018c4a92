"""The first call that a host thread makes: a thread has no CUDA context until a runtime call of its own binds one, and
autograd runs gradients in a thread of its own."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import gated_linear_attention_local_b200 as sg

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.init()


def calls(dtype):
    gen = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(2, 200, 2, 128, generator=gen).to(dtype).cuda() for _ in range(3))
    g = torch.full((2, 200, 2), -0.1, device="cuda")
    n = torch.tensor([200, 17]).cuda()
    cu = torch.tensor([0, 150, 400]).cuda()
    flat = [x.reshape(400, 2, 128) for x in (q, k, v)]
    o, lse = sg.softmax_attention_fwd(q, k, v)
    pos, freq = torch.arange(400).view(2, 200).cuda(), torch.rand(64, generator=gen).cuda()
    first = q[:, 0].contiguous()
    return {
        "softmax_attention_fwd": lambda: sg.softmax_attention_fwd(q, k, v),
        "packed": lambda: sg.softmax_attention_fwd(*flat, cu_seqlens=cu),
        "softmax_attention_bwd": lambda: tuple(sg.softmax_attention_bwd(q, k, v, o, lse, q).values()),
        "softmax_attention_decode_step": lambda: (sg.softmax_attention_decode_step(first, k, v, n),),
        "prefix": lambda: (sg.softmax_attention_decode_step(first, k, v, n, k[0], v[0]),),
        "multi_axis_rotary": lambda: sg.multi_axis_rotary(q, k, pos, freq),
        "simple_gla_fwd": lambda: sg.simple_gla_fwd(q, k, v, g=g, output_final_state=True),
        "simple_gla_fwd_varlen": lambda: sg.simple_gla_fwd_varlen(*(x[None] for x in flat), cu, g=g.view(1, 400, 2)),
        "simple_gla_chunk_final_state": lambda: (sg.simple_gla_chunk_final_state(k, v, g=g),),
        "simple_gla_chunk_bwd": lambda: (sg.simple_gla_chunk_bwd(q, k, v, q, g=g)["dq"],),
        "simple_gla_fused_recurrent": lambda: sg.simple_gla_fused_recurrent(q, k, v, g=g),
        "gla_chunk": lambda: sg.gla_chunk(q, k, v, g[..., None].expand(2, 200, 2, 128).contiguous()),
    }


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("name", ["softmax_attention_fwd", "packed", "softmax_attention_bwd", "softmax_attention_decode_step",
                                  "prefix", "multi_axis_rotary", "simple_gla_fwd", "simple_gla_fwd_varlen",
                                  "simple_gla_chunk_final_state", "simple_gla_chunk_bwd", "simple_gla_fused_recurrent",
                                  "gla_chunk"])
def test_first_call_of_a_thread(name, dtype):
    call = calls(dtype)[name]
    want = call()
    torch.cuda.synchronize()
    got = []

    def work():
        try:
            got.extend(call())
        except Exception as e:  # seen by the test, not only printed by the thread
            got.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert not isinstance(a, Exception), a
        assert a is b is None or torch.equal(a, b)
    assert len(got) == len(want)


def test_gradients_before_anything_else_in_autograds_thread():
    """A process whose first differentiable call is this one (a fresh process: autograd's thread outlives a test)."""
    code = ("import torch, gated_linear_attention_local_b200 as sg\n"
            "x = [torch.randn(1, 300, 2, 64, device='cuda', dtype=torch.bfloat16, requires_grad=True) for _ in range(3)]\n"
            "o = sg.softmax_attention(*x)\n"
            "g = torch.autograd.grad(o, x, torch.ones_like(o))\n"
            "torch.cuda.synchronize()\n"
            "assert all(bool(t.isfinite().all()) for t in g)\n"
            "print('fine')\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("mixer", ["softmax", "packed"])
def test_a_training_step_captured_and_replayed(mixer):
    """Rotation and attention, forward and backward through autograd, in one graph; replayed on new inputs beside an
    eager step on the same leaves."""
    gen = torch.Generator().manual_seed(3)
    lead = (2, 150) if mixer == "softmax" else (300,)
    q, k, v, do = (torch.randn(*lead, h, 64, generator=gen).to(BF16).cuda() for h in (4, 2, 2, 4))
    leaves = [x.requires_grad_() for x in (q, k, v)]
    pos = torch.randint(0, 1000, (*lead, 2), generator=gen).cuda()
    freq, axes = torch.rand(32, generator=gen).cuda(), [i % 2 for i in range(32)]
    cu = None if mixer == "softmax" else torch.tensor([0, 100, 101, 300]).cuda()

    def step():
        qr, kr = sg.multi_axis_rotary(q, k, pos, freq, axes=axes)
        o = sg.softmax_attention(qr, kr, v, cu_seqlens=cu)
        return (o.detach(), *torch.autograd.grad(o, leaves, do))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    with torch.no_grad():
        for x in (q, k, v, do):
            x.copy_(torch.randn(x.shape, generator=gen).to(BF16))
        pos.add_(5)
    graph.replay()
    want = step()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
