"""multi_axis_rotary on the GPU: values against fp64 with counted roundings, layouts, far positions, gradient."""
import pytest
import torch

import attention_ref as ref
import gated_linear_attention_local_b200 as sg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.init()


def make(lead, H, Hk, D, R, A, far, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    q = torch.randn(*lead, H, D, generator=gen).to(dtype).cuda()
    k = torch.randn(*lead, Hk, D, generator=gen).to(dtype).cuda()
    pos = torch.randint(-far, far, (*lead, A), generator=gen).cuda()
    half = R // 2
    freq = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).float().cuda()
    axes = torch.randint(0, A, (half,), generator=gen).tolist()
    return q, k, pos, freq, axes


CASES = [
    # lead, H, Hk, D, R, A, far
    ((1,), 1, 1, 2, 2, 1, 10),
    ((3, 5), 4, 2, 128, 128, 3, 1000),
    ((2500,), 3, 1, 64, 64, 2, 1 << 20),       # four tokens a block, a last block of fewer
    ((7,), 5, 5, 80, 64, 4, 100),
    ((11,), 2, 1, 40, 20, 1, 1 << 30),         # vectors of two
    ((9,), 3, 3, 10, 10, 2, 50),               # odd number of pairs
    ((4,), 2, 2, 512, 512, 8, 5000),
    ((6,), 2, 1, 24, 0, 1, 5),                 # nothing rotates
    ((2401,), 1, 1, 6, 6, 1, 9),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CASES, ids=[f"D{c[3]}R{c[4]}A{c[5]}" for c in CASES])
def test_values(case, dtype, interleaved, inverse):
    lead, H, Hk, D, R, A, far = case
    q, k, pos, freq, axes = make(lead, H, Hk, D, R, A, far, dtype, 5)
    fn = sg.multi_axis_rotary_bwd if inverse else sg.multi_axis_rotary
    qo, ko = fn(q, k, pos, freq, axes=axes, interleaved=interleaved)
    torch.cuda.synchronize()
    for got, x in ((qo, q), (ko, k)):
        ref.check(got, ref.rotary(x, pos, freq, axes, interleaved, inverse), "rotated")


def test_one_axis_without_its_dimension_and_without_k():
    q, _, pos, freq, _ = make((6, 3), 2, 1, 32, 32, 1, 4000, torch.float32, 6)
    qo, ko = sg.multi_axis_rotary(q, None, pos[..., 0].contiguous(), freq)
    assert ko is None
    ref.check(qo, ref.rotary(q, pos, freq, [0] * 16, False), "q")


def test_empty_batch():
    q, k, pos, freq, axes = make((0,), 2, 1, 32, 32, 2, 10, torch.bfloat16, 7)
    qo, ko = sg.multi_axis_rotary(q, k, pos, freq, axes=axes)
    assert qo.shape == q.shape and ko.shape == k.shape


def test_gradient_is_the_rotation_back():
    q, k, pos, freq, axes = make((2, 9), 4, 2, 48, 32, 3, 300, torch.float32, 8)
    q.requires_grad_()
    k.requires_grad_()
    qo, ko = sg.multi_axis_rotary(q, k, pos, freq, axes=axes)
    gq, gk = torch.randn_like(qo), torch.randn_like(ko)
    dq, dk = torch.autograd.grad([qo, ko], [q, k], [gq, gk])
    ref.check(dq, ref.rotary(gq, pos, freq, axes, False, True), "dq")
    ref.check(dk, ref.rotary(gk, pos, freq, axes, False, True), "dk")
    # against differences of the fp64 definition along one direction: the map is linear
    step = torch.randn_like(q)
    (a, _), (b, _) = (ref.rotary(x, pos, freq, axes, False) for x in (q.detach() + step, q.detach()))
    moved = float(((torch.from_numpy(a) - torch.from_numpy(b)) * gq.double().cpu()).sum())
    assert abs(float((dq.double() * step.double()).sum()) - moved) < 1e-4 * dq.numel() ** 0.5


def test_only_one_output_used():
    q, k, pos, freq, axes = make((5,), 2, 1, 16, 16, 2, 30, torch.float32, 9)
    q.requires_grad_()
    k.requires_grad_()
    qo, _ = sg.multi_axis_rotary(q, k, pos, freq, axes=axes)
    qo.sum().backward()
    assert q.grad is not None and float(k.grad.abs().max()) == 0.0


def test_captured_and_replayed():
    q, k, pos, freq, axes = make((33,), 4, 2, 64, 64, 3, 100, torch.bfloat16, 10)
    sg.multi_axis_rotary(q, k, pos, freq, axes=axes)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qo, ko = sg.multi_axis_rotary(q, k, pos, freq, axes=axes)
    q.copy_(torch.randn_like(q))
    pos.add_(7)
    graph.replay()
    torch.cuda.synchronize()
    ref.check(qo, ref.rotary(q, pos, freq, axes, False), "q")
    ref.check(ko, ref.rotary(k, pos, freq, axes, False), "k")
