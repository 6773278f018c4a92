"""softmax_attention as a layer calls it, through autograd, on the GPU: dense and packed, in both types, against fp64 in
the norm of each tensor (attention_norms says how far off a kernel's roundings take it)."""
import numpy as np
import pytest
import torch

import attention_norms as norms
import attention_ref as ref
import gated_linear_attention_local_b200 as sg

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.init()


def normal(gen, *shape, dtype):
    return torch.randn(*shape, generator=gen).to(dtype).cuda()


def compare(got, want, dtype, rows=slice(None), keys=slice(None)):
    for n in want:
        part = keys if n in ("dk", "dv") else rows
        x = got[n][part]
        assert bool(torch.isfinite(x).all()), n
        if float(want[n].norm()) == 0:
            assert float(x.abs().max()) == 0, n
        else:
            assert norms.off(x, want[n]) <= norms.LIMIT[dtype], (n, norms.off(x, want[n]))


def through_autograd(q, k, v, do, **kw):
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    o = sg.softmax_attention(*leaves, **kw)
    return dict(o=o, **dict(zip(("dq", "dk", "dv"), torch.autograd.grad(o, leaves, do))))


# B, T, S, H, Hk, D, causal
DENSE = [(1, 400, 513, 8, 2, 128, False), (1, 1100, 1100, 4, 1, 64, True), (2, 257, 257, 6, 2, 80, True),
         (1, 700, 300, 7, 1, 96, True), (2, 130, 1500, 4, 4, 128, True), (1, 2100, 129, 16, 1, 40, False)]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("case", DENSE, ids=lambda c: "x".join(map(str, c)))
def test_dense(case, dtype):
    B, T, S, H, Hk, D, causal = case
    gen = torch.Generator().manual_seed(T + S)
    q, do = (normal(gen, B, T, H, D, dtype=dtype) for _ in range(2))
    k, v = (normal(gen, B, S, Hk, D, dtype=dtype) for _ in range(2))
    got = through_autograd(q, k, v, do, causal=causal)
    for b in range(B):
        compare({n: x[b] for n, x in got.items()}, norms.attention64(q[b], k[b], v[b], do[b], causal), dtype)


PACKED = [([300, 1, 128, 517], None, 4, 2, 64, True), ([200, 640, 33], [10, 900, 300], 6, 2, 128, True),
          ([129, 400], [257, 64], 3, 3, 80, False), ([1000], [1200], 8, 1, 96, True)]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("case", PACKED, ids=lambda c: f"N{len(c[0])}D{c[4]}")
def test_packed(case, dtype):
    lq, lk, H, Hk, D, causal = case
    gen = torch.Generator().manual_seed(sum(lq))
    cu = np.concatenate(([0], np.cumsum(lq)))
    cu_k = cu if lk is None else np.concatenate(([0], np.cumsum(lk)))
    q, do = (normal(gen, int(cu[-1]), H, D, dtype=dtype) for _ in range(2))
    k, v = (normal(gen, int(cu_k[-1]), Hk, D, dtype=dtype) for _ in range(2))
    word = torch.full((2,), 9, dtype=torch.int32, device="cuda")
    got = through_autograd(q, k, v, do, causal=causal, cu_seqlens=torch.tensor(cu).cuda(), device_status=word,
                           cu_seqlens_k=None if lk is None else torch.tensor(cu_k).cuda())
    assert word.tolist() == [0, 0]
    for n in range(len(lq)):
        a, b = slice(cu[n], cu[n + 1]), slice(cu_k[n], cu_k[n + 1])
        if lq[n] == 1:  # a single key: ds is 0, and only its rounding is left
            continue
        compare(got, norms.attention64(q[a], k[b], v[b], do[a], causal), dtype, a, b)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_one_gradient_asked_for(dtype):
    """One of the operands requires a gradient: its value, and none for the others."""
    gen = torch.Generator().manual_seed(31)
    q, k, v, do = (normal(gen, 1, 300, 2, 64, dtype=dtype) for _ in range(4))
    want = norms.attention64(q[0], k[0], v[0], do[0], True)
    for i, n in enumerate(("dq", "dk", "dv")):
        x = [q.clone(), k.clone(), v.clone()]
        x[i].requires_grad_()
        sg.softmax_attention(*x).backward(do)
        assert [t.grad is not None for t in x] == [j == i for j in range(3)]
        compare({n: x[i].grad[0]}, {n: want[n]}, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_gradients_that_are_not_contiguous(dtype):
    """The gradient of a permuted, and of a summed, output: its strides are whatever autograd makes them."""
    gen = torch.Generator().manual_seed(32)
    q, k, v, do = (normal(gen, 1, 270, 4, 64, dtype=dtype) for _ in range(4))
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    o = sg.softmax_attention(*leaves)
    grads = torch.autograd.grad(o.permute(0, 2, 3, 1), leaves, do.permute(0, 2, 3, 1).contiguous())
    compare({n: x[0] for n, x in zip(("dq", "dk", "dv"), grads)},
            {n: x for n, x in norms.attention64(q[0], k[0], v[0], do[0], True).items() if n != "o"}, dtype)
    o = sg.softmax_attention(*leaves)
    grads = torch.autograd.grad(o.float().sum(), leaves)
    one = norms.attention64(q[0], k[0], v[0], torch.ones_like(do[0]), True)
    # (p sums to 1 and do is constant: dv adds p of one sign, whose roundings cancel no more than those of other sums)
    compare({"dq": grads[0][0], "dk": grads[1][0]}, {n: one[n] for n in ("dq", "dk")}, dtype)
    compare({"dv": grads[2][0]}, {"dv": one["dv"]}, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_gradients_of_large_scores(dtype):
    """Scores up to some hundreds, a key that takes nearly all of a row's weight, and one that nearly all rows see most
    of.  The bounds of attention_ref, and what an fp32 lse adds: it holds a row's sum to 2^-24 of itself twice over (as
    stored, and in units of log2), and s - lse is rounded once, so p is off by the factor 1 + 4 2^-24 |lse|."""
    gen = torch.Generator().manual_seed(33)
    q, k, v, do = (normal(gen, 1, 200, 2, 64, dtype=dtype) for _ in range(4))
    q[:, 3] *= 8
    k[:, 60] *= 8
    q[:, 9] = -k[:, 9]
    o, lse = sg.softmax_attention_fwd(q, k, v, scale=0.7)
    got = sg.softmax_attention_bwd(q, k, v, o, lse, do, scale=0.7)
    want = ref.attention(q, k, v, True, scale=0.7, do=do)
    ref.check(o, want["o"], "o")
    extra = 4 * 2.0 ** -24 * float(np.abs(want["lse"][0]).max())
    Q, K, V, G = (x[0].double().cpu().transpose(0, 1) for x in (q, k, v, do))
    s = 0.7 * (Q @ K.transpose(1, 2))
    s = s.masked_fill(torch.ones(200, 200).triu(1).bool(), float("-inf"))
    p = torch.softmax(s, -1)
    dp = G @ V.transpose(1, 2)
    ds = (p * (dp - (p * dp).sum(-1, keepdim=True))).abs()
    more = {"dq": 0.7 * (ds @ K.abs()), "dk": 0.7 * (ds.transpose(1, 2) @ Q.abs()), "dv": p.transpose(1, 2) @ G.abs()}
    for n, m in more.items():
        value, bound = want[n]
        ref.check(got[n], (value, bound + extra * m.transpose(0, 1)[None].numpy()), n)
