"""Softmax attention at the ends of what its calls allow: very long items, extreme and non-finite values, rows that see
nothing."""
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


def test_a_block_of_keys_that_takes_seconds():
    """128 keys seen by 2^28 rows: one work item of dk dv walks 2^21 tiles (some 4 s), longer than any wait may last
    without progress.  All scores are 0, so p = 2^-7.

    With every row of do 1, dv sums 2^28 terms of 2^-7.  Multiples of 2^-7 up to 2^17 fit the 24 bits of fp32, so the
    running sum is exact to there; from there on a term may vanish beside it (an fp32 sum of n terms is only known to
    n 2^-24 of itself, 16 here), but none lowers it and none is counted for more than it is: 2^17 <= dv <= 2^21.  With
    do = 1 in the last token alone, dv = 128 2^-7 = 1 exactly, which shows the walk's end."""
    T, H, S, D = 1 << 21, 128, 128, 8
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    q = torch.zeros(1, T, H, D, device="cuda", dtype=BF16)
    do = torch.ones_like(q)
    k = torch.randn(1, S, 1, D, device="cuda", dtype=BF16)
    v = torch.zeros_like(k)
    status = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    o, lse = sg.softmax_attention_fwd(q, k, v, causal=False, device_status=status)
    assert int(status) == 0 and float(o.abs().max()) == 0.0
    r = sg.softmax_attention_bwd(q, k, v, o, lse, do, causal=False, device_status=status)
    assert int(status) == 0
    assert 2.0 ** 17 <= float(r["dv"].min()) and float(r["dv"].max()) <= 2.0 ** 21
    assert float(r["dk"].abs().max()) == 0.0 and float(r["dq"].abs().max()) == 0.0
    do[:, :-1] = 0
    r = sg.softmax_attention_bwd(q, k, v, o, lse, do, causal=False, device_status=status)
    assert int(status) == 0 and bool((r["dv"] == 1.0).all())


def test_bad_bounds_show_through_the_differentiable_call():
    gen = torch.Generator().manual_seed(1)
    q, do = (torch.randn(100, 4, 64, generator=gen).to(BF16).cuda() for _ in range(2))
    k, v = (torch.randn(100, 2, 64, generator=gen).to(BF16).cuda() for _ in range(2))
    q.requires_grad_()
    good, bad = (torch.tensor(x).cuda() for x in ([0, 50, 100], [0, 60, 50, 100]))
    word = torch.full((2,), 9, dtype=torch.int32, device="cuda")
    o = sg.softmax_attention(q, k, v, cu_seqlens=good, device_status=word)
    assert word.tolist() == [0, 9]
    torch.autograd.grad(o, q, do)
    assert word.tolist() == [0, 0]
    o = sg.softmax_attention(q, k, v, cu_seqlens=bad, device_status=word)
    assert word.tolist() == [1, 0]
    torch.autograd.grad(o, q, do)
    assert word.tolist() == [1, 1]
    sg.softmax_attention(q.detach(), k, v, cu_seqlens=good, device_status=word[:1])
    assert word.tolist() == [0, 1]


def operands(gen, dtype, Tq, Tk, H, Hk, D):
    q, do = (torch.randn(1, Tq, H, D, generator=gen).to(dtype).cuda() for _ in range(2))
    k, v = (torch.randn(1, Tk, Hk, D, generator=gen).to(dtype).cuda() for _ in range(2))
    return q, k, v, do


def rounding(dtype):
    """One rounding of a result; fp32: with room for its sums."""
    return 2.0 ** -8 if dtype == BF16 else 2.0 ** -16


def minus_infinity(dtype):
    gen = torch.Generator().manual_seed(2)
    q, k, v, do = operands(gen, dtype, 200, 300, 4, 2, 64)
    q[..., 0] = -1.0
    k[..., 0] = 0.0
    want, want_lse = sg.softmax_attention_fwd(q, k[:, 200:].contiguous(), v[:, 200:].contiguous(), causal=False)
    k[:, :200, :, 0] = float("inf")
    v[:, :200] = torch.finfo(dtype).max
    o, lse = sg.softmax_attention_fwd(q, k, v, causal=False)
    # the same 100 keys in one tile or in two: on each side p is rounded, and o
    assert float((o.double() - want.double()).abs().max()) <= 4 * rounding(dtype) * float(v[:, 200:].abs().max())
    assert float((lse - want_lse).abs().max()) <= 2e-4  # sums of p, each to 7.5e-5
    k[..., 0] = float("inf")
    o, lse = sg.softmax_attention_fwd(q, k, v, causal=False)
    assert float(o.abs().max()) == 0.0 and bool((lse == float("-inf")).all())
    v.zero_()
    r = sg.softmax_attention_bwd(q, k, v, o, lse, do, causal=False)
    assert float(r["dk"].abs().max()) == 0.0 and float(r["dv"].abs().max()) == 0.0
    assert float(r["dq"][..., 1:].abs().max()) == 0.0


def test_scores_of_minus_infinity_weigh_nothing():
    """Keys whose score is -inf get the weight 0 in every tile, so values of any size there do not show; rows whose
    visible scores are all -inf come out as rows that see nothing, and add nothing to dk and dv.  (The first column of dq
    is 0 times the infinite key.)"""
    minus_infinity(BF16)


def equal_scores(dtype, value, decode):
    """Every score is value / 8: o is the mean of the values."""
    gen = torch.Generator().manual_seed(3)
    q, k, v, _ = operands(gen, dtype, 1 if decode else 150, 333, 4, 2, 64)
    k.zero_()
    q[..., 0], k[..., 0] = 1.0, value
    if decode:
        o = sg.softmax_attention_decode_step(q[:, 0].contiguous(), k, v, torch.tensor([333]).cuda())[:, None]
    else:
        o, lse = sg.softmax_attention_fwd(q, k, v, causal=False)
        score = float(k[0, 0, 0, 0].double()) / 8
        assert float((lse.double() - score).abs().max()) <= 2.0 ** -20 * abs(score)
    want = v.double().mean(1).repeat_interleave(2, 1)[:, None]
    # p is 1 or a value near 1, the same up to 7.5e-5 for all keys; then o is rounded
    assert float((o.double() - want).abs().max()) <= rounding(dtype) * float(v.double().abs().mean(1).max())


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("value", [-3.38e38, -1e30, 1e12, 2e38])
def test_huge_equal_scores(value, decode):
    """A row whose keys were all given the type's lowest value, or any huge one, is the mean of their values."""
    equal_scores(BF16, value, decode)


def lowest_then_ordinary(dtype):
    gen = torch.Generator().manual_seed(4)
    q, k, v, _ = operands(gen, dtype, 150, 400, 2, 1, 128)
    q[..., 0], k[..., 0] = 1.0, 0.0
    want, _ = sg.softmax_attention_fwd(q, k[:, 256:].contiguous(), v[:, 256:].contiguous(), causal=False)
    k[:, :256, :, 0] = torch.finfo(dtype).min
    o, _ = sg.softmax_attention_fwd(q, k, v, causal=False)
    # the same 144 keys, whole tiles of others in front of them: on each side p is rounded, and o
    off = 4 * rounding(dtype) * float(v.abs().max())
    assert float((o.double() - want.double()).abs().max()) <= off
    step = sg.softmax_attention_decode_step(q[:, 0].contiguous(), k, v, torch.tensor([400]).cuda())
    assert float((step.double() - want[:, 0].double()).abs().max()) <= off


def test_lowest_scores_then_ordinary_ones():
    """Keys of the lowest value weigh nothing beside ordinary ones that come later, whatever their own tiles held."""
    lowest_then_ordinary(BF16)


def test_fp32_operands_to_the_ends_of_their_range():
    """The split of an fp32 operand into two parts holds for the largest finite values (which rounding to 11 bits takes
    past the range) and for infinities."""
    minus_infinity(FP32)
    lowest_then_ordinary(FP32)
    for decode in (False, True):
        for value in (torch.finfo(FP32).min, -1e30, 1e12, torch.finfo(FP32).max):
            equal_scores(FP32, value, decode)


def test_fp32_largest_values_stay():
    """A value of the largest size at the only key that a row sees is the output, and elsewhere reaches no row."""
    top = torch.finfo(FP32).max
    gen = torch.Generator().manual_seed(6)
    q, k, v, _ = operands(gen, FP32, 70, 70, 2, 1, 32)
    want, _ = sg.softmax_attention_fwd(q, k, v)
    v[:, 69, 0, 3], v[:, 0, 0, 4] = top, -top
    o, _ = sg.softmax_attention_fwd(q, k, v)
    # row 0 sees key 0 alone: 1 times its value, a product of three parts, to 2^-21
    assert float((o[0, 0, :, 4].double() / top + 1).abs().max()) <= 2.0 ** -21
    keep = [c for c in range(32) if c != 4]
    assert torch.equal(o[:, :69][..., keep], want[:, :69][..., keep])
    # row 69 sees key 69 too: finite, p times the largest value, p of 70 terms to 2^-16
    p = torch.softmax(torch.einsum("hd,jd->hj", q[0, 69].double(), k[0, :, 0].double()) / 32 ** 0.5, -1)[:, 69]
    assert float((o[0, 69, :, 3].double() / top - p).abs().max()) <= 2.0 ** -16 * float(p.max())


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("H", [1, 4, 7])
def test_rows_that_see_nothing_may_hold_anything(dtype, H):
    """Causal, more queries than keys: what the first rows hold (NaN, infinity) reaches no gradient."""
    gen = torch.Generator().manual_seed(5)
    q, k, v, do = operands(gen, dtype, 333, 200, H, 1, 64)
    o, lse = sg.softmax_attention_fwd(q, k, v)
    want = sg.softmax_attention_bwd(q, k, v, o, lse, do)
    q[:, :133], do[:, :133] = float("nan"), float("-inf")
    o2, lse2 = sg.softmax_attention_fwd(q, k, v)
    got = sg.softmax_attention_bwd(q, k, v, o2, lse2, do)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for n in want:
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_what_a_row_sees_that_is_no_number_shows(dtype):
    """NaN in a query is its row's, NaN in a key every row's that sees it, and no other's."""
    gen = torch.Generator().manual_seed(7)
    q, k, v, _ = operands(gen, dtype, 300, 300, 4, 2, 64)
    want, want_lse = sg.softmax_attention_fwd(q, k, v)
    q2, k2 = q.clone(), k.clone()
    q2[0, 7, 1, 5] = float("nan")
    o, lse = sg.softmax_attention_fwd(q2, k, v)
    hit = torch.zeros(1, 300, 4, dtype=torch.bool, device="cuda")
    hit[0, 7, 1] = True
    assert bool(o[hit].isnan().all()) and bool(lse[hit].isnan().all())
    assert torch.equal(o[~hit], want[~hit]) and torch.equal(lse[~hit], want_lse[~hit])
    k2[0, 150, 0, 63] = float("nan")
    o, lse = sg.softmax_attention_fwd(q, k2, v)
    hit = torch.zeros(1, 300, 4, dtype=torch.bool, device="cuda")
    hit[0, 150:, :2] = True
    assert bool(o[hit].isnan().all()) and bool(lse[hit].isnan().all())
    assert torch.equal(o[~hit], want[~hit]) and torch.equal(lse[~hit], want_lse[~hit])
    n = torch.tensor([150, 151]).cuda()
    first = q[0, :2].contiguous()
    cache = [x.expand(2, 300, 2, 64).contiguous() for x in (k2, v)]
    step = sg.softmax_attention_decode_step(first, *cache, n)
    assert bool(step[1, :2].isnan().all()) and bool(step[1, 2:].isfinite().all()) and bool(step[0].isfinite().all())
    behind = sg.softmax_attention_decode_step(first, cache[0][:, :100].contiguous(), cache[1][:, :100].contiguous(),
                                              torch.tensor([0, 100]).cuda(), cache[0][0], cache[1][0])
    assert bool(behind[:, :2].isnan().all()) and bool(behind[:, 2:].isfinite().all())


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("B,T,S", [(0, 5, 5), (2, 0, 7), (2, 7, 0), (1, 0, 0)])
def test_nothing_to_do(B, T, S, dtype):
    """Empty sides, through the differentiable call: empty or zero results, no error."""
    q, k = (torch.zeros(B, n, h, 64, device="cuda", dtype=dtype, requires_grad=True) for n, h in ((T, 4), (S, 2)))
    v = torch.randn(B, S, 2, 64, device="cuda").to(dtype).requires_grad_()
    o = sg.softmax_attention(q, k, v)
    g = torch.autograd.grad(o, (q, k, v), torch.ones_like(o))
    for got, like in ((o, q), (g[0], q), (g[1], k), (g[2], v)):
        assert got.shape == like.shape and float(got.detach().abs().sum()) == 0.0


def test_a_pack_of_very_many_empty_sequences():
    """2^27 sequences, all but the last empty: a CTA passes hundreds of thousands of blocks without work (some seconds)
    between two items."""
    N = 1 << 27
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GB of device memory")
    gen = torch.Generator().manual_seed(8)
    q, k, v, do = operands(gen, BF16, 128, 128, 1, 1, 64)
    want, lse = sg.softmax_attention_fwd(q, k, v)
    grads = sg.softmax_attention_bwd(q, k, v, want, lse, do)
    cu = torch.zeros(N + 1, dtype=torch.int64, device="cuda")
    cu[N] = 128
    status = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    o, lse2 = sg.softmax_attention_fwd(q, k, v, cu_seqlens=cu, device_status=status)
    assert int(status) == 0
    assert torch.equal(o, want) and torch.equal(lse, lse2)
    got = sg.softmax_attention_bwd(q, k, v, o, lse, do, cu_seqlens=cu, device_status=status)
    assert int(status) == 0
    for n in grads:
        assert torch.equal(got[n], grads[n]), n
