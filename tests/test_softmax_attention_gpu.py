"""Softmax attention on the GPU (forward, gradients, one-token step, shared prefix) against fp64 with counted roundings."""
import numpy as np
import pytest
import torch

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


# B, Tq, Tk, H, Hk, D, causal
DENSE = [
    (1, 1, 1, 1, 1, 8, True),
    (2, 1, 300, 4, 2, 64, True),
    (1, 300, 1, 2, 1, 64, True),          # 299 rows see nothing
    (2, 127, 129, 3, 1, 128, True),
    (1, 128, 128, 2, 2, 128, True),
    (1, 257, 64, 4, 4, 40, True),         # 193 rows see nothing
    (3, 64, 200, 7, 1, 72, False),        # group of 7: 126 rows a tile of 128
    (1, 700, 700, 5, 5, 96, True),
    (1, 400, 513, 8, 2, 128, False),
    (2, 33, 33, 66, 1, 64, True),         # a group of 66: one token a tile
    (1, 5, 260, 128, 1, 120, True),
    (1, 1100, 1100, 4, 1, 64, True),
    (1, 40, 0, 2, 1, 64, False),          # no keys at all
]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("case", DENSE, ids=["x".join(map(str, c)) for c in DENSE])
def test_dense(case, dtype):
    B, Tq, Tk, H, Hk, D, causal = case
    gen = torch.Generator().manual_seed(Tq * 131 + Tk)
    q, do = (normal(gen, B, Tq, H, D, dtype=dtype) for _ in range(2))
    k, v = (normal(gen, B, Tk, Hk, D, dtype=dtype) for _ in range(2))
    o, lse = sg.softmax_attention_fwd(q, k, v, causal=causal)
    r = sg.softmax_attention_bwd(q, k, v, o, lse, do, causal=causal)
    torch.cuda.synchronize()
    want = ref.attention(q, k, v, causal, do=do)
    ref.check(o, want["o"], "o")
    ref.check(lse, want["lse"], "lse")
    for n in ("dq", "dk", "dv"):
        ref.check(r[n], want[n], n)


PACKED = [
    # lengths of q, lengths of k (None: the same), tokens behind the last sequence, H, Hk, D, causal
    ([0, 1, 5, 128, 129, 0, 300], None, 0, 4, 2, 64, True),
    ([37], None, 100, 2, 2, 128, True),
    ([200, 1, 64, 0], [10, 1, 300, 7], 3, 6, 2, 80, True),
    ([3, 130], [0, 257], 0, 3, 3, 128, False),
    ([1] * 70 + [250], None, 9, 2, 1, 64, True),
    ([9] * 1100, None, 0, 1, 1, 32, True),
    ([3] * 200 + [140] + [2] * 54, None, 5, 2, 2, 64, True),
    ([3] * 200 + [140] + [2] * 55, None, 5, 2, 2, 64, True),
    ([1, 700, 40, 390], [800, 1, 0, 400], 11, 4, 1, 96, False),
]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("case", PACKED, ids=[f"N{len(c[0])}D{c[5]}" for c in PACKED])
def test_packed(case, dtype):
    lq, lk, behind, H, Hk, D, causal = case
    gen = torch.Generator().manual_seed(sum(lq))
    cu = torch.tensor([0] + list(np.cumsum(lq)), dtype=torch.int64).cuda()
    cu_k = None if lk is None else torch.tensor([0] + list(np.cumsum(lk)), dtype=torch.int64).cuda()
    Tq, Tk = sum(lq) + behind, sum(lk or lq) + behind
    q, do = (normal(gen, Tq, H, D, dtype=dtype) for _ in range(2))
    k, v = (normal(gen, Tk, Hk, D, dtype=dtype) for _ in range(2))
    if behind:  # what no sequence holds may be anything
        for x in (q, k, v, do):
            x[-behind:] = float("nan")
    status = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    o, lse = sg.softmax_attention_fwd(q, k, v, causal=causal, cu_seqlens=cu, cu_seqlens_k=cu_k, device_status=status)
    assert int(status) == 0
    r = sg.softmax_attention_bwd(q, k, v, o, lse, do, causal=causal, cu_seqlens=cu, cu_seqlens_k=cu_k)
    torch.cuda.synchronize()
    for x in (q, k, v, do):
        x.nan_to_num_(0.0)
    want = ref.attention(q, k, v, causal, cu=cu, cu_k=cu_k, do=do)
    ref.check(o, want["o"], "o")
    ref.check(lse, want["lse"], "lse")
    for n in ("dq", "dk", "dv"):
        ref.check(r[n], want[n], n)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_neighbours_do_not_leak(dtype):
    """NaN and infinity in the next sequence of a pack reach nothing of this one, forward and backward."""
    gen = torch.Generator().manual_seed(3)
    cu = torch.tensor([0, 70, 140, 333], dtype=torch.int64).cuda()
    q, k, v, do = (normal(gen, 333, 2, 64, dtype=dtype) for _ in range(4))
    args = dict(causal=False, cu_seqlens=cu)
    o, lse = sg.softmax_attention_fwd(q, k, v, **args)
    r = sg.softmax_attention_bwd(q, k, v, o, lse, do, **args)
    for x, bad in ((q, float("nan")), (k, float("inf")), (v, float("nan")), (do, float("-inf"))):
        x[70:140] = bad
    o2, lse2 = sg.softmax_attention_fwd(q, k, v, **args)
    r2 = sg.softmax_attention_bwd(q, k, v, o2, lse2, do, **args)
    for a, b in ((o, o2), (lse, lse2), *((r[n], r2[n]) for n in r)):
        for part in (slice(0, 70), slice(140, 333)):
            assert torch.equal(a[part], b[part])


def test_bad_cu_seqlens_is_reported():
    q = torch.randn(100, 2, 64, device="cuda", dtype=BF16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for cu in ([0, 60, 50, 100], [0, 50, 101], [-1, 50, 100], [0, 1 << 40, 100], [1, 50, 100]):
        o, lse = sg.softmax_attention_fwd(q, q, q, cu_seqlens=torch.tensor(cu).cuda(), device_status=status)
        assert int(status) == 1, cu
    good = torch.tensor([0, 50, 100]).cuda()
    o, lse = sg.softmax_attention_fwd(q, q, q, cu_seqlens=good, device_status=status)
    assert int(status) == 0
    sg.softmax_attention_bwd(q, q, q, o, lse, q, cu_seqlens=torch.tensor([0, 120, 100]).cuda(), device_status=status)
    assert int(status) == 1


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_large_scores_and_scale(dtype):
    """Scores far apart (one key takes all the weight), a scale of the caller's, a very negative row."""
    gen = torch.Generator().manual_seed(4)
    q, k, v = (normal(gen, 1, 150, 2, 64, dtype=dtype) for _ in range(3))
    q[:, 3] *= 40
    k[:, 60] *= 40
    q[:, 9] = -k[:, 9]
    o, lse = sg.softmax_attention_fwd(q, k, v, causal=True, scale=0.7)
    want = ref.attention(q, k, v, True, scale=0.7)
    ref.check(o, want["o"], "o")
    ref.check(lse, want["lse"], "lse")


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_repeats_bitwise(dtype):
    gen = torch.Generator().manual_seed(5)
    q, do = (normal(gen, 1, 900, 8, 128, dtype=dtype) for _ in range(2))
    k, v = (normal(gen, 1, 900, 2, 128, dtype=dtype) for _ in range(2))
    first = None
    for _ in range(5):
        o, lse = sg.softmax_attention_fwd(q, k, v)
        r = sg.softmax_attention_bwd(q, k, v, o, lse, do)
        got = [o, lse, r["dq"], r["dk"], r["dv"]]
        if first is not None:
            assert all(torch.equal(a, b) for a, b in zip(first, got))
        first = got


def test_gradients_against_differences():
    """dq, dk, dv of the fp32 form against central differences of the fp64 definition's loss along random directions."""
    gen = torch.Generator().manual_seed(6)
    q, do = (normal(gen, 1, 19, 4, 16, dtype=FP32) for _ in range(2))
    k, v = (normal(gen, 1, 23, 2, 16, dtype=FP32) for _ in range(2))
    for x in (q, k, v):
        x.requires_grad_()
    o = sg.softmax_attention(q, k, v)
    grads = torch.autograd.grad(o, [q, k, v], do)

    def loss(*x):
        return float((ref.attention(*x, True)["o"][0] * do.double().cpu().numpy()).sum())

    for i, g in enumerate(grads):
        step = torch.randn([q, k, v][i].shape, generator=gen).double().cuda()
        h = 1e-4  # difference error h^2 f''' ~ 1e-7, gradient's own fp32 error ~ 1e-5
        args = [[x.detach().double() for x in (q, k, v)] for _ in range(2)]
        args[0][i] = args[0][i] + h * step
        args[1][i] = args[1][i] - h * step
        slope = (loss(*args[0]) - loss(*args[1])) / (2 * h)
        assert abs(float((g.double() * step).sum()) - slope) < 1e-4 * max(1.0, abs(slope))


def test_autograd_without_a_gradient_for_the_keys():
    q, k, v = (torch.randn(1, 50, 2, 32, device="cuda") for _ in range(3))
    q.requires_grad_()
    sg.softmax_attention(q, k, v).sum().backward()
    assert q.grad is not None and k.grad is None


def decode_reference(q, kc, vc, lengths, pk, pv, scale=None):
    """(value, bound) row by row through the fp64 reference: every sequence is one query over its own keys."""
    vals, bounds = [], []
    for n, length in enumerate(lengths):
        ks, vs = kc[n, :length], vc[n, :length]
        if pk is not None:
            ks, vs = torch.cat((pk, ks)), torch.cat((pv, vs))
        a, b = ref.attention(q[n:n + 1, None], ks[None], vs[None], False, scale=scale)["o"]
        vals.append(a[0, 0])
        bounds.append(b[0, 0] + 8 * ref.W * np.abs(a[0, 0]))  # joining the parts
    return np.stack(vals), np.stack(bounds)


DECODE = [
    # N, S, lengths, P, H, Hk, D
    (1, 1, [1], 0, 1, 1, 8),
    (3, 40, [0, 40, 17], 0, 4, 2, 64),
    (2, 2000, [2000, 1999], 0, 8, 8, 128),
    (5, 777, [1, 0, 300, 256, 257], 33, 4, 1, 128),
    (2, 0, [0, 0], 130, 3, 3, 40),
    (4, 64, [64, 1, 0, 63], 0, 16, 16, 96),
    (70, 300, list(range(1, 71)), 1000, 10, 2, 128),
    (1, 9000, [8999], 0, 32, 1, 128),
    (3, 100, [100, 50, 3], 1, 128, 1, 64),
    (2, 500, [431, 500], 260, 7, 1, 72),
]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("case", DECODE, ids=[f"N{c[0]}S{c[1]}P{c[3]}H{c[4]}-{c[5]}D{c[6]}" for c in DECODE])
def test_decode_step(case, dtype):
    N, S, lengths, P, H, Hk, D = case
    gen = torch.Generator().manual_seed(N * 7 + S)
    q = normal(gen, N, H, D, dtype=dtype)
    kc, vc = (normal(gen, N, S, Hk, D, dtype=dtype) for _ in range(2))
    pk, pv = ((normal(gen, P, Hk, D, dtype=dtype) for _ in range(2)) if P else (None, None))
    for n, length in enumerate(lengths):  # a cache holds anything behind its valid tokens
        kc[n, length:] = float("nan")
        vc[n, length:] = float("inf")
    status = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    ln = torch.tensor(lengths, dtype=torch.int64).cuda()
    o = sg.softmax_attention_decode_step(q, kc, vc, ln, prefix_k=pk, prefix_v=pv, device_status=status)
    assert int(status) == 0
    ref.check(o, decode_reference(q, kc, vc, lengths, pk, pv), "o")


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("G,P", [(15, 0), (16, 0), (16, 140), (17, 0), (17, 140)])
def test_decode_group_sizes(G, P, dtype):
    """On both sides of the largest group that the streaming kernel takes."""
    test_decode_step((3, 520, [1, 519, 260], P, 2 * G, 2, 64), dtype)


def test_decode_bad_length_counts_as_empty():
    q = torch.randn(3, 2, 64, device="cuda", dtype=BF16)
    kc = torch.randn(3, 50, 2, 64, device="cuda", dtype=BF16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = sg.softmax_attention_decode_step(q, kc, kc, torch.tensor([51, -1, 50]).cuda(), device_status=status)
    assert int(status) == 1
    assert float(o[:2].abs().max()) == 0.0 and float(o[2].abs().max()) > 0


def test_decode_continues_a_prompt():
    """Prompt through the forward, then token by token through the cache: each row as in the whole sequence."""
    gen = torch.Generator().manual_seed(11)
    T, H, Hk, D = 150, 4, 2, 64
    q = normal(gen, 2, T, H, D, dtype=BF16)
    k, v = (normal(gen, 2, T, Hk, D, dtype=BF16) for _ in range(2))
    kc, vc = torch.zeros(2, T, Hk, D, device="cuda", dtype=BF16), torch.zeros(2, T, Hk, D, device="cuda", dtype=BF16)
    kc[:, :140], vc[:, :140] = k[:, :140], v[:, :140]
    want = ref.attention(q, k, v, True)["o"]
    out = torch.empty(2, H, D, device="cuda", dtype=BF16)
    for t in range(140, T):
        kc[:, t], vc[:, t] = k[:, t], v[:, t]
        ln = torch.full((2,), t + 1, dtype=torch.int64, device="cuda")
        got = sg.softmax_attention_decode_step(q[:, t].contiguous(), kc, vc, ln, out=out)
        assert got is out
        ref.check(got, (want[0][:, t], want[1][:, t] * 1.01), f"token {t}")


def test_decode_cache_past_32_bit_offsets():
    """The last sequence's cache lies more than 2^31 elements into the tensors."""
    N, S, Hk, D = 3, 8200, 1024, 128
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB of device memory")
    kc = torch.zeros(N, S, Hk, D, device="cuda", dtype=BF16)
    vc = torch.zeros(N, S, Hk, D, device="cuda", dtype=BF16)
    gen = torch.Generator().manual_seed(12)
    kc[2, 8000:, 1000:] = normal(gen, 200, 24, D, dtype=BF16)
    vc[2, 8000:, 1000:] = normal(gen, 200, 24, D, dtype=BF16)
    q = normal(gen, N, Hk, D, dtype=BF16)
    o = sg.softmax_attention_decode_step(q, kc, vc, torch.tensor([1, 1, S]).cuda())
    want = ref.attention(q[2:, None, 1000:], kc[2:, :, 1000:], vc[2:, :, 1000:], False)["o"]
    ref.check(o[2, 1000:], tuple(x[0, 0] for x in want), "o")


def test_packed_tokens_past_32_bit_offsets():
    """The last sequence of a pack lies more than 2^31 elements into q, o, do and dq."""
    T, H, D = 132000, 128, 128
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    cu = torch.tensor([*range(0, T - 500, 500), T - 150, T], dtype=torch.int64).cuda()
    gen = torch.Generator().manual_seed(21)
    q, do = (torch.zeros(T, H, D, device="cuda", dtype=BF16) for _ in range(2))
    k, v = (normal(gen, T, 1, D, dtype=BF16) for _ in range(2))
    last = slice(T - 150, T)
    q[last], do[last] = normal(gen, 150, H, D, dtype=BF16), normal(gen, 150, H, D, dtype=BF16)
    o, lse = sg.softmax_attention_fwd(q, k, v, cu_seqlens=cu)
    r = sg.softmax_attention_bwd(q, k, v, o, lse, do, cu_seqlens=cu)
    want = ref.attention(q[None, last], k[None, last], v[None, last], True, do=do[None, last])
    for name, got in (("o", o), ("lse", lse), *r.items()):
        ref.check(got[None, last], want[name], name)


def test_two_streams_at_once():
    """Calls that run at the same time share nothing: each stream's results as alone."""
    gen = torch.Generator().manual_seed(22)
    sets = [[normal(gen, 2, 700, 8, 64, dtype=BF16)] + [normal(gen, 2, 700, 2, 64, dtype=BF16) for _ in range(2)]
            for _ in range(2)]
    kc = normal(gen, 4, 900, 2, 64, dtype=BF16)
    ln = torch.tensor([900, 1, 450, 0]).cuda()

    def work(q, k, v):
        o, lse = sg.softmax_attention_fwd(q, k, v)
        r = sg.softmax_attention_bwd(q, k, v, o, lse, q)
        step = sg.softmax_attention_decode_step(q[0, :4].contiguous(), kc, kc, ln, k[0], v[0])
        return [o, lse, r["dq"], r["dk"], r["dv"], step]

    want = [work(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(10):
        for st, s, out in zip(streams, sets, got):
            with torch.cuda.stream(st):
                out.append(work(*s))
    torch.cuda.synchronize()
    for w, out in zip(want, got):
        for x in out:
            assert all(torch.equal(a, b) for a, b in zip(x, w))


def test_captured_and_replayed():
    """Forward, backward and decode in one graph, replayed on new inputs; a second graph beside it."""
    gen = torch.Generator().manual_seed(13)
    q, do = (normal(gen, 1, 200, 4, 64, dtype=BF16) for _ in range(2))
    k, v = (normal(gen, 1, 200, 2, 64, dtype=BF16) for _ in range(2))
    kc, vc = (normal(gen, 2, 600, 2, 64, dtype=BF16) for _ in range(2))
    pk, pv = (normal(gen, 300, 2, 64, dtype=BF16) for _ in range(2))
    qt = normal(gen, 2, 4, 64, dtype=BF16)
    ln = torch.tensor([600, 20]).cuda()

    def step():
        o, lse = sg.softmax_attention_fwd(q, k, v)
        r = sg.softmax_attention_bwd(q, k, v, o, lse, do)
        return [o, r["dq"], r["dk"], r["dv"], sg.softmax_attention_decode_step(qt, kc, vc, ln, pk, pv)]

    step()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step()
        graphs.append((g, outs))
    for x in (q, k, v, do, kc, vc, qt):
        x.copy_(torch.randn(x.shape, generator=gen).to(BF16))
    ln.copy_(torch.tensor([77, 598]))
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    want = step()
    for _, outs in graphs:
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_on_a_side_stream():
    gen = torch.Generator().manual_seed(14)
    q, k, v = (normal(gen, 1, 260, 2, 64, dtype=BF16) for _ in range(3))
    want, _ = sg.softmax_attention_fwd(q, k, v)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, _ = sg.softmax_attention_fwd(q, k, v)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


@pytest.mark.parametrize("mixer", ["softmax", "linear"])
def test_rotated_layer(mixer):
    """Rotation, then a token mixer, forward and backward through autograd, as a layer of a hybrid model runs them."""
    gen = torch.Generator().manual_seed(15)
    B, T, H, Hk, D = 2, 130, 4, 4, 64
    q, do = (normal(gen, B, T, H, D, dtype=FP32) for _ in range(2))
    k, v = (normal(gen, B, T, Hk, D, dtype=FP32) for _ in range(2))
    pos = torch.stack((torch.arange(T) // 16, torch.arange(T) % 16), -1).expand(B, T, 2).contiguous().cuda()
    freq = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float().cuda()
    axes = [i % 2 for i in range(D // 2)]
    gamma = torch.full((H,), -0.05, device="cuda")
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    qr, kr = sg.multi_axis_rotary(leaves[0], leaves[1], pos, freq, axes=axes)
    if mixer == "softmax":
        o = sg.softmax_attention(qr, kr, leaves[2])
    else:
        o, _ = sg.chunk_simple_gla(qr, kr, leaves[2], g_gamma=gamma)
    grads = torch.autograd.grad(o, leaves, do)

    ls = [x.detach().double().requires_grad_() for x in (q, k, v)]
    theta = pos[..., axes].double() * freq.double()
    c, s = theta.cos()[..., None, :], theta.sin()[..., None, :]

    def turn(x):
        a, b = x.chunk(2, -1)
        return torch.cat((a * c - b * s, a * s + b * c), -1)

    scores = torch.einsum("bihd,bjhd->bhij", turn(ls[0]), turn(ls[1])) * D ** -0.5
    i, j = torch.arange(T, device="cuda")[:, None], torch.arange(T, device="cuda")[None]
    if mixer == "softmax":
        p = torch.softmax(scores.masked_fill(j > i, float("-inf")), -1)
    else:
        p = scores * torch.exp(-0.05 * (i - j).double()).masked_fill(j > i, 0.0)
    oo = torch.einsum("bhij,bjhd->bihd", p, ls[2])
    want = torch.autograd.grad(oo, ls, do.double())
    for a, b in zip((o, *grads), (oo, *want)):  # the fp32 tolerance of the library's other parity tests
        assert float((a.double() - b).abs().max()) <= 1e-4 * float(b.abs().max())


def test_profile_records_the_kernels():
    from gated_linear_attention_local_b200 import _lib
    q = torch.randn(1, 64, 2, 64, device="cuda", dtype=FP32)
    n = _lib.kernel_launch_count()
    _lib.profile_begin()
    o, lse = sg.softmax_attention_fwd(q, q, q)
    sg.softmax_attention_bwd(q, q, q, o, lse, q)
    rec = _lib.profile_end()
    assert _lib.kernel_launch_count() == n + sum(c for c, _ in rec.values())
    assert set(rec) == {"softmax_attention_fwd", "softmax_attention_delta", "softmax_attention_dkdv",
                        "softmax_attention_dq"}


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_output_alone_is_the_forwards(dtype):
    """softmax_attention without gradients (no lse is formed) gives softmax_attention_fwd's output."""
    gen = torch.Generator().manual_seed(23)
    q, k, v = (normal(gen, 2, 200, 2, 64, dtype=dtype) for _ in range(3))
    want, _ = sg.softmax_attention_fwd(q, k, v)
    assert torch.equal(sg.softmax_attention(q, k, v), want)
    with torch.no_grad():
        assert torch.equal(sg.softmax_attention(q.clone().requires_grad_(), k, v), want)
