"""Softmax attention (forward, gradients, one-token step over a cache, shared prefix) and multi-axis rotary positions:
the cases they are measured on, their plain forms, and their definitions in 64 bits.

``run`` computes an operator in elementary torch operations in fp32, rounded once at the end; with ``own`` set it makes
the framework's calls.  ``exact`` computes the definition in fp64, written apart from the plain form.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one new token of 64 running sequences, positions on three axes (time, height, width): latency counts
        dict(name="rotary step", op="rotary", dtype="bf16", tokens=64, heads=32, kv_heads=8, dim=128, rot=128, axes=3,
             interleaved=False, far=100000),
        # a long video prompt: 65536 patches, heads of a 4096-wide layer with shared key heads
        dict(name="rotary prompt", op="rotary", dtype="bf16", tokens=65536, heads=32, kv_heads=8, dim=128, rot=128,
             axes=3, interleaved=False, far=65536),
        # gradient with respect to q and k in fp32, part of each head rotated, interleaved pairs, odd token count
        dict(name="rotary gradient fp32", op="rotary_bwd", dtype="fp32", tokens=8197, heads=16, kv_heads=16, dim=80,
             rot=64, axes=2, interleaved=True, far=4096),
        # prompts of one batch, as many key heads as query heads
        dict(name="attention prompt", op="attention", dtype="bf16", batch=4, tq=2048, tk=2048, heads=16, kv_heads=16,
             dim=128, causal=True),
        # eight packed prompts of 128 to 4096 tokens, four query heads to a key head
        dict(name="attention packed", op="attention", dtype="bf16", packed=8, shortest=128, longest=4096, lengths=3,
             heads=16, kv_heads=4, dim=128, causal=True),
        # one long prompt, shared key heads
        dict(name="attention long", op="attention", dtype="bf16", batch=1, tq=8192, tk=8192, heads=32, kv_heads=8,
             dim=128, causal=True),
        # a training step's attention: output and gradients
        dict(name="train dense", op="train", dtype="bf16", batch=2, tq=4096, tk=4096, heads=16, kv_heads=4, dim=128,
             causal=True),
        # packed training sequences of odd lengths, smaller heads
        dict(name="train packed", op="train", dtype="bf16", packed=13, shortest=1, longest=2047, lengths=5, heads=12,
             kv_heads=12, dim=64, causal=True),
        # the fp32 form, attending to another sequence (no causal mask), odd sizes
        dict(name="train fp32", op="train", dtype="fp32", batch=2, tq=317, tk=501, heads=8, kv_heads=4, dim=64,
             causal=False),
        # one token of 128 sequences with caches of up to 4096 tokens
        dict(name="decode batch", op="decode", dtype="bf16", n=128, cap=4096, heads=32, kv_heads=8, dim=128, prefix=0,
             lengths=7),
        # one token of 64 sequences that share a prompt of 32768 tokens
        dict(name="decode shared prefix", op="decode", dtype="bf16", n=64, cap=512, heads=32, kv_heads=8, dim=128,
             prefix=32768, lengths=9),
        # one token of a few short sequences: latency counts
        dict(name="decode small", op="decode", dtype="bf16", n=4, cap=1000, heads=16, kv_heads=16, dim=128, prefix=0,
             lengths=11),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "rotary_bwd", "attention", "attention", "train", "train", "decode", "decode"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    kv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 1, 2, 4, 5, 8])
    if op in ("rotary", "rotary_bwd"):
        dim = 8 * rng.randint(4, 24)
        return dict(op=op, dtype=dtype, tokens=_log(rng, 1, 30000), heads=kv * group, kv_heads=kv, dim=dim,
                    rot=rng.choice([dim, dim // 2, dim // 4 * 2]), axes=rng.randint(1, 4),
                    interleaved=rng.random() < 0.5, far=_log(rng, 64, 2000000))
    dim = rng.choice([32, 40, 64, 64, 72, 80, 96, 128, 128, 128])
    if op == "decode":
        cap = _log(rng, 1, 8192 if dtype == "bf16" else 2048)
        n = _log(rng, 1, max(1, min(256, 600000 // (cap * kv))))
        prefix = _log(rng, 16, 16384 if dtype == "bf16" else 2048) if rng.random() < 0.4 else 0
        return dict(op=op, dtype=dtype, n=n, cap=cap, heads=kv * group, kv_heads=kv, dim=dim, prefix=prefix,
                    lengths=rng.randint(0, 1 << 20))
    most = 4096 if dtype == "bf16" else 900
    causal = rng.random() < 0.7
    if rng.random() < 0.5:
        return dict(op=op, dtype=dtype, packed=rng.randint(1, 20), shortest=1, longest=_log(rng, 8, most // 3),
                    lengths=rng.randint(0, 1 << 20), heads=kv * group, kv_heads=kv, dim=dim, causal=causal)
    tq, tk = _log(rng, 1, most), _log(rng, 1, most)
    if rng.random() < 0.6:
        tk = tq
    batch = rng.randint(1, max(1, min(4, most * most // (tq * tk * 4))))
    return dict(op=op, dtype=dtype, batch=batch, tq=tq, tk=tk, heads=kv * group, kv_heads=kv, dim=dim, causal=causal)


def _lengths(case):
    """The packed sequences' lengths, or the valid lengths of the caches."""
    rng = random.Random(case["lengths"])
    if case["op"] == "decode":
        return [rng.randint(1, case["cap"]) for _ in range(case["n"])]
    return [rng.randint(case["shortest"], case["longest"]) for _ in range(case["packed"])]


def _spans(case):
    """[(first query, queries, first key, keys)] of every sequence of an attention case, on the flattened token axes."""
    if "packed" in case:
        at, spans = 0, []
        for n in _lengths(case):
            spans.append((at, n, at, n))
            at += n
        return spans
    return [(b * case["tq"], case["tq"], b * case["tk"], case["tk"]) for b in range(case["batch"])]


def _pairs(case):
    """Pairs of a query and a key that it sees, over all sequences, for one head."""
    total = 0
    for _, tq, _, tk in _spans(case):
        if not case["causal"]:
            total += tq * tk
        else:  # query i sees min(tk, i + 1 + tk - tq) keys
            first = max(0, tq - tk)
            total += (first + 1 + 2 * tk - tq) * (tq - first) // 2
    return total


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] in ("rotary", "rotary_bwd"):
        n = case["tokens"] * (h + hk)
        return {"bytes": 2 * n * d * size + case["tokens"] * case["axes"] * 8 + case["rot"] * 2, "flops": 3 * n * case["rot"]}
    if case["op"] == "decode":
        keys = sum(_lengths(case))
        return {"bytes": 2 * (keys + case["prefix"]) * hk * d * size + 2 * case["n"] * h * d * size + 8 * case["n"],
                "flops": 4 * d * h * (keys + case["n"] * case["prefix"])}
    tq, tk = (sum(s[i] for s in _spans(case)) for i in (1, 3))
    q, kv = tq * h * d * size, tk * hk * d * size
    if case["op"] == "attention":
        return {"bytes": 2 * q + 2 * kv, "flops": 4 * d * h * _pairs(case)}
    return {"bytes": 4 * q + 4 * kv, "flops": 14 * d * h * _pairs(case)}  # q, do in, o, dq out; k, v in, dk, dv out


# ------------------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32 if dt == torch.float32 else dt)

    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    state = dict(case=case)
    if case["op"] in ("rotary", "rotary_bwd"):
        half = case["rot"] // 2
        state["q"], state["k"] = normal(case["tokens"], h, d), normal(case["tokens"], hk, d)
        state["positions"] = torch.randint(0, case["far"], (case["tokens"], case["axes"]), generator=gen, device="cuda")
        state["inv_freq"] = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
        state["axes"] = [min(case["axes"] - 1, i * case["axes"] // half) for i in range(half)]  # sections in order
        state["axes_index"] = torch.tensor(state["axes"], device="cuda")
        return state
    if case["op"] == "decode":
        lengths = _lengths(case)
        state["q"] = normal(case["n"], h, d)
        state["k"], state["v"] = normal(case["n"], case["cap"], hk, d), normal(case["n"], case["cap"], hk, d)
        state["lengths"] = torch.tensor(lengths, dtype=torch.int64, device="cuda")
        state["prefix_k"] = normal(case["prefix"], hk, d) if case["prefix"] else None
        state["prefix_v"] = normal(case["prefix"], hk, d) if case["prefix"] else None
        return state
    spans = _spans(case)
    if "packed" in case:
        tokens = sum(s[1] for s in spans)
        lead_q = lead_k = (tokens,)
        state["cu"] = torch.tensor([s[0] for s in spans] + [tokens], dtype=torch.int64, device="cuda")
    else:
        lead_q, lead_k = (case["batch"], case["tq"]), (case["batch"], case["tk"])
        state["cu"] = None
    state["spans"] = spans
    state["q"], state["k"], state["v"] = normal(*lead_q, h, d), normal(*lead_k, hk, d), normal(*lead_k, hk, d)
    if case["op"] == "train":
        state["do"] = normal(*lead_q, h, d)
    return state


# ------------------------------------------------------------------------------------------------ plain forms

def _plain_rotary(state, sign):
    case = state["case"]
    half = case["rot"] // 2
    angle = state["positions"][:, state["axes_index"]].double() * state["inv_freq"].double()  # far positions: the angle in 64 bits
    cos, sin = angle.cos().float()[:, None], (sign * angle.sin()).float()[:, None]
    out = []
    for x in (state["q"], state["k"]):
        y = x.float().clone()
        if case["interleaved"]:
            a, b = x[..., 0:case["rot"]:2].float(), x[..., 1:case["rot"]:2].float()
            y[..., 0:case["rot"]:2], y[..., 1:case["rot"]:2] = a * cos - b * sin, a * sin + b * cos
        else:
            a, b = x[..., :half].float(), x[..., half:case["rot"]].float()
            y[..., :half], y[..., half:case["rot"]] = a * cos - b * sin, a * sin + b * cos
        out.append(y.to(x.dtype))
    return out


def _plain_mask(tq, tk):
    i, j = torch.arange(tq, device="cuda")[:, None], torch.arange(tk, device="cuda")[None]
    return j > i + (tk - tq)


def _plain_softmax(scores, hidden=None):
    """Softmax over the last axis in place; rows that see nothing become zero."""
    if hidden is not None:
        scores.masked_fill_(hidden, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    top.masked_fill_(top == float("-inf"), 0.0)
    p = scores.sub_(top).exp_()
    return p.div_(p.sum(-1, keepdim=True).clamp_min_(1e-30))


def _plain_attention(state):
    """Sequence by sequence: the probabilities of all heads, then their products."""
    case = state["case"]
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    g, scale, train = h // hk, d ** -0.5, case["op"] == "train"
    q, k, v = (state[x].reshape(-1, n, d) for x, n in (("q", h), ("k", hk), ("v", hk)))
    o = torch.empty_like(q)
    grads = [torch.empty_like(x) for x in (q, k, v)] if train else []
    for q0, tq, k0, tk in state["spans"]:
        # [hk, g tq, d] and [hk, tk, d]: the query heads of a key head one after another
        def rows(x):
            return x[q0:q0 + tq].float().view(tq, hk, g, d).permute(1, 2, 0, 3).reshape(hk, g * tq, d)

        def back(x):
            return x.view(hk, g, tq, d).permute(2, 0, 1, 3).reshape(tq, h, d)

        qs, ks, vs = rows(q), k[k0:k0 + tk].float().transpose(0, 1), v[k0:k0 + tk].float().transpose(0, 1)
        s = torch.matmul(qs * scale, ks.transpose(1, 2))
        p = _plain_softmax(s, _plain_mask(tq, tk).repeat(g, 1) if case["causal"] else None)
        os_ = torch.matmul(p, vs)
        o[q0:q0 + tq] = back(os_).to(o.dtype)
        if train:
            dos = rows(state["do"].reshape(-1, h, d))
            grads[2][k0:k0 + tk] = torch.matmul(p.transpose(1, 2), dos).transpose(0, 1).to(o.dtype)
            ds = torch.matmul(dos, vs.transpose(1, 2)).sub_((dos * os_).sum(-1, keepdim=True)).mul_(p)
            grads[0][q0:q0 + tq] = back(torch.matmul(ds, ks) * scale).to(o.dtype)
            grads[1][k0:k0 + tk] = (torch.matmul(ds.transpose(1, 2), qs) * scale).transpose(0, 1).to(o.dtype)
    o = o.view(state["q"].shape)
    if not train:
        return o
    return [o] + [x.view(state[n].shape) for x, n in zip(grads, ("q", "k", "v"))]


def _plain_decode(state):
    case = state["case"]
    n, h, hk, d, cap = case["n"], case["heads"], case["kv_heads"], case["dim"], case["cap"]
    g = h // hk
    q = state["q"].float().view(n, hk, g, d) * d ** -0.5
    s = torch.matmul(q, state["k"].float().permute(0, 2, 3, 1))  # [n, hk, g, cap]
    s.masked_fill_((torch.arange(cap, device="cuda")[None] >= state["lengths"][:, None])[:, None, None], float("-inf"))
    if case["prefix"]:
        rows = q.permute(1, 0, 2, 3).reshape(hk, n * g, d)
        sp = torch.matmul(rows, state["prefix_k"].float().permute(1, 2, 0)).view(hk, n, g, -1).permute(1, 0, 2, 3)
        s = torch.cat((sp, s), -1)
    p = _plain_softmax(s)
    o = torch.matmul(p[..., case["prefix"]:], state["v"].float().permute(0, 2, 1, 3))
    if case["prefix"]:
        pp = p[..., :case["prefix"]].permute(1, 0, 2, 3).reshape(hk, n * g, -1)
        o += torch.matmul(pp, state["prefix_v"].float().transpose(0, 1)).view(hk, n, g, d).permute(1, 0, 2, 3)
    return o.reshape(n, h, d).to(state["q"].dtype)


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import gated_linear_attention_local_b200 as sg
        if op in ("rotary", "rotary_bwd"):
            call = sg.multi_axis_rotary if op == "rotary" else sg.multi_axis_rotary_bwd
            return list(call(state["q"], state["k"], state["positions"], state["inv_freq"], axes=state["axes"],
                             interleaved=case["interleaved"]))
        if op == "decode":
            return sg.softmax_attention_decode_step(state["q"], state["k"], state["v"], state["lengths"],
                                                    prefix_k=state["prefix_k"], prefix_v=state["prefix_v"])
        args = dict(causal=case["causal"], cu_seqlens=state["cu"])
        if op == "attention":
            return sg.softmax_attention(state["q"], state["k"], state["v"], **args)
        o, lse = sg.softmax_attention_fwd(state["q"], state["k"], state["v"], **args)
        r = sg.softmax_attention_bwd(state["q"], state["k"], state["v"], o, lse, state["do"], **args)
        return [o, r["dq"], r["dk"], r["dv"]]
    if op in ("rotary", "rotary_bwd"):
        return _plain_rotary(state, 1.0 if op == "rotary" else -1.0)
    return _plain_decode(state) if op == "decode" else _plain_attention(state)


# ------------------------------------------------------------------------------------------------ definitions in 64 bits

def _exact_rotary(state, inverse):
    case = state["case"]
    rot = case["rot"]
    turn = torch.empty(case["tokens"], rot // 2, dtype=torch.complex128, device="cuda")
    for i, a in enumerate(state["axes"]):
        theta = state["positions"][:, a].double() * state["inv_freq"][i].double()
        turn[:, i] = torch.polar(torch.ones_like(theta), -theta if inverse else theta)
    out = []
    for x in (state["q"].double(), state["k"].double()):
        pairs = x[..., :rot].unflatten(-1, (-1, 2) if case["interleaved"] else (2, -1))
        if not case["interleaved"]:
            pairs = pairs.transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
        if not case["interleaved"]:
            z = z.transpose(-1, -2)
        out.append(torch.cat((z.flatten(-2), x[..., rot:]), -1))
    return out


def _exact_head(q, k, v, causal, do=None):
    """One head of one sequence: o, and with do the gradients, from p = exp(s - log sum exp s)."""
    scale = 1.0 / math.sqrt(q.shape[-1])
    s = torch.einsum("id,jd->ij", q, k) * scale
    if causal:
        seen = torch.ones_like(s, dtype=torch.bool).tril_(k.shape[0] - q.shape[0])
        s = torch.where(seen, s, torch.full_like(s, -math.inf))
    lse = torch.logsumexp(s, 1)
    p = torch.where(torch.isneginf(lse)[:, None], torch.zeros_like(s), torch.exp(s - lse[:, None]))
    o = p @ v
    if do is None:
        return (o,)
    dp = torch.einsum("id,jd->ij", do, v)
    ds = p * (dp - (p * dp).sum(1, keepdim=True))
    return o, scale * (ds @ k), scale * torch.einsum("ij,id->jd", ds, q), torch.einsum("ij,id->jd", p, do)


def _exact_attention(state):
    case = state["case"]
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    train = case["op"] == "train"
    q, k, v = (state[x].reshape(-1, n, d) for x, n in (("q", h), ("k", hk), ("v", hk)))
    do = state["do"].reshape(-1, h, d) if train else None
    outs = [torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in ((q, q, k, v) if train else (q,))]
    for q0, tq, k0, tk in state["spans"]:
        for i in range(h):
            j = i // (h // hk)
            a, b = slice(q0, q0 + tq), slice(k0, k0 + tk)
            got = _exact_head(q[a, i].double(), k[b, j].double(), v[b, j].double(), case["causal"],
                              do[a, i].double() if train else None)
            for out, x, (rows, col) in zip(outs, got, ((a, i), (a, i), (b, j), (b, j))):
                out[rows, col] += x
    outs = [x.view(state[n].shape) for x, n in zip(outs, ("q", "q", "k", "v"))]
    return outs if train else outs[0]


def _exact_decode(state):
    case = state["case"]
    h, hk = case["heads"], case["kv_heads"]
    o = torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda")
    pk, pv = (None if x is None else x.double() for x in (state["prefix_k"], state["prefix_v"]))
    for n, length in enumerate(_lengths(case)):
        k, v = state["k"][n, :length].double(), state["v"][n, :length].double()
        if pk is not None:
            k, v = torch.cat((pk, k)), torch.cat((pv, v))
        q = state["q"][n].double().view(hk, h // hk, -1)
        s = torch.einsum("agd,jad->agj", q, k) / math.sqrt(case["dim"])
        o[n] = torch.einsum("agj,jad->agd", torch.softmax(s, -1), v).reshape(h, -1)
    return o


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] in ("rotary", "rotary_bwd"):
        return _exact_rotary(state, case["op"] == "rotary_bwd")
    return _exact_decode(state) if case["op"] == "decode" else _exact_attention(state)
