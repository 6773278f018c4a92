"""Softmax attention, its gradients and rotary positions in fp64 (numpy), with the error each result may have.

The bounds count the roundings a kernel makes.  u = eps / 2 of the operand type is the relative error of one
rounding to it, w = 2^-24 that of one fp32 operation.
  scores    s = scale sum_d q k: D products and sums in fp32 and the scaling, so |ds| <= (D + 4) w scale sum|q k|;
            p = exp(s - lse) then errs by the factor 1 + e with e <= 2 |ds|max + 8 w + c (both s and lse move; c: the
            exponential and its argument's rounding for |s - lse| < 64, 2^-21 relative in fp32; 2^-12, a sixteenth of
            the rounding of p that follows, with bf16 operands)
  o         sum_j p v over tk terms: |do_| <= (u_p + e + tk w) sum p|v| + u |o|, u_p = 2^-8 where p is rounded to bf16
            for the product with v (bf16 operands), else 0
  gradients the same way through dv = p^T do, ds = p (do v - delta), dq = scale ds k, dk = scale ds^T q, with
            delta = sum_d do o formed from the rounded o.
"""
import numpy as np
import torch

W = 2.0 ** -24


def _f64(t):
    return t.detach().double().cpu().numpy()


def spans(q, k, cu=None, cu_k=None):
    """[(q0, tq, k0, tk)] on the flattened token axes."""
    if cu is None:
        B, T, S = q.shape[0], q.shape[1], k.shape[1]
        return [(b * T, T, b * S, S) for b in range(B)]
    cu = [int(x) for x in cu]
    cu_k = cu if cu_k is None else [int(x) for x in cu_k]
    return [(a, b - a, c, d - c) for a, b, c, d in zip(cu, cu[1:], cu_k, cu_k[1:])]


def attention(q, k, v, causal, scale=None, cu=None, cu_k=None, do=None, o_given=None):
    """dict of (value, bound) for o, lse and, with do, dq, dk, dv; in the operands' shapes."""
    bf16 = q.dtype == torch.bfloat16
    u = 2.0 ** -8 if bf16 else W
    up = 2.0 ** -8 if bf16 else 0.0
    H, D = q.shape[-2:]
    Hk = k.shape[-2]
    G = H // Hk
    scale = D ** -0.5 if scale is None else scale
    Q, K, V = (_f64(t).reshape(-1, t.shape[-2], D) for t in (q, k, v))
    out = {n: [np.zeros(x.shape), np.zeros(x.shape)] for n, x in (("o", Q), ("dq", Q), ("dk", K), ("dv", V))}
    out["lse"] = [np.full(Q.shape[:2], -np.inf), np.zeros(Q.shape[:2])]
    dO = None if do is None else _f64(do).reshape(-1, H, D)
    for q0, tq, k0, tk in spans(q, k, cu, cu_k):
        if tq == 0 or tk == 0:
            continue
        seen = np.ones((tq, tk), bool)
        if causal:
            seen = np.arange(tk)[None] <= np.arange(tq)[:, None] + tk - tq
        some = seen.any(1)
        for h in range(H):
            j = h // G
            qs, ks, vs = Q[q0:q0 + tq, h], K[k0:k0 + tk, j], V[k0:k0 + tk, j]
            s = np.where(seen, scale * (qs @ ks.T), -np.inf)
            top = np.where(some, s.max(1), 0.0)
            p = np.exp(s - top[:, None])
            l = p.sum(1)
            lse = np.where(some, top + np.log(np.where(some, l, 1.0)), -np.inf)
            p = p / np.where(some, l, 1.0)[:, None]
            ds_ = np.where(seen, (D + 4) * W * scale * (np.abs(qs) @ np.abs(ks).T), 0.0)
            e = (2 * ds_.max(1) + 8 * W + (2.0 ** -12 if bf16 else 2.0 ** -21))[:, None]
            o = p @ vs
            pv = p @ np.abs(vs)
            do_err = (up + e + tk * W) * pv
            a, b = slice(q0, q0 + tq), slice(k0, k0 + tk)
            out["o"][0][a, h] = o
            out["o"][1][a, h] = do_err + u * np.abs(o)
            out["lse"][0][a, h] = lse
            out["lse"][1][a, h] = np.where(some, e[:, 0] + (tk + 8) * W + 4 * W * np.abs(np.where(some, lse, 0)), 0)
            if dO is None:
                continue
            g = dO[a, h]
            dp = g @ vs.T
            delta = (g * o).sum(1)[:, None]
            dp_err = (D + 2) * W * (np.abs(g) @ np.abs(vs).T)
            delta_err = (np.abs(g) * out["o"][1][a, h]).sum(1)[:, None] + (D + 2) * W * (np.abs(g) * np.abs(o)).sum(1)[:, None]
            ds = p * (dp - delta)
            ds_err = p * (dp_err + delta_err) + (e + up + 4 * W) * np.abs(ds)
            out["dv"][0][b, j] += p.T @ g
            out["dv"][1][b, j] += (up + tq * G * W) * (p.T @ np.abs(g)) + (p * e).T @ np.abs(g)
            out["dq"][0][a, h] = scale * (ds @ ks)
            out["dq"][1][a, h] = scale * ((ds_err + tk * W * np.abs(ds)) @ np.abs(ks))
            out["dk"][0][b, j] += scale * (ds.T @ qs)
            out["dk"][1][b, j] += scale * ((ds_err + tq * G * W * np.abs(ds)).T @ np.abs(qs))
    for n in ("dq", "dk", "dv"):
        out[n][1] += u * np.abs(out[n][0])
    shapes = dict(o=q, dq=q, dk=k, dv=v)
    res = {n: tuple(x.reshape(shapes[n].shape) for x in out[n]) for n in shapes}
    res["lse"] = tuple(x.reshape(q.shape[:-1]) for x in out["lse"])
    return res


def check(got, want, what, slack=1.05):
    """Every element within its bound (slack: products of two errors), the infinities in the same places."""
    value, bound = want
    x = _f64(got)
    assert x.shape == value.shape, (what, x.shape, value.shape)
    inf = np.isinf(value)
    assert np.array_equal(np.isinf(x), inf) and not np.isnan(x).any(), f"{what}: {np.isnan(x).sum()} NaN"
    assert np.array_equal(x[inf], value[inf])
    off = np.abs(x - np.where(inf, x, value))
    bad = off > slack * bound + 1e-30
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, off / (bound + 1e-30), 0)), off.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off, worst at {i}: {x[i]} for {value[i]} (bound {bound[i]})")


def rotary(x, positions, inv_freq, axes, interleaved, inverse=False):
    """(value, bound): angles p * f in fp64 (f the fp32 table), cos and sin in fp32 (2 ulp and the reduced angle's own
    rounding: 8 w), two products and a sum in fp32, one rounding to the operand type."""
    u = 2.0 ** -8 if x.dtype == torch.bfloat16 else W
    X = _f64(x)
    half = inv_freq.shape[0]
    P = positions.cpu().numpy().reshape(*X.shape[:-2], -1)
    theta = P[..., list(axes)].astype(np.float64) * inv_freq.double().cpu().numpy()
    if inverse:
        theta = -theta
    c, s = np.cos(theta)[..., None, :], np.sin(theta)[..., None, :]
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    y, e = X.copy(), np.zeros_like(X)
    y[..., a], y[..., b] = X[..., a] * c - X[..., b] * s, X[..., a] * s + X[..., b] * c
    mag = np.abs(X[..., a]) + np.abs(X[..., b])
    e[..., a] = e[..., b] = 12 * W * mag
    e[..., :2 * half] += u * (np.abs(y[..., :2 * half]) + 12 * W)
    return y, e
