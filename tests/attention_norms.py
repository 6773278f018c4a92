"""How far the outputs and gradients of softmax attention may be off as whole tensors, |got - want| / |want| in the
Frobenius norm: a wrong or missing term of a few per cent shows, which bounds on single elements (all errors with one
sign) cannot see.

bf16 operands: a kernel rounds p and ds for their products, and its results; o's rounding enters delta.  A rounding to
bf16 is off by at most u = 2^-8 of its value, u / sqrt 3 in the root mean square where errors spread evenly over that
range.  The errors of the terms of a sum are independent, and with values of random signs |sum|^2 is on average the sum
of the terms' squares, so each kind of rounding moves the sum's norm by that part of itself.  o and dv have two kinds (p,
the result), dq and dk three (ds, delta, the result): sqrt 3 u / sqrt 3 = u.  Exponentials to 7.5e-5 and fp32 sums are
small beside it; a quarter is left for tensors of few elements.
fp32 operands: products to 2^-21, sums in fp32, p = 2^x with x to 2^-21: below 2^-18 together.
"""
import torch

LIMIT = {torch.bfloat16: 1.25 * 2.0 ** -8, torch.float32: 2.0 ** -18}


def off(got, want):
    got, want = got.detach().double().cpu(), torch.as_tensor(want).double().cpu()
    return float((got - want).norm() / want.norm())


def attention64(q, k, v, do, causal, scale=None, spoil=None, rounding=None):
    """o, dq, dk, dv of [T,H,D], [S,Hk,D] operands in fp64.  spoil: a mistake ("delta x": delta times x, "tile j": the
    128 keys from 128 j on are left out of dq, "p": every p of dv a hundredth too large).  rounding: a dtype to which p, ds
    and the results are rounded as a kernel does."""
    T, H, D = q.shape
    S, Hk = k.shape[:2]
    scale = D ** -0.5 if scale is None else scale
    rd = (lambda x: x) if rounding is None else (lambda x: x.to(rounding).double())
    q, do = (x.double().transpose(0, 1) for x in (q, do))
    ks, vs = (x.double().repeat_interleave(H // Hk, 1).transpose(0, 1) for x in (k, v))
    s = scale * (q @ ks.transpose(1, 2))
    if causal:
        seen = torch.arange(S, device=q.device)[None] <= torch.arange(T, device=q.device)[:, None] + S - T
        s = s.masked_fill(~seen, float("-inf"))
    lse = torch.logsumexp(s, -1, keepdim=True)
    p = torch.where(lse == float("-inf"), 0.0, torch.exp(s - lse))
    o = rd(rd(p) @ vs)
    delta = (do * o).sum(-1, keepdim=True)
    if spoil and spoil[0] == "delta":
        delta = delta * spoil[1]
    ds = rd(p * (do @ vs.transpose(1, 2) - delta))
    dsq = ds.clone()
    if spoil and spoil[0] == "tile":
        dsq[..., 128 * spoil[1]:128 * (spoil[1] + 1)] = 0
    dv = rd(p).transpose(1, 2) @ do
    if spoil and spoil[0] == "p":
        dv = dv * 1.01
    back = lambda x: x.transpose(0, 1)
    share = lambda x: back(x).reshape(S, Hk, H // Hk, D).sum(2)
    return {"o": back(o), "dq": back(rd(scale * (dsq @ ks))), "dk": rd(share(scale * (ds.transpose(1, 2) @ q))),
            "dv": rd(share(dv))}
