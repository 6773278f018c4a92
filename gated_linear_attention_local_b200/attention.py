"""Softmax attention and multi-axis rotary positions: the token mixer of the layers a hybrid model keeps and the
transform of q and k in front of either mixer ("relinear -- convert pretrained transformers to linear/hybrid-attention
models").  Argument marshalling for the entry points of ``include/simple_gla.h``, as in the package's ``__init__``.

  softmax_attention(q, k, v, causal=True, scale=None, cu_seqlens=None, cu_seqlens_k=None, device_status=None) -> o,
      differentiable
  softmax_attention_fwd(...) -> (o, lse);  softmax_attention_bwd(q, k, v, o, lse, do, ...) -> {dq, dk, dv}
  softmax_attention_decode_step(q, k_cache, v_cache, lengths, prefix_k=None, prefix_v=None, scale=None) -> o
  multi_axis_rotary(q, k, positions, inv_freq, axes=None, interleaved=False) -> (q, k) rotated, differentiable
  multi_axis_rotary_bwd(dq, dk, positions, inv_freq, ...) -> (dq, dk) rotated back
"""
from __future__ import annotations

import math

import torch
from torch.autograd.function import once_differentiable

from . import _DTYPES, _autograd_follows, _check_cuda, _on_tensor_device, _ptr, _scale, _stream, _workspace
from ._lib import SGLA_ERR_WORKSPACE, lib, raise_for_status

__all__ = ["softmax_attention", "softmax_attention_fwd", "softmax_attention_bwd", "softmax_attention_decode_step",
           "SoftmaxAttentionFunction", "multi_axis_rotary", "multi_axis_rotary_bwd", "MultiAxisRotaryFunction"]


def _check(name, t, dtype, ndim=None):
    """_check_cuda, the usual case (nothing wrong) in one expression."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.is_contiguous()):
        _check_cuda(name, t, dtype)
    if ndim is not None and t.dim() != ndim:
        _check_cuda(name, t, dtype, ndim)


def _operands(named):
    """CUDA, contiguous, one of the library's two operand types, one type for all."""
    name, t = named[0]
    _check_cuda(name, t)
    dtype = t.dtype
    if dtype not in _DTYPES:
        raise TypeError(f"{name} must be bfloat16 or float32, got {dtype}")
    for other, t in named[1:]:
        if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.is_contiguous()):
            _check_cuda(other, t)
            raise TypeError(f"{other} must be {dtype} like {name}, got {t.dtype}")
    return _DTYPES[dtype]


def _attention_shapes(q, k, v, cu_seqlens, cu_seqlens_k):
    """Checks of the forward and backward; returns (N, Tq, Tk, H, Hk, D, dtype, cu_k)."""
    dt = _operands((("q", q), ("k", k), ("v", v)))
    qs, ks = q.shape, k.shape
    if cu_seqlens is None:
        if cu_seqlens_k is not None:
            raise ValueError("cu_seqlens_k needs cu_seqlens")
        if len(qs) != 4 or len(ks) != 4 or ks[0] != qs[0]:
            raise ValueError("q must be [B,T,H,D] and k, v [B,S,Hk,D]")
        N = qs[0]
    else:
        _check("cu_seqlens", cu_seqlens, torch.int64, 1)
        _check_cuda("cu_seqlens_k", cu_seqlens_k, torch.int64, 1)
        if len(qs) not in (3, 4) or len(ks) != len(qs):
            raise ValueError("with cu_seqlens q must be [T,H,D] or [1,T,H,D], and k, v alike")
        if len(qs) == 4 and (qs[0] != 1 or ks[0] != 1):
            raise ValueError("with cu_seqlens the batch size must be 1 (flatten the batch first)")
        N = cu_seqlens.shape[0] - 1
        if N < 1:
            raise ValueError("cu_seqlens must hold at least two entries")
        if cu_seqlens_k is None:
            cu_seqlens_k = cu_seqlens
            if ks[-3] != qs[-3]:
                raise ValueError("without cu_seqlens_k, k and v must have as many tokens as q")
        elif cu_seqlens_k.shape[0] != N + 1:
            raise ValueError(f"cu_seqlens_k must hold {N + 1} entries like cu_seqlens")
    H, D, Hk = qs[-2], qs[-1], ks[-2]
    if v.shape != ks or ks[-1] != D:
        raise ValueError("k and v must have one shape, and q, k and v one head dimension")
    if Hk < 1 or H % Hk:
        raise ValueError(f"the {H} query heads must be a multiple of the {Hk} key heads")
    return N, qs[-3], ks[-3], H, Hk, D, dt, cu_seqlens_k


def _check_status(device_status, words=1):
    if device_status is not None:
        _check_cuda("device_status", device_status, torch.int32)
        if device_status.numel() < words:
            raise ValueError(f"device_status must hold {words} element{'s' if words > 1 else ''}")


def _forward(q, k, v, causal, scale, cu_seqlens, cu_seqlens_k, device_status=None, want_lse=True):
    N, Tq, Tk, H, Hk, D, dt, cu_k = _attention_shapes(q, k, v, cu_seqlens, cu_seqlens_k)
    _check_status(device_status)
    o = torch.empty_like(q)
    lse = q.new_empty(q.shape[:-1], dtype=torch.float32) if want_lse else None
    st = lib().softmax_attention_fwd(_ptr(q), _ptr(k), _ptr(v), _scale(scale), int(bool(causal)), _ptr(o), _ptr(lse),
                                     _ptr(cu_seqlens), _ptr(cu_k), N, Tq, Tk, H, Hk, D, dt, _ptr(device_status),
                                     _stream())
    raise_for_status(st, "softmax_attention_fwd")
    return o, lse


@_on_tensor_device
def softmax_attention_fwd(q, k, v, causal=True, scale=None, cu_seqlens=None, cu_seqlens_k=None, device_status=None):
    """Softmax attention.  q [B,T,H,D]; k, v [B,S,Hk,D], H a multiple of Hk; or packed [T,H,D] / [1,T,H,D] with
    cu_seqlens int64 [N+1] on the device (and cu_seqlens_k where the keys are split otherwise).  causal: query i
    of a sequence sees the keys j <= i + S - T.  device_status: optional int32 CUDA tensor of one element that
    receives the cu_seqlens check.  Returns (o shaped like q, lse [..., H] fp32); a query that sees no key has
    o = 0 and lse = -inf."""
    return _forward(q, k, v, causal, scale, cu_seqlens, cu_seqlens_k, device_status)


@_on_tensor_device
def softmax_attention_bwd(q, k, v, o, lse, do, causal=True, scale=None, cu_seqlens=None, cu_seqlens_k=None,
                          device_status=None, workspace=None):
    """Gradients of softmax_attention_fwd for the loss sum(o * do), with its outputs o and lse.  Returns
    dict(dq, dk, dv) in the shapes and dtype of q, k, v."""
    N, Tq, Tk, H, Hk, D, dt, cu_k = _attention_shapes(q, k, v, cu_seqlens, cu_seqlens_k)
    _check_status(device_status)
    for name, t in (("o", o), ("do", do)):
        _check(name, t, q.dtype)
        if t.shape != q.shape:
            raise ValueError(f"{name} must have the shape of q {tuple(q.shape)}, got {tuple(t.shape)}")
    _check("lse", lse, torch.float32)
    if lse.shape != q.shape[:-1]:
        raise ValueError(f"lse must be {tuple(q.shape[:-1])}, got {tuple(lse.shape)}")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    nbytes = max(256, lib().softmax_attention_bwd_workspace_size(q.numel() // (H * D) if H * D else 0, H))
    ws = q.new_empty(nbytes, dtype=torch.uint8) if workspace is None else _workspace(nbytes, q.device, workspace)
    st = lib().softmax_attention_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _scale(scale),
                                     int(bool(causal)), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(cu_seqlens), _ptr(cu_k), N,
                                     Tq, Tk, H, Hk, D, dt, _ptr(device_status), _ptr(ws), ws.numel(), _stream())
    raise_for_status(st, "softmax_attention_bwd")
    return dict(dq=dq, dk=dk, dv=dv)


class SoftmaxAttentionFunction(torch.autograd.Function):
    """softmax_attention_fwd with softmax_attention_bwd as its gradient."""

    @staticmethod
    def forward(ctx, q, k, v, causal, scale, cu_seqlens, cu_seqlens_k, device_status=None):
        _check_status(device_status, 2)
        o, lse = _forward(q, k, v, causal, scale, cu_seqlens, cu_seqlens_k, device_status)
        ctx.save_for_backward(q, k, v, o, lse, cu_seqlens, cu_seqlens_k)
        # (written to, never read here: no saved tensor, so that one word may serve many steps)
        ctx.opts = (causal, scale, None if device_status is None else device_status.flatten()[1:])
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, do):
        q, k, v, o, lse, cu, cu_k = ctx.saved_tensors
        causal, scale, status = ctx.opts
        r = softmax_attention_bwd(q, k, v, o, lse, do.contiguous(), causal, scale, cu, cu_k, status)
        return r["dq"], r["dk"], r["dv"], None, None, None, None, None


@_on_tensor_device
def softmax_attention(q, k, v, causal=True, scale=None, cu_seqlens=None, cu_seqlens_k=None, device_status=None):
    """The output of softmax_attention_fwd alone; differentiable in q, k and v (through softmax_attention_bwd) when
    gradients are enabled and one of them requires gradients.  device_status: optional int32 CUDA tensor that receives
    what the device finds (sequences whose bounds are bad are skipped, their outputs and gradients not written): element
    0 the forward's status, element 1 the gradients' once they run (it is needed when the call is differentiable).
    Forward and gradients can be captured into a graph, as long as no graph that autograd recorded eagerly from the same
    leaves is alive then (torch refuses that for every operator)."""
    if _autograd_follows(q, k, v):
        return SoftmaxAttentionFunction.apply(q, k, v, causal, scale, cu_seqlens, cu_seqlens_k, device_status)
    return _forward(q, k, v, causal, scale, cu_seqlens, cu_seqlens_k, device_status, want_lse=False)[0]


@_on_tensor_device
def softmax_attention_decode_step(q, k_cache, v_cache, lengths, prefix_k=None, prefix_v=None, scale=None, out=None,
                                  device_status=None, workspace=None):
    """One token of N sequences: q [N,H,D] against the first lengths[n] tokens (int64 [N] on the device) of
    k_cache, v_cache [N,S,Hk,D], preceded by prefix_k, prefix_v [P,Hk,D] that all sequences share.  The new
    token's own key belongs in the cache before the call.  Returns o [N,H,D]."""
    dt = _operands((("q", q), ("k_cache", k_cache), ("v_cache", v_cache)))
    if q.dim() != 3 or k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError("q must be [N,H,D] and k_cache, v_cache [N,S,Hk,D]")
    N, H, D = q.shape
    S, Hk = k_cache.shape[1:3]
    if k_cache.shape[0] != N or k_cache.shape[3] != D:
        raise ValueError(f"k_cache must be [{N},S,Hk,{D}], got {tuple(k_cache.shape)}")
    if Hk < 1 or H % Hk:
        raise ValueError(f"the {H} query heads must be a multiple of the {Hk} key heads")
    _check("lengths", lengths, torch.int64, 1)
    if lengths.shape[0] != N:
        raise ValueError(f"lengths must be [{N}], got {tuple(lengths.shape)}")
    P = 0
    if prefix_k is not None or prefix_v is not None:
        if prefix_k is None or prefix_v is None:
            raise ValueError("prefix_k and prefix_v go together")
        for name, t in (("prefix_k", prefix_k), ("prefix_v", prefix_v)):
            _check_cuda(name, t, q.dtype, 3)
            if tuple(t.shape[1:]) != (Hk, D):
                raise ValueError(f"{name} must be [P,{Hk},{D}], got {tuple(t.shape)}")
        if prefix_k.shape != prefix_v.shape:
            raise ValueError("prefix_k and prefix_v must have one shape")
        P = prefix_k.shape[0]
    _check_status(device_status)
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_cuda("out", out, q.dtype, 3)
        if out.shape != q.shape:
            raise ValueError(f"out must be {tuple(q.shape)}, got {tuple(out.shape)}")
    ws = workspace
    if ws is not None:
        _check("workspace", ws, torch.uint8)
    while True:
        st = lib().softmax_attention_decode_step(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(lengths),
                                                 _ptr(prefix_k) if P else None, _ptr(prefix_v) if P else None,
                                                 _scale(scale), _ptr(out), N, S, P, H, Hk, D, dt, _ptr(device_status),
                                                 _ptr(ws), 0 if ws is None else ws.numel(), _stream())
        if st != SGLA_ERR_WORKSPACE or ws is not None:
            break
        # there are parts to join (nothing was launched): only then is a workspace needed
        nbytes = int(lib().softmax_attention_decode_workspace_size(N, S, P, H, Hk, D, dt))
        ws = _workspace(nbytes, q.device, None)
    if st == SGLA_ERR_WORKSPACE:
        raise ValueError("workspace is smaller than softmax_attention_decode_workspace_size")
    raise_for_status(st, "softmax_attention_decode_step")
    return out


def _rotary(q, k, positions, inv_freq, axes, interleaved, inverse, where):
    dt = _operands((("q", q),) if k is None else (("q", q), ("k", k)))
    if q.dim() < 2:
        raise ValueError("q must be [..., H, D]")
    *lead, H, D = q.shape
    Hk = 0
    if k is not None:
        *klead, Hk, Dk = k.shape if k.dim() > 1 else (0, 0)
        if klead != lead or Dk != D:
            raise ValueError(f"k must be [..., Hk, D] with q's leading and last dimensions, got {tuple(k.shape)}")
    _check("positions", positions, torch.int64)
    pshape = [*positions.shape]
    if pshape == lead:
        A = 1
    elif pshape and pshape[:-1] == lead and pshape[-1] >= 1:
        A = pshape[-1]
    else:
        raise ValueError(f"positions must be {tuple(lead)} or {tuple(lead)} + (axes,), got {tuple(pshape)}")
    _check("inv_freq", inv_freq, torch.float32, 1)
    half = inv_freq.shape[0]
    if 2 * half > D:
        raise ValueError(f"inv_freq has {half} pairs, a head of {D} has {D // 2}")
    if isinstance(axes, int):
        raise TypeError("axes must be a sequence of ints")
    # (element by element: bytes() of an array is its memory, of a one-element tensor that many zeros)
    table = bytes(half) if axes is None else bytes(axes if type(axes) in (list, tuple) else list(axes))
    if len(table) != half or A > 255:  # an axis that is not below A is refused by the library
        raise ValueError(f"axes must hold one axis below {A} for each of the {half} pairs, {A} at most 255")
    qo = torch.empty_like(q)
    ko = None if k is None else torch.empty_like(k)
    st = lib().multi_axis_rotary(q.data_ptr(), _ptr(k), positions.data_ptr(), inv_freq.data_ptr(), table, qo.data_ptr(),
                                 _ptr(ko), math.prod(lead), H, Hk, D, 2 * half, A, 1 if interleaved else 0,
                                 1 if inverse else 0, dt, _stream())
    raise_for_status(st, where)
    return qo, ko


class MultiAxisRotaryFunction(torch.autograd.Function):
    """multi_axis_rotary with multi_axis_rotary_bwd as its gradient."""

    @staticmethod
    def forward(ctx, q, k, positions, inv_freq, axes, interleaved):
        ctx.save_for_backward(positions, inv_freq)
        axes = None if axes is None else bytes(list(axes))  # read once: the caller's sequence may change later
        ctx.opts = (axes, interleaved)
        return _rotary(q, k, positions, inv_freq, axes, interleaved, False, "multi_axis_rotary")

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        positions, inv_freq = ctx.saved_tensors
        dq, dk = multi_axis_rotary_bwd(dq.contiguous(), None if dk is None else dk.contiguous(), positions, inv_freq,
                                       *ctx.opts)
        return dq, dk, None, None, None, None


@_on_tensor_device
def multi_axis_rotary(q, k, positions, inv_freq, axes=None, interleaved=False):
    """Rotate q [..., H, D] and k [..., Hk, D] (k may be None) by the tokens' positions: pair i of each head turns by
    positions[..., axes[i]] * inv_freq[i].  positions int64 [..., A], or [...] for one axis; inv_freq fp32 [R/2],
    R <= D (later columns pass unchanged); axes: R/2 ints, the axis of each pair (None: axis 0).  Pairs are
    (i, i + R/2), or (2i, 2i + 1) with interleaved.  Returns (q', k'); differentiable in q and k."""
    if _autograd_follows(q, k):
        return MultiAxisRotaryFunction.apply(q, k, positions, inv_freq, axes, interleaved)
    return _rotary(q, k, positions, inv_freq, axes, interleaved, False, "multi_axis_rotary")


@_on_tensor_device
def multi_axis_rotary_bwd(dq, dk, positions, inv_freq, axes=None, interleaved=False):
    """Gradient of multi_axis_rotary: dq, dk rotated by the opposite angles.  Also undoes the rotation."""
    return _rotary(dq, dk, positions, inv_freq, axes, interleaved, True, "multi_axis_rotary_bwd")
