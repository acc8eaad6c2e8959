"""Binding of libkda's latent attention (the full-attention layers between KDA layers) and of the
root-mean-square norm in front of a layer: argument checks and marshalling only.

Unlike the KDA calls these also take views: ``latent_fwd`` and ``latent_bwd`` accept keys and values
that are slices of one up-projection, ``latent_append`` slices of one down-projection. Tensors must lie
on one CUDA device; the work is enqueued on that device's current stream.
"""
from __future__ import annotations

import functools

import torch

import kimi_delta_attention_25_b200 as _kda

LATENT_DIM, HEAD_DIM = 512, 128
_BF16, _F32, _I32, _I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


def _check(name, t, dtype, dev, shape=None, dense=True):
    """One tensor argument: type, device (by index), shape and (``dense``) contiguity."""
    if t.dtype is dtype and t.get_device() == dev >= 0 and (shape is None or t.shape == shape) and (
            not dense or t.is_contiguous()):
        return
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, str(dtype).replace("torch.", ""), t.dtype))
    if not t.is_cuda or dev < 0:
        raise ValueError("libkda takes CUDA tensors only (no CPU fallback)")
    if t.get_device() != dev:
        raise ValueError("%s is on %s, the call's other tensors on cuda:%d" % (name, t.device, dev))
    if shape is not None and t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    raise ValueError("%s must be contiguous" % name)


_FNS = {}


def _call(name, dev, args):
    """The C entry point on device ``dev`` and its current stream; raises on a status. (The tensors were
    checked to be on that device; torch's context manager is entered only when it is not the current one.)"""
    fn = _FNS.get(name)
    if fn is None:
        fn = _FNS[name] = getattr(_kda.load(), name)
    if dev == torch._C._cuda_getDevice():
        st = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if st != _kda.KDA_OK:
        raise _kda.KDAError(st, name)


@functools.lru_cache(maxsize=256)
def _size(name, *dims):
    """A workspace size, which depends on the arguments alone."""
    return int(getattr(_kda.load(), name)(*dims))


def _p(t):
    return None if t is None else t.data_ptr()


def _rows(name, t, B, L, H, D):
    """Token and head strides of a [B, L, H, D] view whose batch rows follow one another."""
    sb, st, sh, sc = t.stride()
    if L == 1:
        st = sb                           # batch rows of one token: the stride between them is the tokens'
    if sc != 1 or (B > 1 and L > 1 and sb != L * st):
        raise ValueError("%s: channels must be contiguous and batch rows follow one another" % name)
    # a stride along an axis of one element is never used; the library wants a plausible one
    return (st if B * L > 1 else max(st, 8) // 8 * 8), (sh if H > 1 else D)


def _expanded(q, k, v, k_shared, cu_q, cu_k):
    """Checks of the expanded form's inputs; sizes and strides as the C call takes them."""
    shape, k_shape, v_shape = q.shape, k.shape, v.shape
    if len(shape) != 4 or len(k_shape) != 4 or len(v_shape) != 4:
        raise ValueError("q, k and v must be [B, T, H, D]")
    dev = q.get_device()
    B, T, H, _ = shape
    Tk, dk, dv = k_shape[1], k_shape[3], v_shape[3]
    dr = 0 if k_shared is None else k_shared.shape[-1]
    _check("q", q, _BF16, dev, (B, T, H, dk + dr))
    _check("k", k, _BF16, dev, (B, Tk, H, dk), dense=False)
    _check("v", v, _BF16, dev, (B, Tk, H, dv), dense=False)
    ks, vs, rs = _rows("k", k, B, Tk, H, dk), _rows("v", v, B, Tk, H, dv), 0
    if k_shared is not None:
        _check("k_shared", k_shared, _BF16, dev, (B, Tk, dr), dense=False)
        sb, rs, sc = k_shared.stride()
        if Tk == 1:
            rs = sb
        if sc != 1 or (B > 1 and Tk > 1 and sb != Tk * rs):
            raise ValueError("k_shared: channels must be contiguous and batch rows follow one another")
        rs = rs if B * Tk > 1 else dr
    N = B
    if (cu_q is None) != (cu_k is None):
        raise ValueError("give both cu_seqlens and cu_seqlens_k, or neither")
    if cu_q is not None:
        N = cu_q.shape[0] - 1
        _check("cu_seqlens", cu_q, _I32, dev, (N + 1,))
        if cu_k is not cu_q:
            _check("cu_seqlens_k", cu_k, _I32, dev, (N + 1,))
    return dev, (B, T, Tk, H, N, dk, dv, dr), (*ks, *vs, rs)


def _workspace(workspace, size, like):
    if workspace is None:
        return like.new_empty((max(size, 256),), dtype=torch.uint8)
    _check("workspace", workspace, torch.uint8, like.get_device())
    return workspace


def latent_fwd(q, k, v, k_shared=None, cu_seqlens=None, cu_seqlens_k=None, causal=True, scale=None, out=None, lse=None,
               workspace=None, return_workspace=False):
    """``kda_latent_fwd``: softmax attention whose keys are a part per head and a part all heads share.
    q [B,T,H,128+dr] bf16; k, v [B,Tk,H,128] bf16 (views with strides allowed); k_shared [B,Tk,dr] (dr 64)
    or None; cu_seqlens and cu_seqlens_k int32 [N+1] for packed sequences (``cu_seqlens_k`` defaults to
    ``cu_seqlens``). With ``causal`` a sequence's last query sees all its keys, the one before one key
    less, and so on. ``scale`` defaults to (128 + dr) ** -0.5. Returns (out [B,T,H,128] bf16, lse [B,T,H]
    fp32), and the workspace (for ``workspace_status``) as a third element when ``return_workspace``."""
    if cu_seqlens_k is None:
        cu_seqlens_k = cu_seqlens
    dev, dims, strides = _expanded(q, k, v, k_shared, cu_seqlens, cu_seqlens_k)
    B, T, Tk, H, N, _, dv, dr = dims
    if out is None:
        out = q.new_empty((B, T, H, dv))
    else:
        _check("out", out, _BF16, dev, (B, T, H, dv))
    if lse is None:
        lse = q.new_empty((B, T, H), dtype=_F32)
    else:
        _check("lse", lse, _F32, dev, (B, T, H))
    ws = _workspace(workspace, _size("kda_latent_fwd_workspace_size", B, T, Tk, H, N, dr), q)
    _call("kda_latent_fwd", dev, (_p(q), _p(k), _p(v), _p(k_shared), _p(cu_seqlens), _p(cu_seqlens_k), _p(out), _p(lse),
                                  *dims, *strides, 1 if causal else 0, q.shape[-1] ** -0.5 if scale is None else scale,
                                  _kda.KDA_BF16, _p(ws), ws.numel()))
    return (out, lse, ws) if return_workspace else (out, lse)


def latent_bwd_workspace_size(B, T, Tk, H, N, dr=64) -> int:
    return _size("kda_latent_bwd_workspace_size", B, T, Tk, H, N, dr)


def latent_bwd(q, k, v, k_shared, out, lse, dout, cu_seqlens=None, cu_seqlens_k=None, causal=True, scale=None, grads=None,
               workspace=None, return_workspace=False):
    """``kda_latent_bwd``: gradients of ``latent_fwd`` with the same inputs, its ``out`` and ``lse``, and
    ``dout`` [B,T,H,128] bf16. Returns a dict of dense bf16 tensors dq, dk, dv and dk_shared (None without
    a shared key part); ``grads`` may supply them (same keys) to be written in place."""
    if cu_seqlens_k is None:
        cu_seqlens_k = cu_seqlens
    dev, dims, strides = _expanded(q, k, v, k_shared, cu_seqlens, cu_seqlens_k)
    B, T, Tk, H, N, dk, dv, dr = dims
    _check("out", out, _BF16, dev, (B, T, H, dv))
    _check("lse", lse, _F32, dev, (B, T, H))
    _check("dout", dout, _BF16, dev, (B, T, H, dv))
    g = dict(grads) if grads is not None else {}
    for key, like in (("dq", q), ("dk", k), ("dv", v), ("dk_shared", k_shared if dr else None)):
        if like is None:
            g[key] = None
        elif g.get(key) is None:
            g[key] = torch.empty_like(like, memory_format=torch.contiguous_format)
        else:
            _check(key, g[key], _BF16, dev, like.shape)
    ws = _workspace(workspace, latent_bwd_workspace_size(B, T, Tk, H, N, dr), q)
    _call("kda_latent_bwd", dev, (_p(q), _p(k), _p(v), _p(k_shared), _p(cu_seqlens), _p(cu_seqlens_k), _p(out), _p(lse),
                                  _p(dout), _p(g["dq"]), _p(g["dk"]), _p(g["dv"]), _p(g["dk_shared"]), *dims, *strides,
                                  1 if causal else 0, q.shape[-1] ** -0.5 if scale is None else scale, _kda.KDA_BF16,
                                  _p(ws), ws.numel()))
    return (g, ws) if return_workspace else g


def latent_decode_workspace_size(N, Tq, H) -> int:
    return _size("kda_latent_decode_workspace_size", N, Tq, H)


def latent_decode_step(q, cache, page_table, seq_lens, scale=None, out=None, lse=None, workspace=None,
                       return_workspace=False):
    """``kda_latent_decode_step``: the absorbed form over a paged cache. q [N,Tq,H,512+dr] bf16 (Tq new
    tokens per sequence, already in the cache); cache [pages,page_size,512+dr] bf16; page_table int32
    [N,max_pages]; seq_lens int32 [N], the new tokens included. ``scale`` defaults to (128 + dr) ** -0.5,
    that of the expanded form. Returns (out [N,Tq,H,512] bf16, lse [N,Tq,H] fp32), and the workspace as a
    third element when ``return_workspace``."""
    if q.dim() != 4 or cache.dim() != 3 or page_table.dim() != 2:
        raise ValueError("q must be [N, Tq, H, D], cache [pages, page_size, D], page_table [N, max_pages]")
    dev = q.get_device()
    N, Tq, H, W = q.shape
    pages, page = cache.shape[:2]
    _check("q", q, _BF16, dev)
    _check("cache", cache, _BF16, dev, (pages, page, W))
    _check("page_table", page_table, _I32, dev, (N, page_table.shape[1]))
    _check("seq_lens", seq_lens, _I32, dev, (N,))
    if out is None:
        out = q.new_empty((N, Tq, H, LATENT_DIM))
    else:
        _check("out", out, _BF16, dev, (N, Tq, H, LATENT_DIM))
    if lse is None:
        lse = q.new_empty((N, Tq, H), dtype=_F32)
    else:
        _check("lse", lse, _F32, dev, (N, Tq, H))
    dr = W - LATENT_DIM
    ws = _workspace(workspace, latent_decode_workspace_size(N, Tq, H), q)
    _call("kda_latent_decode_step", dev, (_p(q), _p(cache), _p(page_table), _p(seq_lens), _p(out), _p(lse), N, Tq, H,
                                          LATENT_DIM, dr, page, pages, page_table.shape[1],
                                          (HEAD_DIM + dr) ** -0.5 if scale is None else scale, _kda.KDA_BF16, _p(ws),
                                          ws.numel()))
    return (out, lse, ws) if return_workspace else (out, lse)


def latent_append(c, k_shared, cache, slots, weight=None, eps=1e-5):
    """``kda_latent_append``: cache row ``slots[t]`` = [c_t / rms(c_t) * weight, k_shared_t] for new tokens:
    c [T,512] and k_shared [T,dr] or None, bf16 (rows with a stride allowed), cache [pages,page_size,512+dr]
    bf16 (updated in place and returned), slots int64 [T] (rows of the flattened cache, each at most once;
    rows outside it, such as -1, are skipped). ``weight`` fp32 [512], or None for c as it is."""
    shape, rows = c.shape, cache.shape
    if len(shape) != 2 or len(rows) != 3:
        raise ValueError("c must be [T, 512] and cache [pages, page_size, D]")
    dev = c.get_device()
    (T, dc), (pages, page, _) = shape, rows
    dr = 0 if k_shared is None else k_shared.shape[-1]
    _check("c", c, _BF16, dev, dense=False)
    _check("cache", cache, _BF16, dev, (pages, page, dc + dr))
    _check("slots", slots, _I64, dev, (T,))
    cs, step = c.stride()
    rs, step_r = 0, 1
    if k_shared is not None:
        _check("k_shared", k_shared, _BF16, dev, (T, dr), dense=False)
        if dr:
            rs, step_r = k_shared.stride()
    if weight is not None:
        _check("weight", weight, _F32, dev, (dc,))
    if step != 1 or step_r != 1:
        raise ValueError("the channels of c and k_shared must be contiguous")
    if T <= 1:
        cs = rs = 0                       # a stride that is never used
    _call("kda_latent_append", dev, (_p(c), _p(k_shared), _p(slots), _p(weight), _p(cache), cs, rs, pages * page, T, dc, dr,
                                     eps, _kda.KDA_BF16))
    return cache


def _norm_args(x, weight, residual, residual_out):
    dev, dtype, shape = x.get_device(), x.dtype, x.shape
    D = shape[-1]
    if dtype is not _BF16 and dtype is not _F32:
        raise TypeError("x must be float32 or bfloat16, got %s" % dtype)
    _check("x", x, dtype, dev)
    _check("weight", weight, _F32, dev, (D,))
    if residual is None:
        return dev, D, x
    _check("residual", residual, dtype, dev, shape)
    if residual_out is None:
        return dev, D, torch.empty_like(x)
    _check("residual_out", residual_out, dtype, dev, shape)
    return dev, D, residual_out


def rms_norm(x, weight, residual=None, eps=1e-5, out=None, residual_out=None):
    """``kda_rms_norm``: h = x + residual (in x's dtype), y = h / sqrt(mean(h^2) + eps) * weight over the last
    axis. x [..., D] float32 or bfloat16, weight fp32 [D]. Returns (y, h); h is x itself without a residual,
    else a new tensor or ``residual_out`` (which may be ``residual``, updated in place)."""
    dev, D, h = _norm_args(x, weight, residual, residual_out)
    if out is None:
        out = torch.empty_like(x)
    else:
        _check("out", out, x.dtype, dev, x.shape)
    _call("kda_rms_norm", dev, (_p(x), _p(residual), _p(weight), _p(out), _p(h), x.numel() // D if D else 0, D, eps,
                                _kda._dtype_code(x)))
    return out, h


def rms_norm_e4m3(x, weight, residual=None, eps=1e-5, out=None, scale=None, residual_out=None):
    """``kda_rms_norm_e4m3``: ``rms_norm`` with its output in 8 bits. Returns (q [..., D] float8_e4m3fn, scale
    fp32 [..., D/128], h): y = q * scale, each scale over 128 channels."""
    dev, D, h = _norm_args(x, weight, residual, residual_out)
    if out is None:
        out = torch.empty_like(x, dtype=torch.float8_e4m3fn)
    else:
        _check("out", out, torch.float8_e4m3fn, dev, x.shape)
    if scale is None:
        scale = weight.new_empty((*x.shape[:-1], D // 128))
    else:
        _check("scale", scale, _F32, dev, (*x.shape[:-1], D // 128))
    _call("kda_rms_norm_e4m3", dev, (_p(x), _p(residual), _p(weight), _p(out), _p(scale), _p(h),
                                     x.numel() // D if D else 0, D, eps, _kda._dtype_code(x)))
    return out, scale, h


def rms_norm_bwd_workspace_size(rows, D) -> int:
    return _size("kda_rms_norm_bwd_workspace_size", rows, D)


def rms_norm_bwd(dy, h, weight, dh=None, eps=1e-5, dx=None, dweight=None, workspace=None):
    """``kda_rms_norm_bwd``: gradients of ``rms_norm`` at its h: dy [..., D] the gradient of y, ``dh`` that of
    h along the residual stream (or None). Returns (dx, the gradient of x and of the residual, in h's dtype,
    and dweight fp32 [D])."""
    dev, D = h.get_device(), h.shape[-1]
    if h.dtype not in (_F32, _BF16):
        raise TypeError("h must be float32 or bfloat16, got %s" % h.dtype)
    _check("h", h, h.dtype, dev)
    _check("dy", dy, h.dtype, dev, h.shape)
    _check("weight", weight, _F32, dev, (D,))
    if dh is not None:
        _check("dh", dh, h.dtype, dev, h.shape)
    if dx is None:
        dx = torch.empty_like(h)
    else:
        _check("dx", dx, h.dtype, dev, h.shape)
    if dweight is None:
        dweight = torch.empty_like(weight)
    else:
        _check("dweight", dweight, _F32, dev, (D,))
    rows = h.numel() // D if D else 0
    ws = _workspace(workspace, rms_norm_bwd_workspace_size(rows, D), h)
    _call("kda_rms_norm_bwd", dev, (_p(dy), _p(h), _p(weight), _p(dh), _p(dx), _p(dweight), rows, D, eps,
                                    _kda._dtype_code(h), _p(ws), ws.numel()))
    return dx, dweight
