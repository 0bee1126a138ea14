"""Binding of the softmax-attention layer's entry points (declared in include/gdn2.h): norms of
queries and keys with the position rotation, the serving prologue that fills the 8-bit cache,
and attention over that cache.

As in the rest of the binding: argument checks, outputs allocated with torch, one call on
torch's current stream of the inputs' device. Every step of the computation runs in the
library's kernels.
"""
from __future__ import annotations

import functools
import math
from typing import NamedTuple

import torch

from ._lib import GDN2_BF16, GDN2_F32, Gdn2Error, _aligned_gradient, lib

CACHE_BLOCK = 64  # tokens per cache block
_INTERLEAVED, _NO_NORM = 1, 2


class KVCache(NamedTuple):
    """The paged 8-bit cache: k [P, Hk, 64, d] and v [P, Hk, d, 64] (columns permuted, see
    value_columns) float8_e4m3fn, k_scale and v_scale [P, Hk] fp32. Any tuple of four such
    tensors serves as one."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


def kv_cache(num_blocks, num_kv_heads, head_dim, device="cuda"):
    """An empty (zero) cache of num_blocks blocks of 64 tokens."""
    P, Hk, d = num_blocks, num_kv_heads, head_dim
    if d not in (64, 128):
        raise ValueError("head_dim must be 64 or 128")
    codes = [torch.zeros(s, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
             for s in ((P, Hk, CACHE_BLOCK, d), (P, Hk, d, CACHE_BLOCK))]
    scales = [torch.zeros((P, Hk), dtype=torch.float32, device=device) for _ in range(2)]
    return KVCache(*codes, *scales)


def value_columns(device=None):
    """Column of each of a block's 64 tokens in the rows of the value cache (int64 [64]):
    v[..., value_columns()] has its last axis in token order."""
    t = torch.arange(CACHE_BLOCK, device=device)
    return (t // 4 % 4) * 16 + (t // 16) * 4 + t % 4


def _call(name, device, *args):
    """The entry point `name` with torch's current stream of `device` behind args, that device
    being current meanwhile. (The raw getters: torch.cuda's objects for the same cost 2 us of a
    small call's 10.)"""
    fn = getattr(lib(), name)
    index = device.index
    if index == torch._C._cuda_getDevice():
        st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if st != 0:
        raise Gdn2Error(name, st)


def _p(t):
    return None if t is None else t.data_ptr()


def _need_gpu(t):
    if not t.is_cuda:
        raise ValueError("tensors must be on a HIP device")


_CODES = {torch.bfloat16: GDN2_BF16, torch.float32: GDN2_F32}


def _bad(name, t, shape, dtype, device):
    want = f"a {dtype} tensor of shape {tuple(shape)} on {device}"
    err = TypeError if t.dtype != dtype else ValueError
    raise err(f"{name}: expected {want}, got {t.dtype} {tuple(t.shape)} on {t.device}, "
              f"strides {t.stride()}")


def _dense(name, t, shape, dtype, device):
    if not t.is_contiguous() or t.shape != shape or t.dtype != dtype or t.device != device:
        _bad(name + " (contiguous)", t, shape, dtype, device)


def _rows(name, t, shape, dtype, device):
    """Checks [B, T, H, d] rows whose tokens lie at one stride with dense heads; returns that
    stride in elements."""
    if t.shape != shape or t.dtype != dtype or t.device != device:
        _bad(name, t, shape, dtype, device)
    return _token_stride(name, t, shape)


def _token_stride(name, t, shape):
    B, T, H, d = shape
    if t.is_contiguous():
        return H * d
    sb, st, sh, sd = t.stride()
    if T == 1:
        st = sb if B > 1 else H * d
    if (d > 1 and sd != 1) or (H > 1 and sh != d) or (B > 1 and sb != T * st):
        raise ValueError(f"{name}: the rows of a token must be dense and all tokens at one stride, "
                         f"got strides {t.stride()} for shape {tuple(t.shape)}")
    if st < H * d or st % 8:
        raise ValueError(f"{name}: a token stride of {st} elements is not a multiple of 8 "
                         f"of at least {H * d}")
    return st


def _empty(t):
    """A contiguous tensor like t. (A memory format costs the allocation half as much again.)"""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _rotation(inv_freq, d, dev):
    """rot, after a check of inv_freq [rot / 2] (None: no rotation)."""
    if inv_freq is None:
        return 0
    half = inv_freq.numel()
    _dense("inv_freq", inv_freq, (half,), torch.float32, dev)
    if 2 * half > d or half % 4:
        raise ValueError(f"inv_freq: {2 * half} rotated channels; a multiple of 8 up to {d} is "
                         f"needed")
    return 2 * half


def _norm_rope_args(q, k, inv_freq, positions, q_weight, k_weight):
    _need_gpu(q)
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be [B, T, H, d]")
    B, T, Hq, d = shape = q.shape
    Hk = k.shape[2]
    dev, dt = q.device, q.dtype
    code = _CODES.get(dt)
    if code is None:
        raise TypeError(f"unsupported dtype {dt}; use bfloat16 or float32")
    qs = _token_stride("q", q, shape)
    ks = _rows("k", k, (B, T, Hk, d), dt, dev)
    if positions is not None:
        _dense("positions", positions, (B, T), torch.int32, dev)
    if q_weight is not None:
        _dense("q_weight", q_weight, (d,), torch.float32, dev)
    if k_weight is not None:
        _dense("k_weight", k_weight, (d,), torch.float32, dev)
    return B, T, Hq, Hk, d, qs, ks, _rotation(inv_freq, d, dev), code, dev, dt


def _flags(interleaved, norm):
    return (_INTERLEAVED if interleaved else 0) | (0 if norm else _NO_NORM)


def qk_norm_rope_fwd(q, k, inv_freq, positions=None, q_weight=None, k_weight=None, eps=1e-6,
                     interleaved=False, norm=True, out=None):
    """RMS norm of every head row of q [B, T, Hq, d] and k [B, T, Hk, d] (bf16 or fp32), times
    q_weight / k_weight (fp32 [d] or None), then the rotation of its first 2 * len(inv_freq)
    channels by position * inv_freq (fp32 [rot / 2], None: no rotation).

    positions: int32 [B, T] or None (0 .. T - 1 in every sequence). interleaved: pairs
    (2i, 2i + 1) instead of (i, i + rot / 2). norm=False leaves the mean square out. q and k may
    be slices of one projection (a token's rows dense, tokens at one stride). out: optional
    contiguous pair, written and returned (q and k themselves where they are contiguous); not
    tensors that require gradients, unless under no_grad.
    Returns (q_out, k_out)."""
    B, T, Hq, Hk, d, qs, ks, rot, code, dev, dt = _norm_rope_args(q, k, inv_freq, positions,
                                                                  q_weight, k_weight)
    if out is None:
        qo, ko = _empty(q), _empty(k)
    else:
        qo, ko = out
        _dense("out[0]", qo, (B, T, Hq, d), dt, dev)
        _dense("out[1]", ko, (B, T, Hk, d), dt, dev)
        if (qo.requires_grad or ko.requires_grad) and torch.is_grad_enabled():
            raise ValueError("out: the tensors require gradients, which would not know of this "
                             "call; use qk_norm_rope, or no_grad")
    _call("gdn2_qk_norm_rope", dev, q.data_ptr(), k.data_ptr(), _p(q_weight), _p(k_weight),
          _p(positions), _p(inv_freq), qo.data_ptr(), ko.data_ptr(), B, T, Hq, Hk, d, qs, ks, rot,
          eps, _flags(interleaved, norm), code)
    return qo, ko


@functools.lru_cache(maxsize=1024)
def _bwd_workspace(B, T, Hq, Hk, d):
    return int(lib().gdn2_qk_norm_rope_bwd_workspace_bytes(B, T, Hq, Hk, d))


def qk_norm_rope_bwd(q, k, dq_out, dk_out, inv_freq, positions=None, q_weight=None, k_weight=None,
                     eps=1e-6, interleaved=False, norm=True):
    """Gradients of qk_norm_rope_fwd for the gradients dq_out, dk_out (contiguous) of its outputs:
    (dq, dk, dq_weight, dk_weight), the weights' in fp32 [d] (None where the weight is None)."""
    B, T, Hq, Hk, d, qs, ks, rot, code, dev, dt = _norm_rope_args(q, k, inv_freq, positions,
                                                                  q_weight, k_weight)
    _dense("dq_out", dq_out, (B, T, Hq, d), dt, dev)
    _dense("dk_out", dk_out, (B, T, Hk, d), dt, dev)
    dq, dk = torch.empty_like(dq_out), torch.empty_like(dk_out)
    make = torch.empty_like if B * T else torch.zeros_like
    dwq = make(q_weight) if q_weight is not None else None
    dwk = make(k_weight) if k_weight is not None else None
    ws, need = None, 0
    if dwq is not None or dwk is not None:
        need = _bwd_workspace(B, T, Hq, Hk, d)
        ws = (dwk if dwq is None else dwq).new_empty((need + 3) // 4)
    _call("gdn2_qk_norm_rope_bwd", dev, q.data_ptr(), k.data_ptr(), dq_out.data_ptr(),
          dk_out.data_ptr(), _p(q_weight), _p(k_weight), _p(positions), _p(inv_freq),
          dq.data_ptr(), dk.data_ptr(), _p(dwq), _p(dwk), B, T, Hq, Hk, d, qs, ks, rot, eps,
          _flags(interleaved, norm), code, _p(ws), need)
    return dq, dk, dwq, dwk


class _QKNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, inv_freq, positions, eps, interleaved, norm):
        ctx.save_for_backward(q, k, q_weight, k_weight, inv_freq, positions)
        ctx.how = (eps, interleaved, norm)
        return qk_norm_rope_fwd(q, k, inv_freq, positions, q_weight, k_weight, eps, interleaved,
                                norm)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, q_weight, k_weight, inv_freq, positions = ctx.saved_tensors
        eps, interleaved, norm = ctx.how
        dq_out, dk_out = _aligned_gradient(dq_out), _aligned_gradient(dk_out)
        dq, dk, dwq, dwk = qk_norm_rope_bwd(q, k, dq_out, dk_out, inv_freq, positions, q_weight,
                                            k_weight, eps, interleaved, norm)
        return dq, dk, dwq, dwk, None, None, None, None, None


def qk_norm_rope(q, k, inv_freq, positions=None, q_weight=None, k_weight=None, eps=1e-6,
                 interleaved=False, norm=True):
    """Differentiable qk_norm_rope_fwd: gradients flow to q, k and the weights through the
    library's backward. Positions and frequencies are constants. (torch ties a leaf's accumulation
    to the stream of its first use: before a backward pass is captured into a graph, drop eager
    results of the same leaves that are still alive.)"""
    return _QKNormRope.apply(q, k, q_weight, k_weight, inv_freq, positions, eps, interleaved, norm)


def _cache_args(q, cache, block_table, seq_lens, cu_seqlens):
    _need_gpu(q)
    if q.dim() != 4:
        raise ValueError("q must be [B, T, H, d]")
    B, T, Hq, d = q.shape
    dev = q.device
    if q.dtype != torch.bfloat16:
        raise TypeError(f"the cached attention layer is built for bfloat16, got {q.dtype}")
    kc, vc, ks, vs = cache
    if kc.dim() != 4:
        raise ValueError("cache: k must be [P, Hk, 64, d] and v [P, Hk, d, 64]")
    P, Hk = kc.shape[:2]
    _dense("cache.k", kc, (P, Hk, CACHE_BLOCK, d), torch.float8_e4m3fn, dev)
    _dense("cache.v", vc, (P, Hk, d, CACHE_BLOCK), torch.float8_e4m3fn, dev)
    _dense("cache.k_scale", ks, (P, Hk), torch.float32, dev)
    _dense("cache.v_scale", vs, (P, Hk), torch.float32, dev)
    if Hq % Hk:
        raise ValueError(f"{Hq} query heads cannot share {Hk} kv heads evenly")
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.device != dev or cu_seqlens.dim() != 1:
            raise ValueError("cu_seqlens must be a 1-D int32 tensor on the inputs' device")
        if not cu_seqlens.is_contiguous():
            raise ValueError("cu_seqlens must be contiguous")
        if B != 1:
            raise ValueError("packed (cu_seqlens) inputs must have B == 1")
        N = cu_seqlens.numel() - 1
    else:
        N = B
    _dense("seq_lens", seq_lens, (N,), torch.int32, dev)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [N, max_blocks]")
    MB = block_table.shape[1]
    _dense("block_table", block_table, (N, MB), torch.int32, dev)
    return B, T, Hq, Hk, d, N, P, MB, dev


def attn_prologue(q, k, v, cache, block_table, seq_lens, inv_freq, cu_seqlens=None, q_weight=None,
                  k_weight=None, eps=1e-6, interleaved=False, norm=True, out=None):
    """Serving prologue of the attention layer: norm and rotation of the new rows (as
    qk_norm_rope_fwd, at their places in the sequences), queries returned, keys and values
    written into the 8-bit cache.

    q: [N, T, Hq, d], k, v: [N, T, Hk, d] bf16 (slices of one projection are fine), or packed
    [1, T, H, d] with cu_seqlens int32 [N + 1]; cache: a KVCache; block_table: int32
    [N, max_blocks], entries outside [0, P) naming no block; seq_lens: int32 [N], all tokens of
    each sequence with the new ones, which are its last. A sequence with fewer tokens than new
    rows has its leading rows as padding (zeros in the result); rows behind the last packed
    sequence are not written (undefined where out is None). A block that is written must stand in
    the table once. q, k and v are what the projections give: their norm and rotation happen here.
    out: optional contiguous result, which may be q.
    Returns q_out, [.., Hq, d]."""
    B, T, Hq, Hk, d, N, P, MB, dev = _cache_args(q, cache, block_table, seq_lens, cu_seqlens)
    qs = _token_stride("q", q, q.shape)
    ks = _rows("k", k, (B, T, Hk, d), torch.bfloat16, dev)
    vs = _rows("v", v, (B, T, Hk, d), torch.bfloat16, dev)
    if q_weight is not None:
        _dense("q_weight", q_weight, (d,), torch.float32, dev)
    if k_weight is not None:
        _dense("k_weight", k_weight, (d,), torch.float32, dev)
    rot = _rotation(inv_freq, d, dev)
    if out is None:
        out = _empty(q)
    else:
        _dense("out", out, (B, T, Hq, d), torch.bfloat16, dev)
    kc, vc, kcs, vcs = cache
    _call("gdn2_attn_prologue", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), _p(q_weight),
          _p(k_weight), _p(inv_freq), out.data_ptr(), kc.data_ptr(), vc.data_ptr(),
          kcs.data_ptr(), vcs.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
          _p(cu_seqlens), B, T, Hq, Hk, d, N, P, MB, qs, ks, vs, rot, eps,
          _flags(interleaved, norm), GDN2_BF16)
    return out


@functools.lru_cache(maxsize=1024)
def _attention_workspace(packed, B, T, Hq, Hk, d, N, MB, window):
    return int(lib().gdn2_cache_attention_workspace_bytes(packed, B, T, Hq, Hk, d, N, MB, window))


def cache_attention(q, cache, block_table, seq_lens, cu_seqlens=None, window=0, scale=None,
                    out=None, workspace=None):
    """Causal attention of the new rows over the 8-bit cache, which holds their own keys and
    values already (attn_prologue): one token or a few per sequence, or whole prompts.

    q: [N, T, Hq, d] bf16 contiguous, or packed [1, T, Hq, d] with cu_seqlens int32 [N + 1];
    cache, block_table, seq_lens: as for attn_prologue. Query i of a sequence of length S with T
    new rows stands at p = S - T + i and sees the keys j <= p, with window > 0 only those with
    j > p - window. scale: 1 / sqrt(d) where None. Rows that see no key come out zero; rows behind
    the last packed sequence are not written (undefined where out is None). The work is cut by the
    block table's width: a table much wider than the sequences need makes small calls slower. out:
    optional contiguous result (may be q). workspace: optional uint8 device tensor of at least
    cache_attention_workspace_bytes(...), allocated when None; calls that can overlap, captured
    ones among them, need one each.
    Returns o, shaped like q."""
    B, T, Hq, Hk, d, N, P, MB, dev = _cache_args(q, cache, block_table, seq_lens, cu_seqlens)
    if not q.is_contiguous():
        raise ValueError("q: must be contiguous")
    if not 0 <= window < 1 << 31:
        raise ValueError("window must be a token count, or 0 for none")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    elif not 0.0 < scale < math.inf:
        raise ValueError("scale must be positive and finite")
    if out is None:
        out = torch.empty_like(q)
    else:
        _dense("out", out, q.shape, torch.bfloat16, dev)
    need = _attention_workspace(cu_seqlens is not None, B, T, Hq, Hk, d, N, MB, window)
    if workspace is None:
        if need:
            workspace = seq_lens.new_empty((need + 3) // 4)
    elif workspace.device != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the inputs' device")
    else:
        need = workspace.numel()
    kc, vc, ks, vs = cache
    _call("gdn2_cache_attention", dev, q.data_ptr(), kc.data_ptr(), vc.data_ptr(), ks.data_ptr(),
          vs.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), _p(cu_seqlens),
          out.data_ptr(), B, T, Hq, Hk, d, N, P, MB, window, scale, GDN2_BF16, _p(workspace),
          need)
    return out


def cache_attention_workspace_bytes(B, T, Hq, Hk, d, N, max_blocks, window=0, packed=False):
    """Device workspace that cache_attention needs for these sizes (0: none)."""
    return _attention_workspace(bool(packed), B, T, Hq, Hk, d, N, max_blocks, window)
