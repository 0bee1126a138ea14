"""Binding of what stands around the mixer in a stack (declared in include/gdn2.h): the diagonal
gated recurrence, the norm between layers with the residual's addition, and the verification of
drafted tokens.

As in the rest of the binding: argument checks, outputs allocated with torch, one call on
torch's current stream of the inputs' device. Every step of the computation runs in the
library's kernels.
"""
from __future__ import annotations

import functools
import math

import torch

from ._attn import _CODES, _bad, _call, _dense, _empty, _need_gpu, _p
from ._lib import _aligned_gradient, lib


def _code(dt):
    code = _CODES.get(dt)
    if code is None:
        raise TypeError(f"unsupported dtype {dt}; use bfloat16 or float32")
    return code


def _row_stride(name, t):
    """Elements from one row (of the last axis) to the next; rows dense and at one stride."""
    if t.is_contiguous():
        return t.shape[-1]
    *lead, D = t.shape
    *steps, inner = t.stride()
    step = span = None
    good = inner == 1 or D <= 1
    for n, s in zip(reversed(lead), reversed(steps)):  # axes of one are skipped, others follow each other
        if n == 1:
            continue
        if step is None:
            step, span = s, n * s
        else:
            good, span = good and s == span, n * span
    step = D if step is None else step
    if not good or step < D or step % 8:
        raise ValueError(f"{name}: rows must be dense and at one stride, a multiple of 8 elements, "
                         f"got strides {t.stride()} for shape {tuple(t.shape)}")
    return step


def _like(name, t, shape, dtype, device):
    """The row stride of t, after a check of its shape, type and device."""
    if t.shape != shape or t.dtype != dtype or t.device != device:
        _bad(name, t, shape, dtype, device)
    return _row_stride(name, t)


def _no_second(backward):
    """once_differentiable, whose own bookkeeping is skipped where no graph of the gradients is asked
    for."""
    recorded = torch.autograd.function.once_differentiable(backward)

    @functools.wraps(backward)
    def run(ctx, *grads):
        return (recorded if torch.is_grad_enabled() else backward)(ctx, *grads)

    return run


# ---------------------------------------------------------------- diagonal recurrence

def _recurrence_args(v, g, w, cu_seqlens):
    _need_gpu(v)
    if v.dim() != 3:
        raise ValueError("v must be [B, T, D]")
    B, T, D = shape = v.shape
    dev, dt = v.device, v.dtype
    code = _code(dt)
    if D % 8 or not D:
        raise ValueError(f"{D} channels: a multiple of 8 is needed")
    strides = (_row_stride("v", v), _like("g", g, shape, dt, dev),
               0 if w is None else _like("w", w, shape, dt, dev))
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.device != dev or cu_seqlens.dim() != 1:
            raise ValueError("cu_seqlens must be a 1-D int32 tensor on the inputs' device")
        if not cu_seqlens.is_contiguous() or not cu_seqlens.numel():
            raise ValueError("cu_seqlens must be contiguous, [N + 1]")
        if B != 1:
            raise ValueError("packed (cu_seqlens) inputs must have B == 1")
        N = cu_seqlens.numel() - 1
    else:
        N = B
    return B, T, D, N, strides, code, dev, dt


@functools.lru_cache(maxsize=1024)
def _recurrence_sizes(backward, packed, B, T, D, N):
    """Workspace bytes of a call, and slots of its kept states."""
    L = lib()
    return (int(L.gdn2_linear_recurrence_workspace_bytes(backward, packed, B, T, D, N)),
            int(L.gdn2_linear_recurrence_states_bytes(packed, B, T, D, N)) // (4 * D))


def _recurrence(v, g, w, initial_state, cu_seqlens, output_final_state, keep):
    sizes = _recurrence_args(v, g, w, cu_seqlens)
    B, T, D, N, strides, code, dev, dt = sizes
    if initial_state is not None:
        _dense("initial_state", initial_state, (N, D), torch.float32, dev)
    o = _empty(v)
    last = torch.empty((N, D), dtype=torch.float32, device=dev) if output_final_state else None
    need, slots = _recurrence_sizes(False, cu_seqlens is not None, B, T, D, N)
    states = torch.empty((slots, D), dtype=torch.float32, device=dev) if keep else None
    ws = torch.empty(need // 4, dtype=torch.float32, device=dev) if need else None
    _call("gdn2_linear_recurrence", dev, v.data_ptr(), g.data_ptr(), _p(w), _p(initial_state),
          o.data_ptr(), _p(last), _p(states), _p(cu_seqlens), B, T, D, N, *strides, code, _p(ws), need)
    return o, last, states, sizes


def linear_recurrence_fwd(v, g, w=None, initial_state=None, cu_seqlens=None,
                          output_final_state=True):
    """The diagonal gated recurrence h_t = exp(g_t) h_{t-1} + w_t v_t over whole sequences, a state
    per channel; the output is h_t.

    v, g, w: [B, T, D] bf16 or fp32, D a multiple of 8 (slices of one projection are fine: a token's
    channels dense, tokens at one stride); g = log(alpha) <= 0; w: None for ones. initial_state:
    fp32 [N, D] or None. cu_seqlens: int32 [N + 1] (packed batch, B == 1; rows behind the last
    sequence are not written) or None (N = B). (Rows at a power of two of bytes meet on the same
    memory channels: where v, g, w are slices of one projection, 64 columns more than 3 D make a
    layer of 2048 channels 15% faster.)
    Returns (o [B, T, D], final_state [N, D] fp32 or None)."""
    return _recurrence(v, g, w, initial_state, cu_seqlens, output_final_state, False)[:2]


def linear_recurrence_fwd_train(v, g, w=None, initial_state=None, cu_seqlens=None,
                                output_final_state=True):
    """linear_recurrence_fwd for training: (o, final_state, states), the last for
    linear_recurrence_bwd (the fp32 state before every 64th token of every sequence). Rows that belong
    to no packed sequence are zeros."""
    return _recurrence(v, g, w, initial_state, cu_seqlens, output_final_state, True)[:3]


def linear_recurrence_bwd(v, g, w, states, do, d_final_state=None, cu_seqlens=None):
    """Gradients of linear_recurrence_fwd: (dv, dg, dw, d_initial_state), the first three dense in
    the inputs' type (dw None where w is), the last fp32 [N, D].

    states: from linear_recurrence_fwd_train on the same inputs. do: [B, T, D] contiguous;
    d_final_state: fp32 [N, D] or None. Rows that belong to no packed sequence get zeros."""
    sizes = _recurrence_args(v, g, w, cu_seqlens)
    B, T, D, N, strides, code, dev, dt = sizes
    _dense("do", do, (B, T, D), dt, dev)
    slots = _recurrence_sizes(True, cu_seqlens is not None, B, T, D, N)[1]
    _dense("states", states, (slots, D), torch.float32, dev)
    if d_final_state is not None:
        _dense("d_final_state", d_final_state, (N, D), torch.float32, dev)
    return _recurrence_bwd(v, g, w, states, do, d_final_state, cu_seqlens, sizes)


def _recurrence_bwd(v, g, w, states, do, d_final_state, cu_seqlens, sizes):
    """The call itself, of checked tensors."""
    B, T, D, N, strides, code, dev, dt = sizes
    need = _recurrence_sizes(True, cu_seqlens is not None, B, T, D, N)[0]
    dv, dg = torch.empty_like(do), torch.empty_like(do)
    dw = None if w is None else torch.empty_like(do)
    ds0 = states.new_empty((N, D))
    ws = states.new_empty(need // 4) if need else None
    _call("gdn2_linear_recurrence_bwd", dev, v.data_ptr(), g.data_ptr(), _p(w), states.data_ptr(),
          do.data_ptr(), _p(d_final_state), dv.data_ptr(), dg.data_ptr(), _p(dw), ds0.data_ptr(),
          _p(cu_seqlens), B, T, D, N, *strides, code, _p(ws), need)
    return dv, dg, dw, ds0


class _LinearRecurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, v, g, w, initial_state, cu_seqlens):
        o, last, states, ctx.sizes = _recurrence(v, g, w, initial_state, cu_seqlens, True, True)
        ctx.kept = states.shape
        ctx.set_materialize_grads(False)
        ctx.has_s0 = initial_state is not None
        ctx.save_for_backward(v, g, w, states, cu_seqlens)
        return o, last

    @staticmethod
    @_no_second
    def backward(ctx, do, d_last):
        v, g, w, states, cu = ctx.saved_tensors
        # Saved-tensor hooks may hand back another layout (slices come back dense), or anything: what does not
        # lie as the forward's own did goes through the checks from the start.
        B, T, D, N, strides, code, dev, dt = ctx.sizes
        shape, index = (B, T, D), dev.index
        same = (states.shape == ctx.kept and states.dtype is torch.float32 and states.is_contiguous() and
                states.get_device() == index)
        for t, step in zip((v, g, w), strides):
            if t is not None and (t.stride() != (T * step, step, 1) or t.shape != shape or t.dtype is not dt or
                                  t.get_device() != index):
                same = False
        if cu is not None and (cu.shape != (N + 1,) or cu.dtype is not torch.int32 or not cu.is_contiguous() or
                               cu.get_device() != index):
            same = False
        do = torch.zeros_like(v, memory_format=torch.contiguous_format) if do is None else _aligned_gradient(do)
        d_last = None if d_last is None else _aligned_gradient(d_last)
        if same:
            dv, dg, dw, ds0 = _recurrence_bwd(v, g, w, states, do, d_last, cu, ctx.sizes)
        else:
            dv, dg, dw, ds0 = linear_recurrence_bwd(v, g, w, states, do, d_last, cu)
        return dv, dg, dw, ds0 if ctx.has_s0 else None, None


def linear_recurrence(v, g, w=None, initial_state=None, cu_seqlens=None):
    """Differentiable linear_recurrence_fwd: (o, final_state); gradients flow to v, g, w and the
    initial state through the library's backward. Rows that belong to no packed sequence are zeros, and
    so are their gradients. (torch ties a leaf's accumulation to the stream of
    its first use: before a backward pass is captured into a graph, drop eager results of the same
    leaves that are still alive.)"""
    return _LinearRecurrence.apply(v, g, w, initial_state, cu_seqlens)


def linear_recurrence_tokens(v, g, w, state_pool, state_indices=None, commit_len=None,
                             return_step_states=False):
    """L consecutive tokens of every sequence of the diagonal recurrence against a pool of states
    (decode, or verification of draft tokens).

    v, g, w: [N, L, D] (w may be None), strides as for linear_recurrence_fwd; state_pool: [P, D]
    fp32, updated in place for the committed prefix; state_indices: int32 [N] (slot per sequence,
    one outside [0, P) skips it: its outputs are not written) or None (slot n); commit_len: int32
    [N], clamped to [0, L], or None (all L tokens). Two sequences must not share a slot.
    Returns (o [N, L, D], step_states [N, L, D] fp32 or None)."""
    _need_gpu(v)
    if v.dim() != 3:
        raise ValueError("v must be [N, L, D]")
    N, L, D = shape = v.shape
    dev, dt = v.device, v.dtype
    code = _code(dt)
    if D % 8 or not D:
        raise ValueError(f"{D} channels: a multiple of 8 is needed")
    vs, gs = _row_stride("v", v), _like("g", g, shape, dt, dev)
    ws = 0 if w is None else _like("w", w, shape, dt, dev)
    if state_pool.dim() != 2:
        raise ValueError("state_pool must be [P, D]")
    P = state_pool.shape[0]
    _dense("state_pool", state_pool, (P, D), torch.float32, dev)
    if state_indices is not None:
        _dense("state_indices", state_indices, (N,), torch.int32, dev)
    elif P < N:
        raise ValueError(f"{N} sequences without state_indices need as many states, got {P}")
    if commit_len is not None:
        _dense("commit_len", commit_len, (N,), torch.int32, dev)
    o = _empty(v)
    steps = torch.empty(shape, dtype=torch.float32, device=dev) if return_step_states else None
    _call("gdn2_linear_recurrence_tokens", dev, v.data_ptr(), g.data_ptr(), _p(w),
          state_pool.data_ptr(), _p(state_indices), _p(commit_len), o.data_ptr(), _p(steps), N, L,
          D, P, vs, gs, ws, code)
    return o, steps


# ---------------------------------------------------------------- norm between layers

_NORM_WIDTH = 16384


def _norm_args(x, residual, weight):
    _need_gpu(x)
    if x.dim() < 1:
        raise ValueError("x must be [..., D]")
    shape, dev, dt = x.shape, x.device, x.dtype
    D = shape[-1]
    code = _code(dt)
    if not D or D % 8 or D > _NORM_WIDTH:
        raise ValueError(f"{D} channels: a multiple of 8 up to {_NORM_WIDTH} is needed")
    xs, rs, rcode = _row_stride("x", x), 0, code
    if residual is not None:
        rcode = _code(residual.dtype)
        if code > rcode:
            raise TypeError(f"residual: {residual.dtype} is narrower than x's {dt}")
        rs = _like("residual", residual, shape, residual.dtype, dev)
    _dense("weight", weight, (D,), torch.float32, dev)
    return shape, D, x.numel() // D, xs, rs, code, rcode, dev, dt


def _norm(x, residual, weight, eps, group, out):
    shape, D, rows, xs, rs, code, rcode, dev, dt = _norm_args(x, residual, weight)
    scale = None
    if group is not None:
        if group not in (0, 32, 64, 128) or (group and D % group):
            raise ValueError(f"group: 0 (a scale for every row), 32, 64 or 128 dividing {D} channels, got {group}")
        scale = weight.new_empty(shape[:-1] + (D // (group or D),))
    if out is None:
        kind = dt if group is None else torch.float8_e4m3fn
        y = torch.empty_like(x, dtype=kind) if x.is_contiguous() else x.new_empty(shape, dtype=kind)
        h = x if residual is None else _empty(residual)
    else:
        y, h = out
        _dense("out[0]", y, shape, dt if group is None else torch.float8_e4m3fn, dev)
        if residual is None:
            if h is not None and h is not x:
                raise ValueError("out[1]: without a residual the stream is x itself")
            h = x
        else:
            _dense("out[1]", h, shape, residual.dtype, dev)
        if torch.is_grad_enabled() and (y.requires_grad or (residual is not None and h.requires_grad)):
            raise ValueError("out: the tensors require gradients, which would not know of this "
                             "call; use residual_norm, or no_grad")
    _call("gdn2_residual_norm", dev, x.data_ptr(), _p(residual), weight.data_ptr(), y.data_ptr(),
          None if residual is None else h.data_ptr(), _p(scale), rows, D, xs, rs, group or 0, eps,
          code, rcode)
    return y, scale, h


def residual_norm_fwd(x, residual, weight, eps=1e-6, out=None):
    """The norm between layers: h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight over the
    last axis.

    x: [..., D] bf16 or fp32, D a multiple of 8 up to 16384 (rows dense and at one stride);
    residual: like x, or fp32 where x is bf16 (the stream in more bits), or None: h = x; weight:
    fp32 [D]. h is rounded to the residual's type, and the norm is of h as it is stored. out:
    optional contiguous (y, h), written and returned; h may be residual itself (the stream in
    place); not tensors that require gradients, unless under no_grad.
    Returns (y [..., D] in x's type, h)."""
    y, _, h = _norm(x, residual, weight, eps, None, out)
    return y, h


def residual_norm_8bit(x, residual, weight, eps=1e-6, group=0, out=None):
    """residual_norm_fwd with y in 8 bits, for a projection that reads e4m3: the value of a code is
    code * scale, with one power-of-two scale (the smallest s >= 2^-64 with max|y| <= 448 s) for
    every group of 32, 64 or 128 channels, or for every row (group 0).

    out: optional contiguous (codes, h).
    Returns (codes [..., D] float8_e4m3fn, scale [..., D / group] fp32, h)."""
    return _norm(x, residual, weight, eps, group, out)


@functools.lru_cache(maxsize=1024)
def _norm_workspace(rows, D):
    return int(lib().gdn2_residual_norm_bwd_workspace_bytes(rows, D))


def residual_norm_bwd(dy, dh, h, weight, eps=1e-6):
    """Gradients of residual_norm_fwd for the gradients dy (contiguous, x's type) and dh (contiguous,
    h's type; None: zero) of its outputs, from h as it returned it: (dx, dresidual, dweight). dx and
    dresidual are the same values (one tensor where the types agree), dweight is fp32 [D]."""
    shape, _, _, _, _, hcode, _, dev, ht = _norm_args(h, None, weight)
    if _code(dy.dtype) > hcode:
        raise TypeError(f"dy: {dy.dtype} is wider than h's {ht}")
    _dense("dy", dy, shape, dy.dtype, dev)
    if dh is not None:
        _dense("dh", dh, shape, ht, dev)
    return _norm_bwd(dy, dh, h, weight, eps)


def _norm_bwd(dy, dh, h, weight, eps):
    """The call itself, of checked tensors."""
    D = weight.numel()
    rows, code, hcode = dy.numel() // D, _CODES[dy.dtype], _CODES[h.dtype]
    dx = torch.empty_like(dy)
    dr = dx if code == hcode else torch.empty_like(dy, dtype=h.dtype)
    dw = torch.empty_like(weight) if rows else torch.zeros_like(weight)
    need = _norm_workspace(rows, D)
    ws = weight.new_empty(need // 4)
    _call("gdn2_residual_norm_bwd", dy.device, dy.data_ptr(), _p(dh), h.data_ptr(),
          weight.data_ptr(), dx.data_ptr(), None if code == hcode else dr.data_ptr(),
          dw.data_ptr(), rows, D, _row_stride("h", h), eps, code, hcode, ws.data_ptr(), need)
    return dx, dr, dw


class _ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps):
        y, _, h = _norm(x, residual, weight, eps, None, None)
        ctx.set_materialize_grads(False)
        ctx.eps = eps
        ctx.save_for_backward(h, weight)
        ctx.dt, ctx.ht = x.dtype, h.dtype
        return y if residual is None else (y, h)

    @staticmethod
    @_no_second
    def backward(ctx, dy, dh=None):
        h, weight = ctx.saved_tensors
        # (as for the recurrence: what saved-tensor hooks have changed is checked from the start)
        out = dh if dy is None else dy  # of the forward's shape and device
        index = out.device.index
        same = (h.shape == out.shape and h.dtype is ctx.ht and h.get_device() == index and weight.dtype is torch.float32 and
                weight.shape == out.shape[-1:] and weight.is_contiguous() and weight.get_device() == index)
        dy = torch.zeros(h.shape, dtype=ctx.dt, device=h.device) if dy is None else _aligned_gradient(dy)
        dh = None if dh is None else _aligned_gradient(dh)
        dx, dr, dw = (_norm_bwd if same else residual_norm_bwd)(dy, dh, h, weight, ctx.eps)
        return dx, dr if ctx.needs_input_grad[1] else None, dw, None


def residual_norm(x, residual, weight, eps=1e-6):
    """Differentiable residual_norm_fwd: (y, h); gradients flow to x, the residual and the weight
    through the library's backward. (torch ties a leaf's accumulation to the stream of its first
    use: before a backward pass is captured into a graph, drop eager results of the same leaves that
    are still alive.)"""
    if residual is None:
        return _ResidualNorm.apply(x, None, weight, eps), x
    return _ResidualNorm.apply(x, residual, weight, eps)


# ---------------------------------------------------------------- verification of drafts

@functools.lru_cache(maxsize=1024)
def _verify_workspace(N, V):
    return int(lib().gdn2_verify_drafts_workspace_bytes(N, V))


def verify_drafts(target_probs, drafts, uniforms, draft_probs=None, draft_len=None, workspace=None):
    """Verification of drafted tokens against the target's probabilities, from given random numbers.

    target_probs: [N, L + 1, V] bf16 or fp32, in front of every draft and behind the last; drafts:
    int32 [N, L]; uniforms: fp32 [N, L + 1] in [0, 1), the last one for the drawn token;
    draft_probs: [N, L, V] like target_probs, or None for drafts that were certain (greedy or
    copied ones); draft_len: int32 [N], clamped to [0, L], or None (L drafts each). All contiguous.
    Draft i is accepted where uniforms[i] q_i(x_i) < p_i(x_i) and all before it were; the next token
    is drawn from max(p - q, 0) at the first draft that was not, or from p behind the last.
    workspace: optional uint8 device tensor of at least verify_drafts_workspace_bytes(N, V),
    allocated when None; calls that can overlap, captured ones among them, need one each.
    Returns (tokens int32 [N, L + 1]: the accepted drafts, the next token, -1 behind it; commit_len
    int32 [N]: how many of the L + 1 tokens that went through the target - the last known one, then
    the drafts - are to be committed, as decode_tokens and linear_recurrence_tokens take it)."""
    _need_gpu(target_probs)
    if target_probs.dim() != 3 or drafts.dim() != 2:
        raise ValueError("target_probs must be [N, L + 1, V] and drafts [N, L]")
    N, L = drafts.shape
    V = target_probs.shape[2]
    dev, dt = target_probs.device, target_probs.dtype
    code = _code(dt)
    if not 0 < V <= 1 << 28:
        raise ValueError(f"a vocabulary of 1 to 2^28 entries is needed, got {V}")
    _dense("target_probs", target_probs, (N, L + 1, V), dt, dev)
    _dense("drafts", drafts, (N, L), torch.int32, dev)
    _dense("uniforms", uniforms, (N, L + 1), torch.float32, dev)
    if draft_probs is not None:
        _dense("draft_probs", draft_probs, (N, L, V), dt, dev)
    if draft_len is not None:
        _dense("draft_len", draft_len, (N,), torch.int32, dev)
    need = _verify_workspace(N, V)
    if workspace is None:
        workspace = uniforms.new_empty(need // 4)
    elif workspace.device != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the inputs' device")
    else:
        need = workspace.numel()
    tokens = drafts.new_empty((N, L + 1))
    commit = drafts.new_empty(N)
    _call("gdn2_verify_drafts", dev, target_probs.data_ptr(), _p(draft_probs), drafts.data_ptr(),
          _p(draft_len), uniforms.data_ptr(), tokens.data_ptr(), commit.data_ptr(), N, L, V, code,
          workspace.data_ptr(), need)
    return tokens, commit


def verify_drafts_workspace_bytes(N, V):
    """Device workspace that verify_drafts needs for N sequences and a vocabulary of V."""
    return _verify_workspace(N, V)
