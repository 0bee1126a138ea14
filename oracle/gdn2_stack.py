"""Float64 oracle of what stands around the mixer in a stack: the diagonal gated recurrence (forward,
backward, tokens against a pool), the norm between layers (forward, backward, 8-bit output) and the
verification of drafted tokens. Token by token, entry by entry; plain numpy."""
import numpy as np

from .gdn2_attn import block_scale, round_e4m3


# ---- diagonal recurrence: h_t = exp(g_t) h_{t-1} + w_t v_t

def recurrence(v, g, w=None, s0=None, cu=None):
    """v, g, w: [B, T, D]; s0: [N, D]. Returns (o, final [N, D]); rows outside cu stay NaN."""
    o = np.full(v.shape, np.nan)
    spans = _spans(v, cu)
    last = np.zeros((len(spans), v.shape[2]))
    for n, (b, i, j) in enumerate(spans):
        h = np.zeros(v.shape[2]) if s0 is None else s0[n].astype(np.float64)
        for t in range(i, j):
            h = np.exp(g[b, t]) * h + (1.0 if w is None else w[b, t]) * v[b, t]
            o[b, t] = h
        last[n] = h
    return o, last


def recurrence_backward(v, g, w, do, s0=None, d_last=None, cu=None):
    """(dv, dg, dw, ds0) by the reverse of every step; rows outside cu get zeros."""
    spans = _spans(v, cu)
    dv, dg, dw = (np.zeros(v.shape) for _ in range(3))
    ds0 = np.zeros((len(spans), v.shape[2]))
    for n, (b, i, j) in enumerate(spans):
        h = [np.zeros(v.shape[2]) if s0 is None else s0[n].astype(np.float64)]
        for t in range(i, j):
            h.append(np.exp(g[b, t]) * h[-1] + (1.0 if w is None else w[b, t]) * v[b, t])
        e = np.zeros(v.shape[2]) if d_last is None else d_last[n].astype(np.float64)
        for t in range(j - 1, i - 1, -1):
            d = do[b, t] + e
            dv[b, t] = d if w is None else d * w[b, t]
            dw[b, t] = d * v[b, t]
            e = d * np.exp(g[b, t])
            dg[b, t] = e * h[t - i]
        ds0[n] = e
    return dv, dg, None if w is None else dw, ds0


def recurrence_tokens(pool, v, g, w=None, indices=None, commit=None):
    """(o [N, L, D], states [N, L, D], pool after); skipped sequences stay NaN."""
    N, L, _ = v.shape
    o = np.full(v.shape, np.nan)
    pool = pool.astype(np.float64).copy()
    for n in range(N):
        slot = n if indices is None else int(indices[n])
        if not 0 <= slot < len(pool):
            continue
        h = pool[slot].copy()
        keep = L if commit is None else min(max(int(commit[n]), 0), L)
        for t in range(L):
            h = np.exp(g[n, t]) * h + (1.0 if w is None else w[n, t]) * v[n, t]
            o[n, t] = h
            if t + 1 == keep:
                pool[slot] = h
    return o, o.copy(), pool


def _spans(v, cu):
    if cu is None:
        return [(b, 0, v.shape[1]) for b in range(v.shape[0])]
    return [(0, int(i), int(j)) for i, j in zip(cu[:-1], cu[1:])]


# ---- norm between layers: y = h / sqrt(mean(h^2) + eps) * weight, of the stored h

def norm(h, weight, eps):
    return h / np.sqrt(np.mean(h * h, -1, keepdims=True) + eps) * weight


def norm_backward(dy, dh, h, weight, eps):
    """(gradient of h, gradient of the weight), from the Jacobian of every row."""
    D = h.shape[-1]
    rho = 1 / np.sqrt(np.mean(h * h, -1, keepdims=True) + eps)
    u = dy * weight
    dx = rho * u - rho ** 3 / D * h * np.sum(u * h, -1, keepdims=True)
    return dx + (0 if dh is None else dh), (dy * h * rho).reshape(-1, D).sum(0)


def norm_8bit(h, weight, eps, group):
    """(codes, scale [..., D / group], y)."""
    y = norm(h, weight, eps)
    parts = y.reshape(*y.shape[:-1], -1, group or y.shape[-1])
    with np.errstate(invalid="ignore"):
        big = np.abs(parts).max(-1)
        scale = np.vectorize(lambda a: block_scale(a) if a > 0 else 2.0 ** -64)(big)
        codes = round_e4m3(parts / scale[..., None]).reshape(y.shape)
    return codes, scale, y


# ---- verification of drafts

def verify(p, drafts, u, q=None, draft_len=None):
    """(tokens [N, L + 1], commit [N]). p [N, L + 1, V], q [N, L, V] in float64."""
    p = np.where(p > 0, p, 0.0)
    q = None if q is None else np.where(q > 0, q, 0.0)
    N, L = drafts.shape
    V = p.shape[2]
    tokens = np.full((N, L + 1), -1, np.int32)
    commit = np.zeros(N, np.int32)
    for n in range(N):
        length = L if draft_len is None else min(max(int(draft_len[n]), 0), L)
        a = 0
        while a < length:
            x = int(drafts[n, a])
            if not 0 <= x < V or not float(u[n, a]) * (1.0 if q is None else q[n, a, x]) < p[n, a, x]:
                break
            tokens[n, a] = x
            a += 1
        weight = p[n, a].copy()
        if a < length:
            if q is not None:
                weight = np.maximum(weight - q[n, a], 0)
            elif 0 <= drafts[n, a] < V:
                weight[drafts[n, a]] = 0
        if not weight.any():
            weight = p[n, a]
        c = np.cumsum(weight)
        past = np.flatnonzero((c > float(u[n, L]) * c[-1]) & (weight > 0))
        some = np.flatnonzero(weight)
        tokens[n, a] = past[0] if len(past) else some[-1] if len(some) else -1
        commit[n] = a + 1
    return tokens, commit
