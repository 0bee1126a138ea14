"""Tolerances of the tests of what stands around the mixer. `U` is half a step of fp32; `half(dtype)`
the relative bound of one rounding to dtype."""
import numpy as np

from oracle import gdn2_stack as R
from tests.attn_util import U, half

TINY = 1e-38


def _swept(x, g, w_err, start, spans, reverse):
    """Majorants along time: m_t = alpha m_{t-1} + |x_t| and the error e_t = alpha e_{t-1} + w_err_t,
    from `start` (no error); as arrays like x, zero outside the spans, and their last values."""
    m_out, e_out = np.zeros(x.shape), np.zeros(x.shape)
    last = np.zeros((2, len(spans), x.shape[2]))
    for n, (b, i, j) in enumerate(spans):
        m, e = np.abs(start[n]), np.zeros(x.shape[2])
        for t in (range(j - 1, i - 1, -1) if reverse else range(i, j)):
            al = np.exp(g[b, t])
            if reverse:  # e_{t-1} = alpha_t (do_t + e_t): the value at t is what do_t meets
                m = m + np.abs(x[b, t])
                e = e + w_err * m * (1 + np.minimum(np.abs(g[b, t]), 100))
                m_out[b, t], e_out[b, t] = m, e
                m, e = al * m, al * e
            else:
                m = al * m + np.abs(x[b, t])
                e = al * e + w_err * m * (1 + np.minimum(np.abs(g[b, t]), 100))
                m_out[b, t], e_out[b, t] = m, e
        last[:, n] = m, e
    return m_out, e_out, last


# Roundings that a token meets on its way into the states behind it, of U each and of the state's
# majorant: the gate's product 1, its own decay 3 (the logarithm's product with log2 e, |g| U, counted
# apart; exp2 2 U) and 2 in the product and sum; then for every 2 tokens (a run in fp32; 4 in bf16) the
# run's decay, 3, and at most 3 levels of products and sums, 6, and for every wave in between (16 tokens or
# more) 2, so that the number of waves does not matter: 6 + 9 / 2 + 2 / 16 < 16.
STEP = 16 * U


def recurrence_bounds(v, g, w, s0, cu, dtype):
    """(o, bound of o, last, bound of last, majorants, errors)."""
    spans = R._spans(v, cu)
    start = np.zeros((len(spans), v.shape[2])) if s0 is None else s0
    o, last = R.recurrence(v, g, w, s0, cu)
    z = v if w is None else v * w
    m, e, (lm, le) = _swept(z, g, STEP, start, spans, False)
    return o, e + half(dtype) * np.abs(o) + TINY, last, le + U * np.abs(last) + TINY, m, e


def recurrence_grad_bounds(v, g, w, do, s0, ds, cu, dtype):
    """((dv, bound), (dg, bound), (dw, bound), (ds0, bound))."""
    spans = R._spans(v, cu)
    N, D = len(spans), v.shape[2]
    start = np.zeros((N, D)) if s0 is None else s0
    grads = R.recurrence_backward(v, g, w, do, s0, ds, cu)
    z = v if w is None else v * w
    mh, eh, _ = _swept(z, g, STEP, start, spans, False)
    md, ed, (lm, le) = _swept(do, g, STEP, np.zeros((N, D)) if ds is None else ds, spans, True)
    # the state before every token
    mb, eb = np.zeros(v.shape), np.zeros(v.shape)
    for n, (b, i, j) in enumerate(spans):
        if j > i:
            mb[b, i], mb[b, i + 1:j], eb[b, i + 1:j] = np.abs(start[n]), mh[b, i:j - 1], eh[b, i:j - 1]
    al = np.exp(g)
    hb = half(dtype)
    wt = 1.0 if w is None else np.abs(w)
    out = [(grads[0], ed * wt + U * md * wt + hb * np.abs(grads[0]) + TINY),
           (grads[1], al * (ed * mb + md * eb + (4 + np.minimum(np.abs(g), 100)) * U * md * mb) + hb * np.abs(grads[1]) + TINY)]
    if w is not None:
        out.append((grads[2], ed * np.abs(v) + U * md * np.abs(v) + hb * np.abs(grads[2]) + TINY))
    return out + [(grads[3], le + U * np.abs(grads[3]) + TINY)]


def norm_bound(h, weight, eps, dtype):
    """y and its bound. The mean square: a lane's sum of at most 64 squares, 6 exchanges, 3 waves, the
    division: 75 U at most, half of it in the root; the root 2 U, two products: 42 U, one rounding."""
    y = R.norm(h, weight, eps)
    return y, 42 * U * np.abs(y) + half(dtype) * np.abs(y) + TINY


def norm_grad_bounds(dy, dh, h, weight, eps, dtype, htype):
    """(dh_total, bound in dtype, bound in htype, dweight, bound). rho 40 U; the sum u h 76 U of its
    absolute terms, three products behind it: 240 U of |rho^3 h| mean|u h|, 45 U of |rho u|; the weight's
    terms 42 U each, their sum over rows at most U for every row and partial sum of them."""
    dx, dw = R.norm_backward(dy, dh, h, weight, eps)
    D = h.shape[-1]
    rho = 1 / np.sqrt(np.mean(h * h, -1, keepdims=True) + eps)
    u = np.abs(dy * weight)
    size = 45 * rho * u + 240 * rho ** 3 * np.abs(h) * np.mean(u * np.abs(h), -1, keepdims=True)
    size = U * (size + np.abs(dx))
    terms = np.abs(dy * h * rho).reshape(-1, D)
    return (dx, size + half(dtype) * np.abs(dx) + TINY, size + half(htype) * np.abs(dx) + TINY, dw,
            (42 + min(len(terms), 4096) + 64) * U * terms.sum(0) + U * np.abs(dw) + TINY)
