"""Pins of the float64 oracle of what stands around the mixer: the recurrence against the mixer's own
oracle and against a closed form, gradients against differences, the verification against counting
every draw of small distributions."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import gdn2_forward
from oracle import gdn2_stack as R


def _rec(seed, B=2, T=9, D=5, N=None):
    r = np.random.default_rng(seed)
    v, g, w = r.standard_normal((B, T, D)), -np.abs(r.standard_normal((B, T, D))), r.random((B, T, D))
    return v, g, w, r.standard_normal((N or B, D)), r


def test_recurrence_is_the_mixer_with_one_key_channel():
    """One key channel, k = q = 1, no erase: the mixer's state row is the recurrence's."""
    v, g, w, s0, _ = _rec(1)
    for c in range(v.shape[2]):
        one = np.ones(v.shape[:2] + (1, 1))
        o, s = gdn2_forward(one, one, v[..., None, c:c + 1], g[..., None, c:c + 1], 0 * one, w[..., None, c:c + 1],
                            s0=s0[:, None, None, c:c + 1])
        ref, last = R.recurrence(v, g, w, s0)
        assert np.allclose(o[:, :, 0, 0], ref[..., c], atol=1e-13) and np.allclose(s[:, 0, 0, 0], last[:, c], atol=1e-13)


def test_recurrence_closed_form_and_packed():
    v, g, w, s0, r = _rec(2, B=1, T=12, N=4)
    cu = np.array([0, 5, 5, 6, 12])
    o, last = R.recurrence(v, g, w, s0, cu)
    for n, (i, j) in enumerate(zip(cu, cu[1:])):
        for t in range(i, j):
            G = np.array([g[0, s + 1:t + 1].sum(0) for s in range(i, t + 1)])
            ref = np.exp(g[0, i:t + 1].sum(0)) * s0[n] + (np.exp(G) * w[0, i:t + 1] * v[0, i:t + 1]).sum(0)
            assert np.allclose(o[0, t], ref, atol=1e-13)
    assert np.array_equal(last[1], s0[1])


def test_recurrence_tokens_are_the_forward():
    v, g, w, _, r = _rec(3, B=4, T=3)
    pool = r.standard_normal((6, 5))
    idx, commit = np.array([5, -1, 2, 0]), np.array([3, 1, 0, 2])
    o, states, after = R.recurrence_tokens(pool, v, g, w, idx, commit)
    ref = R.recurrence(v[[0, 2, 3]], g[[0, 2, 3]], w[[0, 2, 3]], pool[[5, 2, 0]])[0]
    assert np.allclose(o[[0, 2, 3]], ref) and np.isnan(o[1]).all()
    assert np.allclose(after[5], ref[0, 2]) and np.array_equal(after[2], pool[2]) and np.allclose(after[0], ref[2, 1])
    assert np.array_equal(after[[1, 3, 4]], pool[[1, 3, 4]])


@pytest.mark.parametrize("gate", [True, False])
def test_recurrence_gradient_equals_differences(gate):
    v, g, w, s0, r = _rec(4, B=1, T=7, D=2, N=3)
    cu = np.array([0, 3, 3, 6])  # the last row belongs to no sequence
    do, ds = r.standard_normal(v.shape), r.standard_normal(s0.shape)

    def loss(v, g, w, s0):
        o, last = R.recurrence(v, g, w if gate else None, s0, cu)
        return np.nansum(o * do) + np.sum(last * ds)

    grads = R.recurrence_backward(v, g, w if gate else None, do, s0, ds, cu)
    args = [v, g, w, s0]
    for k in range(4):
        if grads[k] is None:
            assert k == 2 and not gate
            continue
        for at in np.ndindex(args[k].shape):
            e = np.zeros_like(args[k])
            e[at] = 1e-6
            up, down = (loss(*(a + s * e if i == k else a for i, a in enumerate(args))) for s in (1, -1))
            assert abs((up - down) / 2e-6 - grads[k][at]) < 1e-7


def test_norm_gradient_equals_differences():
    r = np.random.default_rng(5)
    h, w, dy, dh = r.standard_normal((3, 8)), 1 + r.standard_normal(8), r.standard_normal((3, 8)), r.standard_normal((3, 8))

    def loss(h, w):
        return np.sum(R.norm(h, w, 1e-3) * dy) + np.sum(h * dh)

    gh, gw = R.norm_backward(dy, dh, h, w, 1e-3)
    for x, g, other in ((h, gh, False), (w, gw, True)):
        for at in np.ndindex(x.shape):
            e = np.zeros_like(x)
            e[at] = 1e-6
            d = (loss(h, w + e) - loss(h, w - e)) if other else (loss(h + e, w) - loss(h - e, w))
            assert abs(d / 2e-6 - g[at]) < 1e-7


def test_norm_8bit_groups():
    r = np.random.default_rng(6)
    h, w = r.standard_normal((4, 64)) * np.exp(3 * r.standard_normal((4, 1))), 1 + 0.1 * r.standard_normal(64)
    for group in (0, 32):
        codes, scale, y = R.norm_8bit(h, w, 1e-6, group)
        parts = np.abs(y).reshape(4, -1, group or 64).max(-1)
        assert np.array_equal(np.log2(scale), np.floor(np.log2(scale)))
        assert (parts <= 448 * scale).all() and (parts > 224 * scale).all()
        held = codes.reshape(4, -1, group or 64) * scale[..., None]
        assert np.all(np.abs(held.reshape(4, 64) - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * np.repeat(scale, group or 64, -1)))


def _emitted(p, q, certain, steps):
    """Distribution of the first emitted token over a grid of draws: the draft from q, u_0 for its
    acceptance, u_1 for the token, all on `steps` equal cells."""
    V = len(p)
    out = [Fraction(0)] * V
    u = (np.arange(steps) + 0.5) / steps
    for x in range(V):
        if q[x] == 0:
            continue
        drafts = np.full((steps * steps, 1), x, np.int32)
        grid = np.stack(np.meshgrid(u, u, indexing="ij"), -1).reshape(-1, 2).astype(np.float32)
        P = np.repeat(np.stack([p, p])[None], steps * steps, 0)
        Q = None if certain else np.repeat(q[None, None], steps * steps, 0)
        tokens, _ = R.verify(P, drafts, grid, Q)
        for t in range(V):
            out[t] += Fraction(int((tokens[:, 0] == t).sum()), steps * steps) * Fraction(float(q[x]))
    return [float(f) for f in out]


def test_verification_keeps_the_targets_distribution():
    """Whatever the draft's distribution is, the first emitted token follows the target's; for
    probabilities on the grid's cells the count is exact."""
    p = np.array([0.25, 0.5, 0.125, 0.125])
    for q in ([0.5, 0.25, 0.25, 0.0], [0.25, 0.25, 0.25, 0.25], [0.125, 0.125, 0.25, 0.5], [0.25, 0.5, 0.125, 0.125]):
        assert np.allclose(_emitted(p, np.array(q), False, 48), p, atol=1e-12), q
    for x, steps in ((0, 48), (1, 48), (2, 56), (3, 56)):  # certain drafts: what is left has 6ths or 7ths
        assert np.allclose(_emitted(p, np.eye(4)[x], True, steps), p, atol=1e-12), x


def test_verification_edges():
    p = np.array([[[0.5, 0.5, 0], [0, 0, 1], [0, 0, 0]]])
    u = np.array([[0.4, 0.999, 0.0]], np.float32)
    tokens, commit = R.verify(p, np.array([[1, 2]]), u)
    assert tokens.tolist() == [[1, 2, -1]] and commit.tolist() == [3]          # both accepted, an empty row behind
    tokens, commit = R.verify(p, np.array([[2, 2]]), u)
    assert tokens.tolist() == [[0, -1, -1]] and commit.tolist() == [1]         # p(x) = 0: rejected
    tokens, commit = R.verify(p, np.array([[7, 2]]), u)
    assert tokens.tolist() == [[0, -1, -1]] and commit.tolist() == [1]         # no such token
    tokens, _ = R.verify(p, np.array([[1, 0]]), u, draft_len=np.array([1]))
    assert tokens.tolist() == [[1, 2, -1]]
    q = p[:, :2].copy()
    tokens, _ = R.verify(p, np.array([[2, 2]]), u, q)                           # q(x) = 0, p(x) = 0: rejected, nothing left: p
    assert tokens.tolist() == [[0, -1, -1]]
