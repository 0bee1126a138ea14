"""Pins of the attention layer's float64 oracle: the gradient against differences, the rotation
against complex numbers, the e4m3 rounding and the block scale against their definitions, the
cache against a one-call append, attention against a loop."""
import itertools

import numpy as np
import pytest
import torch

from oracle import gdn2_attn as R
from tests.attn_util import Paged, draw, f64, few_rows_ref


def _rows(seed, T=3, H=2, d=16):
    rng = np.random.default_rng(seed)
    return rng.standard_normal((T, H, d)), 1 + 0.3 * rng.standard_normal(d), rng.integers(-50, 50, T), rng


@pytest.mark.parametrize("il,norm,rot", [(False, True, 16), (True, True, 8), (False, False, 8), (True, True, 0)])
def test_gradient_equals_differences(il, norm, rot):
    x, w, pos, rng = _rows(1)
    fr = 100.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    dy = rng.standard_normal(x.shape)
    dx, dw = R.norm_rope_backward(x, dy, w, pos, fr, 1e-3, il, norm)

    def loss(x, w):
        return np.sum(R.norm_rope(x, w, pos, fr, 1e-3, il, norm) * dy)

    h = 1e-6
    for at in itertools.product(range(3), range(2), range(16)):
        e = np.zeros_like(x)
        e[at] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[at]) < 1e-7
    for c in range(16):
        e = np.zeros_like(w)
        e[c] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[c]) < 1e-7


@pytest.mark.parametrize("il", [False, True])
def test_rotation_is_a_complex_product(il):
    x, _, pos, _ = _rows(2)
    fr = 10.0 ** -np.arange(4.0)
    y = R.rotate(x, pos, fr, il)
    for t, h, i in itertools.product(range(3), range(2), range(4)):
        a, b = (2 * i, 2 * i + 1) if il else (i, i + 4)
        z = (x[t, h, a] + 1j * x[t, h, b]) * np.exp(1j * pos[t] * fr[i])
        assert abs(y[t, h, a] + 1j * y[t, h, b] - z) < 1e-12
    assert np.array_equal(y[..., 8:], x[..., 8:])
    assert np.allclose(R.rotate(y, pos, fr, il, back=True), x, atol=1e-13)


def test_norm_of_a_row():
    x, w, _, _ = _rows(3)
    n = R.norm_rope(x, None, np.zeros(3), np.zeros(0), eps=0.0)
    assert np.allclose(np.mean(n * n, -1), 1)
    assert np.allclose(R.norm_rope(x, w, np.zeros(3), np.zeros(0), 0.0), n * w)


def _all_e4m3():
    vals = []
    for e, m in itertools.product(range(16), range(8)):
        if (e, m) != (15, 7):
            vals.append(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(sorted(vals))


def test_e4m3_rounding_is_nearest_even():
    vals = _all_e4m3()
    assert vals[-1] == 448 and np.array_equal(R.round_e4m3(vals), vals)
    rng = np.random.default_rng(4)
    x = np.concatenate([rng.uniform(0, 448, 500), np.exp(rng.uniform(-8, 6, 500)), (vals[1:] + vals[:-1]) / 2])
    for v in x:
        y = R.round_e4m3(v)
        gap = np.abs(vals - v)
        assert abs(y - v) == gap.min() and y in vals
        near = np.flatnonzero(gap == gap.min())
        if len(near) == 2:  # a tie goes to the even code
            assert near[np.flatnonzero(vals[near] == y)[0]] % 2 == 0
        assert R.round_e4m3(-v) == -y


def test_block_scale_is_the_smallest():
    for a in (0.0, 1e-30, 1.0, 447.9, 448.0, 448.1, 896.0, 1e30):
        s = R.block_scale(a)
        assert np.log2(s) == round(np.log2(s)) and a <= 448 * s
        assert s == 2.0 ** -64 or a > 448 * s / 2


def test_append_piecewise_equals_at_once_where_scales_stay():
    """Tokens appended one by one hold what one call holds, once the largest comes first; a
    growing scale rescales the older codes."""
    rng = np.random.default_rng(5)
    k, v = rng.standard_normal((100, 2, 8)), rng.standard_normal((100, 2, 8))
    for b in (0, 64):
        k[b], v[b] = 10.0, -10.0
    whole, parts = R.Cache(3, 2, 8), R.Cache(3, 2, 8)
    row = [2, 0]
    R.append(whole, row, 100, k, v)
    for t in range(100):
        R.append(parts, row, t + 1, k[t:t + 1], v[t:t + 1])
    for a, b in zip((whole.k, whole.v, whole.k_scale, whole.v_scale), (parts.k, parts.v, parts.k_scale, parts.v_scale)):
        assert np.array_equal(a, b)
    held = (parts.k * parts.k_scale[..., None, None])[2, 0, :64]
    assert np.abs(held - k[:64, 0]).max() <= 10 * 2 ** -4
    R.append(parts, row, 101, np.full((1, 2, 8), 1000.0), v[:1])
    grown = (parts.k * parts.k_scale[..., None, None])[0, 0, :36]
    assert parts.k_scale[0, 0] > whole.k_scale[0, 0]
    assert np.abs(grown - k[64:100, 0]).max() <= 10 * 2 ** -4 + parts.k_scale[0, 0] * 2 ** -9


def test_append_clears_values_behind_the_largest_scale():
    """What lies behind the new tokens stays, whatever the scales do, except for values whose scale
    grows to 2^120."""
    c = R.Cache(1, 1, 8)
    one = lambda x: np.full((1, 1, 8), x)
    R.append(c, [0], 5, np.ones((5, 1, 8)), np.ones((5, 1, 8)))
    R.append(c, [0], 3, one(1.0), one(1e4))
    held = c.v[0, 0] * c.v_scale[0, 0]
    assert (held[:2] == 1).all() and (np.abs(held[2] - 1e4) <= 1e4 / 16).all() and (c.v[0, 0, 3:5] > 0).all()
    R.append(c, [0], 3, one(1.0), one(448 * 2.0 ** 119))
    assert c.v_scale[0, 0] == 2.0 ** 119 and (c.v[0, 0, 3:5] > 0).all()
    R.append(c, [0], 3, one(1.0), one(240 * 2.0 ** 120))
    assert c.v_scale[0, 0] == 2.0 ** 120 and (c.v[0, 0, 2] == 240).all() and not c.v[0, 0, 3:].any()
    assert (c.k[0, 0, 3:5] > 0).all()


def test_attention_equals_a_loop():
    rng = np.random.default_rng(6)
    c = R.Cache(4, 2, 8)
    c.k[:], c.v[:] = rng.standard_normal(c.k.shape), rng.standard_normal(c.v.shape)
    c.k_scale[:], c.v_scale[:] = 0.5, 2.0
    row, total, q = [3, 1, 0], 150, rng.standard_normal((5, 6, 8))
    for window in (0, 1, 70):
        o, _ = R.attention(q, c, row, total, window, 0.3)
        for i, h in itertools.product(range(5), range(6)):
            p = total - 5 + i
            keys = [j for j in range(total) if j <= p and (not window or j > p - window)]
            kk = np.array([c.k[row[j // 64], h // 3, j % 64] * 0.5 for j in keys])
            vv = np.array([c.v[row[j // 64], h // 3, j % 64] * 2.0 for j in keys])
            w = np.exp(kk @ q[i, h] * 0.3)
            assert np.allclose(o[i, h], w @ vv / w.sum(), atol=1e-12)
    o, _ = R.attention(q, c, [-1, 9, 77], total)
    assert not o.any()
    o, _ = R.attention(q, c, row, 3)  # two rows of padding
    assert not o[:2].any() and o[2:].any()


def test_attention_over_missing_blocks_is_that_over_the_rest():
    """Whatever the pool holds elsewhere."""
    rng = np.random.default_rng(7)
    c = R.Cache(4, 1, 8)
    c.k[:], c.v[:] = rng.standard_normal(c.k.shape), rng.standard_normal(c.v.shape)
    c.k_scale[:], c.v_scale[:] = 1.0, 1.0
    for x in (c.k, c.v, c.k_scale, c.v_scale):
        x[0] = np.nan
    q = rng.standard_normal((2, 3, 8))
    o, spread = R.attention(q, c, [3, -1, 1], 150)
    for i in range(2):
        keys = [j for j in range(149 + i) if j // 64 != 1]
        kk, vv = (np.array([x[[3, -1, 1][j // 64], 0, j % 64] for j in keys]) for x in (c.k, c.v))
        for h in range(3):
            w = np.exp(kk @ q[i, h] * 8 ** -0.5)
            assert np.allclose(o[i, h], w @ vv / w.sum(), atol=1e-12)
    assert np.isfinite(spread).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,L,window", [(4, 1, 0), (3, 5, 70), (8, 4, 0)])
def test_few_rows_bound_tells_one_rounding_of_the_weights_from_two_terms(G, L, window, d):
    """The bound that the few-row kernel is held to takes weights as two bf16 terms and rejects
    weights rounded once."""
    rng = np.random.default_rng(G * 7 + L + d + window)
    lens = [L, 64, 65, 127 + L, 449]
    paged = Paged(rng, lens, 2, d, device="cpu")
    paged.fill(rng, spread=0.3)
    q = f64(draw(rng, len(lens), L, 2 * G, d))
    bf = lambda x: torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    ref, bound = few_rows_ref(q, paged, lens, L, window)
    for n, total in enumerate(lens):
        assert np.allclose(R.attention(q[n], paged.ref, paged.table[n], total, window)[0], ref[n], atol=1e-12)
    two, _ = few_rows_ref(q, paged, lens, L, window, lambda w: bf(w) + bf(w - bf(w)))
    assert (np.abs(bf(two) - ref) <= bound).all()
    one, _ = few_rows_ref(q, paged, lens, L, window, bf)
    assert (np.abs(bf(one) - ref) > 3 * bound).any()
