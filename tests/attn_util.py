"""Inputs, transfer and tolerances of the attention-layer tests. `U` is half a step of fp32;
`half(dtype)` the relative bound of one rounding to dtype."""
import numpy as np
import torch

from oracle import gdn2_attn as R

U = 2.0 ** -24
B64 = R.BLOCK


def half(dtype):
    return torch.finfo(dtype).eps / 2


def inv_freq(rot):
    return (10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32)


def draw(rng, *shape, dtype=torch.bfloat16, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(dtype)


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def assert_within(name, got, ref, bound):
    """|got - ref| <= bound elementwise; NaN where the reference is NaN and nowhere else."""
    got, ref = f64(got) if isinstance(got, torch.Tensor) else got, np.asarray(ref)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{name}: NaN in other places"
    off = np.nan_to_num(np.abs(got - ref)) - np.nan_to_num(np.broadcast_to(bound, ref.shape))
    at = np.unravel_index(np.argmax(off), off.shape) if off.size else None
    assert not off.size or off.max() <= 0, (
        f"{name}: at {at} got {got[at]!r} for {ref[at]!r}, bound {np.broadcast_to(bound, ref.shape)[at]!r}")


def rows_bound(x, w, positions, freq, dtype, eps, interleaved, norm):
    """Bound of a normed and rotated row. fp32: the mean square 12 U (7 additions a lane, 4
    exchanges, 1 product; its root halves it), root and division 2 U, products with the root and
    the weight 2 U, cosine and sine 4 U, the two-term rotation 2 U: 16 U of |a| + |b|, which a
    rotation by absolute values bounds; then one rounding."""
    y = R.norm_rope(x, w, positions, freq, eps, interleaved, norm)
    n = np.abs(R.norm_rope(x, w, positions, freq[:0], eps, interleaved, norm))
    rot = 2 * len(freq)
    a, b = R._split(n, rot, interleaved)
    size = R._join(n, a + b, a + b, rot, interleaved)
    return y, 16 * U * size + half(dtype) * np.abs(y) + 1e-38


class Paged:
    """A cache on the device and its oracle twin, with a table of shuffled blocks."""

    def __init__(self, rng, lens, Hk, d, spare=2, table_width=None, device="cuda"):
        import gated_delta_rule_36_amd as G
        self.Hk, self.d, self.device = Hk, d, device
        need = [-(-int(n) // B64) for n in lens]
        self.P = sum(need) + spare
        order = rng.permutation(self.P)
        width = table_width or max(need + [1])
        self.table = np.full((len(lens), width), -1, np.int32)
        at = 0
        for i, n in enumerate(need):
            m = min(n, width)
            self.table[i, :m] = order[at:at + m]
            at += n
        self.ref = R.Cache(self.P, Hk, d)
        self.dev = G.kv_cache(self.P, Hk, d, device=device)
        self.cols = G.value_columns("cpu").numpy()

    def table_t(self):
        return torch.from_numpy(self.table).to(self.device)

    def fill(self, rng, spread=1.0):
        """Random codes and scales in every block, the same on both sides."""
        for held, scale in ((self.ref.k, self.ref.k_scale), (self.ref.v, self.ref.v_scale)):
            x = rng.standard_normal(held.shape) * np.exp(spread * rng.standard_normal(scale.shape))[..., None, None]
            scale[:] = np.vectorize(R.block_scale)(np.abs(x).max((2, 3)))
            held[:] = R.round_e4m3(x / scale[..., None, None])
        self.push()

    def push(self):
        """The oracle's cache to the device."""
        k = torch.from_numpy(self.ref.k).float().to(torch.float8_e4m3fn)
        v = np.empty((self.P, self.Hk, self.d, B64))
        v[..., self.cols] = self.ref.v.transpose(0, 1, 3, 2)
        v = torch.from_numpy(v).float().to(torch.float8_e4m3fn)
        self.dev.k.view(torch.uint8).copy_(k.view(torch.uint8))
        self.dev.v.view(torch.uint8).copy_(v.view(torch.uint8))
        self.dev.k_scale.copy_(torch.from_numpy(self.ref.k_scale))
        self.dev.v_scale.copy_(torch.from_numpy(self.ref.v_scale))

    def pull(self):
        """The device's cache in the oracle's layout: k, v codes, k_scale, v_scale."""
        k, v = f64(self.dev.k.float()), f64(self.dev.v.float())
        return k, v[..., self.cols].transpose(0, 1, 3, 2), f64(self.dev.k_scale), f64(self.dev.v_scale)


def attention_ref(q, paged, lens, spans, window=0, scale=None, few=False):
    """Oracle and bound for packed rows q [tokens, Hq, d] (float64), spans = [(first, count)].

    Scores: exact bf16 products summed in fp32, at most d U sum|q k| scale; exp2 of a
    difference 4 U more and 2 U of the scores' size for the scaled operands; weights thus off by
    at most e = 2 (d U A + 4 U + 2 U A) with A = max sum|q k| scale, relative to p and to their
    sum alike. The weight's rounding: half a step of bf16, or its square where the weight goes as
    two terms (few rows). Output sums: 2 U per key of the longest run in one accumulator, here
    taken as 64 U + U sqrt(keys). Then one rounding of the output."""
    n, Hq, d = q.shape
    o, bound = np.zeros(q.shape), np.zeros(q.shape)
    sc = d ** -0.5 if scale is None else scale
    P = paged.P
    for i, (first, count) in enumerate(spans):
        if count == 0:
            continue
        rows = q[first:first + count]
        total = int(lens[i])
        o_i, spread = R.attention(rows, paged.ref, paged.table[i], total, window, scale)
        kmax = np.nanmax(np.abs(paged.ref.k) * paged.ref.k_scale[..., None, None], initial=0.0)
        A = np.abs(rows).sum(-1, keepdims=True) * kmax * sc
        e = 2 * (d * U * A + 4 * U + 2 * U * A)
        hb = half(torch.bfloat16)
        w = hb * hb if few else hb
        o[first:first + count] = o_i
        bound[first:first + count] = (e + w + 64 * U + U * max(total, 1) ** 0.5) * spread + hb * np.abs(o_i) + 1e-38
    return o, bound


def half_step(x, dtype):
    """Half the distance of dtype's values around |x|."""
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(x), torch.finfo(dtype).tiny)))) * torch.finfo(dtype).eps
    return step / 2


def few_rows_ref(q, paged, lens, L, window=0, round_weights=None):
    """Rows q [N, L, Hq, d] (float64) over blocks that all exist, and a bound near the output's own
    rounding, for kernels whose weights keep more bits than the output's type. As in attention_ref
    the weights are off by at most e = 2 (d U A + 4 U + 2 U A) and the sums by 64 U + U sqrt(keys),
    and the square of bf16's half step for a weight as two terms, but A is the largest sum|q k| scale
    of a key that the row sees, and the output's rounding the half step around its own value. round_weights: applied to the weights (relative to the row's
    largest) of the product, their sum staying as it is."""
    N, _, Hq, d = q.shape
    G = Hq // paged.Hk
    o, bound = np.zeros(q.shape), np.zeros(q.shape)
    for n in range(N):
        total = int(lens[n])
        slots = paged.table[n, : -(-total // B64)]
        for i in range(L):
            p = total - L + i
            low = max(0, p + 1 - window) if window else 0
            if p < 0:
                continue
            for h in range(Hq):
                k, v = ((x[slots, h // G] * s[slots, h // G][:, None, None]).reshape(-1, d)[low:p + 1] for x, s in
                        ((paged.ref.k, paged.ref.k_scale), (paged.ref.v, paged.ref.v_scale)))
                x = k @ q[n, i, h] * d ** -0.5
                w = np.exp(x - x.max())
                wr = w if round_weights is None else round_weights(w)
                o[n, i, h] = wr @ v / w.sum()
                A = (np.abs(k) @ np.abs(q[n, i, h])).max() * d ** -0.5
                e = 2 * (d * U * A + 4 * U + 2 * U * A) + half(torch.bfloat16) ** 2 + 64 * U + U * total ** 0.5
                b = e * (w @ np.abs(v)) / w.sum()
                bound[n, i, h] = b + half_step(np.abs(o[n, i, h]) + b, torch.bfloat16) + 1e-38
    return o, bound
