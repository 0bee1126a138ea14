"""GPU tests of the serving prologue and of attention over the 8-bit cache against the float64
oracle, apart and as they are used together."""
import numpy as np
import pytest
import torch

from oracle import gdn2_attn as R
from tests.attn_util import (B64, U, Paged, assert_within, attention_ref, draw, f64, few_rows_ref, half,
                             inv_freq, rows_bound)
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _layout(new, packed, behind=0):
    """Row spans of the new tokens, the leading shape and cu_seqlens."""
    if packed:
        cu = np.concatenate([[0], np.cumsum(new)])
        return [(int(c), int(n)) for c, n in zip(cu, new)], (1, int(cu[-1]) + behind), _i32(cu)
    assert len(set(new)) == 1
    return [(i * new[0], new[0]) for i in range(len(new))], (len(new), new[0]), None


# ---------------------------------------------------------------- prologue

def _prologue(rng, paged, new, lens, Hq, packed, rot, il=False, norm=True, spoil=None, strided=True, behind=0,
              sizes=1.0):
    """One call on the device and in the oracle; checks q_out and the whole cache."""
    import gated_delta_rule_36_amd as G
    Hk, d = paged.Hk, paged.d
    spans, lead, cu = _layout(new, packed, behind)
    w = (Hq + 2 * Hk) * d
    qkv = draw(rng, *lead, w + (8 if strided else 0), scale=sizes)
    if spoil is not None:
        spoil(qkv)
    qkv = qkv.cuda()
    q = qkv[..., : Hq * d].view(*lead, Hq, d)
    k = qkv[..., Hq * d: (Hq + Hk) * d].view(*lead, Hk, d)
    v = qkv[..., (Hq + Hk) * d: w].view(*lead, Hk, d)
    wq, wk = (torch.from_numpy((1 + 0.2 * rng.standard_normal(d)).astype(np.float32)).cuda() for _ in range(2))
    fr = inv_freq(rot)
    out = torch.full((*lead, Hq, d), 7.0, dtype=BF, device="cuda")
    before = paged.pull()
    G.attn_prologue(q, k, v, paged.dev, paged.table_t(), _i32(lens), torch.from_numpy(fr).cuda() if rot else None,
                    cu_seqlens=cu, q_weight=wq, k_weight=wk, interleaved=il, norm=norm, out=out)
    torch.cuda.synchronize()
    flat = {n: f64(t).reshape(-1, t.shape[2], d) for n, t in (("q", q), ("k", k), ("v", v))}
    got = f64(out).reshape(-1, Hq, d)
    ref, bound = np.full_like(got, 7.0), np.zeros_like(got)
    errs = {}
    for i, (first, n) in enumerate(spans):
        if n == 0:
            continue
        pos = int(lens[i]) - n + np.arange(n)
        rows = slice(first, first + n)
        with np.errstate(invalid="ignore"):
            y, b = rows_bound(flat["q"][rows], f64(wq), np.maximum(pos, 0), fr, BF, 1e-6, il, norm)
            kn, kb = rows_bound(flat["k"][rows], f64(wk), np.maximum(pos, 0), fr, torch.float64, 1e-6, il, norm)
        none = (pos < 0)[:, None, None]
        ref[rows], bound[rows] = np.where(none, 0.0, y), np.where(none, 0.0, b)
        R.append(paged.ref, paged.table[i], int(lens[i]), kn, flat["v"][rows])
        errs[i] = kb
    assert_within("q_out", got, ref, bound)
    # scales are powers of two and equal; codes of the values are roundings of exact inputs and
    # equal; a key's code may fall to the other side of a rounding border by fp32's error
    # (16 U of the row), so it is at most one step off, and only where it is that near a border
    k_, v_, ks_, vs_ = paged.pull()
    assert np.array_equal(ks_, paged.ref.k_scale) and np.array_equal(vs_, paged.ref.v_scale)
    wrong = np.argwhere(v_ != paged.ref.v)
    assert len(wrong) == 0, wrong[:4]
    assert np.array_equal(np.isnan(k_), np.isnan(paged.ref.k))
    off = np.argwhere((k_ != paged.ref.k) & ~np.isnan(k_))
    assert len(off) <= 1 + k_.size // 10000, len(off)
    for at in off[:50]:
        a, b = k_[tuple(at)], paged.ref.k[tuple(at)]
        assert abs(a - b) <= 2 ** -3 * max(abs(a), abs(b)) + 2 ** -9, (at, a, b)
    paged.ref.k[:] = k_  # the device's roundings from here on
    return before, (k_, v_, ks_, vs_)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("total", [1, 2, 64, 65, 66, 100, 128, 129])
def test_prologue_single_token(total, d):
    """One token at every kind of place in a block, behind random older ones."""
    rng = np.random.default_rng(total * 3 + d)
    lens = [total, 70]
    paged = Paged(rng, lens, 2, d)
    paged.fill(rng)
    say("attn_prologue one token", total, d)
    _prologue(rng, paged, [1, 1], lens, 6, False, d, il=total % 2 == 0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,lens,packed", [
    ([5] * 3, [5, 66, 200], False),
    ([64] * 2, [64, 128], False),
    ([70] * 2, [70, 133], False),
    ([9] * 2, [60, 73], False),          # more tokens than go out as single bytes
    ([3, 0, 150, 1, 64], [3, 0, 150, 90, 64], True),
    ([1, 1, 1], [1, 64, 65], True),
    ([130, 2], [131, 2], True),
    ([300], [300], True),
])
def test_prologue_rows(new, lens, packed, d):
    rng = np.random.default_rng(sum(new) + d)
    paged = Paged(rng, lens, 3, d)
    paged.fill(rng)
    say("attn_prologue", new, lens, packed, d)
    _prologue(rng, paged, new, lens, 3, packed, d // 2, behind=4 if packed else 0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [2, 3, 4, 5, 8, 9])
def test_prologue_few_tokens(T, d):
    """Drafts: over a block's edge, in a new block, behind older ones, fewer tokens than rows, an empty
    sequence, a missing block, values whose scales grow."""
    rng = np.random.default_rng(T * 5 + d)
    lens = [T, 64, 63 + T, 65, 127 + T // 2, 200, 1, 0, 40 + T, 130]
    paged = Paged(rng, lens, 2, d)
    paged.fill(rng)
    paged.table[9, 2] = -1
    say("attn_prologue few tokens", T, d)
    _prologue(rng, paged, [T] * len(lens), lens, 4, False, d // 2, il=T % 2 == 0)
    for size in (1e-2, 50.0):
        _prologue(rng, paged, [T] * len(lens), lens, 4, False, d, norm=False, sizes=size)


@pytest.mark.parametrize("d", [64, 128])
def test_prologue_few_tokens_packed(d):
    """Blocks of few and of many new tokens in one packed call, scales that grow and ones that do not."""
    rng = np.random.default_rng(d + 1)
    new = [1, 4, 5, 8, 9, 2, 70, 3, 0, 64]
    lens = [64, 66, 5, 71, 200, 127, 134, 131, 0, 100]
    paged = Paged(rng, lens, 2, d)
    paged.fill(rng)
    say("attn_prologue few tokens packed", d)
    for size in (1.0, 1e-2, 50.0):
        _prologue(rng, paged, new, lens, 4, True, d, norm=False, sizes=size, behind=2)


def test_prologue_many_sequences_packed():
    """More sequences than one round of the 64-way search, empty ones among them."""
    rng = np.random.default_rng(5)
    new = [int(x) for x in rng.integers(0, 4, 150)]
    lens = [n + int(x) for n, x in zip(new, rng.integers(0, 130, 150))]
    paged = Paged(rng, lens, 1, 64)
    paged.fill(rng)
    say("attn_prologue 150 packed sequences")
    _prologue(rng, paged, new, lens, 2, True, 64, behind=3)


def test_prologue_scales_grow_and_shrink():
    """Tokens of rising size into one block: the scale grows and older codes follow; a block
    begun anew drops its old scale."""
    rng = np.random.default_rng(6)
    lens = [130]
    paged = Paged(rng, lens, 2, 128)
    say("attn_prologue growth")
    scales = []
    for t, size in ((3, 1e-3), (4, 1e-2), (6, 1.0), (7, 300.0), (9, 1e4), (30, 1.0), (64, 1.0)):
        _prologue(rng, paged, [t - (paged.t if hasattr(paged, "t") else 0)], [t], 2, False, 128, norm=False, sizes=size)
        paged.t = t
        scales.append(paged.ref.k_scale[paged.table[0, 0], 0])
    assert scales == sorted(scales) and scales[-1] > 1000 * scales[0]
    _prologue(rng, paged, [2], [2], 2, False, 128, norm=False, sizes=1e-3)  # the block again, from its start
    assert paged.ref.k_scale[paged.table[0, 0], 0] < 1e-4


def test_prologue_padding_rows_and_missing_blocks():
    rng = np.random.default_rng(7)
    # more new rows than tokens; an empty sequence; a sequence past its table; a hole in a table
    lens = [3, 0, 200, 130]
    paged = Paged(rng, [3, 0, 200, 130], 2, 64, table_width=2)
    paged.fill(rng)
    paged.table[3, 1] = paged.P + 5
    paged.table[2, 0] = -7
    say("attn_prologue padding and missing blocks")
    _prologue(rng, paged, [80] * 4, lens, 4, False, 64)


def test_prologue_not_finite_tokens():
    rng = np.random.default_rng(8)
    lens = [70, 70]
    Hq, Hk, d = 2, 2, 64
    paged = Paged(rng, lens, Hk, d)

    def spoil(x):
        x[0, 5, (Hq + 1) * d + 3] = float("nan")           # key of head 1
        x[0, 9, (Hq + Hk) * d + 1] = float("inf")          # value of head 0
        x[1, 0, (Hq + Hk + 1) * d] = float("-inf")         # value of head 1
        x[0, 68, Hq * d + 8] = float("inf")                # key of head 0, the last block

    say("attn_prologue not finite")
    _prologue(rng, paged, [70, 70], lens, Hq, False, d, norm=False, spoil=spoil)
    assert np.isnan(paged.ref.k).any() and not np.isnan(paged.ref.v).any()


def test_prologue_largest_and_smallest_values():
    """Values near the ends of the range: bf16's largest (stored as a marked token), large ones
    whose scale is 2^119, and ones below the smallest scale's codes."""
    rng = np.random.default_rng(18)
    Hq, Hk, d = 2, 2, 64
    paged = Paged(rng, [40], Hk, d)

    def spoil(x):
        x[0, 3, Hq * d] = torch.finfo(BF).max
        x[0, 7, (Hq + Hk) * d] = -torch.finfo(BF).max
        x[0, 8, (Hq + Hk) * d] = 3.0e38
        x[0, 9, (Hq + 1) * d: (Hq + 2) * d] *= 2.0 ** -80

    say("attn_prologue largest values")
    _prologue(rng, paged, [40], [40], Hq, False, 0, norm=False, spoil=spoil)
    assert np.isnan(paged.ref.k[paged.table[0, 0], 0, [3, 7]]).all()
    assert paged.ref.v_scale[paged.table[0, 0], 0] == 2.0 ** 120


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kept", [30, 1, 60])
def test_prologue_scale_grows_before_dropped_drafts(kept, d):
    """Drafts are dropped and the next token's values raise the block's scale to its largest: what the
    drafts left behind it must not stand for infinities, which weights of zero do not mask."""
    rng = np.random.default_rng(kept + d)
    Hq, Hk = 4, 2
    paged = Paged(rng, [64], Hk, d)
    first = (Hq + Hk) * d  # of the values

    def drafts(x):
        x[0, kept:, first:] = 448.0

    def large(x):
        x[0, 0, first:] = 3.0e38

    say("attn_prologue scale grows before dropped drafts", kept, d)
    _prologue(rng, paged, [kept + 3], [kept + 3], Hq, False, d, spoil=drafts)
    assert paged.ref.v_scale[paged.table[0, 0], 0] == 1.0
    _prologue(rng, paged, [1], [kept + 1], Hq, False, d, spoil=large)
    assert paged.ref.v_scale[paged.table[0, 0], 0] == 2.0 ** 120
    out = _attention(rng, paged, [1], [kept + 1], Hq, q=draw(rng, 1, 1, Hq, d, scale=0.1))
    assert out.isfinite().all()


def test_prologue_leaves_other_blocks():
    rng = np.random.default_rng(9)
    lens = [100, 300]
    paged = Paged(rng, lens, 2, 128, spare=5)
    paged.fill(rng)
    say("attn_prologue other blocks")
    before, after = _prologue(rng, paged, [3, 3], lens, 4, False, 128)
    touched = {paged.table[0, 1], paged.table[1, 4]}
    for b, a in zip(before, after):
        for s in range(paged.P):
            if s not in touched:
                assert np.array_equal(b[s], a[s]), s


# ---------------------------------------------------------------- attention

def _attention(rng, paged, new, lens, Hq, packed=False, window=0, scale=None, behind=0, q=None, alias=False):
    import gated_delta_rule_36_amd as G
    spans, lead, cu = _layout(new, packed, behind)
    q = draw(rng, *lead, Hq, paged.d) if q is None else q
    qd = q.cuda()
    out = qd if alias else torch.full_like(qd, 7.0)
    G.cache_attention(qd, paged.dev, paged.table_t(), _i32(lens), cu_seqlens=cu, window=window, scale=scale,
                      out=out)
    torch.cuda.synchronize()
    rows = f64(q).reshape(-1, Hq, paged.d)
    few = max(lead[1] if packed else new[0], 1) * (Hq // paged.Hk) <= 32
    ref, bound = attention_ref(rows, paged, lens, spans, window, scale, few=few)
    if behind:
        ref[-behind:] = rows[-behind:] if alias else 7.0
    assert_within("o", f64(out).reshape(ref.shape), ref, bound)
    return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,L", [(1, 1), (4, 1), (3, 5), (8, 2), (8, 4), (16, 1), (1, 32)])
@pytest.mark.parametrize("window", [0, 1, 70])
def test_attention_few_rows(G, L, d, window):
    rng = np.random.default_rng(G * 7 + L + d + window)
    lens = [L, 64, 65, 1000, 127 + L, 449]
    paged = Paged(rng, lens, 2, d)
    paged.fill(rng)
    say("cache_attention few rows", G, L, d, window)
    _attention(rng, paged, [L] * len(lens), lens, 2 * G, window=window, alias=L == 1)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,L,longest,window", [(4, 1, 449, 0), (4, 1, 449, 70), (3, 5, 1000, 0), (8, 4, 1000, 70),
                                                (16, 1, 1000, 0), (2, 2, 6001, 0)])
def test_attention_few_rows_at_the_outputs_rounding(G, L, longest, window, d):
    """Single tokens and drafts are off by the output's own rounding and little more: weights rounded
    once to bf16 would be 4 to 35 times the bound somewhere."""
    import gated_delta_rule_36_amd as G_
    rng = np.random.default_rng(G * 7 + L + d + window)
    lens = [L, 64, 65, 127 + L, longest]
    paged = Paged(rng, lens, 2, d)
    paged.fill(rng, spread=0.3)
    say("cache_attention few rows at the output's rounding", G, L, longest, window, d)
    q = draw(rng, len(lens), L, 2 * G, d)
    got = G_.cache_attention(q.cuda(), paged.dev, paged.table_t(), _i32(lens), window=window)
    torch.cuda.synchronize()
    ref, bound = few_rows_ref(f64(q), paged, lens, L, window)
    assert_within("o", got, ref, bound)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,L", [(1, 33), (4, 40), (3, 130), (5, 200)])
@pytest.mark.parametrize("window", [0, 1, 100])
def test_attention_many_rows(G, L, d, window):
    rng = np.random.default_rng(G * 7 + L + d + window)
    lens = [L, L + 64, L + 333]
    paged = Paged(rng, lens, 2, d)
    paged.fill(rng)
    say("cache_attention many rows", G, L, d, window)
    _attention(rng, paged, [L] * len(lens), lens, 2 * G, window=window, alias=G == 4)


@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("new,lens,Hq,Hk", [
    ([1, 0, 200, 33, 64], [300, 0, 200, 40, 1000], 6, 2),
    ([3, 0, 4, 1], [70, 9, 4, 1], 4, 4),             # packed, few rows in all
    ([700], [700], 4, 1),
    ([1] * 70 + [90], [200] * 70 + [90], 2, 2),
])
def test_attention_packed(new, lens, Hq, Hk, window):
    rng = np.random.default_rng(len(new) + window)
    paged = Paged(rng, lens, Hk, 64)
    paged.fill(rng)
    say("cache_attention packed", len(new), Hq, Hk, window)
    _attention(rng, paged, new, lens, Hq, packed=True, window=window, behind=5)


@pytest.mark.parametrize("new,lens,Hq,Hk,d,width,window", [
    ([1, 0, 200, 3, 4, 16, 5, 1], [300, 0, 900, 70, 4, 2600, 33, 0], 8, 2, 128, 50, 0),
    ([2, 3, 1, 40], [700, 64, 2100, 40], 16, 1, 64, 40, 0),       # 32 rows, and 48
    ([16, 17, 1, 60], [16, 17, 129, 1000], 2, 2, 128, 32, 0),     # 16 rows, and 17
    ([1] * 40, [61 * i for i in range(40)], 4, 2, 128, 40, 0),    # single tokens alone
    ([5, 100, 6, 1], [2500, 2500, 333, 2400], 6, 2, 64, 50, 2100),
    ([1, 130, 1, 60], [3000, 500, 64, 2000], 8, 4, 128, 64, 0),   # both kernels cut the key axis
    ([1, 50], [2200, 50], 32, 1, 128, 40, 0),                     # one token fills the rows
    ([1, 2, 33], [100, 200, 300], 33, 1, 64, 40, 0),              # no token fits them
    ([1] * 299 + [70], [i % 150 + 1 for i in range(299)] + [200], 6, 2, 64, 5, 50),  # short, but many
])
def test_attention_mixed_batches(new, lens, Hq, Hk, d, width, window):
    """Packed batches over wide tables: sequences of few rows beside long ones, holes in a table."""
    rng = np.random.default_rng(len(new) + Hq + window)
    paged = Paged(rng, lens, Hk, d, table_width=width)
    paged.fill(rng)
    paged.table[0, 1] = -1
    paged.table[-1, 2] = paged.P
    say("cache_attention mixed", new, Hq, Hk, d, window)
    for alias in (False, True):
        _attention(rng, paged, new, lens, Hq, packed=True, window=window, behind=3, alias=alias)


@pytest.mark.parametrize("new,Hq,d,blocks", [([1, 33], 1, 128, 143), ([1, 34], 1, 64, 143), ([64, 2, 35], 3, 128, 254)])
def test_attention_mixed_batches_with_odd_rows(new, Hq, d, blocks):
    """Both passes with pieces of the key axis and an odd number of partial rows in the first, in a
    workspace of just the size that was asked for."""
    import gated_delta_rule_36_amd as G
    rng = np.random.default_rng(blocks + d)
    lens = [blocks * 64 - 5, 700, 9000][: len(new)]
    T = 35 if len(new) == 2 else 101
    paged = Paged(rng, lens, Hq, d, table_width=blocks)
    paged.fill(rng)
    say("cache_attention mixed, odd rows", new, Hq, d, blocks)
    behind = T - sum(new)
    spans, lead, cu = _layout(new, True, behind)
    q = draw(rng, *lead, Hq, d)
    need = G.cache_attention_workspace_bytes(1, T, Hq, Hq, d, len(new), blocks, packed=True)
    room = torch.full((need + 256,), 0x5a, dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 7.0, device="cuda")
    G.cache_attention(q.cuda(), paged.dev, paged.table_t(), _i32(lens), cu_seqlens=cu, out=out, workspace=room[:need])
    torch.cuda.synchronize()
    assert (room[need:] == 0x5a).all()
    rows = f64(q).reshape(-1, Hq, d)
    ref, bound = attention_ref(rows, paged, lens, spans)
    ref[sum(new):] = 7.0
    assert_within("o", f64(out).reshape(ref.shape), ref, bound)


@pytest.mark.parametrize("L", [2, 90])
def test_attention_padding_and_missing_blocks(L):
    """Padding rows, an empty sequence, holes in a table, a table too short for its sequence, a
    sequence none of whose blocks exist."""
    rng = np.random.default_rng(L)
    lens = [1, 0, 500, 700, 64]
    paged = Paged(rng, lens, 2, 128, table_width=9)
    paged.fill(rng)
    paged.table[2, 1] = -1
    paged.table[2, 4] = paged.P
    paged.table[4, :] = 2 ** 31 - 1
    say("cache_attention padding and missing blocks", L)
    for window in (0, 40):
        _attention(rng, paged, [L] * 5, lens, 4, window=window)


@pytest.mark.parametrize("N,L,total,Hq,Hk,d,window,packed", [
    (2, 1, 500, 4, 2, 128, 0, False),       # few rows: 8 waves, one piece
    (2, 1, 3000, 4, 2, 64, 0, False),       # pieces of the key axis
    (2, 1, 500, 4, 2, 64, 130, False),
    (2, 6, 500, 8, 2, 128, 0, False),       # two tiles of rows
    (2, 90, 500, 4, 2, 128, 0, False),      # many rows
    (2, 90, 500, 4, 2, 64, 200, False),
    (1, 40, 5000, 4, 2, 128, 0, False),     # pieces of the key axis
    (16, 512, 1601, 16, 16, 128, 0, False),  # 8 waves
    (3, 70, 2500, 4, 2, 128, 0, True),      # single tokens beside a prompt
])
def test_attention_missing_blocks_read_nothing(N, L, total, Hq, Hk, d, window, packed):
    """Holes in the table where no block of the pool but the sequences' own holds numbers: what they
    do not name cannot show, so the rows are those over a pool of zeros."""
    import gated_delta_rule_36_amd as G
    rng = np.random.default_rng(N + L)
    say("cache_attention missing blocks read nothing", N, L, total, Hq, Hk, d, window, packed)
    nb = -(-total // B64)
    gen = torch.Generator(device="cuda").manual_seed(N + L)
    P = N * nb + 2  # block 0 and the last one are no sequence's
    cache = G.kv_cache(P, Hk, d)
    for codes, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        codes[1:-1].view(torch.uint8).copy_(torch.randn(codes[1:-1].shape, generator=gen, device="cuda").mul(50).to(
            torch.float8_e4m3fn).view(torch.uint8))
        scale[1:-1] = 2.0 ** -6
    table = 1 + rng.permutation(N * nb).astype(np.int32).reshape(N, nb)
    for row in table:  # the first and the last block, a neighbour pair and every seventh
        row[[0, 2, 3, nb - 1]] = [-1, P, 2 ** 31 - 1, -2 ** 31]
        row[6::7] = -1
    lens = np.full(N, total)
    lens[0] -= 70
    q = torch.randn(1 if packed else N, L, Hq, d, generator=gen, device="cuda").to(BF)
    cu = _i32([0, 1, 2, L]) if packed else None
    call = lambda: G.cache_attention(q, cache, _i32(table), _i32(lens), cu_seqlens=cu, window=window)
    ref = call()
    torch.cuda.synchronize()
    assert ref.isfinite().all() and ref.any()
    for codes, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        codes.view(torch.uint8)[[0, P - 1]] = 0x7f
        scale[[0, P - 1]] = float("nan")
    got = call()
    torch.cuda.synchronize()
    assert torch.equal(got, ref)


def test_attention_missing_blocks_in_an_unused_pool():
    """The oracle's rows, with a first block of the pool that no one has written."""
    rng = np.random.default_rng(51)
    lens = [300, 128]
    paged = Paged(rng, lens, 2, 128, spare=3)
    paged.fill(rng)
    unused = max(set(range(paged.P)) - set(paged.table[paged.table >= 0].tolist()))
    paged.table[paged.table == 0] = unused
    paged.table[0, 1] = -1
    paged.table[1, 0] = paged.P
    for x in (paged.ref.k, paged.ref.v, paged.ref.k_scale, paged.ref.v_scale):
        x[0] = np.nan
    paged.push()
    say("cache_attention missing blocks, block 0 not written")
    for L in (1, 10, 90):
        for window in (0, 100):
            _attention(rng, paged, [L] * 2, lens, 4, window=window)


@pytest.mark.parametrize("L", [1, 6, 100])
def test_attention_not_finite_keys(L):
    """A marked token makes NaN of the rows that see it, and of no others."""
    rng = np.random.default_rng(L)
    lens = [150, 150]
    paged = Paged(rng, lens, 2, 64)
    paged.fill(rng)
    for pos in (40, 148):
        paged.ref.k[paged.table[0, pos // B64], 1, pos % B64] = np.nan
    paged.push()
    say("cache_attention not finite", L)
    for window in (0, 3):
        out = _attention(rng, paged, [L] * 2, lens, 4, window=window)
        assert out.isnan().any() and not out[1].isnan().any()


@pytest.mark.parametrize("L", [1, 100])
def test_attention_stale_bytes_behind_a_sequence(L):
    """Keys of any code, and finite values, behind the last token of a block are never seen."""
    rng = np.random.default_rng(L + 1)
    lens = [130, 101]
    paged = Paged(rng, lens, 1, 128)
    paged.fill(rng)
    for i, n in enumerate(lens):
        paged.ref.k[paged.table[i, n // B64], :, n % B64:] = np.nan
        paged.ref.v[paged.table[i, n // B64], :, n % B64:] = 448.0
    paged.push()
    say("cache_attention stale bytes", L)
    _attention(rng, paged, [L] * 2, lens, 3)


def test_attention_shared_blocks():
    """Sequences that share their first blocks, and one that names a block twice."""
    rng = np.random.default_rng(41)
    lens = [200, 200, 129]
    paged = Paged(rng, lens, 2, 64)
    paged.fill(rng)
    paged.table[1, :2] = paged.table[0, :2]
    paged.table[2, 1] = paged.table[2, 0]
    say("cache_attention shared blocks")
    for L in (1, 60):
        _attention(rng, paged, [L] * 3, lens, 4)


def test_attention_scales_far_apart():
    """Blocks whose scales differ by many powers of two, tiny and large scores."""
    rng = np.random.default_rng(21)
    lens = [400, 257]
    paged = Paged(rng, lens, 2, 64)
    paged.fill(rng, spread=4.0)
    say("cache_attention scales")
    for L in (1, 64):
        _attention(rng, paged, [L] * 2, lens, 4, scale=0.01)
        _attention(rng, paged, [L] * 2, lens, 4, scale=1.0, q=draw(rng, 2, L, 4, 64, scale=0.05))


def test_attention_long_context():
    """Many pieces of the key axis, odd lengths."""
    rng = np.random.default_rng(22)
    lens = [9001, 4133]
    paged = Paged(rng, lens, 1, 64)
    paged.fill(rng)
    say("cache_attention long")
    for L, window in ((1, 0), (3, 5000), (40, 0)):
        _attention(rng, paged, [L] * 2, lens, 4, window=window)


def _plain64(q, cache, table, lens, window=0):
    """Attention in 64-bit torch on the device, [N, T, Hq, d] queries, and the sum of p |v|."""
    import gated_delta_rule_36_amd as G
    N, T, Hq, d = q.shape
    Hk = cache.k.shape[1]
    cols = G.value_columns("cuda")
    out, spread = torch.empty(q.shape, dtype=torch.float64, device="cuda"), torch.empty(q.shape, dtype=torch.float64, device="cuda")
    for n in range(N):
        total = int(lens[n])
        blocks = table[n, : -(-total // B64)].long()
        k = (cache.k[blocks].double() * cache.k_scale[blocks].double()[..., None, None]).transpose(0, 1).reshape(Hk, -1, d)
        v = (cache.v[blocks].float()[..., cols].double() * cache.v_scale[blocks].double()[..., None, None])
        v = v.permute(1, 0, 3, 2).reshape(Hk, -1, d)
        p = total - T + torch.arange(T, device="cuda")[:, None]
        j = torch.arange(k.shape[1], device="cuda")
        hide = (j > p) | ((j <= p - window) if window else (j < 0))
        for h in range(Hq):
            x = q[n, :, h].double() @ k[h // (Hq // Hk)].t().contiguous() / d ** 0.5
            w = torch.softmax(x.masked_fill(hide, float("-inf")), -1)
            out[n, :, h], spread[n, :, h] = w @ v[h // (Hq // Hk)], w @ v[h // (Hq // Hk)].abs()
    return f64(out), f64(spread)


@pytest.mark.parametrize("N,T,total,Hq,Hk,d,window", [
    (16, 512, 1601, 16, 16, 128, 0),   # tiles of 256 rows, 8 waves
    (8, 1000, 1900, 16, 16, 128, 1700),
    (70, 1, 400, 8, 4, 128, 0),        # 280 (sequence, head) pairs: 8 waves, one piece
    (70, 2, 1500, 8, 4, 64, 0),
    (3, 1, 450, 4, 2, 64, 0),          # 8 blocks: a block a wave
    (260, 3, 333, 4, 4, 64, 100),
    (1, 40, 20000, 8, 2, 128, 0),      # a few tiles, the key axis cut many times
    (1, 9, 20011, 16, 2, 128, 0),      # one tile a head: pieces of 4 blocks
    (2, 35, 9000, 2, 2, 64, 0),
    (1, 700, 700, 4, 1, 64, 0),        # cut in pieces that the short tiles do not reach
    (1, 500, 3001, 4, 2, 128, 1000),   # pieces of a window
    (1, 1300, 1333, 8, 8, 128, 0),
])
def test_attention_variants_at_size(N, T, total, Hq, Hk, d, window):
    """Every way a call is cut, at the sizes that choose it, against 64-bit torch on the device."""
    import gated_delta_rule_36_amd as G
    rng = np.random.default_rng(N + total)
    say("cache_attention at size", N, T, total, Hq, Hk, d, window)
    nb = -(-total // B64)
    gen = torch.Generator(device="cuda").manual_seed(N + total)
    P = N * nb
    cache = G.kv_cache(P, Hk, d)
    for codes, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        codes.view(torch.uint8).copy_(torch.randn(codes.shape, generator=gen, device="cuda").mul(50).clamp(-448, 448).to(
            torch.float8_e4m3fn).view(torch.uint8))
        scale.copy_(torch.exp2(torch.randint(-7, -4, scale.shape, generator=gen, device="cuda").float()))
    table = torch.from_numpy(rng.permutation(P).astype(np.int32).reshape(N, nb)).cuda()
    lens = rng.integers(max(T, total * 3 // 4), total + 1, N)
    q = torch.randn(N, T, Hq, d, generator=gen, device="cuda").to(BF)
    got = G.cache_attention(q, cache, table, _i32(lens), window=window)
    torch.cuda.synchronize()
    ref, spread = _plain64(q, cache, table, lens, window)
    # the bound of attention_ref, with |k| at most 448 * 2^-5
    qs = np.abs(f64(q)).sum(-1, keepdims=True)
    A = qs * 448 * 2.0 ** -5 * d ** -0.5
    hb = half(BF)
    w = hb * hb if T * (Hq // Hk) <= 32 else hb
    e = 2 * (d * U * A + 4 * U + 2 * U * A)
    assert_within("o", got, ref, (e + w + 64 * U + U * total ** 0.5) * spread + hb * np.abs(ref) + 1e-38)


def test_attention_offsets_past_32_bits():
    """Blocks past 2^31 bytes of a cache."""
    import gated_delta_rule_36_amd as G
    rng = np.random.default_rng(23)
    P, Hk, d = 34000, 8, 128  # 2.2 GB of keys
    lens = [150]
    say("cache_attention large pool")
    small = Paged(rng, lens, Hk, d, spare=0)
    small.fill(rng)
    big = [torch.zeros((P, Hk, *s), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
           for s in ((64, d), (d, 64))] + [torch.zeros((P, Hk), device="cuda") for _ in range(2)]
    place = [P - 1 - i for i in range(small.P)]
    for b, s in zip(big, small.dev):
        b.view(torch.uint8)[place] = s.view(torch.uint8)
    table = np.array([[place[t] for t in small.table[0]]], np.int32)
    fr = torch.from_numpy(inv_freq(d)).cuda()
    for L in (1, 70):
        q, k, v = (draw(rng, 1, L, h, d).cuda() for h in (16, Hk, Hk))
        outs = []
        for cache, tb in ((big, _i32(table)), (small.dev, small.table_t())):
            qo = G.attn_prologue(q, k, v, cache, tb, _i32(lens), fr)
            outs.append(G.cache_attention(qo, cache, tb, _i32(lens)))
        torch.cuda.synchronize()
        assert torch.equal(*outs)
        for b, s in zip(big, small.dev):
            assert torch.equal(b.view(torch.uint8)[place], s.view(torch.uint8))


# ---------------------------------------------------------------- together

def test_serving_run():
    """Packed prompts, single tokens, drafts with a rollback, as a serving loop makes them; then the
    same tokens through attention at once give the same rows within the bounds."""
    import gated_delta_rule_36_amd as G
    rng = np.random.default_rng(31)
    Hq, Hk, d, window = 4, 2, 64, 90
    lens = np.array([130, 61, 5])
    paged = Paged(rng, lens + 20, Hk, d, spare=1)
    say("serving run")
    fr = inv_freq(d)
    frt = torch.from_numpy(fr).cuda()

    def step(new, total, packed):
        spans, lead, cu = _layout(new, packed)
        q, k, v = (draw(rng, *lead, h, d).cuda() for h in (Hq, Hk, Hk))
        qo = G.attn_prologue(q, k, v, paged.dev, paged.table_t(), _i32(total), frt, cu_seqlens=cu)
        o = G.cache_attention(qo, paged.dev, paged.table_t(), _i32(total), cu_seqlens=cu, window=window)
        torch.cuda.synchronize()
        kf, vf = f64(k).reshape(-1, Hk, d), f64(v).reshape(-1, Hk, d)
        for i, (first, n) in enumerate(spans):
            p = int(total[i]) - n + np.arange(n)
            R.append(paged.ref, paged.table[i], int(total[i]), R.norm_rope(kf[first:first + n], None, p, fr),
                     vf[first:first + n])
        kd, vd, ksd, vsd = paged.pull()
        assert np.array_equal(ksd, paged.ref.k_scale) and np.array_equal(vsd, paged.ref.v_scale)
        assert np.array_equal(vd, paged.ref.v)
        assert np.count_nonzero(kd != paged.ref.k) <= 4
        paged.ref.k[:] = kd
        few = (lead[1] if packed else new[0]) * (Hq // Hk) <= 32
        ref, bound = attention_ref(f64(qo).reshape(-1, Hq, d), paged, total, spans, window, few=few)
        assert_within("o", f64(o).reshape(ref.shape), ref, bound)

    step([int(n) for n in lens], lens, True)
    for _ in range(4):
        lens = lens + 1
        step([1] * 3, lens, False)
    step([4] * 3, lens + 4, False)      # drafts
    lens = lens + np.array([4, 1, 0])   # accepted
    step([1] * 3, lens + 1, False)
    step([3] * 3, lens + 4, False)


def test_serving_step_captured():
    """Prologue and attention in one graph; tokens, lengths and table change between replays."""
    import gated_delta_rule_36_amd as G
    rng = np.random.default_rng(32)
    Hq, Hk, d = 8, 2, 128
    lens = np.array([130, 610, 5, 0])
    paged = Paged(rng, lens + 70, Hk, d)
    paged.fill(rng)
    say("serving step captured")
    fr = torch.from_numpy(inv_freq(d)).cuda()
    q, k, v = (draw(rng, 4, 1, h, d).cuda() for h in (Hq, Hk, Hk))
    lt, tb = _i32(lens), paged.table_t()

    def step(cache):
        qo = G.attn_prologue(q, k, v, cache, tb, lt, fr)
        return qo, G.cache_attention(qo, cache, tb, lt)

    twin = G.KVCache(*(t.clone() for t in paged.dev))
    step(G.KVCache(*(t.clone() for t in paged.dev)))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(paged.dev)
    for i in range(4):
        lens = lens + np.array([1, 1, 20, 1])
        lt.copy_(_i32(lens))
        for t in (q, k, v):
            t.copy_(draw(rng, *t.shape))
        ref = step(twin)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, ref)), i
        for a, b in zip(paged.dev, twin):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_mixed_batch_captured():
    """A packed call in a graph: which sequences hold single tokens changes between replays."""
    import gated_delta_rule_36_amd as G
    rng = np.random.default_rng(35)
    T, Hq, Hk, d = 200, 8, 2, 64
    lens = [2100, 900, 64, 300, 0]
    paged = Paged(rng, lens, Hk, d, table_width=40)
    paged.fill(rng)
    say("mixed batch captured")
    q, out = draw(rng, 1, T, Hq, d).cuda(), torch.empty(1, T, Hq, d, dtype=torch.bfloat16, device="cuda")
    cu, lt, tb = _i32([0, 1, 2, 66, 196, 196]), _i32(lens), paged.table_t()
    call = lambda o: G.cache_attention(q, paged.dev, tb, lt, cu_seqlens=cu, out=o)
    call(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    for i, new in enumerate([[1, 1, 64, 130, 0], [150, 4, 5, 1, 0], [1, 1, 1, 1, 0], [0, 160, 1, 39, 0],
                             [1, 0, 0, 0, 0]]):
        cu.copy_(_i32(np.concatenate([[0], np.cumsum(new)])))
        q.copy_(draw(rng, 1, T, Hq, d))
        out.fill_(5.0)
        graph.replay()
        ref = call(torch.full_like(out, 5.0))
        torch.cuda.synchronize()
        assert torch.equal(out, ref), i
        assert (out[0, sum(new):] == 5.0).all()
        spans = [(sum(new[:n]), c) for n, c in enumerate(new)]
        exact, bound = attention_ref(f64(q).reshape(-1, Hq, d), paged, lens, spans, 0, None, few=False)
        n = sum(new)
        assert_within("o", f64(out).reshape(exact.shape)[:n], exact[:n], bound[:n])


def test_serving_many_packed_sequences():
    """More sequences than one round of the search, in both kernels of a serving step."""
    rng = np.random.default_rng(34)
    new = [int(x) for x in rng.integers(0, 5, 90)]
    lens = [n + int(x) for n, x in zip(new, rng.integers(0, 150, 90))]
    paged = Paged(rng, lens, 2, 64)
    paged.fill(rng)
    say("serving 90 packed sequences")
    _prologue(rng, paged, new, lens, 4, True, 64, behind=2)
    _attention(rng, paged, new, lens, 4, packed=True, behind=2)


def test_two_streams():
    """Two calls in flight on streams of their own, each with its own workspace."""
    import gated_delta_rule_36_amd as G
    rng = np.random.default_rng(33)
    lens = [5000, 3000]
    paged = Paged(rng, lens, 2, 64)
    paged.fill(rng)
    say("cache_attention two streams")
    qs = [draw(rng, 2, n, 4, 64).cuda() for n in (1, 50)]
    tb, lt = paged.table_t(), _i32(lens)
    ref = [G.cache_attention(q, paged.dev, tb, lt) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = []
    for q, st in zip(qs, streams):
        with torch.cuda.stream(st):
            got.append([G.cache_attention(q, paged.dev, tb, lt) for _ in range(5)])
    torch.cuda.synchronize()
    for r, many in zip(ref, got):
        assert all(torch.equal(r, g) for g in many)


@pytest.mark.parametrize("seed", range(16))
def test_sweep(seed):
    """Seeded mixed shapes: prologue, then attention on the result."""
    rng = np.random.default_rng(1000 + seed)
    d = int(rng.choice([64, 128]))
    Hk, G = int(rng.choice([1, 2, 3, 5])), int(rng.choice([1, 2, 3, 4, 7]))
    N = int(rng.integers(1, 6))
    packed = bool(rng.random() < 0.5)
    if packed:
        new = [int(x) for x in rng.integers(0, 140, N)]
        new[0] = max(new[0], 1)
    else:
        new = [int(rng.choice([1, 2, 3, 8, 20, 65, 129]))] * N
    lens = [max(0, n + int(x)) for n, x in zip(new, rng.integers(-3, 300, N))]
    window = int(rng.choice([0, 0, 1, 33, 64, 200]))
    paged = Paged(rng, lens, Hk, d)
    paged.fill(rng)
    say("attention layer sweep", seed, d, Hk, G, new, lens, window)
    _prologue(rng, paged, new, lens, Hk * G, packed, int(rng.choice([0, 16, d])), il=bool(rng.random() < 0.5))
    _attention(rng, paged, new, lens, Hk * G, packed=packed, window=window)
