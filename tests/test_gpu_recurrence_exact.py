"""GPU tests of the diagonal recurrence that no long memory blunts: decays of one and of zero over small whole
numbers, where every sum is exact, so that a token lost, doubled or carried over a reset at any border of a
run, tile, segment or sequence shows; and 2-norms over slow decays."""
import numpy as np
import pytest
import torch

from oracle import gdn2_stack as R
from tests.attn_util import U, assert_within, f64, half
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _cu(lens):
    return None if lens is None else np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def _whole(rng, low, high, shape, dtype, stride=0):
    x = torch.from_numpy(rng.integers(low, high + 1, shape[:-1] + (shape[-1] + stride,)).astype(np.float32)).to(dtype).cuda()
    return x[..., :shape[-1]]


# B, T, D, lens, chance of a reset
CASES = [
    (2, 37, 64, None, 0.0), (2, 257, 8, None, 0.05), (1, 1000, 72, None, 0.0), (3, 500, 2048, None, 0.002),
    (130, 400, 8, None, 0.0),                                                        # not cut
    (1, 2048, 64, None, 0.0), (1, 9000, 64, None, 0.0), (3, 2000, 136, None, 0.001),  # cut
    (1, 8192, 2048, None, 0.0), (1, 80000, 136, None, 0.0), (1, 80000, 136, None, 1e-4),  # in two passes
    (1, 0, 64, [256, 0, 1025, 1, 512, 257], 0.0), (1, 0, 8, [3, 9000] + 80 * [7], 0.0), (1, 0, 136, [3000, 0, 7, 70000], 3e-4),
]


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,D,lens,resets", CASES)
@pytest.mark.parametrize("stride", [0, 40])
def test_sums_of_whole_numbers(B, T, D, lens, resets, dt, stride):
    """|h| and |d| stay below 80000 times 6, 2^19: exact, as are their products with v and w. dg = d h takes
    one rounding."""
    import gated_delta_rule_36_amd as G
    rng = np.random.default_rng(T + D)
    cu = _cu(lens)
    N = B if lens is None else len(lens)
    T = T if lens is None else int(sum(lens))
    dtype, shape = DT[dt], (B, T, D)
    v, w, do = _whole(rng, -3, 3, shape, dtype, stride), _whole(rng, 0, 2, shape, dtype, stride), _whole(rng, -2, 2, shape, dtype)
    g = torch.zeros(B, T, D + stride, dtype=dtype, device="cuda")[..., :D]
    if resets:
        g.masked_fill_(torch.from_numpy(rng.random(shape) < resets).cuda(), float("-inf"))
    s0, ds = (_whole(rng, -9, 9, (N, D), torch.float32) for _ in range(2))
    cut = None if cu is None else torch.from_numpy(cu).cuda()
    say("linear_recurrence of whole numbers", B, T, D, lens, resets, dt, stride)
    o, last, states = G.linear_recurrence_fwd_train(v, g, w, initial_state=s0, cu_seqlens=cut)
    dv, dg, dw, ds0 = G.linear_recurrence_bwd(v, g, w, states, do, d_final_state=ds, cu_seqlens=cut)
    torch.cuda.synchronize()
    ref, lref = R.recurrence(f64(v), f64(g), f64(w), f64(s0), cu)
    rv, rg, rw, r0 = R.recurrence_backward(f64(v), f64(g), f64(w), f64(do), f64(s0), f64(ds), cu)
    assert max(np.abs(x).max() for x in (ref, lref, rv, rw, r0)) < 2 ** 24
    for name, x, r in (("o", o, ref), ("final", last, lref), ("dv", dv, rv), ("dw", dw, rw), ("ds0", ds0, r0)):
        exact = torch.from_numpy(r).to(x.dtype)
        assert torch.equal(x.cpu(), exact), f"{name}: {int((x.cpu() != exact).sum())} values of {x.numel()}"
    # (an fp32 rounding, in bf16 another)
    assert_within("dg", dg, rg, (U if dt == "fp32" else (U + half(dtype)) * 1.001) * np.abs(rg))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("gate", [True, False])
def test_tokens_of_whole_numbers(dt, gate):
    import gated_delta_rule_36_amd as G
    rng = np.random.default_rng(3)
    N, L, D = 33, 6, 72
    v, w = _whole(rng, -3, 3, (N, L, D), DT[dt], 8), _whole(rng, 0, 2, (N, L, D), DT[dt]) if gate else None
    g = torch.zeros(N, L, D, dtype=DT[dt], device="cuda")
    g.masked_fill_(torch.from_numpy(rng.random((N, L, D)) < 0.1).cuda(), float("-inf"))
    pool = _whole(rng, -9, 9, (N + 2, D), torch.float32).contiguous()
    idx, commit = rng.permutation(N + 2)[:N].astype(np.int32), rng.integers(-1, L + 2, N).astype(np.int32)
    ref, steps, after = R.recurrence_tokens(f64(pool), f64(v), f64(g), None if w is None else f64(w), idx, commit)
    say("linear_recurrence_tokens of whole numbers", dt, gate)
    o, got = G.linear_recurrence_tokens(v, g, w, pool, state_indices=torch.from_numpy(idx).cuda(),
                                        commit_len=torch.from_numpy(commit).cuda(), return_step_states=True)
    torch.cuda.synchronize()
    for x, r in ((o, ref), (got, steps), (pool, after)):
        assert np.array_equal(f64(x), r)


@pytest.mark.parametrize("B,T,D,lens", [(1, 777, 64, None), (1, 9000, 64, None), (1, 80000, 72, None), (1, 0, 64, [3, 9000, 500]),
                                        (16, 1500, 1024, None)])
def test_slow_decays_in_the_2_norm(B, T, D, lens):
    """Decays of 0.999 on average, fp32. A token's way into the states behind it takes at most 11 roundings
    for every token (tests/stack_util.py: 6 + 9 / 2 + 2 / 16), each of at most U of the state and of
    changing sign, U / sqrt(3) in the root mean square. They decay with the state: 500 tokens' squares are
    left of them. sqrt(11 * 500) / sqrt(3) = 43 U; a token lost at one border is 10^-3 and more. A gradient
    that is the product of two such states has both errors."""
    import gated_delta_rule_36_amd as G
    rng = np.random.default_rng(T + D)
    cu = _cu(lens)
    N = B if lens is None else len(lens)
    T = T if lens is None else int(sum(lens))
    v, g, do = (torch.from_numpy(rng.standard_normal((B, T, D)).astype(np.float32)).cuda() for _ in range(3))
    g = -1e-3 * g.abs()
    s0, ds = (torch.from_numpy(10 * rng.standard_normal((N, D)).astype(np.float32)).cuda() for _ in range(2))
    cut = None if cu is None else torch.from_numpy(cu).cuda()
    say("linear_recurrence 2-norm", B, T, D, lens)
    o, last, states = G.linear_recurrence_fwd_train(v, g, None, initial_state=s0, cu_seqlens=cut)
    dv, dg, _, ds0 = G.linear_recurrence_bwd(v, g, None, states, do, d_final_state=ds, cu_seqlens=cut)
    torch.cuda.synchronize()
    ref, lref = R.recurrence(f64(v), f64(g), None, f64(s0), cu)
    rv, rg, _, r0 = R.recurrence_backward(f64(v), f64(g), None, f64(do), f64(s0), f64(ds), cu)
    for name, x, r, k in (("o", o, ref, 43), ("final", last, lref, 43), ("dv", dv, rv, 43), ("dg", dg, rg, 86), ("ds0", ds0, r0, 43)):
        off = np.linalg.norm(f64(x) - r) / np.linalg.norm(r)
        assert off < k * U, f"{name}: {off / U:.1f} U in the 2-norm"
