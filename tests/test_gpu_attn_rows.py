"""GPU tests of the norms of queries and keys with the position rotation (forward, backward,
autograd) against the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import gdn2_attn as R
from tests.attn_util import U, assert_within, draw, f64, half, inv_freq, rows_bound
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _case(seed, B, T, Hq, Hk, d, rot, dt, weights=True, far=0, strided=False):
    rng = np.random.default_rng(seed)
    dtype = DT[dt]
    if strided:  # slices of one projection, with a gap behind
        qkv = draw(rng, B, T, (Hq + 2 * Hk) * d + 8, dtype=dtype).cuda()
        q = qkv[..., : Hq * d].view(B, T, Hq, d)
        k = qkv[..., Hq * d: (Hq + Hk) * d].view(B, T, Hk, d)
    else:
        q, k = draw(rng, B, T, Hq, d, dtype=dtype).cuda(), draw(rng, B, T, Hk, d, dtype=dtype).cuda()
    pos = (rng.integers(-far, far + 1, (B, 1)) + np.arange(T)).astype(np.int32)
    w = [torch.from_numpy((1 + 0.2 * rng.standard_normal(d)).astype(np.float32)).cuda() if weights else None
         for _ in range(2)]
    return q, k, pos, w, rng


def _np(w):
    return None if w is None else f64(w)


CASES = [
    # B, T, Hq, Hk, d, rot, dtype, interleaved, norm, weights, far, strided
    (2, 37, 4, 4, 128, 128, "bf16", False, True, True, 0, False),
    (2, 37, 4, 2, 128, 128, "bf16", True, True, True, 0, True),
    (1, 1, 1, 1, 64, 64, "bf16", False, True, True, 5, False),
    (1, 5, 33, 17, 64, 32, "bf16", False, True, False, 1000, False),
    (3, 7, 17, 1, 128, 64, "bf16", True, True, True, 2 ** 30, True),
    (1, 130, 16, 4, 128, 40, "bf16", False, False, True, 0, True),
    (1, 9, 3, 5, 64, 8, "bf16", True, False, False, 0, False),
    (2, 6, 2, 2, 128, 0, "bf16", False, True, True, 0, False),
    (1, 255, 2, 2, 64, 32, "fp32", True, True, True, 10 ** 6, False),
    (2, 33, 5, 3, 128, 128, "fp32", False, True, True, 2 ** 30, True),
    (1, 1, 1, 1, 128, 120, "fp32", False, True, False, 0, False),
]


@pytest.mark.parametrize("case", CASES)
def test_forward(case):
    import gated_delta_rule_36_amd as G
    B, T, Hq, Hk, d, rot, dt, il, norm, weights, far, strided = case
    q, k, pos, w, _ = _case(7, B, T, Hq, Hk, d, rot, dt, weights, far, strided)
    fr = inv_freq(rot)
    say("qk_norm_rope_fwd", case)
    got = G.qk_norm_rope_fwd(q, k, torch.from_numpy(fr).cuda() if rot else None,
                             positions=torch.from_numpy(pos).cuda(), q_weight=w[0], k_weight=w[1],
                             eps=1e-5, interleaved=il, norm=norm)
    torch.cuda.synchronize()
    for name, x, y, wt in (("q", q, got[0], w[0]), ("k", k, got[1], w[1])):
        assert y.dtype == DT[dt] and y.is_contiguous()
        ref, bound = rows_bound(f64(x), _np(wt), pos, fr, DT[dt], 1e-5, il, norm)
        assert_within(name, y, ref, bound)


def test_forward_frequencies_past_a_turn():
    """Frequencies of several turns a position, negative ones, zero, at the ends of int32."""
    import gated_delta_rule_36_amd as G
    rng = np.random.default_rng(16)
    fr = (rng.standard_normal(32) * np.array([0.0, 1e-3, 1.0, 50.0] * 8)).astype(np.float32)
    pos = np.array([[-2 ** 31, -2 ** 31 + 1, -1, 0, 1, 2 ** 30, 2 ** 31 - 2, 2 ** 31 - 1]], np.int32)
    q = draw(rng, 1, 8, 3, 64, dtype=torch.float32).cuda()
    say("qk_norm_rope_fwd frequencies past a turn")
    got, _ = G.qk_norm_rope_fwd(q, q, torch.from_numpy(fr).cuda(), positions=torch.from_numpy(pos).cuda())
    torch.cuda.synchronize()
    # the reference's own angle in 64 bits: the product of a 24-bit frequency and a 32-bit position
    # needs 56 bits, so the largest angles (2^31 * 100 rad) are off by 2^-53 of them, 2.4e-5
    ref, bound = rows_bound(f64(q), None, pos, fr, torch.float32, 1e-6, False, True)
    size = np.abs(R.norm_rope(f64(q), None, pos, fr[:0]))
    slack = 2.0 ** -52 * np.abs(pos[..., None].astype(np.float64)) * np.abs(fr).max()
    assert_within("q", got, ref, bound + 2 * size.max(-1, keepdims=True) * slack[..., None])


def test_forward_default_positions_and_in_place():
    import gated_delta_rule_36_amd as G
    q, k, _, w, _ = _case(8, 3, 20, 4, 2, 64, 64, "bf16")
    fr = torch.from_numpy(inv_freq(64)).cuda()
    say("qk_norm_rope_fwd positions None, out=(q, k)")
    pos = torch.arange(20, dtype=torch.int32, device="cuda").repeat(3, 1)
    ref = G.qk_norm_rope_fwd(q, k, fr, positions=pos, q_weight=w[0], k_weight=w[1])
    got = G.qk_norm_rope_fwd(q, k, fr, q_weight=w[0], k_weight=w[1], out=(q, k))
    torch.cuda.synchronize()
    assert got[0] is q and got[1] is k
    assert torch.equal(q, ref[0]) and torch.equal(k, ref[1])


def test_forward_zero_rows_and_no_tokens():
    import gated_delta_rule_36_amd as G
    fr = torch.from_numpy(inv_freq(128)).cuda()
    say("qk_norm_rope_fwd zero rows, B T = 0")
    z = torch.zeros(1, 3, 2, 128, dtype=torch.bfloat16, device="cuda")
    q, k = G.qk_norm_rope_fwd(z, z[:, :, :1], fr, eps=1e-6)
    torch.cuda.synchronize()
    assert not q.any() and not k.any()
    e = torch.empty(2, 0, 4, 128, dtype=torch.bfloat16, device="cuda")
    q, k = G.qk_norm_rope_fwd(e, e, fr)
    assert q.shape == e.shape
    wt = torch.ones(128, device="cuda")
    g = G.qk_norm_rope_bwd(e, e, e, e, fr, q_weight=wt, k_weight=wt)
    assert g[0].shape == e.shape and not g[2].any() and not g[3].any()


def test_forward_keeps_bad_rows_apart():
    """NaN and infinity stay in their own head row."""
    import gated_delta_rule_36_amd as G
    q, k, pos, w, _ = _case(9, 1, 6, 5, 2, 128, 128, "bf16")
    fr = torch.from_numpy(inv_freq(128)).cuda()
    good = G.qk_norm_rope_fwd(q, k, fr, q_weight=w[0], k_weight=w[1])
    q2 = q.clone()
    q2[0, 3, 2, 17] = float("nan")
    q2[0, 4, 0, 1] = float("inf")
    got = G.qk_norm_rope_fwd(q2, k, fr, q_weight=w[0], k_weight=w[1])
    torch.cuda.synchronize()
    bad = torch.zeros(1, 6, 5, dtype=torch.bool)
    bad[0, 3, 2] = bad[0, 4, 0] = True
    assert torch.equal(got[0][~bad.cuda()], good[0][~bad.cuda()]) and torch.equal(got[1], good[1])
    assert got[0][0, 3, 2].isnan().all()


def _bwd_bound(x, dy, w, pos, fr, dtype, eps, il, norm):
    """dn 8 U of |a| + |b| of dy; with the root's 10 U, the products' and the two sums' (12 U of
    their absolute values) at most 40 U of r (|w dn| + |x| r^2 / d sum |w dn x|); one rounding.
    dw: terms off by 24 U, the sums over rows by U per addition in fp32 lanes (at most 64 here
    a lane, then 10 to the partial row): 100 U of the sum of absolute terms, one rounding."""
    dx, dw = R.norm_rope_backward(x, dy, w, pos, fr, eps, il, norm)
    d, rot = x.shape[-1], 2 * len(fr)
    a, b = R._split(np.abs(dy), rot, il)
    dn = R._join(np.abs(dy), a + b, a + b, rot, il)
    wt = np.ones(d) if w is None else np.abs(w)
    r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) if norm else np.ones_like(x[..., :1])
    back = r * r / d * np.sum(wt * dn * np.abs(x), -1, keepdims=True) if norm else 0.0
    bx = 40 * U * r * (wt * dn + np.abs(x) * back) + half(dtype) * np.abs(dx) + 1e-38
    bw = 100 * U * (dn * np.abs(x) * r).reshape(-1, d).sum(0) + U * np.abs(dw)
    return dx, dw, bx, bw


@pytest.mark.parametrize("case", CASES)
def test_backward(case):
    import gated_delta_rule_36_amd as G
    B, T, Hq, Hk, d, rot, dt, il, norm, weights, far, strided = case
    q, k, pos, w, rng = _case(11, B, T, Hq, Hk, d, rot, dt, weights, far, strided)
    gq, gk = draw(rng, B, T, Hq, d, dtype=DT[dt]).cuda(), draw(rng, B, T, Hk, d, dtype=DT[dt]).cuda()
    fr = inv_freq(rot)
    say("qk_norm_rope_bwd", case)
    got = G.qk_norm_rope_bwd(q, k, gq, gk, torch.from_numpy(fr).cuda() if rot else None,
                             positions=torch.from_numpy(pos).cuda(), q_weight=w[0], k_weight=w[1],
                             eps=1e-5, interleaved=il, norm=norm)
    torch.cuda.synchronize()
    for i, (name, x, g, wt) in enumerate((("q", q, gq, w[0]), ("k", k, gk, w[1]))):
        dx, dw, bx, bw = _bwd_bound(f64(x), f64(g), _np(wt), pos, fr, DT[dt], 1e-5, il, norm)
        assert_within("d" + name, got[i], dx, bx)
        if weights:
            assert_within(f"d{name}_weight", got[2 + i], dw, bw)
        else:
            assert got[2 + i] is None


def test_backward_many_tokens_and_same_bits():
    """More tokens than the backward's waves (each wave then walks several), twice."""
    import gated_delta_rule_36_amd as G
    q, k, pos, w, rng = _case(12, 1, 4096 * 2 + 77, 3, 1, 64, 64, "bf16")
    gq, gk = draw(rng, *q.shape).cuda(), draw(rng, *k.shape).cuda()
    fr = inv_freq(64)
    say("qk_norm_rope_bwd 8269 tokens")
    runs = [G.qk_norm_rope_bwd(q, k, gq, gk, torch.from_numpy(fr).cuda(), q_weight=w[0], k_weight=w[1])
            for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    for i, (x, g, wt) in enumerate(((q, gq, w[0]), (k, gk, w[1]))):
        dx, dw, bx, bw = _bwd_bound(f64(x), f64(g), f64(wt), np.arange(x.shape[1])[None], fr, torch.bfloat16,
                                    1e-6, False, True)
        assert_within("dx", runs[0][i], dx, bx)
        assert_within("dw", runs[0][2 + i], dw, bw)


def test_autograd_equals_the_calls():
    import gated_delta_rule_36_amd as G
    q, k, pos, w, rng = _case(13, 2, 19, 4, 2, 64, 32, "fp32", strided=True)
    gq, gk = draw(rng, 2, 19, 4, 64, dtype=torch.float32).cuda(), draw(rng, 2, 19, 2, 64, dtype=torch.float32).cuda()
    fr, p = torch.from_numpy(inv_freq(32)).cuda(), torch.from_numpy(pos).cuda()
    say("qk_norm_rope autograd")
    leaves = [t.detach().clone().requires_grad_() for t in (q, k, *w)]
    y = G.qk_norm_rope(leaves[0], leaves[1], fr, positions=p, q_weight=leaves[2], k_weight=leaves[3])
    torch.autograd.backward(y, (gq, gk))
    ref = G.qk_norm_rope_bwd(q, k, gq, gk, fr, positions=p, q_weight=w[0], k_weight=w[1])
    torch.cuda.synchronize()
    for leaf, r in zip(leaves, ref):
        assert torch.equal(leaf.grad, r)
    # one output only, an expanded gradient
    leaf = q.detach().clone().requires_grad_()
    G.qk_norm_rope(leaf, k, fr, positions=p)[0].sum().backward()
    one = G.qk_norm_rope_bwd(leaf.detach(), k, torch.ones_like(gq), torch.zeros_like(gk), fr, positions=p)[0]
    assert torch.equal(leaf.grad, one)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_autograd_through_one_projection(dt):
    """Queries and keys as slices of a projection that is the leaf, with the values between them and
    the gradient, which comes back as views of one flat tensor."""
    import gated_delta_rule_36_amd as G
    B, T, Hq, Hk, d, rot = 2, 21, 4, 2, 64, 64
    rng = np.random.default_rng(17)
    x = draw(rng, B, T, (Hq + 2 * Hk) * d + 8, dtype=DT[dt]).cuda().requires_grad_()
    w = [torch.from_numpy((1 + 0.2 * rng.standard_normal(d)).astype(np.float32)).cuda().requires_grad_() for _ in range(2)]
    fr = inv_freq(rot)
    say("qk_norm_rope autograd through a projection", dt)
    q = x[..., : Hq * d].view(B, T, Hq, d)
    k = x[..., Hq * d: (Hq + Hk) * d].view(B, T, Hk, d)
    v = x[..., (Hq + Hk) * d: (Hq + 2 * Hk) * d]
    y = G.qk_norm_rope(q, k, torch.from_numpy(fr).cuda(), q_weight=w[0], k_weight=w[1])
    lead = torch.zeros(3, dtype=DT[dt], device="cuda")
    flat = torch.cat([lead, y[0].flatten(), y[1].flatten(), v.flatten()])
    grad = draw(rng, flat.numel(), dtype=DT[dt]).cuda()
    flat.backward(grad)
    torch.cuda.synchronize()
    gq, gk, gv = (f64(g) for g in grad[3:].split([B * T * h * d for h in (Hq, Hk, Hk)]))
    got = f64(x.grad)
    pos = np.tile(np.arange(T), (B, 1))
    for i, (name, t, g, H, at) in enumerate((("q", q, gq, Hq, 0), ("k", k, gk, Hk, Hq * d))):
        dx, dw, bx, bw = _bwd_bound(f64(t), g.reshape(B, T, H, d), f64(w[i]), pos, fr, DT[dt], 1e-6, False, True)
        assert_within("d" + name, got[..., at: at + H * d].reshape(dx.shape), dx, bx)
        assert_within(f"d{name}_weight", w[i].grad, dw, bw)
    assert np.array_equal(got[..., (Hq + Hk) * d: -8].ravel(), gv) and not got[..., -8:].any()


def test_second_derivatives_are_refused():
    import gated_delta_rule_36_amd as G
    q, k, pos, w, rng = _case(15, 1, 3, 2, 2, 64, 64, "fp32")
    fr = torch.from_numpy(inv_freq(64)).cuda()
    q.requires_grad_()
    (g,) = torch.autograd.grad(G.qk_norm_rope(q, k, fr)[0].sum(), q, create_graph=True)
    with pytest.raises(RuntimeError):
        g.square().sum().backward()


def test_capture_and_replay():
    """Forward and backward in one graph, replayed on new inputs."""
    import gated_delta_rule_36_amd as G
    q, k, pos, w, rng = _case(14, 2, 50, 4, 2, 128, 128, "bf16")
    gq, gk = draw(rng, *q.shape).cuda(), draw(rng, *k.shape).cuda()
    fr = torch.from_numpy(inv_freq(128)).cuda()
    say("qk_norm_rope capture")

    def both():
        return (*G.qk_norm_rope_fwd(q, k, fr, q_weight=w[0], k_weight=w[1]),
                *G.qk_norm_rope_bwd(q, k, gq, gk, fr, q_weight=w[0], k_weight=w[1]))

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for seed in range(3):
        r = np.random.default_rng(seed)
        q.copy_(draw(r, *q.shape))
        gk.copy_(draw(r, *gk.shape))
        ref = both()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, ref))
