"""GPU tests of the norm between layers with the residual's addition (forward, backward, autograd,
8-bit output) against the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import gdn2_stack as R
from tests.attn_util import assert_within, draw, f64
from tests.gpu_util import say
from tests.stack_util import TINY, U, norm_bound, norm_grad_bounds

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _case(seed, rows, D, dt, rt, strided=False, spread=1.0):
    rng = np.random.default_rng(seed)
    size = torch.from_numpy(np.exp(spread * rng.standard_normal((rows, 1))).astype(np.float32))
    x = (draw(rng, rows, D + 16, dtype=torch.float32) * size).to(DT[dt]).cuda()
    x = x[:, 8:8 + D] if strided else x[:, :D].contiguous()
    r = None
    if rt is not None:
        r = (draw(rng, rows, 2 * D, dtype=torch.float32) * size).to(DT[rt]).cuda()
        r = r[:, D:] if strided else r[:, :D].contiguous()
    w = torch.from_numpy((1 + 0.3 * rng.standard_normal(D)).astype(np.float32)).cuda()
    return x, r, w, rng


def _stream(x, r):
    """h as the definition stores it: the sum in fp32, rounded once to the residual's type."""
    return x.cpu() if r is None else (x.cpu().float() + r.cpu().float()).to(r.dtype)


# rows, D, x, residual, strided: one and four waves a row, every number of steps a lane, odd widths
CASES = [
    (1, 8, "bf16", "bf16", False), (3, 64, "fp32", "fp32", False), (5, 520, "bf16", "fp32", True),
    (7, 1000, "bf16", None, True), (2, 2048, "bf16", "bf16", False), (3, 2056, "fp32", "fp32", True),
    (2, 4104, "bf16", "fp32", False), (1, 8200, "bf16", "bf16", True), (2, 16384, "fp32", "fp32", False),
    (2, 16384, "bf16", "fp32", False), (1027, 64, "bf16", "bf16", True), (1025, 512, "fp32", "fp32", False),
    (1030, 520, "bf16", "fp32", False), (1024, 1032, "bf16", "bf16", False), (1029, 2048, "bf16", "fp32", True),
    (1031, 2040, "fp32", None, False),
    # several rows a wave
    (37, 56, "bf16", "bf16", True), (29, 128, "fp32", "fp32", False), (31, 104, "bf16", "fp32", True),
    (9, 256, "bf16", "fp32", False), (2050, 136, "bf16", None, True), (3, 512, "bf16", "bf16", False),
]


@pytest.mark.parametrize("case", CASES)
def test_forward(case):
    import gated_delta_rule_36_amd as G
    x, r, w, _ = _case(1, *case)
    say("residual_norm_fwd", case)
    y, h = G.residual_norm_fwd(x, r, w, eps=1e-5)
    torch.cuda.synchronize()
    ref = _stream(x, r)
    assert torch.equal(h.cpu(), ref) and (h is x if r is None else h.is_contiguous())
    assert y.dtype == x.dtype and y.is_contiguous()
    assert_within("y", y, *norm_bound(f64(ref), f64(w), 1e-5, x.dtype))


@pytest.mark.parametrize("case", CASES)
def test_backward(case):
    import gated_delta_rule_36_amd as G
    rows, D, dt, rt, strided = case
    x, r, w, rng = _case(2, *case)
    h = x if r is None else _stream(x, r).cuda()
    dy = draw(rng, rows, D, dtype=torch.float32).to(x.dtype).cuda()
    dh = None if r is None else draw(rng, rows, D, dtype=torch.float32).to(r.dtype).cuda()
    say("residual_norm_bwd", case)
    dx, dr, dw = G.residual_norm_bwd(dy, dh, h, w, eps=1e-5)
    again = G.residual_norm_bwd(dy, dh, h, w, eps=1e-5)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((dx, dr, dw), again))
    ref, bx, br, rw, bw = norm_grad_bounds(f64(dy), None if dh is None else f64(dh), f64(h), f64(w), 1e-5, x.dtype, h.dtype)
    assert dx.dtype == x.dtype and dr.dtype == h.dtype
    assert_within("dx", dx, ref, bx)
    assert_within("dr", dr, ref, br)
    assert_within("dweight", dw, rw, bw)


def test_backward_many_rows():
    """More rows than the backward's waves: each then walks several."""
    import gated_delta_rule_36_amd as G
    for rows, D, rt in ((20000, 24, "bf16"), (9000, 128, "fp32"), (5000, 200, "bf16"), (2500, 520, "bf16"), (1100, 2056, "fp32"), (600, 9000, "bf16")):
        x, r, w, rng = _case(3, rows, D, "bf16", rt)
        h, dy = _stream(x, r).cuda(), draw(rng, rows, D).cuda()
        say("residual_norm_bwd", rows, D)
        dx, dr, dw = G.residual_norm_bwd(dy, None, h, w)
        torch.cuda.synchronize()
        ref, bx, br, rw, bw = norm_grad_bounds(f64(dy), None, f64(h), f64(w), 1e-6, x.dtype, h.dtype)
        assert_within("dx", dx, ref, bx)
        assert_within("dr", dr, ref, br)
        assert_within("dweight", dw, rw, bw)


GROUPS = [(1, 32, 32), (5, 96, 32), (3, 64, 0), (7, 1000, 0), (2, 2048, 64), (4, 2048, 0), (3, 4096, 128), (2, 4224, 32),
          (1, 8192, 0), (1, 16384, 64), (2, 128, 128), (67, 64, 64), (70, 64, 0), (41, 128, 32), (18, 256, 0), (33, 256, 128), (1030, 512, 32), (1026, 1024, 0), (1025, 1920, 128), (1024, 520, 0)]


@pytest.mark.parametrize("dt,rt", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32"), ("bf16", None)])
@pytest.mark.parametrize("rows,D,group", GROUPS)
def test_8bit(rows, D, group, dt, rt):
    import gated_delta_rule_36_amd as G
    x, r, w, _ = _case(4, rows, D, dt, rt, spread=3.0)
    say("residual_norm_8bit", rows, D, group, dt, rt)
    codes, scale, h = G.residual_norm_8bit(x, r, w, group=group)
    torch.cuda.synchronize()
    ref = _stream(x, r)
    assert torch.equal(h.cpu(), ref)
    assert codes.dtype == torch.float8_e4m3fn and codes.shape == x.shape and scale.shape == (rows, D // (group or D))
    _, s, y = R.norm_8bit(f64(ref), f64(w), 1e-6, group)
    assert np.array_equal(f64(scale), s)
    wide = np.repeat(s, group or D, -1)
    # one rounding to e4m3: half a step, of normal codes 2^-4 relative, below them 2^-10; y itself 42 U
    assert_within("codes", f64(codes.float()) * wide, y, np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * wide) * (1 + 1e-6) + 42 * U * np.abs(y))


def test_8bit_scale_steps():
    """Rows whose largest value stands at 448 times a power of two, and one step of the input to
    either side: the scale steps behind it and not before."""
    import gated_delta_rule_36_amd as G
    D = 64
    h = torch.zeros(64, D)
    w = torch.ones(D)
    # one value a row: y = sqrt(D) * weight = 8 w exactly but for eps, here zero: w at 3.5 2^k borders
    for i in range(64):
        h[i, i] = 2.0 ** (i % 5 - 2)
    base = torch.tensor([3.5 * 2.0 ** (i % 7 - 3) for i in range(D)])
    for step in (-1, 0, 1):
        w = base if step == 0 else torch.nextafter(base, torch.full_like(base, float("inf") * step))
        say("residual_norm_8bit scale at its border", step)
        codes, scale, _ = G.residual_norm_8bit(h.cuda(), None, w.cuda(), eps=0.0)
        torch.cuda.synchronize()
        ref, s, _ = R.norm_8bit(f64(h), f64(w), 0.0, 0)
        assert np.array_equal(f64(scale), s)
        assert np.array_equal(f64(codes.float()), ref)


def test_empty_zero_and_bad_rows():
    import gated_delta_rule_36_amd as G
    x, r, w, rng = _case(5, 6, 96, "bf16", "bf16")
    say("residual_norm zero, NaN and infinite rows")
    good = G.residual_norm_8bit(x, r, w, group=32) + G.residual_norm_fwd(x, r, w)[:1]
    x2 = x.clone()
    x2[0], r[0] = 0, 0
    x2[2, 5], x2[4, 90] = float("nan"), float("inf")
    got = G.residual_norm_8bit(x2, r, w, group=32) + G.residual_norm_fwd(x2, r, w)[:1]
    dy = draw(rng, 6, 96).cuda()
    dx, _, dw = G.residual_norm_bwd(dy, None, got[2], w)
    torch.cuda.synchronize()
    for a, b in zip(got, good):
        for i in (1, 3, 5):
            assert torch.equal(a[i].float(), b[i].float())
    assert not got[0][0].float().any() and (got[1][0] == 2.0 ** -64).all() and not got[3][0].any()
    assert got[0][2].float().isnan().all() and got[3][2].isnan().all() and (got[1][2] == 2.0 ** -64).all()
    y = got[3][4].float()
    assert y[90].isnan() and not y[:90].any() and got[0][4, 90].float().isnan() and not got[0][4, :64].float().any()
    assert dx[[0, 1, 3, 5]].isfinite().all() and dx[2].isnan().all()
    e = torch.empty(0, 3, 96, device="cuda")
    y, h = G.residual_norm_fwd(e, e, w)
    assert y.shape == h.shape == e.shape
    codes, scale, _ = G.residual_norm_8bit(e, e, w, group=32)
    assert codes.shape == e.shape and scale.shape == (0, 3, 3)
    dx, dr, dw = G.residual_norm_bwd(e, e, e, w)
    assert dx.shape == e.shape and not dw.any()


def test_in_place_and_shapes():
    """The stream in place of the residual; any leading axes."""
    import gated_delta_rule_36_amd as G
    x, r, w, _ = _case(6, 24, 256, "bf16", "fp32")
    say("residual_norm_fwd in place")
    y, h = G.residual_norm_fwd(x, r, w)
    y3, h3 = G.residual_norm_fwd(x.view(2, 3, 4, 256), r.view(2, 3, 4, 256), w)
    out = torch.empty_like(y)
    got = G.residual_norm_fwd(x, r, w, out=(out, r))
    torch.cuda.synchronize()
    assert got[0] is out and got[1] is r and torch.equal(out, y) and torch.equal(r, h)
    assert torch.equal(y3.view_as(y), y) and torch.equal(h3.view_as(h), h)
    one = G.residual_norm_fwd(x[0], h[0], w)
    assert one[0].shape == (256,)


@pytest.mark.parametrize("dt,rt", [("bf16", "fp32"), ("fp32", "fp32"), ("bf16", None)])
def test_autograd(dt, rt):
    import gated_delta_rule_36_amd as G
    x, r, w, rng = _case(7, 50, 128, dt, rt)
    x, w = x.requires_grad_(), w.requires_grad_()
    if r is not None:
        r.requires_grad_()
    say("residual_norm autograd", dt, rt)
    y, h = G.residual_norm(x, r, w)
    dy, dh = draw(rng, 50, 128, dtype=y.dtype).cuda(), draw(rng, 50, 128, dtype=h.dtype).cuda()
    torch.autograd.backward((y, h), (dy, dh))
    torch.cuda.synchronize()
    ref, bx, br, rw, bw = norm_grad_bounds(f64(dy), f64(dh), f64(h), f64(w), 1e-6, x.dtype, h.dtype)
    if r is None:  # two gradients of x, each rounded, and their sum's rounding
        bx = bx + (torch.finfo(x.dtype).eps / 2) * (2 * np.abs(ref - f64(dh)) + np.abs(ref)) * 1.1
    assert_within("dx", x.grad, ref, bx)
    if r is not None:
        assert_within("dr", r.grad, ref, br)
    assert_within("dweight", w.grad, rw, bw)
    y, h = G.residual_norm(x, r, w)   # the stream alone: a sum
    x.grad = None
    if r is not None:
        h.backward(dh)
        torch.cuda.synchronize()
        assert torch.equal(x.grad, dh.to(x.dtype))
    (g,) = torch.autograd.grad(G.residual_norm(x, r, w)[0].sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.square().sum().backward()


def test_capture_and_replay():
    import gated_delta_rule_36_amd as G
    x, r, w, rng = _case(8, 1500, 264, "bf16", "fp32")
    x2, r2, w2, _ = _case(9, 9, 512, "bf16", "bf16")
    dy = draw(rng, 1500, 264).cuda()
    say("residual_norm capture")

    def all_of():
        y, h = G.residual_norm_fwd(x, r, w)
        return (y, h, *G.residual_norm_bwd(dy, h, h, w), *(t.float() for t in G.residual_norm_8bit(x2, r2, w2, group=32)))

    all_of()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = all_of()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, all_of()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = all_of()
    for seed in range(3):
        g = np.random.default_rng(seed)
        x.copy_(draw(g, *x.shape))
        x2.copy_(draw(g, *x2.shape))
        dy.copy_(draw(g, *dy.shape))
        ref = all_of()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, ref))


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows, which alone have a gradient."""
    import gated_delta_rule_36_amd as G
    rows, D, n = 530000, 4096, 50
    say("residual_norm offsets past 32 bits")
    torch.manual_seed(5)
    x, r = (torch.empty(rows, D, dtype=torch.bfloat16, device="cuda").normal_() for _ in range(2))
    w = 1 + 0.3 * torch.randn(D, device="cuda")
    y, h = G.residual_norm_fwd(x, r, w)
    codes, scale, h8 = G.residual_norm_8bit(x, r, w, group=32)
    dy = torch.zeros_like(x)
    dy[-n:].normal_()
    dx, dr, dw = G.residual_norm_bwd(dy, None, h, w)
    torch.cuda.synchronize()
    ref = _stream(x[-n:], r[-n:])
    assert torch.equal(h[-n:].cpu(), ref) and torch.equal(h8[-n:].cpu(), ref)
    assert_within("y", y[-n:], *norm_bound(f64(ref), f64(w), 1e-6, x.dtype))
    _, s, _ = R.norm_8bit(f64(ref), f64(w), 1e-6, 32)
    assert np.array_equal(f64(scale[-n:]), s)
    small = G.residual_norm_8bit(x[-n:], r[-n:], w, group=32)[0]
    assert torch.equal(codes[-n:].view(torch.uint8), small.view(torch.uint8))
    gx, bx, _, rw, bw = norm_grad_bounds(f64(dy[-n:]), None, f64(ref), f64(w), 1e-6, x.dtype, x.dtype)
    assert_within("dx", dx[-n:], gx, bx)
    assert_within("dweight", dw, rw, bw)
