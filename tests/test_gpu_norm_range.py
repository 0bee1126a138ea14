"""GPU tests of the norm between layers at the ends of its range: rows whose root mean square is near 2^-126 or
2^126, whose squares and their sums leave fp32."""
import numpy as np
import pytest
import torch

from oracle import gdn2_stack as R
from tests.attn_util import assert_within, f64
from tests.gpu_util import say
from tests.stack_util import U, norm_bound, norm_grad_bounds

pytestmark = pytest.mark.gpu
TYPES = [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float32, torch.float32), (torch.bfloat16, None)]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# a power of two that every value is multiplied by, and eps (0: the rows' own sizes count)
SIZES = [(124, 1e-6), (63, 1e-6), (58, 0.0), (-63, 0.0), (-75, 0.0), (-120, 0.0), (-75, 2.0 ** -149)]


def _case(rows, D, dt, rt, size, seed):
    """Values of a mean square near 1 and none of them small, times 2^size."""
    rng = np.random.default_rng(seed)
    h = rng.uniform(0.5, 1.4, (rows, D)) * rng.choice([-1, 1], (rows, D))
    h[0] = np.abs(h[0])  # whole rows of one sign
    x = torch.from_numpy(h * 2.0 ** size).to(dt)
    r = None
    if rt is not None:
        r = (0.5 * x.double()).to(rt)
        x = (0.5 * x.double()).to(dt)
    w = torch.from_numpy((1 + 0.3 * rng.standard_normal(D)).astype(np.float32))
    h = x if r is None else (x.float() + r.float()).to(r.dtype)
    return x.cuda(), None if r is None else r.cuda(), w.cuda(), h, rng


@pytest.mark.parametrize("size,eps", SIZES)
@pytest.mark.parametrize("dt,rt", TYPES)
@pytest.mark.parametrize("rows,D", [(3, 64), (5, 520), (2, 2048), (1025, 1024), (3, 4096), (2, 16384)])
def test_forward(rows, D, dt, rt, size, eps):
    import gated_delta_rule_36_amd as G
    x, r, w, h, _ = _case(rows, D, dt, rt, size, rows + D)
    say("residual_norm range", rows, D, dt, rt, size, eps)
    y, got = G.residual_norm_fwd(x, r, w, eps=eps)
    codes, scale, got8 = G.residual_norm_8bit(x, r, w, eps=eps)
    torch.cuda.synchronize()
    assert torch.equal(got.cpu(), h) and torch.equal(got8.cpu(), h)
    e = float(np.float32(eps))
    assert_within("y", y, *norm_bound(f64(h), f64(w), e, dt))
    _, s, ref = R.norm_8bit(f64(h), f64(w), e, 0)
    assert np.array_equal(f64(scale), s)
    # one rounding to e4m3 (half a step: 2^-4 relative, below normal codes 2^-10), y itself 42 U
    bound = np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * s) * (1 + 1e-6) + 42 * U * np.abs(ref)
    assert_within("codes", f64(codes.float()) * s, ref, bound)


@pytest.mark.parametrize("size,eps", SIZES)
@pytest.mark.parametrize("dt,rt", TYPES)
@pytest.mark.parametrize("rows,D", [(3, 64), (5, 520), (2, 2048), (1025, 1024), (3, 4096), (2, 16384)])
def test_backward(rows, D, dt, rt, size, eps):
    """The gradient of y of such a size that dx is of the size of 1 (2^100 at most), dh likewise."""
    import gated_delta_rule_36_amd as G
    x, r, w, h, rng = _case(rows, D, dt, rt, size, rows + D + 1)
    big = 2.0 ** min(size, 100)
    dy = torch.from_numpy(rng.standard_normal((rows, D)) * big).to(dt).cuda()
    dh = torch.from_numpy(rng.standard_normal((rows, D)) * big * 2.0 ** -size).to(h.dtype).cuda()
    say("residual_norm_bwd range", rows, D, dt, rt, size, eps)
    for g in (dh, None):
        dx, dr, dw = G.residual_norm_bwd(dy, g, h.cuda(), w, eps=eps)
        torch.cuda.synchronize()
        ref, bx, br, rw, bw = norm_grad_bounds(f64(dy), None if g is None else f64(g), f64(h), f64(w), float(np.float32(eps)), dt, h.dtype)
        assert_within("dx", dx, ref, bx)
        assert_within("dr", dr, ref, br)
        assert_within("dweight", dw, rw, bw)


def test_small_gradients_of_large_rows():
    """Rows of a size that fp32 squares, gradients whose products with them fp32 does not hold."""
    import gated_delta_rule_36_amd as G
    for size, grad in ((40, 100), (-40, -100), (0, -120), (20, -120)):
        _, _, w, h, rng = _case(3, 2048, torch.float32, None, size, 9)
        dy = torch.from_numpy(rng.standard_normal((3, 2048)) * 2.0 ** grad).float().cuda()
        say("residual_norm_bwd", size, grad)
        dx, dr, dw = G.residual_norm_bwd(dy, None, h.cuda(), w, eps=0.0)
        torch.cuda.synchronize()
        ref, bx, br, rw, bw = norm_grad_bounds(f64(dy), None, f64(h), f64(w), 0.0, torch.float32, torch.float32)
        assert_within("dx", dx, ref, bx)
        assert_within("dweight", dw, rw, bw)
