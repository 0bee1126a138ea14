"""The operators around the mixer together, as a hybrid stack uses them: two layers trained through
autograd, and drafted tokens verified and committed to the states of both kinds of layer."""
import numpy as np
import pytest
import torch

from oracle import gdn2_decode_tokens
from oracle import gdn2_stack as R
from tests.attn_util import f64
from tests.gpu_util import TOL, assert_close, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _stack_ref(x, h, wv, wg, ww, weights, cu, dtype):
    """The two layers in float64, with the roundings of what is stored."""
    for k in range(2):
        h = h + x
        n = R.norm(h, weights[k], 1e-6)
        g = -np.logaddexp(0, n @ wg[k])
        x, _ = R.recurrence(n @ wv[k], g, 1 / (1 + np.exp(-(n @ ww[k]))), None, cu)
    return x, h


def test_two_layers_train():
    """norm -> projections -> recurrence, twice, in fp32: the loss and its gradients by differences of
    the float64 stack."""
    import gated_delta_rule_36_amd as G
    rng = np.random.default_rng(1)
    T, D = 40, 32
    cu = np.array([0, 13, 13, 40], np.int32)
    t = lambda a: torch.from_numpy(a.astype(np.float32)).cuda().requires_grad_()  # noqa: E731
    x, h = rng.standard_normal((1, T, D)), rng.standard_normal((1, T, D))
    wv, wg, ww = (0.3 * rng.standard_normal((2, D, D)) for _ in range(3))
    weights = 1 + 0.2 * rng.standard_normal((2, D))
    mix = rng.standard_normal((1, T, D))
    leaves = dict(x=t(x), h=t(h), wv=t(wv), wg=t(wg), ww=t(ww), weights=t(weights))
    say("two layers of norm and recurrence, autograd")
    a, s = leaves["x"], leaves["h"]
    for k in range(2):
        n, s = G.residual_norm(a, s, leaves["weights"][k])
        g = -torch.nn.functional.softplus(n @ leaves["wg"][k])
        a, _ = G.linear_recurrence(n @ leaves["wv"][k], g, torch.sigmoid(n @ leaves["ww"][k]), cu_seqlens=torch.from_numpy(cu).cuda())
    loss = ((a + 0.5 * s) * torch.from_numpy(mix).float().cuda()).sum()
    loss.backward()
    torch.cuda.synchronize()
    names = list(leaves)
    exact = {n: f64(leaves[n]) for n in names}

    def f(args):
        y, st = _stack_ref(args["x"], args["h"], args["wv"], args["wg"], args["ww"], args["weights"], cu, None)
        return np.sum((y + 0.5 * st) * mix)

    size = np.abs(f64(a)).mean() * a.numel()
    assert abs(float(loss.detach()) - f(exact)) < 1e-4 * size
    for name in names:
        grad, val = f64(leaves[name].grad), exact[name]
        for _ in range(3):  # along random directions
            d = rng.standard_normal(val.shape)
            up, down = (f({**exact, name: val + e * d}) for e in (1e-5, -1e-5))
            got, ref = float(np.sum(grad * d)), (up - down) / 2e-5
            # fp32 through two layers, about 10 products deep: 1e-4 of the gradient's length along d
            assert abs(got - ref) < 1e-4 * np.linalg.norm(grad) * np.linalg.norm(d), name


def test_drafts_verified_and_committed():
    """The last token and 3 drafts through a mixer layer and a recurrent layer without committing, the
    verification, then the commit: states after the accepted tokens and no others."""
    import gated_delta_rule_36_amd as G
    rng = np.random.default_rng(2)
    N, L, H, d, D, V, P = 5, 4, 2, 64, 128, 700, 7
    names = ("q", "k", "v", "g", "b", "w")
    m = {n: rng.standard_normal((N, L, H, d)).astype(np.float32) * 0.3 for n in names}
    m["g"], m["b"], m["w"] = -np.abs(m["g"]), 1 / (1 + np.exp(-m["b"])), 1 / (1 + np.exp(-m["w"]))
    r = {n: rng.standard_normal((N, L, D)).astype(np.float32) for n in "vg"}
    r["g"] = -np.abs(r["g"])
    mp, rp = (0.1 * rng.standard_normal((P, H, d, d))).astype(np.float32), rng.standard_normal((P, D)).astype(np.float32)
    idx = rng.permutation(P)[:N].astype(np.int32)
    c = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    say("drafts through a mixer and a recurrence, verified, committed")
    mt, rt, mpool, rpool, it = {n: c(a.astype(np.float32)) for n, a in m.items()}, {n: c(a) for n, a in r.items()}, c(mp), c(rp), c(idx)
    none = torch.zeros(N, dtype=torch.int32, device="cuda")
    o, _ = G.decode_tokens(*(mt[n] for n in names), mpool, state_indices=it, commit_len=none)
    y, _ = G.linear_recurrence_tokens(rt["v"], rt["g"], None, rpool, state_indices=it, commit_len=none)
    assert torch.equal(mpool, c(mp)) and torch.equal(rpool, c(rp))
    head = c(rng.standard_normal((D, V)).astype(np.float32) * 0.2)
    hidden = y + o.flatten(2)
    n8, scale, _ = G.residual_norm_8bit(hidden, y, torch.ones(D, device="cuda"), group=32)
    read = (n8.float().unflatten(-1, (-1, 32)) * scale[..., None]).flatten(-2)
    p = torch.softmax(read @ head, -1).contiguous()
    q = torch.softmax(read[:, :L - 1] @ head + 0.5 * c(rng.standard_normal((N, L - 1, V)).astype(np.float32)), -1).contiguous()
    drafts = q.argmax(-1).to(torch.int32)
    u = c(rng.random((N, L)).astype(np.float32))
    tokens, commit = G.verify_drafts(p, drafts, u, draft_probs=q)
    G.decode_tokens(*(mt[n] for n in names), mpool, state_indices=it, commit_len=commit)
    G.linear_recurrence_tokens(rt["v"], rt["g"], None, rpool, state_indices=it, commit_len=commit)
    torch.cuda.synchronize()
    ref_t, ref_c = R.verify(f64(p), drafts.cpu().numpy(), u.cpu().numpy(), f64(q))
    assert np.array_equal(tokens.cpu().numpy(), ref_t) and np.array_equal(commit.cpu().numpy(), ref_c)
    _, _, m_after = gdn2_decode_tokens(mp, *(m[n] for n in names), indices=idx, commit=ref_c)
    _, _, r_after = R.recurrence_tokens(rp, r["v"].astype(np.float64), r["g"].astype(np.float64), None, idx, ref_c)
    assert_close("mixer states", f64(mpool), m_after, TOL["fp32"])
    assert_close("recurrent states", f64(rpool), r_after, 1e-6)
