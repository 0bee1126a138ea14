"""GPU tests of the verification of drafted tokens against the float64 oracle: equal, entry by entry."""
import numpy as np
import pytest
import torch

from oracle import gdn2_stack as R
from tests.attn_util import f64
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _case(seed, N, L, V, dt, draft="model", near=0.7, sparse=False):
    rng = np.random.default_rng(seed)
    logits = 2 * rng.standard_normal((N, L + 1, V))
    if sparse:  # a few entries hold everything
        logits[rng.random(logits.shape) > 4.0 / V] = -np.inf
        logits[..., V // 2] = np.maximum(logits[..., V // 2], 0)

    def probs(x):
        x = np.exp(x - x.max(-1, keepdims=True))
        return torch.from_numpy((x / x.sum(-1, keepdims=True)).astype(np.float32)).to(DT[dt])

    p = probs(logits)
    q = probs(logits[:, :L] + near * rng.standard_normal((N, L, V))) if L else None
    drafts = np.zeros((N, L), np.int32)
    for n in range(N):
        for i in range(L):
            c = np.cumsum(f64(q[n, i]))
            drafts[n, i] = min(np.searchsorted(c, rng.random() * c[-1], "right"), V - 1)
    u = rng.random((N, L + 1)).astype(np.float32)
    u = np.minimum(u, np.float32(1 - 2.0 ** -24))
    return p, q if draft == "model" else None, drafts, u, rng


def _check(p, q, drafts, u, draft_len=None):
    import gated_delta_rule_36_amd as G
    to = lambda x: None if x is None else (x if isinstance(x, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(x))).cuda()  # noqa: E731
    tokens, commit = G.verify_drafts(to(p), to(drafts), to(u), draft_probs=to(q), draft_len=to(draft_len))
    torch.cuda.synchronize()
    ref = R.verify(f64(p), drafts, u, None if q is None else f64(q), draft_len)
    assert np.array_equal(commit.cpu().numpy(), ref[1])
    assert np.array_equal(tokens.cpu().numpy(), ref[0])
    return ref


# vocabularies around a lane's 8 entries, a piece's 4096, and past 64 pieces; odd ones
@pytest.mark.parametrize("N,L,V,dt,draft,sparse", [
    (1, 0, 1, "fp32", "model", False), (3, 1, 7, "fp32", "model", False), (5, 4, 8, "bf16", "model", False),
    (9, 3, 257, "fp32", "model", False), (7, 2, 4096, "fp32", "none", False), (6, 5, 4097, "bf16", "model", False),
    (4, 0, 12289, "fp32", "none", False), (33, 3, 1001, "bf16", "none", False), (2, 2, 300007, "fp32", "model", False),
    (3, 1, 262145, "bf16", "none", False), (20, 7, 5003, "fp32", "model", True), (2, 1, 300001, "fp32", "model", True),
    (2, 70, 65, "fp32", "model", False), (2, 130, 9, "bf16", "none", False),
])
def test_verify(N, L, V, dt, draft, sparse):
    say("verify_drafts", N, L, V, dt, draft, sparse)
    p, q, drafts, u, rng = _case(N + V, N, L, V, dt, draft, sparse=sparse)
    _check(p, q, drafts, u)
    _check(p, q, drafts, u, rng.integers(-1, L + 2, N).astype(np.int32))


def test_long_accepted_runs():
    """Draft and target agree: everything is accepted, past the 64 drafts that a wave looks at at once."""
    say("verify_drafts 150 drafts, all accepted")
    p, _, drafts, u, _ = _case(3, 2, 150, 17, "fp32")
    ref = _check(p, p[:, :150].contiguous(), drafts % 17, u)
    assert (ref[1] == 151).all()
    u[1, 149] = 0.9999
    p[1, 149] = 0
    p[1, 149, 3] = 0.5
    q = p[:, :150].clone()
    q[1, 149, :] = 0.25
    drafts[1, 149] = 3
    assert _check(p, q, drafts, u)[1].tolist() in ([151, 151], [151, 150])


def test_borders():
    """Weights that are powers of two, draws at the borders themselves: the first entry whose sum passes
    the border, never one that holds nothing."""
    say("verify_drafts borders")
    V = 9000
    p = torch.zeros(16, 1, V)
    at = [0, 1, 15, 16, 4095, 4096, 4097, 8191, 8192, 8999]
    for k in range(16):
        for a in at[: 8]:
            p[k, 0, (a + 3 * k) % V] = 0.125
    u = np.arange(16, dtype=np.float32)[:, None] / 16
    _check(p, None, np.zeros((16, 0), np.int32), u)
    u[:] = np.float32(1 - 2.0 ** -24)
    _check(p, None, np.zeros((16, 0), np.int32), u)
    u[:] = 0
    _check(p, None, np.zeros((16, 0), np.int32), u)
    u[:] = 1.0  # past the range: the last entry that holds anything
    _check(p, None, np.zeros((16, 0), np.int32), u)


def test_edges():
    """Empty rows, rows where the draft covers the target, drafts that do not exist, values that are
    no probabilities."""
    say("verify_drafts edges")
    p, q, drafts, u, _ = _case(5, 8, 2, 5000, "fp32")
    p[0] = 0                                  # nothing anywhere
    q[1] = 1.0                                # larger than p everywhere: the draw is from p
    drafts[2, 0], drafts[3, 0] = -1, 5000
    p[4, 0, 10:2000] = float("nan")
    q[5, 0, :100] = float("nan")
    p[6, 0, 7] = -0.5
    q[7, 0] = 0
    u[1] = 0.75
    ref = _check(p, q, drafts, u)
    assert ref[0][0].tolist() == [-1, -1, -1] and ref[1][0] == 1
    _check(p, None, drafts, u)
    p[4, 1, 4999] = float("inf")              # stays in range
    import gated_delta_rule_36_amd as G
    t, c = G.verify_drafts(p.cuda(), torch.from_numpy(drafts).cuda(), torch.from_numpy(u).cuda(), draft_probs=q.cuda())
    torch.cuda.synchronize()
    assert (t.cpu() < 5000).all() and (t.cpu() >= -1).all() and (c.cpu() >= 1).all() and (c.cpu() <= 3).all()
    empty = G.verify_drafts(p[:0].cuda(), torch.zeros(0, 2, dtype=torch.int32, device="cuda"), torch.zeros(0, 3, device="cuda"))
    assert empty[0].shape == (0, 3) and empty[1].shape == (0,)


def test_many_sequences():
    say("verify_drafts 70000 sequences")
    N, V = 70000, 5
    rng = np.random.default_rng(6)
    p = torch.from_numpy(rng.random((N, 2, V)).astype(np.float32))
    q = torch.from_numpy(rng.random((N, 1, V)).astype(np.float32))
    _check(p, q, rng.integers(0, V, (N, 1)).astype(np.int32), rng.random((N, 2)).astype(np.float32))


def test_workspace_stream_capture():
    """A workspace of the caller's, shared by calls in a row; a side stream; a captured call replayed
    on new inputs."""
    import gated_delta_rule_36_amd as G
    p, q, drafts, u, _ = _case(7, 6, 3, 9001, "fp32")
    p, q, drafts, u = p.cuda(), q.cuda(), torch.from_numpy(drafts).cuda(), torch.from_numpy(u).cuda()
    ws = torch.full((G.verify_drafts_workspace_bytes(6, 9001),), 255, dtype=torch.uint8, device="cuda")
    say("verify_drafts capture")
    ref = G.verify_drafts(p, drafts, u, draft_probs=q)
    own = G.verify_drafts(p, drafts, u, draft_probs=q, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = G.verify_drafts(p, drafts, u, draft_probs=q)
    torch.cuda.synchronize()
    for got in (own, other):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = G.verify_drafts(p, drafts, u, draft_probs=q, workspace=ws)
    for seed in range(3):
        a, b, c, d, _ = _case(20 + seed, 6, 3, 9001, "fp32")
        p.copy_(a), q.copy_(b), drafts.copy_(torch.from_numpy(c)), u.copy_(torch.from_numpy(d))
        ref = G.verify_drafts(p, drafts, u, draft_probs=q)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held[0], ref[0]) and torch.equal(held[1], ref[1])


def test_offsets_past_32_bits():
    """The widest vocabulary, 2^31 probabilities: a draft accepted and one rejected at the rows' ends; a
    sequence without drafts."""
    import gated_delta_rule_36_amd as G
    N, L, V = 2, 3, 1 << 28
    say("verify_drafts offsets past 32 bits")
    p, q = torch.zeros(N, L + 1, V, device="cuda"), torch.zeros(N, L, V, device="cuda")
    p[0, 0, V - 1] = 1
    p[1, 0, V - 3], q[1, 0, V - 3] = 0.5, 0.25
    p[1, 1, V - 5], p[1, 1, V - 2], q[1, 1, V - 5] = 0.6, 0.4, 0.6
    drafts = torch.tensor([[0, 0, 0], [V - 3, 7, 0]], dtype=torch.int32, device="cuda")
    u = torch.full((N, L + 1), 0.9, device="cuda")
    lens = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    tokens, commit = G.verify_drafts(p, drafts, u, draft_probs=q, draft_len=lens)
    torch.cuda.synchronize()
    assert tokens.tolist() == [[V - 1, -1, -1, -1], [V - 3, V - 2, -1, -1]] and commit.tolist() == [1, 2]
