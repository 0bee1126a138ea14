"""Host-only checks of the entry points around the mixer: every refusal of the C ABI, before anything
is launched, and of the binding."""
import math
import os

import pytest
import torch

from gated_delta_rule_36_amd import _lib, _stack

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.lib_path()),
                                reason="libgdn2.so not built (run __graft_entry__.build())")

F = 0x100000    # 16-byte aligned, never dereferenced on error paths
M4 = 0x100004   # 4-byte aligned
M2 = 0x100002


def _rec(what, **kw):
    a = dict(v=F, g=F, w=F, s0=F, o=F, sN=F, st=F, cu=None, do=F, ds=F, dv=F, dg=F, dw=F, d0=F, B=2, T=8, D=64, N=2, ws_=F, wsz=1 << 30,
             vs=64, gs=64, ws=64, dtype=0, pool=F, idx=None, com=None, steps=None, L=3, P=2)
    a.update(kw)
    L = _lib.lib()
    tail = [a["vs"], a["gs"], a["ws"], a["dtype"], a["ws_"], a["wsz"], None]
    if what == "fwd":
        return L.gdn2_linear_recurrence(a["v"], a["g"], a["w"], a["s0"], a["o"], a["sN"], a["st"], a["cu"], a["B"],
                                        a["T"], a["D"], a["N"], *tail)
    if what == "bwd":
        return L.gdn2_linear_recurrence_bwd(a["v"], a["g"], a["w"], a["st"], a["do"], a["ds"], a["dv"], a["dg"], a["dw"],
                                            a["d0"], a["cu"], a["B"], a["T"], a["D"], a["N"], *tail)
    return L.gdn2_linear_recurrence_tokens(a["v"], a["g"], a["w"], a["pool"], a["idx"], a["com"], a["o"], a["steps"],
                                           a["N"], a["L"], a["D"], a["P"], *tail[:4], None)


@pytest.mark.parametrize("what", ["fwd", "bwd", "tokens"])
def test_recurrence_refusals(what):
    bad = [(1, dict(dtype=2)), (1, dict(dtype=-1)), (1, dict(N=-1)), (1, dict(D=0)), (1, dict(D=-8)), (2, dict(D=60)),
           (1, dict(vs=56)), (1, dict(gs=68)), (1, dict(ws=0)), (1, dict(vs=(1 << 21) + 8)), (1, dict(ws=1 << 32)), (1, dict(v=None)), (1, dict(g=None)), (1, dict(v=M4)),
           (1, dict(w=M4))]
    if what == "tokens":
        bad += [(1, dict(pool=None)), (1, dict(pool=M4)), (1, dict(o=None)), (1, dict(o=M4)), (1, dict(L=-1)), (1, dict(P=1)),
                (1, dict(P=-1)), (1, dict(idx=M2)), (1, dict(com=M2)), (1, dict(steps=M4)), (1, dict(N=1 << 16, L=1 << 16, P=1 << 16))]
    else:
        bad += [(1, dict(N=3)), (1, dict(B=-1, N=-1)), (1, dict(T=-1)), (1, dict(cu=F)), (1, dict(cu=M2, B=1)),
                (1, dict(B=1 << 16, N=1 << 16, T=1 << 16)), (1, dict(B=1 << 23, N=1 << 23, T=1)),
                (1, dict(cu=F, B=1, N=(1 << 31) - 1, T=1000))]
    if what == "fwd":
        bad += [(1, dict(o=None, st=None)), (1, dict(o=M4)), (1, dict(s0=M4)), (1, dict(sN=M4)), (1, dict(st=M4))]
    if what == "bwd":
        bad += [(1, dict(st=None)), (1, dict(do=None)), (1, dict(dv=None)), (1, dict(dg=M4)), (1, dict(dw=None)),
                (1, dict(ds=M4)), (1, dict(d0=M4)), (1, dict(st=M4))]
    for status, kw in bad:
        assert _rec(what, **kw) == status, kw
    none = dict(v=None, g=None, w=None, o=None, st=None, do=None, dv=None, dg=None, dw=None, pool=None, s0=None, sN=None,
                ds=None, d0=None)
    assert _rec(what, B=0, N=0, T=0, **none) == 0
    if what == "tokens":
        assert _rec(what, L=0, **none) == 0


@pytest.mark.parametrize("what", ["fwd", "bwd"])
def test_recurrence_workspace(what):
    """One long sequence of few channels is cut into segments, which need room for their maps; many
    sequences, short ones, none are not."""
    back = what == "bwd"
    ask = lambda *a: _lib.lib().gdn2_linear_recurrence_workspace_bytes(back, *a)  # noqa: E731
    strip = 2 * 64 * 4 + 4  # a map and a count
    need = ask(0, 1, 5000, 64, 1)
    assert need == 20 * strip  # 20 segments of 256 tokens
    one = dict(B=1, N=1, T=5000)
    assert _rec(what, ws_=None, **one) == 3
    assert _rec(what, wsz=need - 1, **one) == 3
    assert _rec(what, ws_=M4, **one) == 1
    assert ask(0, 1, 300, 64, 1) == ask(0, 200, 5000, 64, 200) == ask(0, 1, 5000, 64, 2) == ask(0, 1, 5000, 60, 1) == 0
    assert (ask(0, 1, 700, 64, 1) > 0) == back        # backward from 384 tokens, forward from 768
    assert (ask(0, 140, 5000, 64, 140) > 0) == back   # and up to a larger part of the card
    assert ask(1, 1, 5000, 64, 3) == (5000 // 256 + 3) * strip
    # packed batches of many sequences: one of them may be much longer than the others
    assert ask(1, 1, 200000, 64, 200) == (200000 // 896 + 200) * strip
    # a fair share of 1024 workgroups; forward, where that of 256 is 1024 tokens or more, of 256
    assert ask(0, 1, 200000, 64, 1) == -(-200000 // 256) * strip
    assert ask(0, 1, 300000, 64, 1) == -(-300000 // (384 if back else 1280)) * strip
    assert ask(0, 1, -1, 64, 1) == ask(0, 1, (1 << 31) - 1, 64, 1) == 0


def test_recurrence_states():
    ask = _lib.lib().gdn2_linear_recurrence_states_bytes
    assert ask(0, 3, 129, 64, 3) == 3 * 3 * 64 * 4
    assert ask(1, 1, 129, 64, 5) == (2 + 5) * 64 * 4
    assert ask(0, 3, 129, 60, 3) == ask(0, 3, 129, 64, 4) == ask(1, 2, 129, 64, 4) == ask(0, 3, -1, 64, 3) == 0


def _norm(bwd=False, **kw):
    a = dict(x=F, r=F, w=F, y=F, h=F, s=None, dy=F, dh=F, dx=F, dr=None, dw=F, rows=4, D=64, xs=64, rs=64, hs=64,
             group=0, eps=1e-6, dtype=0, rt=0, ws=F, wsz=1 << 30)
    a.update(kw)
    L = _lib.lib()
    if bwd:
        return L.gdn2_residual_norm_bwd(a["dy"], a["dh"], a["h"], a["w"], a["dx"], a["dr"], a["dw"], a["rows"], a["D"],
                                        a["hs"], a["eps"], a["dtype"], a["rt"], a["ws"], a["wsz"], None)
    return L.gdn2_residual_norm(a["x"], a["r"], a["w"], a["y"], a["h"], a["s"], a["rows"], a["D"], a["xs"], a["rs"],
                                a["group"], a["eps"], a["dtype"], a["rt"], None)


@pytest.mark.parametrize("bwd", [False, True])
def test_norm_refusals(bwd):
    bad = [(1, dict(dtype=3)), (1, dict(rt=2)), (2, dict(dtype=1, rt=0)), (1, dict(rows=-1)), (1, dict(rows=1 << 31)), (1, dict(rows=1 << 23)),
           (1, dict(D=0)), (2, dict(D=60)), (2, dict(D=16392, xs=16392, rs=16392, hs=16392)), (1, dict(eps=-1.0)),
           (1, dict(eps=math.nan)), (1, dict(eps=math.inf)), (1, dict(w=None)), (1, dict(w=M4)), (1, dict(h=None)), (1, dict(h=M4))]
    if bwd:
        ask = _lib.lib().gdn2_residual_norm_bwd_workspace_bytes
        need = ask(4, 64)
        assert need == 64 * 4 and ask(33, 64) == 2 * need          # 32 rows a workgroup
        assert ask(7, 1000) == 7 * 1000 * 4 and ask(100000, 2048) == 512 * 2048 * 4
        assert _lib.lib().gdn2_residual_norm_bwd_workspace_bytes(4, 60) == 0
        assert _lib.lib().gdn2_residual_norm_bwd_workspace_bytes(0, 64) == 0
        bad += [(1, dict(hs=60)), (1, dict(dy=None)), (1, dict(dx=None)), (1, dict(dw=None)), (1, dict(dh=M4)), (1, dict(dr=F)),
                (1, dict(rt=1)), (3, dict(ws=None)), (3, dict(wsz=need - 1)), (1, dict(ws=M4))]
    else:
        bad += [(1, dict(xs=60)), (1, dict(xs=56)), (1, dict(rs=68)), (1, dict(x=None)), (1, dict(y=None)), (1, dict(y=M4)),
                (1, dict(r=M4)), (1, dict(group=32)), (1, dict(s=F, group=-1)), (2, dict(s=F, group=16)),
                (1, dict(s=F, group=128)), (1, dict(s=M2)), (1, dict(r=None, rt=1))]
    for status, kw in bad:
        assert _norm(bwd, **kw) == status, kw
    assert _norm(bwd, rows=0, x=None, r=None, y=None, h=None, dy=None, dx=None, dw=None) == 0


def _verify(**kw):
    a = dict(p=F, q=F, x=F, dl=F, u=F, t=F, c=F, N=2, L=3, V=100, dtype=1, ws=F, wsz=1 << 30)
    a.update(kw)
    return _lib.lib().gdn2_verify_drafts(a["p"], a["q"], a["x"], a["dl"], a["u"], a["t"], a["c"], a["N"], a["L"], a["V"],
                                         a["dtype"], a["ws"], a["wsz"], None)


def test_verify_refusals():
    need = _lib.lib().gdn2_verify_drafts_workspace_bytes(2, 100)
    assert need == 2 * 16 and _lib.lib().gdn2_verify_drafts_workspace_bytes(2, 4097) == 2 * need
    assert _lib.lib().gdn2_verify_drafts_workspace_bytes(0, 100) == _lib.lib().gdn2_verify_drafts_workspace_bytes(2, 0) == 0
    for status, kw in [(1, dict(dtype=2)), (1, dict(N=-1)), (1, dict(L=-1)), (1, dict(V=0)), (1, dict(V=(1 << 28) + 1)),
                       (1, dict(L=(1 << 20) + 1)), (1, dict(p=None)), (1, dict(x=None)), (1, dict(u=None)), (1, dict(t=None)),
                       (1, dict(c=None)), (1, dict(p=M2)), (1, dict(q=M2)), (1, dict(dtype=0, p=0x100001)), (1, dict(x=M2)),
                       (1, dict(dl=M2)), (1, dict(u=M2)), (1, dict(t=M2)), (1, dict(c=M2)), (1, dict(ws=M4)),
                       (3, dict(ws=None)), (3, dict(wsz=need - 1)), (1, dict(N=1 << 20, V=1 << 28)), (1, dict(N=1 << 23))]:
        assert _verify(**kw) == status, kw
    assert _verify(N=0, p=None, q=None, x=None, u=None, t=None, c=None, ws=None) == 0


# ---------------------------------------------------------------- the binding

@pytest.fixture
def anywhere(monkeypatch):
    """The binding's checks on host tensors; a call that passes them all fails the test."""
    monkeypatch.setattr(_stack, "_need_gpu", lambda t: None)

    class Reached(Exception):
        pass

    def reached(*a):
        raise Reached

    monkeypatch.setattr(_stack, "_call", reached)
    return Reached


def test_host_tensors_are_refused():
    import gated_delta_rule_36_amd as G
    x = torch.zeros(1, 2, 64)
    for call in (lambda: G.linear_recurrence_fwd(x, x), lambda: G.linear_recurrence_tokens(x, x, None, x[0]),
                 lambda: G.residual_norm_fwd(x, x, x[0, 0]), lambda: G.residual_norm_bwd(x, x, x, x[0, 0]),
                 lambda: G.verify_drafts(x, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 2))):
        with pytest.raises(ValueError, match="HIP device"):
            call()


def test_recurrence_binding_refusals(anywhere):
    import gated_delta_rule_36_amd as G
    v = torch.zeros(2, 5, 64, dtype=torch.bfloat16)
    one, cu = v.view(1, 10, 64), torch.tensor([0, 4, 10], dtype=torch.int32)
    s0 = torch.zeros(2, 64)
    wide = torch.zeros(2, 5, 200, dtype=torch.bfloat16)
    for args, kw in [((v, v), {}), ((v, v, v), dict(initial_state=s0)), ((one, one), dict(cu_seqlens=cu, initial_state=s0)),
                     ((wide[..., :64], wide[..., 64:128], wide[..., 128:192]), {}), ((v[:0], v[:0]), {})]:
        with pytest.raises(anywhere):
            G.linear_recurrence_fwd(*args, **kw)
        with pytest.raises(anywhere):
            G.linear_recurrence(*args, **kw)
    for args, kw in [
        ((v.half(), v.half()), {}), ((v, v.float()), {}), ((v[0], v[0]), {}), ((v, v[:1]), {}), ((v, v, v[..., :32]), {}),
        ((v[..., :60], v[..., :60]), {}), ((v.transpose(1, 2), v.transpose(1, 2)), {}), ((v[:, ::2], v[:, ::2]), {}),
        ((wide[..., 1:65][..., ::1][:, :, :64], v.transpose(0, 1).contiguous().transpose(0, 1)), {}),
        ((torch.zeros(2, 5, 68, dtype=torch.bfloat16)[..., :64], v), {}),
        ((v, v), dict(initial_state=s0[:1])), ((v, v), dict(initial_state=s0.double())), ((v, v), dict(cu_seqlens=cu)),
        ((one, one), dict(cu_seqlens=cu.long())), ((one, one), dict(cu_seqlens=cu[None])),
        ((one, one), dict(cu_seqlens=cu[:0])), ((one, one), dict(cu_seqlens=torch.zeros(6, dtype=torch.int32)[::2])),
    ]:
        with pytest.raises((ValueError, TypeError)):
            G.linear_recurrence_fwd(*args, **kw)
    states = torch.zeros(2, 64)
    with pytest.raises(anywhere):
        G.linear_recurrence_bwd(v, v, v, states, v, d_final_state=s0)
    for args, kw in [((v, v, v, states[:1], v), {}), ((v, v, v, states.bfloat16(), v), {}), ((v, v, v, states, v.float()), {}),
                     ((v, v, v, states, wide[..., :64]), {}), ((v, v, v, states, v), dict(d_final_state=s0[:1]))]:
        with pytest.raises((ValueError, TypeError)):
            G.linear_recurrence_bwd(*args, **kw)


def test_row_strides():
    """Rows of a tensor's last axis at one stride, whatever the axes in front are."""
    x = torch.zeros(4, 3, 5, 64)
    for t, step in [(x, 64), (x[..., :32], 64), (x[:, :, :1], 320), (x[:, :1, :1, 8:24], 960), (x[2, 1, 3, 8:16], 8),
                    (x[:1, :1, :1, :40], 40), (x.transpose(0, 1)[:, :1], 64), (x[1:3, :, :, 32:], 64)]:
        assert _stack._row_stride("x", t) == step, (t.shape, t.stride())
    for t in (x.transpose(0, 1), x[:, :, ::2, :32], x[:, ::2], x[..., ::2], x.expand(4, 3, 5, 64).transpose(-1, -2),
              torch.zeros(2, 1, 64).expand(2, 3, 64), torch.zeros(3, 68)[:, :64], torch.zeros(4, 32).as_strided((3, 32), (16, 1))):
        with pytest.raises(ValueError):
            _stack._row_stride("x", t)


def test_recurrence_tokens_binding_refusals(anywhere):
    import gated_delta_rule_36_amd as G
    v, pool, n = torch.zeros(3, 2, 64), torch.zeros(4, 64), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(anywhere):
        G.linear_recurrence_tokens(v, v, None, pool, state_indices=n, commit_len=n, return_step_states=True)
    for args, kw in [((v.half(), v.half(), None, pool), {}), ((v[0], v[0], None, pool), {}), ((v, v[:1], None, pool), {}),
                     ((v, v, v.bfloat16(), pool), {}), ((v, v, None, pool[0]), {}), ((v, v, None, pool[:, :32]), {}),
                     ((v, v, None, pool.bfloat16()), {}), ((v, v, None, pool[:2]), {}),
                     ((v, v, None, pool), dict(state_indices=n.long())), ((v, v, None, pool), dict(state_indices=n[:2])),
                     ((v, v, None, pool), dict(commit_len=n.float())), ((v, v, None, pool), dict(commit_len=n[None]))]:
        with pytest.raises((ValueError, TypeError)):
            G.linear_recurrence_tokens(*args, **kw)


def test_norm_binding_refusals(anywhere):
    import gated_delta_rule_36_amd as G
    x, w = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.ones(64)
    for args in [(x, x, w), (x, None, w), (x, x.float(), w), (x.float(), x.float(), w), (x[0, 0], x[0, 0], w),
                 (torch.zeros(3, 2, 72, dtype=torch.bfloat16)[..., :64], x, w)]:
        with pytest.raises(anywhere):
            G.residual_norm_fwd(*args)
        with pytest.raises(anywhere):
            G.residual_norm(*args)
        for group in (0, 32, 64):
            with pytest.raises(anywhere):
                G.residual_norm_8bit(*args, group=group)
    for args, kw in [((x.half(), x.half(), w), {}), ((x.float(), x, w), {}), ((x, x[:1], w), {}), ((x, x, w[:32]), {}),
                     ((x, x, w.bfloat16()), {}), ((x[..., :60], x[..., :60], w[:60]), {}), ((x.transpose(1, 2), x, w), {}),
                     ((x[:, :, ::2], x[:, :, ::2], w[:32]), {}), ((torch.zeros(3, 2, 68, dtype=torch.bfloat16)[..., :64], x, w), {}),
                     ((torch.zeros(4, 16392), torch.zeros(4, 16392), torch.ones(16392)), {}),
                     ((x, x, w), dict(out=(x, x[:1]))), ((x, x, w), dict(out=(x.float(), x))), ((x, None, w), dict(out=(x, w)))]:
        with pytest.raises((ValueError, TypeError)):
            G.residual_norm_fwd(*args, **kw)
    for group in (16, 128, -32, 8):
        with pytest.raises(ValueError):
            G.residual_norm_8bit(x, x, w, group=group)
    with pytest.raises((ValueError, TypeError)):
        G.residual_norm_8bit(x, x, w, out=(x, x))
    with pytest.raises(anywhere):
        G.residual_norm_bwd(x, x.float(), x.float(), w)
    for args in [(x.float(), x, x, w), (x[:1], x, x, w), (x, x[:1], x, w), (x, x.float(), x, w), (x.transpose(0, 1), x, x, w)]:
        with pytest.raises((ValueError, TypeError)):
            G.residual_norm_bwd(*args)


def test_norm_in_place_under_autograd_is_refused(anywhere):
    import gated_delta_rule_36_amd as G
    leaf = torch.zeros(2, 64, requires_grad=True)
    h, w = leaf * 1, torch.ones(64)
    with pytest.raises(ValueError, match="gradients"):
        G.residual_norm_fwd(h, h, w, out=(torch.empty(2, 64), h))
    with torch.no_grad(), pytest.raises(anywhere):
        G.residual_norm_fwd(h, h, w, out=(torch.empty(2, 64), h))


def test_verify_binding_refusals(anywhere):
    import gated_delta_rule_36_amd as G
    p, x, u = torch.zeros(2, 4, 33), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 4)
    q, dl = p[:, :3].contiguous(), torch.zeros(2, dtype=torch.int32)
    for kw in (dict(), dict(draft_probs=q, draft_len=dl), dict(workspace=torch.zeros(64, dtype=torch.uint8))):
        with pytest.raises(anywhere):
            G.verify_drafts(p, x, u, **kw)
    for args, kw in [((p[0], x, u), {}), ((p, x[0], u), {}), ((p[:, :3], x, u), {}), ((p.double(), x, u), {}), ((p, x.long(), u), {}),
                     ((p, x, u[:, :3]), {}), ((p, x, u.double()), {}), ((p.transpose(0, 1), x, u), {}), ((p[..., :0], x, u), {}),
                     ((p, x, u), dict(draft_probs=q.bfloat16())), ((p, x, u), dict(draft_probs=p)), ((p, x, u), dict(draft_probs=p[:, :3])),
                     ((p, x, u), dict(draft_len=dl.long())), ((p, x, u), dict(draft_len=dl[:1])), ((p, x, u), dict(workspace=u))]:
        with pytest.raises((ValueError, TypeError)):
            G.verify_drafts(*args, **kw)


@pytest.mark.parametrize("shift", [0, 3, 5])
def test_gradients_at_any_offset(monkeypatch, shift):
    """Autograd's gradients may be views that start anywhere: the entry points get them contiguous
    and aligned, with their values."""
    import gated_delta_rule_36_amd as G
    held = {}
    monkeypatch.setattr(_stack, "_need_gpu", lambda t: None)
    monkeypatch.setattr(_stack, "_call", lambda *a: None)
    real = {n: getattr(_stack, n) for n in ("_recurrence_bwd", "_norm_bwd")}

    def rec(v, g, w, states, do, d_last, *rest):
        held.update(a=do, b=d_last)
        return real["_recurrence_bwd"](v, g, w, states, do, d_last, *rest)

    def norm(dy, dh, h, w, eps):
        held.update(a=dy, b=dh)
        return real["_norm_bwd"](dy, dh, h, w, eps)

    monkeypatch.setattr(_stack, "_recurrence_bwd", rec)
    monkeypatch.setattr(_stack, "_norm_bwd", norm)
    x = torch.zeros(1, 3, 64, requires_grad=True)
    for pair in (G.linear_recurrence(x, x), G.residual_norm(x, x * 1, torch.ones(64))):
        flat = torch.cat([torch.zeros(shift), pair[0].flatten(), pair[1].flatten()])
        grad = torch.arange(flat.numel(), dtype=torch.float32)
        flat.backward(grad)
        for t, at in ((held["a"], shift), (held["b"], shift + pair[0].numel())):
            assert t.is_contiguous() and t.data_ptr() % 16 == 0
            assert torch.equal(t.flatten(), grad[at:at + t.numel()])


def test_missing_gradients_are_zeros(monkeypatch):
    """An output that the loss does not use reaches the entry points as zeros or as nothing."""
    import gated_delta_rule_36_amd as G
    seen = []
    monkeypatch.setattr(_stack, "_need_gpu", lambda t: None)
    monkeypatch.setattr(_stack, "_call", lambda name, dev, *a: seen.append((name, a)))
    x = torch.zeros(1, 3, 64, requires_grad=True)
    G.linear_recurrence(x, x)[0].sum().backward()
    assert seen[-1][0].endswith("bwd") and seen[-1][1][5] is None
    G.linear_recurrence(x, x)[1].sum().backward()
    assert seen[-1][0].endswith("bwd") and seen[-1][1][5] is not None
    G.residual_norm(x, x * 1, torch.ones(64))[0].sum().backward()
    assert seen[-1][0].endswith("bwd") and seen[-1][1][1] is None
    G.residual_norm(x, None, torch.ones(64))[0].sum().backward()
    assert seen[-1][0].endswith("bwd") and seen[-1][1][1] is None
