"""Host-only checks of the attention layer's entry points: every refusal of the C ABI, before
anything is launched, and of the binding."""
import math
import os

import pytest
import torch

from gated_delta_rule_36_amd import _attn, _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.lib_path()),
                                reason="libgdn2.so not built (run __graft_entry__.build())")

F = 0x100000    # 16-byte aligned, never dereferenced on error paths
M4 = 0x100004   # 4-byte aligned
M2 = 0x100002


def _rope(bwd=False, **kw):
    a = dict(q=F, k=F, gq=F, gk=F, wq=F, wk=F, pos=F, fr=F, qo=F, ko=F, dwq=F, dwk=F, B=2, T=8, Hq=4, Hk=2,
             d=128, qs=512, ks=256, rot=64, eps=1e-6, flags=0, dtype=0, ws=F, wsz=1 << 30)
    a.update(kw)
    L = _lib.lib()
    size = [a[n] for n in ("B", "T", "Hq", "Hk", "d", "qs", "ks", "rot", "eps", "flags", "dtype")]
    if bwd:
        return L.gdn2_qk_norm_rope_bwd(a["q"], a["k"], a["gq"], a["gk"], a["wq"], a["wk"], a["pos"], a["fr"],
                                       a["qo"], a["ko"], a["dwq"], a["dwk"], *size, a["ws"], a["wsz"], None)
    return L.gdn2_qk_norm_rope(a["q"], a["k"], a["wq"], a["wk"], a["pos"], a["fr"], a["qo"], a["ko"], *size, None)


@pytest.mark.parametrize("bwd", [False, True])
def test_norm_rope_refusals(bwd):
    for status, bad in [
        (1, dict(dtype=2)), (1, dict(flags=4)), (1, dict(flags=-1)), (1, dict(Hq=0)), (1, dict(Hk=-1)),
        (1, dict(B=-1)), (1, dict(T=-1)), (1, dict(B=1 << 16, T=1 << 16)), (2, dict(d=96)), (2, dict(d=256)),
        (1, dict(rot=4)), (1, dict(rot=136)), (1, dict(rot=-8)), (1, dict(fr=None)), (1, dict(fr=M2)),
        (1, dict(eps=-1.0)), (1, dict(eps=math.nan)), (1, dict(eps=math.inf)),
        (1, dict(qs=511)), (1, dict(qs=504)), (1, dict(ks=252)), (1, dict(qs=516)),
        (1, dict(q=None)), (1, dict(ko=None)), (1, dict(q=M4)), (1, dict(qo=M4)), (1, dict(wq=M4)),
        (1, dict(pos=M2)),
    ]:
        assert _rope(bwd, **bad) == status, bad
    assert _rope(bwd, T=0, q=None, k=None, qo=None, ko=None, gq=None, gk=None) == 0
    assert _rope(bwd, B=0, q=None, k=None, qo=None, ko=None, gq=None, gk=None) == 0
    if bwd:
        need = _lib.lib().gdn2_qk_norm_rope_bwd_workspace_bytes(2, 8, 4, 2, 128)
        assert need == 4 * 2 * 128 * 4  # 4 groups of 4 tokens, one chunk each of q and k, fp32
        for status, bad in [(1, dict(gq=None)), (1, dict(gk=M4)), (3, dict(ws=None)), (3, dict(wsz=need - 1)),
                            (1, dict(ws=M4)), (1, dict(dwq=M2)), (3, dict(ws=None, dwk=None))]:
            assert _rope(True, **bad) == status, bad
        assert _lib.lib().gdn2_qk_norm_rope_bwd_workspace_bytes(2, 8, 4, 2, 96) == 0
        assert _lib.lib().gdn2_qk_norm_rope_bwd_workspace_bytes(2, 0, 4, 2, 64) == 0


def _serve(attention, **kw):
    a = dict(q=F, k=F, v=F, wq=F, wk=F, fr=F, o=F, kc=F, vc=F, ks=F, vs=F, bt=F, sl=F, cu=None, B=2, T=1, Hq=4,
             Hk=2, d=128, N=2, P=10, MB=4, sq=512, sk=256, sv=256, rot=128, eps=1e-6, flags=0, dtype=0, window=0,
             scale=0.1, ws=F, wsz=1 << 40)
    a.update(kw)
    L = _lib.lib()
    size = [a[n] for n in ("B", "T", "Hq", "Hk", "d", "N", "P", "MB")]
    cache = [a[n] for n in ("kc", "vc", "ks", "vs", "bt", "sl", "cu")]
    if attention:
        return L.gdn2_cache_attention(a["q"], *cache, a["o"], *size, a["window"], a["scale"], a["dtype"], a["ws"],
                                      a["wsz"], None)
    return L.gdn2_attn_prologue(a["q"], a["k"], a["v"], a["wq"], a["wk"], a["fr"], a["o"], *cache, *size, a["sq"],
                                a["sk"], a["sv"], a["rot"], a["eps"], a["flags"], a["dtype"], None)


COMMON = [
    (1, dict(dtype=5)), (2, dict(dtype=1)), (2, dict(d=96)), (1, dict(Hq=3)), (1, dict(Hk=0)), (1, dict(Hq=-4)),
    (1, dict(N=3)), (1, dict(N=-1, B=-1)), (1, dict(T=-1)), (1, dict(cu=F)), (1, dict(cu=M2, B=1)),
    (1, dict(P=0)), (1, dict(P=-1)), (1, dict(MB=0)), (1, dict(MB=-1)), (1, dict(MB=1 << 26)),
    (1, dict(q=None)), (1, dict(q=M4)), (1, dict(o=None)), (1, dict(o=M4)), (1, dict(kc=None)), (1, dict(vc=None)),
    (1, dict(kc=M4)), (1, dict(vc=M4)), (1, dict(ks=None)), (1, dict(vs=M2)), (1, dict(bt=None)), (1, dict(bt=M2)),
    (1, dict(sl=None)), (1, dict(sl=M2)), (1, dict(B=1 << 16, N=1 << 16, T=1 << 16)),
]


@pytest.mark.parametrize("attention", [False, True])
def test_serving_refusals(attention):
    for status, bad in COMMON:
        assert _serve(attention, **bad) == status, bad
    none = dict(q=None, k=None, v=None, o=None, kc=None, vc=None, ks=None, vs=None, bt=None, sl=None)
    assert _serve(attention, T=0, **none) == 0
    assert _serve(attention, B=0, N=0, **none) == 0


def test_prologue_refusals():
    for status, bad in [(1, dict(k=None)), (1, dict(v=None)), (1, dict(v=M4)), (1, dict(sv=255)), (1, dict(sk=248)),
                        (1, dict(sq=508)), (1, dict(rot=12)), (1, dict(fr=None)), (1, dict(eps=-1.0)),
                        (1, dict(flags=8)), (1, dict(wk=M4))]:
        assert _serve(False, **bad) == status, bad


def test_attention_refusals():
    L = _lib.lib()
    for status, bad in [(1, dict(window=-1)), (1, dict(scale=0.0)), (1, dict(scale=-1.0)), (1, dict(scale=math.nan)),
                        (1, dict(scale=math.inf)), (1, dict(ws=M4))]:
        assert _serve(True, **bad) == status, bad
    # two sequences of up to 64 blocks: the key axis is cut, and needs its workspace
    need = L.gdn2_cache_attention_workspace_bytes(0, 2, 1, 4, 2, 128, 2, 64, 0)
    assert need > 0 and need % (2 * 4 * 130 * 4) == 0
    assert _serve(True, MB=64, ws=None) == 3
    assert _serve(True, MB=64, wsz=need - 1) == 3
    ask = L.gdn2_cache_attention_workspace_bytes
    assert ask(0, 2, 1, 4, 2, 128, 2, 1, 0) == 0        # one block: nothing to join
    assert ask(0, 2, 1, 4, 2, 128, 2, 1 << 10, 16) == 0  # a window of one or two blocks
    assert ask(0, 2, 1, 4, 3, 128, 2, 64, 0) == 0
    assert ask(0, 2, 1, 4, 2, 96, 2, 64, 0) == 0
    assert ask(0, 2, 1, 4, 2, 128, 3, 64, 0) == 0
    assert ask(1, 2, 1, 4, 2, 128, 3, 64, 0) == 0
    # the pieces times the rows stay bounded for very long tables
    assert ask(0, 1, 1, 16, 1, 128, 1, 1 << 20, 0) <= 260 * 16 * 130 * 4


def test_mixed_batch_workspace():
    """A packed batch over long tables needs room for its sequences of few rows as well: 16 pieces of
    4 blocks, 16 rows for each of 8 x 2 (sequence, kv head)."""
    ask = _lib.lib().gdn2_cache_attention_workspace_bytes
    row = 130 * 4
    need = ask(1, 1, 4000, 8, 2, 128, 8, 64, 0)
    assert need == 16 * 8 * 2 * 16 * row
    packed = dict(B=1, T=4000, Hq=8, N=8, MB=64, cu=F)
    assert _serve(True, ws=None, **packed) == 3
    assert _serve(True, wsz=need - 1, **packed) == 3
    more = ask(1, 1, 200, 8, 2, 128, 8, 64, 0) - need   # a few tiles: the key axis of those as well
    assert more > 0 and more % (200 * 8 * row) == 0
    assert ask(1, 1, 4000, 8, 2, 128, 8, 64, 512) == 0   # ten blocks in reach: one pass
    assert ask(1, 1, 4000, 8, 2, 128, 8, 16, 0) == 0
    # rows of a group past 32: no sequence fits the few-row kernel
    assert ask(1, 1, 4000, 80, 2, 128, 8, 64, 0) == 0
    # many sequences: one piece each
    assert ask(1, 1, 4000, 8, 2, 128, 256, 64, 0) == 0


@pytest.mark.parametrize("T,Hq,Hk,d,N,blocks,pieces,few_pieces", [
    (35, 1, 1, 128, 2, 143, 29, 36),
    (101, 3, 3, 128, 3, 254, 51, 32),
    (35, 1, 1, 64, 2, 143, 29, 36),
])
def test_mixed_batch_workspace_regions_are_aligned(T, Hq, Hk, d, N, blocks, pieces, few_pieces):
    """The two passes' partial results lie one behind the other and are read 16 bytes at a time: the
    second starts at a multiple of 16 bytes also where the first holds an odd number of rows."""
    need = _lib.lib().gdn2_cache_attention_workspace_bytes(1, 1, T, Hq, Hk, d, N, blocks, 0)
    row = (d + 2) * 4
    first, second = pieces * T * Hq * row, few_pieces * N * Hk * 16 * row
    assert first % 16 == 8 and need == first + 8 + second


def test_few_tiles_over_a_long_context_are_cut():
    """64 query rows a kv head make one tile: its key axis is cut however long it is, into pieces of
    at least 4 blocks, and the room stays bounded."""
    ask = _lib.lib().gdn2_cache_attention_workspace_bytes
    row = 130 * 4
    for blocks in (16, 65, 130, 512, 4096, 1 << 20):
        need = ask(0, 1, 8, 16, 2, 128, 1, blocks, 0)
        assert need > 0 and need % (8 * 16 * row) == 0, blocks
        assert need // (8 * 16 * row) <= min(blocks // 4 + 1, 512), blocks


# ---------------------------------------------------------------- the binding

@pytest.fixture
def anywhere(monkeypatch):
    """The binding's checks on host tensors; a call that passes them all fails the test."""
    monkeypatch.setattr(_attn, "_need_gpu", lambda t: None)

    class Reached(Exception):
        pass

    def reached(*a):
        raise Reached

    monkeypatch.setattr(_attn, "_call", reached)
    return Reached


def test_host_tensors_are_refused():
    import gated_delta_rule_36_amd as G
    x = torch.zeros(1, 2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="HIP device"):
        G.qk_norm_rope_fwd(x, x, None)
    with pytest.raises(ValueError, match="HIP device"):
        G.cache_attention(x, G.kv_cache(2, 1, 64, device="cpu"), torch.zeros(1, 1, dtype=torch.int32),
                          torch.zeros(1, dtype=torch.int32))


def test_norm_rope_binding_refusals(anywhere):
    import gated_delta_rule_36_amd as G
    q, k = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)
    fr = torch.ones(16)
    with pytest.raises(anywhere):
        G.qk_norm_rope_fwd(q, k, fr, positions=torch.zeros(2, 3, dtype=torch.int32))
    for err, args, kw in [
        (TypeError, (q.half(), k.half(), fr), {}),
        (TypeError, (q, k.float(), fr), {}),
        (ValueError, (q[0], k, fr), {}),
        (ValueError, (q, k[:1], fr), {}),
        (ValueError, (q, k[..., :32], fr), {}),
        (ValueError, (q.transpose(1, 2), k.transpose(1, 2), fr), {}),
        (ValueError, (torch.zeros(2, 3, 4, 68, dtype=torch.bfloat16)[..., :64], k, fr), {}),
        (ValueError, (torch.zeros(2, 3, 260, dtype=torch.bfloat16)[..., :256].view(2, 3, 4, 64), k, fr), {}),
        (ValueError, (q[:, ::2], k[:, ::2], fr), {}),  # batch stride no multiple of the tokens'
        (ValueError, (q, k, fr[:3]), {}),
        (ValueError, (q, k, torch.ones(40)), {}),
        (ValueError, (q, k, fr.double()), {}),
        (ValueError, (q, k, fr), dict(positions=torch.zeros(2, 3))),
        (ValueError, (q, k, fr), dict(positions=torch.zeros(2, 4, dtype=torch.int32))),
        (ValueError, (q, k, fr), dict(q_weight=torch.ones(32))),
        (ValueError, (q, k, fr), dict(k_weight=torch.ones(64, dtype=torch.bfloat16))),
        (ValueError, (q, k, fr), dict(out=(q, q))),
    ]:
        with pytest.raises((ValueError, TypeError)):
            G.qk_norm_rope_fwd(*args, **kw)
    with pytest.raises(ValueError):
        G.qk_norm_rope_bwd(q, k, q.transpose(1, 2), k, fr)
    with pytest.raises(TypeError):
        G.qk_norm_rope_bwd(q, k, q, k.float(), fr)


def test_norm_rope_in_place_under_autograd_is_refused(anywhere):
    """Written in place, tensors with a history would keep the gradients of the unrotated rows."""
    import gated_delta_rule_36_amd as G
    leaf = torch.zeros(1, 2, 2, 64, requires_grad=True)
    q, k = leaf * 1, torch.zeros(1, 2, 2, 64)
    for out in ((q, k), (k, q)):
        with pytest.raises(ValueError, match="gradients"):
            G.qk_norm_rope_fwd(q, k, None, out=out)
        with torch.no_grad(), pytest.raises(anywhere):
            G.qk_norm_rope_fwd(q, k, None, out=out)
    with pytest.raises(anywhere):
        G.qk_norm_rope_fwd(q, k, None, out=(torch.empty_like(k), k))


@pytest.mark.parametrize("shift", [0, 3, 5])
def test_gradients_at_any_offset(monkeypatch, shift):
    """Autograd's gradients may be views that start anywhere (here behind `shift` elements of one flat
    tensor): the entry point gets them contiguous and aligned, with their values."""
    import gated_delta_rule_36_amd as G
    seen = []
    monkeypatch.setattr(_attn, "_need_gpu", lambda t: None)
    monkeypatch.setattr(_attn, "_call", lambda name, dev, *a: seen.append((name, a)))
    q = torch.zeros(1, 3, 2, 64, requires_grad=True)
    k = torch.zeros(1, 3, 1, 64, requires_grad=True)
    lead = torch.zeros(shift)
    qo, ko = G.qk_norm_rope(q, k, None)
    flat = torch.cat([lead, qo.flatten(), ko.flatten()])
    held = {}
    bwd = _attn.qk_norm_rope_bwd

    def spy(q, k, dq, dk, *a, **kw):
        held.update(dq=dq, dk=dk)
        return bwd(q, k, dq, dk, *a, **kw)

    monkeypatch.setattr(_attn, "qk_norm_rope_bwd", spy)
    grad = torch.arange(flat.numel(), dtype=torch.float32)
    flat.backward(grad)
    (name, args), = [x for x in seen if x[0].endswith("bwd")]
    assert [args[2], args[3]] == [held["dq"].data_ptr(), held["dk"].data_ptr()]
    for t, at in ((held["dq"], shift), (held["dk"], shift + qo.numel())):
        assert t.is_contiguous() and t.data_ptr() % 16 == 0
        assert torch.equal(t.flatten(), grad[at:at + t.numel()])


@pytest.mark.parametrize("shift", [0, 3])
def test_mixer_gradients_at_any_offset(monkeypatch, shift):
    """The same for the mixer's gradients of outputs and final states."""
    import gated_delta_rule_36_amd as G
    held = {}
    x = torch.zeros(1, 3, 2, 64, dtype=torch.bfloat16, requires_grad=True)
    s0 = torch.zeros(1, 2, 64, 64)
    monkeypatch.setattr(_lib, "chunk_fwd_train",
                        lambda q, *a, **kw: (torch.zeros_like(q), torch.zeros_like(s0), None))

    def spy(q, k, v, g, b, w, do, d_final_state=None, **kw):
        held.update(do=do, ds=d_final_state)
        return (torch.zeros_like(q),) * 6 + (torch.zeros_like(s0),)

    monkeypatch.setattr(_lib, "chunk_bwd", spy)
    o, s = G.gated_delta_rule2(x, x, x, x, x, x)
    flat = torch.cat([torch.zeros(shift, dtype=torch.bfloat16), o.flatten()])
    states = torch.cat([torch.zeros(shift), s.flatten()])
    grads = [(torch.arange(t.numel()) % 251).to(t.dtype) for t in (flat, states)]
    torch.autograd.backward((flat, states), grads)
    for t, g in ((held["do"], grads[0]), (held["ds"], grads[1])):
        assert t.is_contiguous() and t.data_ptr() % 16 == 0 and torch.equal(t.flatten(), g[shift:])


def test_serving_binding_refusals(anywhere):
    import gated_delta_rule_36_amd as G
    cache = G.kv_cache(6, 2, 64, device="cpu")
    q = torch.zeros(3, 1, 4, 64, dtype=torch.bfloat16)
    k = torch.zeros(3, 1, 2, 64, dtype=torch.bfloat16)
    tb, sl = torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    fr, cu = torch.ones(32), torch.tensor([0, 1, 2, 3], dtype=torch.int32)
    one = (q.view(1, 3, 4, 64), k.view(1, 3, 2, 64))
    with pytest.raises(anywhere):
        G.attn_prologue(q, k, k, cache, tb, sl, fr)
    with pytest.raises(anywhere):
        G.cache_attention(one[0], tuple(cache), tb, sl, cu_seqlens=cu)
    for err, args, kw in [
        (TypeError, (q.float(), cache, tb, sl), {}),
        (ValueError, (q[0], cache, tb, sl), {}),
        (ValueError, (q[:, :, :3], cache, tb, sl), {}),
        (ValueError, (q, cache, tb[:2], sl), {}),
        (ValueError, (q, cache, tb.long(), sl), {}),
        (ValueError, (q, cache, tb.t().contiguous().t(), sl), {}),
        (ValueError, (q, cache, tb, sl[:2]), {}),
        (ValueError, (q, cache, tb, sl.long()), {}),
        (ValueError, (q, cache, tb, sl), dict(cu_seqlens=cu)),
        (ValueError, (one[0], cache, tb, sl), dict(cu_seqlens=cu.long())),
        (ValueError, (one[0], cache, tb, sl), dict(cu_seqlens=cu[:3])),
        (ValueError, (q, cache._replace(k=cache.k.view(torch.uint8)), tb, sl), {}),
        (ValueError, (q, cache._replace(v=cache.v[:5]), tb, sl), {}),
        (ValueError, (q, cache._replace(k_scale=cache.k_scale[0]), tb, sl), {}),
        (ValueError, (q, cache._replace(v_scale=cache.v_scale.double()), tb, sl), {}),
    ]:
        with pytest.raises((ValueError, TypeError)):
            G.cache_attention(*args, **kw)
        with pytest.raises((ValueError, TypeError)):
            G.attn_prologue(args[0], k if args[0].dim() == 4 and args[0].shape[0] == 3 else one[1],
                            k if args[0].dim() == 4 and args[0].shape[0] == 3 else one[1], *args[1:], fr, **kw)
    for kw in (dict(window=-1), dict(scale=0.0), dict(scale=-0.1), dict(scale=math.nan), dict(out=q[:2]),
               dict(workspace=torch.zeros(4))):
        with pytest.raises((ValueError, TypeError)):
            G.cache_attention(q, cache, tb, sl, **kw)
    with pytest.raises(ValueError):
        G.cache_attention(torch.zeros(3, 1, 8, 64, dtype=torch.bfloat16)[:, :, ::2], cache, tb, sl)
    with pytest.raises(ValueError):
        G.attn_prologue(q, q, k, cache, tb, sl, fr)
    with pytest.raises(ValueError):
        G.attn_prologue(q, k, k, cache, tb, sl, fr[:30])
    with pytest.raises(ValueError):
        G.kv_cache(4, 2, 96, device="cpu")


def test_value_columns_are_a_permutation():
    import gated_delta_rule_36_amd as G
    c = G.value_columns("cpu")
    assert sorted(c.tolist()) == list(range(64))
    # 16 neighbouring columns hold 4 neighbouring tokens of each quarter of the block
    inv = torch.argsort(c).view(4, 4, 4)
    for lane in range(4):
        for t in range(4):
            assert inv[lane, t].tolist() == [t * 16 + lane * 4 + i for i in range(4)]
