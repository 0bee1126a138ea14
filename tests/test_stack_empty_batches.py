"""Packed batches of no sequences: the training forward and the gradients write zeros to all rows, also where
these are too few for a kept state."""
import os

import numpy as np
import pytest
import torch

from gated_delta_rule_36_amd import _lib, _stack
from tests.gpu_util import say


@pytest.mark.skipif(not os.path.exists(_lib.lib_path()), reason="libgdn2.so not built (run __graft_entry__.build())")
def test_kept_states_have_room(monkeypatch):
    """The pointer of the kept states says that they are wanted: never that of nothing."""
    import gated_delta_rule_36_amd as G
    ask = _lib.lib().gdn2_linear_recurrence_states_bytes
    for T in (1, 63, 64, 127):
        assert ask(1, 1, T, 64, 0) == 64 * 4
        assert ask(1, 1, T, 64, 1) == (T // 64 + 1) * 64 * 4
    assert ask(1, 1, 128, 64, 0) == 2 * 64 * 4
    assert ask(0, 0, 5, 64, 0) == ask(0, 3, 0, 64, 3) == 0
    seen = []
    monkeypatch.setattr(_stack, "_need_gpu", lambda t: None)
    monkeypatch.setattr(_stack, "_call", lambda name, dev, *a: seen.append(a))
    v, cu = torch.zeros(1, 40, 64), torch.zeros(1, dtype=torch.int32)
    states = G.linear_recurrence_fwd_train(v, v, cu_seqlens=cu)[2]
    assert states.shape == (1, 64) and seen[-1][6] == states.data_ptr() != 0
    G.linear_recurrence_bwd(v, v, None, states, v, cu_seqlens=cu)
    assert seen[-1][3] == states.data_ptr()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,D", [(1, 8), (40, 72), (63, 64), (64, 64)])
def test_rows_are_zeros(T, D, dt):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_36_amd as G
    v, g, w, do = (torch.from_numpy(np.random.default_rng(T + k).standard_normal((1, T, D)).astype(np.float32)).to(dt).cuda()
                   for k in range(4))
    g = -g.abs()
    cu = torch.tensor([T // 2], dtype=torch.int32, device="cuda")
    say("linear_recurrence, no sequences", T, D, dt)
    for gate in (w, None):
        # the outputs' memory holds something before
        for _ in range(6):
            torch.full((1, T, D), 7.0, dtype=dt, device="cuda")
        o, last, states = G.linear_recurrence_fwd_train(v, g, gate, cu_seqlens=cu)
        grads = G.linear_recurrence_bwd(v, g, gate, states, do, cu_seqlens=cu)
        torch.cuda.synchronize()
        assert last.shape == grads[3].shape == (0, D)
        for x in (o, *grads[:3]):
            assert x is None or (x.shape == v.shape and not x.any())
        leaves = [t.clone().requires_grad_() for t in (v, g, w) if t is not w or gate is not None]
        o, last = G.linear_recurrence(*leaves, cu_seqlens=cu)
        got = torch.autograd.grad(o, leaves, do)
        torch.cuda.synchronize()
        assert not o.any() and not any(x.any() for x in got)
