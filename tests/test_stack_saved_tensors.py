"""Saved-tensor hooks around the autograd of the recurrence and the norm on the host (the entry points replaced): what the
hooks hand back need not have the layout, nor the type, of what was saved."""
import pytest
import torch

from gated_delta_rule_36_amd import _stack


@pytest.fixture
def calls(monkeypatch):
    """The entry points' calls, (name, arguments), none of them made."""
    seen = []
    monkeypatch.setattr(_stack, "_need_gpu", lambda t: None)
    monkeypatch.setattr(_stack, "_call", lambda name, dev, *a: seen.append((name, a)))
    return seen


def _slices(gate, lead=(2, 5)):
    x = torch.zeros(*lead, 56).requires_grad_()
    return [x[..., :16], x[..., 16:32], x[..., 32:48] if gate else None]


def _dense_copy(t):
    return t.clone(memory_format=torch.contiguous_format)


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("packed", [True, False])
def test_strides_are_those_of_the_unpacked_inputs(calls, gate, packed):
    import gated_delta_rule_36_amd as G
    cu = torch.tensor([0, 2, 10], dtype=torch.int32) if packed else None
    inputs = _slices(gate, (1, 10) if packed else (2, 5))
    held = {}

    def unpack(t):
        held[t.data_ptr()] = t
        return t

    with torch.autograd.graph.saved_tensors_hooks(_dense_copy, unpack):
        o, _ = G.linear_recurrence(*inputs, cu_seqlens=cu)
    assert calls[-1][1][12:15] == (56, 56, 56 if gate else 0)
    o.sum().backward()
    name, a = calls[-1]
    assert name == "gdn2_linear_recurrence_bwd"
    for pointer, stride in zip(a[:3], a[15:18]):
        if pointer is not None:
            assert held[pointer].shape[-1] == 16 and stride == held[pointer].stride(1) == 16
    assert (a[2] is None) == (not gate) and a[17] == (16 if gate else 0)
    # without hooks the slices themselves
    o, _ = G.linear_recurrence(*inputs, cu_seqlens=cu)
    o.sum().backward()
    assert calls[-1][1][15:18] == (56, 56, 56 if gate else 0)


@pytest.mark.parametrize("change", [lambda t: t.bfloat16(), lambda t: t[..., :8], lambda t: t[:1], lambda t: t.to("meta")])
@pytest.mark.parametrize("dims", [2, 3])
def test_recurrence_refuses_other_tensors_than_it_saved(calls, change, dims):
    """The inputs (3 axes) or the kept states (2) in another type or shape, or on another device."""
    import gated_delta_rule_36_amd as G
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, lambda t: change(t) if t.dim() == dims else t):
        o, _ = G.linear_recurrence(*_slices(True))
    made = len(calls)
    with pytest.raises((TypeError, ValueError)):
        o.sum().backward()
    assert len(calls) == made


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("change", [lambda t: t.double(), lambda t: t.float() if t.dtype == torch.bfloat16 else t.bfloat16(),
                                    lambda t: t[..., :8], lambda t: t[:1], lambda t: t.to("meta")])
@pytest.mark.parametrize("dims", [1, 2])
def test_norm_refuses_other_tensors_than_it_saved(calls, change, dims, wide):
    """The stream (2 axes) or the weight (1) in another type or shape, or on another device: the gradients
    are of the saved ones."""
    import gated_delta_rule_36_amd as G
    x = torch.zeros(3, 16, dtype=torch.bfloat16)
    r = torch.zeros(3, 16, dtype=torch.float32 if wide else torch.bfloat16, requires_grad=True)
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, lambda t: change(t) if t.dim() == dims else t):
        y, h = G.residual_norm(x, r, torch.ones(16))
    made = len(calls)
    with pytest.raises((TypeError, ValueError)):
        torch.autograd.backward((y, h), (torch.zeros_like(y), torch.zeros_like(h)))
    assert len(calls) == made


def test_norm_reads_the_unpacked_stream_at_its_stride(calls):
    import gated_delta_rule_36_amd as G
    x = torch.zeros(3, 40).requires_grad_()
    with torch.autograd.graph.saved_tensors_hooks(_dense_copy, lambda t: t):
        y, _ = G.residual_norm(x[:, :16], None, torch.ones(16))
    y.sum().backward()
    name, a = calls[-1]
    assert name == "gdn2_residual_norm_bwd" and a[7:10] == (3, 16, 16)
