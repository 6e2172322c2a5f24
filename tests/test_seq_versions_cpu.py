"""Tensors that a call writes have a new version, by which autograd finds a saved tensor that has changed.

Calls of no batch entry: all of the binding runs, and nothing is launched."""
import pytest
import torch

import dynamic_convolution_amd._sequence as S
from test_seq_abi_cpu import no_gpu


def call(name, tensors, numbers):
    assert getattr(S._binding(), name)(S._numbers(*numbers), *tensors, 1.0, 0) == 0


# entry point, tensors, which of them it writes, the ABI's integers
CALLS = [
    ("attn_fwd", 9, (6, 7, 8), (0, 1, 1, 1, 1, 1, 8, 8, 0) + (8,) * 9),
    ("attn_bwd", 13, (8, 9, 10, 11, 12), (0, 1, 1, 1, 1, 1, 8, 8, 0) + (8,) * 12),
    ("attn_step", 6, (4, 5), (0, 1, 1, 1, 1, 8, 8, 64, 0) + (8,) * 6),
    ("pack", 3, (1, 2), (0, 8, 0)),
    ("unpack", 3, (2,), (0, 8, 0)),
    ("norm_fwd", 9, (3, 4, 5, 6, 7, 8), (0, 1, 8, 1, 0, 0)),
    ("norm_bwd", 12, (8, 9, 10, 11), (0, 1, 8, 1, 0, 0)),
]


@no_gpu
@pytest.mark.parametrize("name,count,written,numbers", CALLS)
def test_what_is_written(name, count, written, numbers):
    tensors = [torch.zeros(8) for _ in range(count)]
    call(name, tensors, numbers)
    assert [i for i, t in enumerate(tensors) if t._version] == list(written)


@no_gpu
def test_a_saved_state_is_found_changed():
    """d(state^2)/dstate needs the state as it was: torch refuses once a token has been added to it."""
    name, count, written, numbers = CALLS[2]
    leaf = torch.ones(8, requires_grad=True)
    state = leaf * 2
    loss = (state * state).sum()
    call(name, [torch.zeros(8) for _ in range(4)] + [state.detach(), torch.zeros(8)], numbers)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@no_gpu
def test_inference_tensors_have_no_version():
    with torch.inference_mode():
        tensors = [torch.zeros(8) for _ in range(6)]
    call("attn_step", tensors, CALLS[2][3])
    with torch.inference_mode():
        call("attn_step", tensors, CALLS[2][3])


def test_tensors_that_are_negated_later_are_refused():
    """Such a view's memory holds the values before torch negates them."""
    x = torch.ones((2, 3))
    with pytest.raises(TypeError, match="resolve_neg"):
        S._binding().key(torch._neg_view(x))
    name, _, _, numbers = CALLS[4]
    with pytest.raises(TypeError, match="resolve_neg"):
        call(name, [torch.zeros(8), torch.zeros(8), torch._neg_view(torch.zeros(8))], numbers)
    assert S._binding().key(torch._neg_view(x).resolve_neg()) == S._binding().key(x)
