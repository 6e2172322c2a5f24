"""The sizes of the long walks on the GPU are ones that the plan does not cut: their workspace holds no segment's state."""
import pytest
import torch

from test_gpu_decayattn_walks import AGES, TYPES, sizes, whole


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [32, 64])
def test_sequences_are_taken_whole(d, dtype):
    b, t, h, d = sizes(dtype, d)
    assert t > 2 * AGES * (64 if dtype == torch.bfloat16 else 32)
    assert whole(b, t, h, d, dtype, 0) and whole(b, t, h, d, dtype, 1)
    # the second of a sequence's two parts; its gradients are not taken
    assert whole(b, t - t // 3, h, d, dtype, 0) and whole(b, t // 3, h, d, dtype, 0)


def test_few_heads_are_cut():
    assert not whole(1, 4096, 1, 64, torch.bfloat16, 0)
