"""What torch knows of the sequence operators' calls: its out-of-memory error."""
import pytest
import torch

import dynamic_convolution_amd as dc

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_no_memory_for_the_outputs():
    """Outputs of 1 TB from inputs of a kilobyte: the type that a caller catches to try a smaller batch."""
    print("[case] out of memory", flush=True)
    x = torch.zeros((1, 1, 1, 256), device=DEV).expand(1, 1 << 30, 1, 256)
    with pytest.raises(torch.OutOfMemoryError):
        dc.decayattn_fwd(x, x, x, torch.zeros((1,), device=DEV))
    torch.cuda.synchronize()
