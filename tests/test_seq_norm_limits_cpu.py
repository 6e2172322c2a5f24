"""How large a norm may be: what its own kernels' launches hold, and no less."""
import pytest
import torch

import dynamic_convolution_amd as dc
from dynamic_convolution_amd import _native as N
from test_seq_abi_cpu import no_gpu, norm_fwd

TOO_LARGE = -6


@pytest.mark.parametrize("pass_", [0, 1])
@pytest.mark.parametrize("n,l,c,groups", [
    (262145, 1, 512, 64),      # tokens whose heads are normed: more than 2^24 groups in all
    (1 << 20, 1, 1024, 32),
    (1 << 23, 1, 256, 8),
    (1 << 15, 5000, 2048, 1024),  # maps in two passes
    (1 << 20, 4, 256, 32),     # maps that fit
])
def test_many_groups(n, l, c, groups, pass_):
    assert dc.groupnorm_act_workspace_bytes(pass_, n, l, c, groups, torch.bfloat16) >= 0


@pytest.mark.parametrize("n,l,c,groups", [
    (1 << 24, 2, 1, 1),                # 2^24 workgroups of 256 threads
    (1, 1, 1 << 28, 1 << 25),          # 2^17 workgroups along the groups
])
def test_launches_that_are_none(n, l, c, groups):
    with pytest.raises(dc.DwconvError, match="DW_ETOOLARGE"):
        dc.groupnorm_act_workspace_bytes(0, n, l, c, groups, torch.bfloat16)


@no_gpu
def test_status():
    """The message fits the operators whose tensors may be larger than the convolutions'."""
    assert norm_fwd(n=1 << 24, l=2, c=1, groups=1) == TOO_LARGE
    assert "2^31" not in N.status_str(TOO_LARGE)


def test_the_headers_limits_are_served():
    """Any n of single positions in groups of up to 512, n < 2^24 of others, c up to 2^24 - 256: every width of a group, alone and as many as fit."""
    most, widest = (1 << 24) - 1, (1 << 24) - 256
    for cg in (1, 2, 3, 7, 8, 12, 31, 32, 100, 256, 512, 513, 1024, 2048, 2049, 5000, 1 << 20):
        for groups in (1, widest // cg):
            c = cg * groups
            for n, l in ((1, 1), (1 << 30 if cg <= 512 else most, 1), (most, 2), (most, 3), (1, 1 << 20), (most, 40), (1 << 12, 4000)):
                if n * l * c <= 1 << 46:
                    for pass_ in (0, 1):
                        dc.groupnorm_act_workspace_bytes(pass_, n, l, c, groups, torch.float32)
                        dc.groupnorm_act_workspace_bytes(pass_, n, l, c, groups, torch.float16)


@no_gpu
def test_the_checkpoints_limit():
    from test_seq_abi_cpu import F, STEP
    import dynamic_convolution_amd._sequence as S
    assert S._lib().act8_pack(F, F + STEP, F + 2 * STEP, (1 << 32) - 255, 32, 0, None) == TOO_LARGE
    assert S._lib().act8_pack(F, F, F, (1 << 32) - 256, 32, 0, None) == -7  # overlapping: past the limits' check


def test_column_sums_launch():
    """32 of the 2 c columns of the gradients' sums go to 1024 threads: 2^32 of them at c = 2^26, which the forward serves."""
    for c, groups, fits in (((1 << 26) - 2048, (1 << 15) - 1, True), (1 << 26, 1 << 15, False)):
        dc.groupnorm_act_workspace_bytes(0, 1, 1, c, groups, torch.float16)
        if fits:
            dc.groupnorm_act_workspace_bytes(1, 1, 1, c, groups, torch.float16)
        else:
            with pytest.raises(dc.DwconvError, match="DW_ETOOLARGE"):
                dc.groupnorm_act_workspace_bytes(1, 1, 1, c, groups, torch.float16)
