"""8-bit checkpoints of blocks at the upper end of fp32's and bf16's range, unpacked and read by the norm's gradients.

A block whose largest magnitude is 2^127 or more has a step of 2^121 or 2^122: 128 of the first are 2^128, which is no
fp32 value, so a decoder may not form that product."""
import numpy as np
import pytest
import torch

import dynamic_convolution_amd as dc
from seq_reference import checkpoint, close, half_step, randn, smallest

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
# under, at and past 2^127, and the largest values of bf16 and fp32
TOPS = [2.0 ** 126, 1.99 * 2.0 ** 126, 2.0 ** 127, 2e38, 1.99 * 2.0 ** 127, 3.3895e38, 1.0]


def ends(rows, c, dtype, seed):
    """Each block of 32 has one of TOPS (of either sign) as its largest magnitude, beside zeros, ones and some between."""
    top = torch.tensor(TOPS, dtype=torch.float64)
    blocks = -(-c // 32)
    which = torch.arange(rows * blocks) % len(TOPS)
    x = randn((rows * blocks, 32), torch.float64, seed).clamp(-3, 3) / 4
    x = x * top[which][:, None]
    x[:, 1], x[:, 2], x[:, 3] = 0.0, -1.0, 1.0
    x[:, 0] = top[which] * (1 - 2 * (torch.arange(rows * blocks) // len(TOPS) % 2))
    x = x.view(rows, blocks * 32)[:, :c].to(dtype)
    assert x.isfinite().all()
    return x


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(7, 32), (9, 64), (14, 100), (21, 7), (30, 13)])
def test_unpacked(shape, dtype):
    """Codes, steps and values are whole numbers of steps: equal to the last bit."""
    print("[case] act8 ends", shape, dtype, flush=True)
    x = ends(*shape, dtype, 500)
    codes, exps, values = checkpoint(x)
    assert (exps == 121).any()
    p = dc.act8_pack(x.to(DEV))
    y = dc.act8_unpack(p, dtype)
    torch.cuda.synchronize()
    assert np.array_equal(p.codes.cpu().numpy(), codes) and np.array_equal(p.exps.cpu().numpy(), exps)
    most = torch.finfo(dtype).max
    assert torch.equal(y.cpu(), torch.from_numpy(np.clip(values, -most, most)).to(dtype))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(14, 1, 64, 2), (14, 1, 56, 8), (1, 9000, 72, 8), (2, 11, 21, 3), (3, 40, 64, 4)])
def test_norm_gradients_from_it(shape, dtype):
    """mean 0 and rstd 2^-120: xhat is a whole number of steps times a power of two, at most 2^8, and exact.  What is left
    is the rounding of fp32 sums of m terms, at most m 2^-24 of their magnitudes, and of a few products."""
    print("[case] act8 ends norm", shape, dtype, flush=True)
    n, l, c, groups = shape
    x = ends(n * l, c, dtype, 510).view(n, l, c)
    dy, gamma = randn((n, l, c), dtype, 511), (1 + 0.2 * randn((c,), torch.float32, 512)).to(dtype)
    beta = torch.zeros((c,), dtype=dtype)
    mean, rstd = torch.zeros((n, groups)), torch.full((n, groups), 2.0 ** -120)
    kept = dc.act8_pack(x.to(DEV))
    got = dc.groupnorm_act_bwd(dy.to(DEV), kept, mean.to(DEV), rstd.to(DEV), gamma.to(DEV), beta.to(DEV), groups)
    torch.cuda.synchronize()
    values = np.clip(checkpoint(x.view(n * l, c))[2], -torch.finfo(torch.float32).max, torch.finfo(torch.float32).max)
    xhat = torch.from_numpy(values).view(n, l, c) * 2.0 ** -120
    dz = dy.double()
    g = dz * gamma.double()

    def mean_of(v):
        return v.view(n, l, groups, -1).mean((1, 3)).repeat_interleave(c // groups, 1)[:, None, :]

    dx = (g - mean_of(g) - xhat * mean_of(g * xhat)) * 2.0 ** -120
    size = (g.abs() + mean_of(g.abs()) + xhat.abs() * mean_of((g * xhat).abs())) * 2.0 ** -120
    least, half = smallest(dtype), half_step(dtype)
    close(got[0], dx, (l * c // groups + 8) * 2.0 ** -24 * size + half * dx.abs() + least, "dx")
    for y, terms, name in ((got[1], dz * xhat, "dgamma"), (got[2], dz, "dbeta")):
        want = terms.sum((0, 1))
        close(y, want, (n * l + 8) * 2.0 ** -24 * terms.abs().sum((0, 1)) + half * want.abs() + least, name)
