"""A norm of more than 2^24 groups in all: many tokens of many heads."""
import pytest
import torch

import dynamic_convolution_amd as dc
from seq_reference import randn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_tokens_of_many_heads():
    """A token's results are those of a call on fewer tokens, to the bit; the sums over all tokens against 64 bits: about
    100 additions follow each other in fp32, each off by 2^-24 of the terms' magnitudes at most."""
    n, c, groups = 262145, 512, 64
    print("[case] norm of many groups", flush=True)
    x = torch.randn((n, 1, c), generator=torch.Generator(DEV).manual_seed(800), device=DEV)
    dy = torch.randn((n, 1, c), generator=torch.Generator(DEV).manual_seed(801), device=DEV)
    gamma, beta = 1 + 0.2 * randn((c,), torch.float32, 802, DEV), 0.2 * randn((c,), torch.float32, 803, DEV)
    y, mean, rstd, _ = dc.groupnorm_act_fwd(x, gamma, beta, groups)
    dx, dgamma, dbeta = dc.groupnorm_act_bwd(dy, x, mean, rstd, gamma, beta, groups)
    torch.cuda.synchronize()
    sums, sizes = torch.zeros((2, c), dtype=torch.float64, device=DEV), torch.zeros((2, c), dtype=torch.float64, device=DEV)
    for at in (slice(0, n // 2), slice(n // 2, n)):
        part = dc.groupnorm_act_fwd(x[at], gamma, beta, groups)
        assert torch.equal(part[0], y[at]) and torch.equal(part[1], mean[at]) and torch.equal(part[2], rstd[at])
        assert torch.equal(dc.groupnorm_act_bwd(dy[at], x[at], mean[at], rstd[at], gamma, beta, groups)[0], dx[at])
        by = x[at].double().view(-1, groups, c // groups)
        by = (by - by.mean(-1, keepdim=True)) / (by.var(-1, unbiased=False, keepdim=True) + 1e-5).sqrt()
        d, xhat = dy[at].double().view(-1, c), by.view(-1, c)
        sums += torch.stack([(d * xhat).sum(0), d.sum(0)])
        sizes += torch.stack([(d.abs() * (xhat.abs() + 1)).sum(0), d.abs().sum(0)])
    for got, want, size in zip((dgamma, dbeta), sums, sizes):
        assert bool(((got.double() - want).abs() <= 256 * 2.0 ** -24 * size).all())
