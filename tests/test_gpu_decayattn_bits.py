"""16-bit attention's values between its products: rounded to nearest, so that no output leans to one side.

All inputs are positive, so an operand that was cut off instead would make every output too small by a part of the same
sign.  The mean over N = 2^19 outputs of (result - exact value rounded once) / exact value separates that from rounding:
an output differs from the exact one's rounding only where that lay near a border, in at most one of 2^6 cases, and then
by a step of at most 2^-7 (bf16), so the mean of N errors of either sign has a deviation under 2^-7 2^-3 / 2^9.5 < 2^-19.
Two planes cut off are 2^-17.1 short on average, in each product that they enter."""
import pytest
import torch

import dynamic_convolution_amd as dc

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
MOST = 2.0 ** -18


def positive(shape, dtype, seed):
    return (0.5 + torch.rand(shape, generator=torch.Generator().manual_seed(seed))).to(dtype)


def exact(q, k, v, do, g, scale):
    """(o, dq, dk, dv) in float64 as products over the whole sequence."""
    q, k, v, do = (x.double().transpose(1, 2).contiguous() for x in (q, k, v, do))
    i = torch.arange(q.shape[2])
    far = (i[:, None] - i[None, :]).clamp(min=0)
    keep = torch.exp(g.double()[:, None, None] * far) * (i[:, None] >= i[None, :]) * scale
    p, w = (q @ k.transpose(2, 3).contiguous()) * keep, (do @ v.transpose(2, 3).contiguous()) * keep
    pt, wt = p.transpose(2, 3).contiguous(), w.transpose(2, 3).contiguous()
    return [x.transpose(1, 2) for x in (p @ v, w @ k, wt @ q, pt @ do)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("b,t,h", [(4, 256, 8), (1, 4096, 2)])
def test_no_side_is_favoured(b, t, h, dtype):
    """Few chunks in one workgroup, and many over segments whose states come from a pass of their own."""
    print("[case] attention bits", b, t, h, dtype, flush=True)
    d = 64
    q, k, v, do = (positive((b, t, h, d), dtype, 600 + i) for i in range(4))
    g = torch.linspace(-0.05, -0.001, h)
    want = exact(q, k, v, do, g, d ** -0.5 / 64)
    a = [x.to(DEV) for x in (q, k, v)]
    got = [dc.decayattn_fwd(*a, g.to(DEV), d ** -0.5 / 64)[0], *dc.decayattn_bwd(*a, g.to(DEV), do.to(DEV), d ** -0.5 / 64)[:3]]
    torch.cuda.synchronize()
    for x, w, name in zip(got, want, ("o", "dq", "dk", "dv")):
        lean = ((x.cpu().double() - w.to(dtype).double()) / w).mean().item()
        print("[lean] %s 2^18 x %.3f" % (name, lean / MOST), flush=True)
        assert abs(lean) <= MOST, (name, lean)
