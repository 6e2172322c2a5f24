"""Decayed attention where a workgroup walks a whole long sequence: more (batch, head) pairs than the plan cuts, and more
chunks than the table of a state's ages holds, with a rest of a chunk."""
import pytest
import torch

import dynamic_convolution_amd as dc
from seq_reference import attention_bounds, close, randn, scale_of

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.float32, torch.float16, torch.bfloat16]
AGES = 16  # entries of the kernel's table

# keeps everything; keeps most over thousands of tokens; falls under 2^-20 after some chunks; within one; keeps nothing
DECAYS = [0.0, -2.0 ** -12, -0.03, -0.5, float("-inf"), -0.002, -0.2, -2.0 ** -9]


def sizes(dtype, d):
    """Tokens of a chunk are 64 (bf16) or 32; two tables' length and a rest of 7 tokens."""
    chunk = 64 if dtype == torch.bfloat16 else 32
    return 64, 2 * AGES * chunk + 7, len(DECAYS), d


def whole(b, t, h, d, dtype, pass_):
    """Whether a call of these sizes takes its sequences whole: segments would have states in the workspace."""
    return dc.decayattn_workspace_bytes(pass_, b, t, h, h, h, h, d, d, dtype) == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,ragged", [(32, False), (64, True)])
def test_long_walks(d, ragged, dtype):
    b, t, h, d = sizes(dtype, d)
    print("[case] attention walk", b, t, h, d, ragged, dtype, flush=True)
    assert whole(b, t, h, d, dtype, 0) and whole(b, t, h, d, dtype, 1)
    g = torch.tensor(DECAYS)
    q, k, v, do = (randn((b, t, h, d), dtype, 700 + i, DEV) for i in range(4))
    state, ds = (randn((b, h, d, d), torch.float32, 710 + i, DEV) for i in range(2)) if ragged else (None, None)
    n = torch.randint(1, t + 1, (b,), generator=torch.Generator().manual_seed(720), dtype=torch.int32)
    n[0], n[b // 2], n[b - 1] = t, 0, t - 7
    lengths = n if ragged else None
    some = [0, 17, b // 2, b - 1]  # sequences that are compared

    def pick(x):
        return None if x is None else x[some].cpu()

    want, tol = attention_bounds((pick(q), pick(k), pick(v), g, scale_of(d), pick(state), pick(lengths), pick(do), pick(ds)), dtype)
    on = None if lengths is None else lengths.to(DEV)
    got = [*dc.decayattn_fwd(q, k, v, g.to(DEV), state=state, lengths=on),
           *dc.decayattn_bwd(q, k, v, g.to(DEV), do, state=state, lengths=on, dstate=ds)]
    torch.cuda.synchronize()
    for x, w, e, name in zip(got, want, tol, ("o", "state", "dq", "dk", "dv", "dstate")):
        if x is not None:
            close(x[some], w, e, name)


@pytest.mark.parametrize("dtype", TYPES)
def test_a_sequence_in_two_parts(dtype):
    """A sequence in two calls, the second from the first's state, against one call: both within the bounds of the recurrence,
    here of a walk that starts in the middle of the table."""
    b, t, h, d = sizes(dtype, 32)
    print("[case] attention walk in parts", dtype, flush=True)
    g = torch.tensor(DECAYS, device=DEV)
    q, k, v = (randn((b, t, h, d), dtype, 730 + i, DEV) for i in range(3))
    cut = t // 3
    first, state = dc.decayattn_fwd(q[:, :cut], k[:, :cut], v[:, :cut], g)
    second, state = dc.decayattn_fwd(q[:, cut:], k[:, cut:], v[:, cut:], g, state=state)
    torch.cuda.synchronize()
    some = [3, b - 2]
    want, tol = attention_bounds((q[some].cpu(), k[some].cpu(), v[some].cpu(), g.cpu(), scale_of(d), None, None), dtype)
    close(torch.cat([first, second], 1)[some], want[0], tol[0], "o")
    close(state[some], want[1], tol[1], "state")
