"""Binding to the sequence operators of libdwconv.so (the C ABI in include/dwseq.h).

Argument marshalling only, as in _native: shapes and strides become the ABI's integers, and a
nonzero status becomes an exception.  Outputs and workspaces that the caller does not pass are
allocated by torch on the stream that the call is enqueued on.

The checks are here; what every call repeats (reading its tensors' forms, making its outputs, the
call itself) is in csrc/seq_bind.cpp, because single tokens and small tensors wait for the host.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
from typing import NamedTuple

from . import _native
from ._native import _I64, _VP, DwconvError

# every exported symbol that include/dwseq.h declares
EXPORTS = ("decayattn_fwd", "decayattn_bwd", "decayattn_step", "decayattn_workspace_bytes", "act8_pack", "act8_unpack",
           "groupnorm_act_fwd", "groupnorm_act_bwd", "groupnorm_act_workspace_bytes")
ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2}
ACT8_BLOCK = 32  # values of a row that share a step in an 8-bit checkpoint

_SZ = ctypes.c_size_t
_INT = ctypes.c_int
_F = ctypes.c_float
_seq = None
_bind = None
torch = None  # imported with the library, by the first call


def _lib():
    """libdwconv.so with the sequence operators' argument types declared."""
    global _seq, torch, _raw_stream, _current_device
    if _seq is not None:
        return _seq
    import torch as torch_
    torch = torch_
    # torch's own ways to the current stream's handle and device, without the objects around them
    # (2 us a call); where they are missing, the public ones
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    L = _native.lib()
    L.decayattn_workspace_bytes.argtypes = [_INT] + [_I64] * 8 + [_INT, ctypes.POINTER(_SZ)]
    L.decayattn_fwd.argtypes = [_VP] * 9 + [_SZ] + [_I64] * 8 + [_VP, _F, _INT, _VP]
    L.decayattn_bwd.argtypes = [_VP] * 13 + [_SZ] + [_I64] * 8 + [_VP, _F, _INT, _VP]
    L.decayattn_step.argtypes = [_VP] * 6 + [_I64] * 7 + [_VP, _I64, _F, _INT, _VP]
    L.act8_pack.argtypes = [_VP] * 3 + [_I64] * 2 + [_INT, _VP]
    L.act8_unpack.argtypes = [_VP] * 3 + [_I64] * 2 + [_INT, _VP]
    L.groupnorm_act_fwd.argtypes = [_VP] * 9 + [_SZ] + [_I64] * 4 + [_F, _INT, _INT, _VP]
    L.groupnorm_act_bwd.argtypes = [_VP] * 12 + [_SZ] + [_I64] * 4 + [_INT, _INT, _VP]
    L.groupnorm_act_workspace_bytes.argtypes = [_INT] + [_I64] * 4 + [_INT, ctypes.POINTER(_SZ)]
    for name in EXPORTS:
        getattr(L, name).restype = _INT
    _seq = L
    return L


def _binding():
    """csrc/seq_bind.cpp, built beside the library."""
    global _bind
    if _bind is None:
        _lib()
        if not os.path.exists(os.path.join(os.path.dirname(__file__), "_seqbind.so")):
            raise RuntimeError("_seqbind.so is not built; run dynamic_convolution_amd/build.py")
        from . import _seqbind
        _bind = _seqbind
    return _bind


# A call's checks depend on its tensors' shapes, strides, types and devices alone, so their outcome, a plan, is
# kept by those (never by a tensor's address or contents).  `_form` is what a check sees of a tensor.
def _form(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.device)


class _Plans(dict):
    """Plans by key; all are dropped when there are many."""
    MOST = 1024

    def add(self, key, plan):
        if len(self) >= self.MOST:
            self.clear()
        self[key] = plan
        return plan


class _Plan(NamedTuple):
    numbers: bytes    # the ABI's integers, as csrc/seq_bind.cpp passes them on
    index: int        # the device
    dtype: object
    device: object
    outs: bytes       # forms of the outputs that the call makes
    shapes: tuple     # shapes of those that the caller may pass
    need: int = 0     # bytes of workspace
    scale: float = 0.0


def _numbers(*n):
    return struct.pack("%dq" % len(n), *n)


def _forms(*outs):
    """What seq_bind's empty() makes: (type code, shape) of each."""
    return b"".join(_numbers(code, len(shape), *shape) for code, shape in outs)


_I8, _U8 = 3, 4  # type codes beside the ABI's


def _call(fn, where, plan, *args):
    """Enqueues on the device's current stream; raises on a nonzero status."""
    index = plan[1]
    if _current_device() == index:
        rc = fn(plan[0], *args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(plan[0], *args, _raw_stream(index))
    if rc != 0:
        raise DwconvError(rc, where)


def _gpu(device, name):
    if device.type != "cuda":
        raise ValueError("%s must be a GPU tensor: there is no CPU path" % name)


@functools.lru_cache(maxsize=64)
def _code(dtype):
    codes = {torch.float32: _native.DW_F32, torch.float16: _native.DW_F16, torch.bfloat16: _native.DW_BF16}
    if dtype not in codes:
        raise TypeError("unsupported dtype %s (float32, float16, bfloat16)" % dtype)
    return codes[dtype]


def _like(form, name, shape, dtype, device):
    """Raises unless the form is that of a tensor of exactly this shape, type and device."""
    if tuple(form[0]) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(form[0]), tuple(shape)))
    if form[2] != dtype:
        raise TypeError("%s dtype %s != %s" % (name, form[2], dtype))
    if form[3] != device:
        raise ValueError("%s is on %s, expected %s" % (name, form[3], device))


def _is_dense(shape, strides):
    want = 1
    for n, st in zip(reversed(shape), reversed(strides)):
        if n == 0:
            return True
        if n != 1 and st != want:
            return False
        want *= n
    return True


def _dense(form, name, shape, dtype, device):
    """_like, and contiguous; a form of None passes."""
    if form is None:
        return
    _like(form, name, shape, dtype, device)
    if 0 not in form[0] and not _is_dense(form[0], form[1]):
        raise ValueError("%s must be contiguous" % name)


def _given(t, name, shape, dtype, device):
    """An output that the caller passes, checked; or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _dense(_form(t), name, shape, dtype, device)
    return t


def _workspace(workspace, plan, like):
    """The workspace to pass: the caller's, or one of the bytes that the plan needs."""
    if workspace is None:
        if plan.need:
            workspace = _bind.empty(_forms((_U8, (plan.need,))), like)[0]
    elif workspace.device != plan.device:
        raise ValueError("workspace is on %s, expected %s" % (workspace.device, plan.device))
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace


# ---------------------------------------------------------------- decayed linear attention
def _attn_shapes(q, k, v, g, step):
    """(b, t, h, hq, hk, hv, dk, dv) of a call; raises where the tensors do not fit together."""
    dims = 3 if step else 4
    if len(q[0]) != dims or len(k[0]) != dims or len(v[0]) != dims:
        raise ValueError("q, k and v have %d dimensions: %s" % (dims, "(b, heads, size)" if step else "(b, t, heads, size)"))
    lead = 1 if step else 2
    if q[0][:lead] != k[0][:lead] or q[0][:lead] != v[0][:lead]:
        raise ValueError("q %s, k %s and v %s differ in batch or length" % (tuple(q[0]), tuple(k[0]), tuple(v[0])))
    if q[0][-1] != k[0][-1]:
        raise ValueError("q and k have head sizes %d and %d" % (q[0][-1], k[0][-1]))
    _gpu(q[3], "q")
    for x, name in ((k, "k"), (v, "v")):
        if x[2] != q[2]:
            raise TypeError("%s dtype %s != %s" % (name, x[2], q[2]))
        if x[3] != q[3]:
            raise ValueError("%s is on %s, expected %s" % (name, x[3], q[3]))
    for x, name in ((q, "q"), (k, "k"), (v, "v")):
        _rows(x, name)
    if len(g[0]) != 1:
        raise ValueError("log_decay has one value for each head")
    h = g[0][0]
    hq, hk, hv = q[0][-2], k[0][-2], v[0][-2]
    if not h or not hq or not hk or not hv or h % hq or h % hk or h % hv:
        raise ValueError("%d, %d and %d heads of q, k and v do not divide the %d of log_decay" % (hq, hk, hv, h))
    _dense(g, "log_decay", (h,), torch.float32, q[3])
    return (q[0][0], 1 if step else q[0][1], h, hq, hk, hv, q[0][-1], v[0][-1])


def _rows(form, name):
    if form[1][-1] != 1 and form[0][-1] != 1:
        raise ValueError("%s must be contiguous along its last dimension" % name)


@functools.lru_cache(maxsize=4096)
def _attn_space(pass_, sizes, code):
    need = _SZ()
    rc = _lib().decayattn_workspace_bytes(pass_, *sizes, code, ctypes.byref(need))
    if rc != 0:
        raise DwconvError(rc, "decayattn_workspace_bytes")
    return need.value


def decayattn_workspace_bytes(pass_, b, t, h, hq, hk, hv, dk, dv, dtype):
    """Bytes of workspace that decayattn_fwd (pass_ 0) or decayattn_bwd (pass_ 1) takes for these sizes."""
    _lib()
    return _attn_space(int(pass_), tuple(int(x) for x in (b, t, h, hq, hk, hv, dk, dv)), _code(dtype))


_fwd_plans, _bwd_plans, _step_plans = _Plans(), _Plans(), _Plans()


def _attn_plan(q, k, v, g, state, lengths, do, dstate):
    """The plan of a whole sequence's call: the forward, or where `do` is given the gradients."""
    sizes = b, t, h, _, _, _, dk, dv = _attn_shapes(q, k, v, g, False)
    dtype, dev = q[2], q[3]
    code = _code(dtype)
    _dense(state, "state", (b, h, dk, dv), torch.float32, dev)
    _dense(dstate, "dstate", (b, h, dk, dv), torch.float32, dev)
    _dense(lengths, "lengths", (b,), torch.int32, dev)
    strides = [*q[1][:3], *k[1][:3], *v[1][:3]]
    o, s = (b, t, h, dv), (b, h, dk, dv)
    if do is None:
        outs = _forms((code, o), (_native.DW_F32, s))
    else:
        _like(do, "do", o, dtype, dev)
        _rows(do, "do")
        strides += do[1][:3]
        outs = _forms((code, q[0]), (code, k[0]), (code, v[0]), *([] if state is None else [(_native.DW_F32, s)]))
    return _Plan(_numbers(*sizes, code, *strides), dev.index, dtype, dev, outs, (o, s),
                 _attn_space(0 if do is None else 1, sizes, code), dk ** -0.5)


def decayattn_fwd(q, k, v, log_decay, scale=None, state=None, lengths=None, out=None, out_state=None, workspace=None):
    """(o, state) of causal linear attention whose head j forgets by exp(log_decay[j]) a token:
    S_i = exp(log_decay) S_(i-1) + k_i v_i', o_i = scale q_i S_i.

    q (b, t, hq, dk), k (b, t, hk, dk), v (b, t, hv, dv): float32, float16 or bfloat16, any
    strides but contiguous in the last dimension; hq, hk and hv divide the heads h of log_decay
    (float32).  scale: dk ** -0.5 if None.  state (b, h, dk, dv) float32: before the first token,
    zeros if None.  lengths (b) int32: tokens of each sequence, the rest is padding, whose output
    is zero.  Returns o (b, t, h, dv) and the float32 state after each sequence's last token.
    A value that is not finite spreads over its 64-token chunk, to the tokens before it too, and after it.
    """
    B = _bind or _binding()
    key = B.key(q, k, v, log_decay, state, lengths)
    plan = _fwd_plans.get(key) or _fwd_plans.add(key, _attn_plan(
        _form(q), _form(k), _form(v), _form(log_decay), _form(state), _form(lengths), None, None))
    if out is None and out_state is None:
        out, out_state = B.empty(plan.outs, q)
    else:
        out = _given(out, "out", plan.shapes[0], plan.dtype, plan.device)
        out_state = _given(out_state, "out_state", plan.shapes[1], torch.float32, plan.device)
    _call(B.attn_fwd, "decayattn_fwd", plan, q, k, v, log_decay, state, lengths, out, out_state,
          _workspace(workspace, plan, q), plan.scale if scale is None else float(scale))
    return out, out_state


def decayattn_bwd(q, k, v, log_decay, do, scale=None, state=None, lengths=None, dstate=None, workspace=None):
    """(dq, dk, dv, dstate) of decayattn_fwd for o's gradient do (b, t, h, dv).

    `dstate` (b, h, dk, dv) float32 is the gradient of the returned state, zeros if None; the
    returned one is that of `state`, None where that is None.  Gradients of heads that several
    of the h share are summed.  log_decay is a constant and gets none.
    """
    B = _bind or _binding()
    key = B.key(q, k, v, log_decay, state, lengths, do, dstate)
    plan = _bwd_plans.get(key) or _bwd_plans.add(key, _attn_plan(
        _form(q), _form(k), _form(v), _form(log_decay), _form(state), _form(lengths), _form(do), _form(dstate)))
    grads = B.empty(plan.outs, q)
    if state is None:
        grads += (None,)
    _call(B.attn_bwd, "decayattn_bwd", plan, q, k, v, log_decay, do, state, lengths, dstate, *grads,
          _workspace(workspace, plan, q), plan.scale if scale is None else float(scale))
    return grads


def _step_plan(q, k, v, g, state):
    """The plan of a single token's call."""
    b, _, h, hq, hk, hv, dk, dv = _attn_shapes(q, k, v, g, True)
    dtype, dev = q[2], q[3]
    code, o = _code(dtype), (b, h, dv)
    _like(state, "state", (b, h, dk, dv), torch.float32, dev)
    if b and not _is_dense(state[0][1:], state[1][1:]):
        raise ValueError("state must be contiguous but for its first dimension")
    return _Plan(_numbers(b, h, hq, hk, hv, dk, dv, state[1][0] if b > 1 else h * dk * dv, code, *q[1][:2], *k[1][:2], *v[1][:2]),
                 dev.index, dtype, dev, _forms((code, o)), (o,), 0, dk ** -0.5)


def decayattn_step(q, k, v, log_decay, state, scale=None, out=None):
    """o (b, h, dv) of one more token; `state` is updated in place.

    q (b, hq, dk), k (b, hk, dk), v (b, hv, dv) as in decayattn_fwd without the token dimension;
    state (b, h, dk, dv) float32, contiguous but for the stride of its first dimension.
    """
    B = _bind or _binding()
    key = B.key(q, k, v, log_decay, state)
    plan = _step_plans.get(key) or _step_plans.add(key, _step_plan(_form(q), _form(k), _form(v), _form(log_decay), _form(state)))
    if out is None:
        out, = B.empty(plan.outs, q)
    else:
        _dense(_form(out), "out", plan.shapes[0], plan.dtype, plan.device)
    _call(B.attn_step, "decayattn_step", plan, q, k, v, log_decay, state, out, plan.scale if scale is None else float(scale))
    return out


# ---------------------------------------------------------------- 8-bit checkpoints
class Act8(NamedTuple):
    """An activation tensor in 8 bits: `codes` (int8, the tensor's shape) and `exps` (int8, the shape
    with the last dimension in blocks of 32).  A value is code * 2 ** exp of its block."""
    codes: object
    exps: object

    @property
    def shape(self):
        return self.codes.shape


def _blocks(shape):
    return (*shape[:-1], -(-shape[-1] // ACT8_BLOCK))


def _count(shape):
    n = 1
    for d in shape:
        n *= d
    return n


def _act8_dense(p, name, shape, device):
    if not isinstance(p, Act8):
        raise TypeError("%s must be an Act8" % name)
    _dense(_form(p.codes), name + ".codes", shape, torch.int8, device)
    _dense(_form(p.exps), name + ".exps", _blocks(shape), torch.int8, device)


_pack_plans, _unpack_plans, _norm_fwd_plans, _norm_bwd_plans = _Plans(), _Plans(), _Plans(), _Plans()


def _act8_sizes(x, name):
    """(rows, c) of a tensor's checkpoint."""
    _gpu(x[3], name)
    shape = x[0]
    if len(shape) < 1 or shape[-1] < 1:
        raise ValueError("%s needs a last dimension of at least one value" % name)
    _dense(x, name, shape, x[2], x[3])
    return _count(shape[:-1]), shape[-1]


def _pack_plan(x):
    rows, c = _act8_sizes(x, "x")
    code = _code(x[2])
    return _Plan(_numbers(rows, c, code), x[3].index, x[2], x[3], _forms((_I8, x[0]), (_I8, _blocks(x[0]))), (x[0],))


def _unpack_plan(codes, exps, dtype):
    rows, c = _act8_sizes(codes, "packed.codes")
    code = _code(dtype)
    if codes[2] != torch.int8:
        raise TypeError("packed.codes dtype %s != %s" % (codes[2], torch.int8))
    _dense(exps, "packed.exps", _blocks(codes[0]), torch.int8, codes[3])
    return _Plan(_numbers(rows, c, code), codes[3].index, dtype, codes[3], _forms((code, codes[0])), (codes[0],))


def act8_pack(x, out=None):
    """The 8-bit checkpoint (Act8) of x, whose last dimension is cut into blocks of 32 values that share
    a power-of-two step: a finite value comes back within half a step, 1/254 of its block's largest to
    1/128; what is not finite comes back as NaN."""
    B = _bind or _binding()
    key = B.key(x)
    plan = _pack_plans.get(key) or _pack_plans.add(key, _pack_plan(_form(x)))
    if out is None:
        out = Act8(*B.empty(plan.outs, x))
    else:
        _act8_dense(out, "out", plan.shapes[0], plan.device)
    _call(B.pack, "act8_pack", plan, x, *out, 0.0)
    return out


def act8_unpack(packed, dtype, out=None):
    """The tensor of `dtype` that an 8-bit checkpoint stands for."""
    B = _bind or _binding()
    if not isinstance(packed, Act8):
        raise TypeError("packed must be an Act8")
    codes, exps = packed
    key = B.key(codes, exps), dtype
    plan = _unpack_plans.get(key) or _unpack_plans.add(key, _unpack_plan(_form(codes), _form(exps), dtype))
    if out is None:
        out, = B.empty(plan.outs, codes)
    else:
        _dense(_form(out), "out", plan.shapes[0], dtype, plan.device)
    _call(B.unpack, "act8_unpack", plan, codes, exps, out, 0.0)
    return out


# ---------------------------------------------------------------- group norm with an activation
@functools.lru_cache(maxsize=4096)
def _norm_space(pass_, sizes, code):
    need = _SZ()
    rc = _lib().groupnorm_act_workspace_bytes(pass_, *sizes, code, ctypes.byref(need))
    if rc != 0:
        raise DwconvError(rc, "groupnorm_act_workspace_bytes")
    return need.value


def groupnorm_act_workspace_bytes(pass_, n, l, c, groups, dtype):
    """Bytes of workspace that groupnorm_act_fwd (pass_ 0) or groupnorm_act_bwd (pass_ 1) takes."""
    _lib()
    return _norm_space(int(pass_), (int(n), int(l), int(c), int(groups)), _code(dtype))


def _norm_sizes(x, name, gamma, beta, groups, act):
    """((n, l, c, groups), dtype code, activation code) of a call on x (n, ..., c)."""
    _gpu(x[3], name)
    shape, dtype, dev = x[0], x[2], x[3]
    if len(shape) < 2:
        raise ValueError("%s has dimensions (n, ..., c)" % name)
    n, c, l, groups = shape[0], shape[-1], _count(shape[1:-1]), int(groups)
    if groups < 1 or c < 1 or c % groups:
        raise ValueError("%d groups do not divide %d channels" % (groups, c))
    if l < 1:
        raise ValueError("a sample has no positions")
    code = _code(dtype)
    if act is not None and act not in ACTIVATIONS:
        raise ValueError("activation %r is none of %s" % (act, ", ".join(ACTIVATIONS)))
    if 0 not in shape and not _is_dense(shape, x[1]):
        raise ValueError("%s must be contiguous, channels last" % name)
    _dense(gamma, "gamma", (c,), dtype, dev)
    _dense(beta, "beta", (c,), dtype, dev)
    return (n, l, c, groups), code, ACTIVATIONS[act or "none"]


def _norm_fwd_plan(x, gamma, beta, groups, act, checkpoint):
    sizes, code, a = _norm_sizes(x, "x", gamma, beta, groups, act)
    stat = (_native.DW_F32, (sizes[0], sizes[3]))
    outs = [(code, x[0]), stat, stat] + ([(_I8, x[0]), (_I8, _blocks(x[0]))] if checkpoint else [])
    return _Plan(_numbers(*sizes, a, code), x[3].index, x[2], x[3], _forms(*outs), (_forms(*outs[1:]), x[0]),
                 _norm_space(0, sizes, code))


def _norm_bwd_plan(dy, x, codes, exps, mean, rstd, gamma, beta, groups, act):
    """The plan of a backward call whose input has form x or, packed, forms codes and exps."""
    sizes, code, a = _norm_sizes(dy, "dy", gamma, beta, groups, act)
    shape, dtype, dev = dy[0], dy[2], dy[3]
    if codes is None:
        _dense(x, "x", shape, dtype, dev)
    else:
        _dense(codes, "x.codes", shape, torch.int8, dev)
        _dense(exps, "x.exps", _blocks(shape), torch.int8, dev)
    n, _, c, g = sizes
    _dense(mean, "mean", (n, g), torch.float32, dev)
    _dense(rstd, "rstd", (n, g), torch.float32, dev)
    return _Plan(_numbers(*sizes, a, code), dev.index, dtype, dev, _forms((code, shape), (code, (c,)), (code, (c,))), (shape,),
                 _norm_space(1, sizes, code))


def groupnorm_act_fwd(x, gamma, beta, groups, eps=1e-5, act="none", checkpoint=False, out=None, workspace=None):
    """(y, mean, rstd, kept): y = act(xhat gamma + beta) with x (n, ..., c), channels last, normalised
    over the positions and the channels of each of `groups` groups.

    act: "none", "silu" or "gelu" (by erf).  gamma and beta (c) are of x's type; mean and rstd
    (n, groups) float32 are what the backward takes.  kept is x's 8-bit checkpoint (Act8) if
    `checkpoint` is true, else None.
    """
    B = _bind or _binding()
    key = B.key(x, gamma, beta), groups, act, bool(checkpoint)
    plan = _norm_fwd_plans.get(key) or _norm_fwd_plans.add(key, _norm_fwd_plan(
        _form(x), _form(gamma), _form(beta), groups, act, checkpoint))
    if out is None:
        out, mean, rstd, *kept = B.empty(plan.outs, x)
    else:
        _dense(_form(out), "out", plan.shapes[1], plan.dtype, plan.device)
        mean, rstd, *kept = B.empty(plan.shapes[0], x)
    kept = Act8(*kept) if checkpoint else None
    _call(B.norm_fwd, "groupnorm_act_fwd", plan, x, gamma, beta, out, mean, rstd, *(kept or (None, None)),
          _workspace(workspace, plan, x), float(eps))
    return out, mean, rstd, kept


def groupnorm_act_bwd(dy, x, mean, rstd, gamma, beta, groups, act="none", workspace=None):
    """(dx, dgamma, dbeta) of groupnorm_act_fwd for y's gradient dy.

    x is the forward's input, or its 8-bit checkpoint (Act8), from which xhat is then taken.
    """
    B = _bind or _binding()
    x, codes, exps = (None, *x) if isinstance(x, Act8) else (x, None, None)
    key = B.key(dy, x, codes, exps, mean, rstd, gamma, beta), groups, act
    plan = _norm_bwd_plans.get(key) or _norm_bwd_plans.add(key, _norm_bwd_plan(
        _form(dy), _form(x), _form(codes), _form(exps), _form(mean), _form(rstd), _form(gamma), _form(beta), groups, act))
    dx, dgamma, dbeta = B.empty(plan.outs, dy)
    if not plan.shapes[0][0]:
        dgamma.zero_()
        dbeta.zero_()
    _call(B.norm_bwd, "groupnorm_act_bwd", plan, dy, x, codes, exps, mean, rstd, gamma, beta, dx, dgamma, dbeta,
          _workspace(workspace, plan, dy), 0.0)
    return dx, dgamma, dbeta
