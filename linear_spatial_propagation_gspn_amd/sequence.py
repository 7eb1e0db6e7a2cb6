"""Thin ctypes binding of libgspn's sequence operators (include/gspn_sequence.h).

The short causal convolution, the selective state space scan and the join of
a block's output to the residual stream, over token rows: prompts, single
tokens, gradients.  As in ``gspn``: argument marshalling only, torch tensors
supply device memory and the current HIP stream, every step of the
computation runs in libgspn's HIP kernels, and a missing library raises.

Rows.  x and its companions are [rows, channels] tensors with unit column
stride (a row stride is taken as it is, so the halves of a projection's
output need no copy), or [batch, length, channels] tensors of evenly spaced
rows, whose batch entries are the sequences.  For 2-D tensors ``cu`` (int32
offsets, nseq + 1 of them, on the device) packs ragged sequences, or ``nseq``
cuts the rows into equal ones (default: one).

Pools.  ``state`` is a pool that the call reads and updates in place;
``slots`` (int32 [nseq]) names each sequence's entry (negative: padding; an
index out of range or named twice makes that sequence's output NaN and leaves
the pool alone), ``resume`` (bool [nseq]) says which prompts continue their
entry.

Gradients have autograd forms (``causal_conv``, ``selective_scan``,
``block_join``) on top of the ``_fwd`` / ``_bwd`` calls, reverse mode only: a
tensor with a forward-mode tangent is refused.  Nothing here
synchronises; outputs and workspaces are allocated by torch unless given, so
every call can be captured in a HIP graph.  As for any autograd node, a backward
is captured with no eager graph of the same leaves alive: torch would tie the
capture to the stream on which that graph found them.
"""
from __future__ import annotations

import ctypes
import math

import torch
from torch.autograd import forward_ad

from . import gspn as G

GSPN_CONV_MIN_WIDTH, GSPN_CONV_MAX_WIDTH = 2, 4
GSPN_SCAN_MAX_STATE = 16
GSPN_JOIN_MAX_CHANNELS = 16384
GSPN_SCAN_CHECKPOINT_ROWS = 8

# Symbols declared in include/gspn_sequence.h.
EXPORTS = ("gspn_causal_conv_fwd", "gspn_causal_conv_step", "gspn_causal_conv_bwd_workspace_bytes",
           "gspn_causal_conv_bwd", "gspn_selective_scan_workspace_bytes", "gspn_selective_scan_checkpoint_bytes",
           "gspn_selective_scan_fwd", "gspn_selective_scan_step", "gspn_selective_scan_bwd_workspace_bytes",
           "gspn_selective_scan_bwd", "gspn_block_join_fwd", "gspn_block_join_bwd_workspace_bytes",
           "gspn_block_join_bwd")

_i64, _vp = ctypes.c_int64, ctypes.c_void_p


class Sequences(ctypes.Structure):
    _fields_ = [("rows", _i64), ("nseq", _i64), ("cu", _vp), ("slots", _vp), ("resume", _vp), ("nslots", _i64)]


def _fields(text: str) -> list:
    """Fields of an argument struct: names ending in ``*`` are pointers, the others 64-bit integers."""
    return [(f.rstrip("*"), _vp if f.endswith("*") else _i64) for f in text.split()]


class ConvArgs(ctypes.Structure):
    _fields_ = [("seq", Sequences)] + _fields(
        "c width silu x* ldx weight* bias* y* ldy state* gy* ldgy dx* lddx dweight* dbias* workspace* workspace_bytes")


class SelscanArgs(ctypes.Structure):
    _fields_ = [("seq", Sequences)] + _fields(
        "channels groups n softplus x* ldx dt* lddt z* ldz B* ldb C* ldc A* D* dt_bias* out* ldo state* checkpoints* "
        "workspace* workspace_bytes gy* ldgy dx* lddx ddt* ldddt dz* lddz dB* dC* dA* dD* ddt_bias*")


class JoinArgs(ctypes.Structure):
    _fields_ = _fields("rows c residual_dtype") + [("eps", ctypes.c_double)] + _fields(
        "h* ldh gate* ldgate residual* ldres post* scale* pre* joined* ldjoined normed* ldnormed gjoined* ldgjoined "
        "gnormed* ldgnormed dh* lddh dgate* lddgate dresidual* lddres dpost* dscale* dpre* workspace* workspace_bytes")


_calls: dict = {}


def lib() -> ctypes.CDLL:
    """libgspn with the sequence calls' argument types set."""
    h = G.lib()
    if not _calls:
        ready = {}
        for name in EXPORTS:
            f = getattr(h, name)
            if name.endswith("_bytes"):
                f.restype = _i64
                f.argtypes = [_i64] * {"gspn_causal_conv_bwd_workspace_bytes": 4,
                                       "gspn_selective_scan_checkpoint_bytes": 4,
                                       "gspn_block_join_bwd_workspace_bytes": 2}.get(name, 5)
                if "selective" in name:
                    f.argtypes = list(f.argtypes) + [ctypes.c_int]
            else:
                f.restype = ctypes.c_int
                f.argtypes = [_vp, ctypes.c_int, _vp]
            ready[name] = f
        _calls.update(ready)
    return h


def _bytes(name: str, *args) -> int:
    if not _calls:
        lib()
    return _calls[name](*args)


# The current stream's handle without building a Stream object, and the current device, where torch offers them.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(name: str, args: ctypes.Structure, dtype: int, index: int) -> None:
    if not _calls:
        lib()
    # the launches go to the tensors' device whatever the current one is
    if index == _current_device():
        st = _calls[name](ctypes.byref(args), dtype, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = _calls[name](ctypes.byref(args), dtype, _raw_stream(index))
    if st:
        G._raise(st, name)


def _tensor(t, name: str, dtype, index: int) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype is not dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if index < 0 or t.get_device() != index:
        raise ValueError("%s must live on HIP device %d, not on %s" % (name, index, t.device))


def _rows(t, name: str, shape: tuple, dtype, index: int, tail: int = 1) -> int:
    """Checks a row tensor (``tail`` contiguous trailing dimensions) and returns its row stride in elements."""
    _tensor(t, name, dtype, index)
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    stride = t.stride()
    if t.numel() == 0:  # whose strides mean nothing
        return max(math.prod(shape[-tail:]), 1)
    want = 1
    for d in range(tail):
        if stride[-1 - d] != want and shape[-1 - d] != 1:
            raise ValueError("%s must have contiguous columns (strides %s)" % (name, stride))
        want *= shape[-1 - d]
    lead = len(shape) - tail
    ld = stride[lead - 1] if shape[lead - 1] != 1 else want
    if lead == 2:
        n, length = shape[0], shape[1]
        if length == 1 and n > 1:
            ld = stride[0]
        elif n > 1 and stride[0] != length * ld:
            raise ValueError("%s must have evenly spaced rows over the batch (strides %s)" % (name, stride))
    if ld < want:
        raise ValueError("%s must not repeat or interleave its rows (strides %s)" % (name, stride))
    return ld


def _ptr_rows(t, name: str, shape: tuple, dtype, index: int, tail: int = 1) -> tuple:
    """A checked row tensor's pointer and row stride."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index >= 0 and t.shape == shape:
        stride = t.stride()  # the usual layouts at once; anything else, and every error, below
        if tail == 1:
            if len(shape) == 2 and stride[1] == 1 and stride[0] >= shape[1] > 0 and shape[0] > 1:
                return t.data_ptr(), stride[0]
        elif len(shape) == 3 and stride[2] == 1 and stride[1] == shape[2] and shape[0] > 1:
            if stride[0] >= shape[1] * shape[2] > 0:
                return t.data_ptr(), stride[0]
    ld = _rows(t, name, shape, dtype, index, tail)
    return t.data_ptr(), ld


def _flat(t, name: str, shape: tuple, dtype, index: int):
    """Checks a contiguous tensor (or None) and returns its pointer."""
    if t is None:
        return None
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index >= 0 and t.shape == shape
            and t.is_contiguous()):
        return t.data_ptr()
    _tensor(t, name, dtype, index)
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _new_like(x, dtype=None) -> torch.Tensor:
    """New contiguous rows of x's shape."""
    return torch.empty_like(x, dtype=dtype, memory_format=torch.contiguous_format)


def _zeros_like(x) -> torch.Tensor:
    return torch.zeros_like(x, memory_format=torch.contiguous_format)


def _need_rows(x, name: str) -> int:
    if not isinstance(x, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if x.dim() not in (2, 3):
        raise ValueError("%s must be [rows, channels] or [batch, length, channels], got %s" % (name, tuple(x.shape)))
    if x.get_device() < 0:
        raise ValueError("%s must live on a HIP device" % name)
    return G._dtype_code(x)


def _sequences(x, cu, nseq, state=None, slots=None, resume=None) -> Sequences:
    """The sequences of rows x, and their pool's entries."""
    dev = x.get_device()
    s = Sequences()
    if x.dim() == 3:
        if cu is not None or nseq not in (None, x.shape[0]):
            raise ValueError("cu / nseq go with [rows, channels] tensors: a 3-D tensor's batch entries are its sequences")
        s.rows, s.nseq = x.shape[0] * x.shape[1], x.shape[0]
    else:
        s.rows = x.shape[0]
        if cu is not None:
            _tensor(cu, "cu", torch.int32, dev)
            if cu.dim() != 1 or cu.numel() < 1 or not cu.is_contiguous():
                raise ValueError("cu must be a contiguous vector of nseq + 1 offsets")
            s.nseq = cu.numel() - 1
            if nseq not in (None, s.nseq):
                raise ValueError("nseq is %d, but cu holds %d sequences" % (nseq, s.nseq))
            s.cu = cu.data_ptr()
        else:
            s.nseq = 1 if nseq is None else int(nseq)
            if s.nseq < 1 or s.rows % s.nseq:
                raise ValueError("%d rows are not %d equal sequences" % (s.rows, s.nseq))
    if state is None:
        if slots is not None or resume is not None:
            raise ValueError("slots and resume name entries of a state pool: pass state")
        return s
    s.nslots = state.shape[0]
    if slots is not None:
        s.slots = _flat(slots, "slots", (s.nseq,), torch.int32, dev)
    elif s.nslots < s.nseq:
        raise ValueError("state holds %d entries for %d sequences" % (s.nslots, s.nseq))
    if resume is not None:
        if not isinstance(resume, torch.Tensor) or resume.dtype not in (torch.bool, torch.uint8):
            raise TypeError("resume must be a bool (or uint8) tensor")
        s.resume = _flat(resume, "resume", (s.nseq,), resume.dtype, dev)
    return s


def _workspace(a, workspace, nbytes: int, x):
    """Points the arguments at the given workspace, or at a new one, which is returned to be kept alive."""
    if workspace is None:
        workspace = x.new_empty(nbytes if nbytes > 4 else 4, dtype=torch.uint8)
    elif workspace.get_device() != x.get_device() or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % x.device)
    a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    return workspace


# ------------------------------------------------------------------------------------------------ causal conv

def _conv_args(x, weight, bias, silu, seq) -> ConvArgs:
    c = x.shape[-1]
    a = ConvArgs()
    a.seq = seq
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a [channels, width] tensor")
    a.c, a.width, a.silu = c, weight.shape[1], 1 if silu else 0
    dev = x.get_device()
    a.weight = _flat(weight, "weight", (c, weight.shape[1]), torch.float32, dev)
    a.bias = _flat(bias, "bias", (c,), torch.float32, dev)
    a.x, a.ldx = _ptr_rows(x, "x", x.shape, x.dtype, dev)
    return a


def _conv_out(a: ConvArgs, x, state, out):
    if state is not None:
        a.state = _flat(state, "state", (state.shape[0], a.width - 1, a.c), x.dtype, x.get_device())
    if out is None:
        out = _new_like(x)
        a.y, a.ldy = out.data_ptr(), max(a.c, 1)
    else:
        a.y, a.ldy = _ptr_rows(out, "out", x.shape, x.dtype, x.get_device())
    return out


def _pool(state, dims: int):
    if state is not None and (not isinstance(state, torch.Tensor) or state.dim() != dims):
        raise ValueError("state must be a %d-D pool, its entries first" % dims)
    return state


def gspn_causal_conv_fwd(x, weight, bias=None, silu: bool = True, cu=None, nseq=None, state=None, slots=None,
                         resume=None, out=None) -> torch.Tensor:
    """Depthwise causal convolution along each sequence's rows, width 2 to 4
    (weight fp32 [channels, width], bias fp32 [channels]), then silu.
    ``state`` ([slots, width - 1, channels], x's dtype): continued where
    ``resume`` says so, and left holding the last width - 1 rows.  Rows outside
    the sequences of ``cu`` are left as they are in ``out``."""
    dt = _need_rows(x, "x")
    a = _conv_args(x, weight, bias, silu, _sequences(x, cu, nseq, _pool(state, 3), slots, resume))
    out = _conv_out(a, x, state, out)
    _call("gspn_causal_conv_fwd", a, dt, x.get_device())
    return out


def gspn_causal_conv_step(x, weight, bias, state, slots=None, silu: bool = True, out=None) -> torch.Tensor:
    """One row per sequence (x [nseq, channels]), each continuing its entry of
    the pool.  Padding rows (negative slot) are left as they are in ``out``."""
    dt = _need_rows(x, "x")
    if x.dim() != 2:
        raise ValueError("a step takes one row per sequence: x [nseq, channels]")
    if state is None:
        raise ValueError("a step continues a state pool: pass state")
    seq = _sequences(x, None, x.shape[0] if x.shape[0] else None, _pool(state, 3), slots)
    a = _conv_args(x, weight, bias, silu, seq)
    out = _conv_out(a, x, state, out)
    if x.shape[0]:
        _call("gspn_causal_conv_step", a, dt, x.get_device())
    return out


def gspn_causal_conv_bwd(x, weight, bias, gy, silu: bool = True, cu=None, nseq=None, workspace=None) -> tuple:
    """Gradients of gspn_causal_conv_fwd without a state: (dx, dweight, dbias),
    dbias None without a bias.  Rows outside the sequences of ``cu`` have a zero dx."""
    dt = _need_rows(x, "x")
    a = _conv_args(x, weight, bias, silu, _sequences(x, cu, nseq))
    a.gy, a.ldgy = _ptr_rows(gy, "gy", x.shape, x.dtype, x.get_device())
    if a.seq.nseq == 0:
        return _zeros_like(x), _zeros_like(weight), None if bias is None else _zeros_like(bias)
    dx = _new_like(x)
    a.dx, a.lddx = dx.data_ptr(), max(a.c, 1)
    dweight = _new_like(weight)
    dbias = None if bias is None else _new_like(bias)
    a.dweight, a.dbias = dweight.data_ptr(), None if dbias is None else dbias.data_ptr()
    ws = _workspace(a, workspace, _bytes("gspn_causal_conv_bwd_workspace_bytes", a.seq.rows, a.seq.nseq, a.c, a.width),
                    x)
    _call("gspn_causal_conv_bwd", a, dt, x.get_device())
    return dx, dweight, dbias


# --------------------------------------------------------------------------------------------- selective scan

def _scan_args(x, dt, A, B, C, D, z, dt_bias, softplus, seq) -> SelscanArgs:
    shape, dtype, dev = x.shape, x.dtype, x.get_device()
    c = shape[-1]
    a = SelscanArgs()
    a.seq = seq
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be a [channels, n] tensor")
    if not isinstance(B, torch.Tensor) or B.dim() != x.dim() + 1:
        raise ValueError("B must be [rows, groups, n] (or [batch, length, groups, n]) beside x")
    n, groups = A.shape[1], B.shape[-2]
    if groups < 1 or c % groups:
        raise ValueError("%d channels are not %d equal groups" % (c, groups))
    a.channels, a.groups, a.n, a.softplus = c, groups, n, 1 if softplus else 0
    a.x, a.ldx = _ptr_rows(x, "x", shape, dtype, dev)
    a.dt, a.lddt = _ptr_rows(dt, "dt", shape, dtype, dev)
    if z is not None:
        a.z, a.ldz = _ptr_rows(z, "z", shape, dtype, dev)
    bshape = (*shape[:-1], groups, n)
    a.B, a.ldb = _ptr_rows(B, "B", bshape, dtype, dev, 2)
    a.C, a.ldc = _ptr_rows(C, "C", bshape, dtype, dev, 2)
    a.A = _flat(A, "A", (c, n), torch.float32, dev)
    a.D = _flat(D, "D", (c,), torch.float32, dev)
    a.dt_bias = _flat(dt_bias, "dt_bias", (c,), torch.float32, dev)
    return a


def _checkpoint_floats(a: SelscanArgs) -> int:
    nbytes = _bytes("gspn_selective_scan_checkpoint_bytes", a.seq.rows, a.seq.nseq, a.channels, a.n,
                    1 if a.seq.cu else 0)
    return max(nbytes, 0) // 4


def gspn_selective_scan_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus: bool = True, cu=None, nseq=None,
                            state=None, slots=None, resume=None, checkpoints=None, out=None, workspace=None):
    """The selective scan along each sequence's rows:
    d = softplus(dt + dt_bias); h = exp(d A) h + d x B; y = <C, h> + D x; out = y silu(z).
    x, dt, z [rows, channels]; B, C [rows, groups, n]; A fp32 [channels, n], n
    1 to 16; D, dt_bias fp32 [channels].  ``state`` (fp32 [slots, channels,
    n]): continued where ``resume`` says so, left holding the last states.
    ``checkpoints`` (True, or a buffer a former call returned): also keeps the
    states before every 8th row for gspn_selective_scan_bwd; the call then
    returns (out, checkpoints).  Rows outside the sequences of ``cu`` are left
    as they are in ``out``."""
    code = _need_rows(x, "x")
    dev = x.get_device()
    a = _scan_args(x, dt, A, B, C, D, z, dt_bias, softplus, _sequences(x, cu, nseq, _pool(state, 3), slots, resume))
    if state is not None:
        a.state = _flat(state, "state", (state.shape[0], a.channels, a.n), torch.float32, dev)
    if out is None:
        out = _new_like(x)
        a.out, a.ldo = out.data_ptr(), max(a.channels, 1)
    else:
        a.out, a.ldo = _ptr_rows(out, "out", x.shape, x.dtype, dev)
    keep = checkpoints is not None and checkpoints is not False
    if keep:
        floats = _checkpoint_floats(a)
        if checkpoints is True:
            checkpoints = x.new_empty(floats, dtype=torch.float32)
        a.checkpoints = _flat(checkpoints, "checkpoints", (floats,), torch.float32, dev)
    need = _bytes("gspn_selective_scan_workspace_bytes", a.seq.rows, a.seq.nseq, a.channels, a.groups, a.n,
                  1 if cu is not None else 0)
    ws = _workspace(a, workspace, need, x) if need > 0 else None
    _call("gspn_selective_scan_fwd", a, code, dev)
    return (out, checkpoints) if keep else out


def gspn_selective_scan_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, softplus: bool = True, slots=None,
                             out=None) -> torch.Tensor:
    """One row per sequence (x [nseq, channels]), each continuing its entry of
    the pool.  Padding rows (negative slot) are left as they are in ``out``."""
    code = _need_rows(x, "x")
    if x.dim() != 2:
        raise ValueError("a step takes one row per sequence: x [nseq, channels]")
    if state is None:
        raise ValueError("a step continues a state pool: pass state")
    a = _scan_args(x, dt, A, B, C, D, z, dt_bias, softplus,
                   _sequences(x, None, x.shape[0] if x.shape[0] else None, _pool(state, 3), slots))
    dev = x.get_device()
    a.state = _flat(state, "state", (state.shape[0], a.channels, a.n), torch.float32, dev)
    if out is None:
        out = _new_like(x)
        a.out, a.ldo = out.data_ptr(), max(a.channels, 1)
    else:
        a.out, a.ldo = _ptr_rows(out, "out", x.shape, x.dtype, dev)
    if x.shape[0]:
        _call("gspn_selective_scan_step", a, code, dev)
    return out


def gspn_selective_scan_bwd(x, dt, A, B, C, gy, D=None, z=None, dt_bias=None, softplus: bool = True, cu=None,
                            nseq=None, checkpoints=None, workspace=None) -> tuple:
    """Gradients of gspn_selective_scan_fwd without a state, for dL/dout = gy:
    (dx, ddt, dA, dB, dC, dD, dz, ddt_bias), None for what was not given.
    ``checkpoints``: what the forward kept for the same inputs; without it the
    forward runs again here.  Rows outside the sequences of ``cu`` have zero
    gradients."""
    code = _need_rows(x, "x")
    dev = x.get_device()
    a = _scan_args(x, dt, A, B, C, D, z, dt_bias, softplus, _sequences(x, cu, nseq))
    a.gy, a.ldgy = _ptr_rows(gy, "gy", x.shape, x.dtype, dev)
    none = a.seq.nseq == 0
    like = _zeros_like if none else _new_like
    dx, ddt, dB, dC, dA = (like(t) for t in (x, x, B, B, A))
    dD, dz, dbias = (None if t is None else like(t) for t in (D, z, dt_bias))
    grads = (dx, ddt, dA, dB, dC, dD, dz, dbias)
    if none:
        return grads
    if checkpoints is None:
        checkpoints = gspn_selective_scan_fwd(x, dt, A, B, C, D, z, dt_bias, softplus, cu, nseq, checkpoints=True)[1]
    a.checkpoints = _flat(checkpoints, "checkpoints", (_checkpoint_floats(a),), torch.float32, dev)
    a.dx, a.ddt, a.dB, a.dC, a.dA = (t.data_ptr() for t in (dx, ddt, dB, dC, dA))
    a.dz, a.dD, a.ddt_bias = (None if t is None else t.data_ptr() for t in (dz, dD, dbias))
    a.lddx = a.ldddt = a.lddz = a.channels
    ws = _workspace(a, workspace, _bytes("gspn_selective_scan_bwd_workspace_bytes", a.seq.rows, a.seq.nseq,
                                         a.channels, a.groups, a.n, 1 if cu is not None else 0), x)
    _call("gspn_selective_scan_bwd", a, code, dev)
    return grads


# ------------------------------------------------------------------------------------------------- block join

def _join_args(h, gate, residual, post, scale, pre, eps, wide) -> JoinArgs:
    c, dev = h.shape[-1], h.get_device()
    a = JoinArgs()
    a.rows, a.c = h.numel() // c if c else 0, c
    a.residual_dtype, a.eps = G.GSPN_F32 if wide == torch.float32 else G.GSPN_BF16, float(eps)
    a.h, a.ldh = _ptr_rows(h, "h", h.shape, h.dtype, dev)
    if gate is not None:
        a.gate, a.ldgate = _ptr_rows(gate, "gate", h.shape, h.dtype, dev)
    if residual is not None:
        a.residual, a.ldres = _ptr_rows(residual, "residual", h.shape, wide, dev)
    a.post = _flat(post, "post", (c,), torch.float32, dev)
    a.scale = _flat(scale, "scale", (c,), torch.float32, dev)
    a.pre = _flat(pre, "pre", (c,), torch.float32, dev)
    return a


def _wide(h, residual):
    if residual is None:
        return h.dtype
    if not isinstance(residual, torch.Tensor) or residual.dtype not in (h.dtype, torch.float32):
        raise TypeError("residual must be a float32 tensor or one of h's dtype")
    return residual.dtype


def gspn_block_join_fwd(h, gate=None, residual=None, post=None, scale=None, pre=None, eps: float = 1e-6, out=None,
                        normed=None) -> tuple:
    """joined = residual + scale * (norm(h) * post) * silu(gate), each part
    where it is given (no post: h itself), and normed = norm(joined) * pre
    (None without pre).  Norms are root mean square norms over the channels.
    h, gate [rows, channels]; post, scale, pre fp32 [channels]; residual in
    h's dtype or float32, which joined then has.  Returns (joined, normed)."""
    dt = _need_rows(h, "h")
    wide = _wide(h, residual)
    a = _join_args(h, gate, residual, post, scale, pre, eps, wide)
    dev = h.get_device()
    if out is None:
        out = _new_like(h, wide)
        a.joined, a.ldjoined = out.data_ptr(), max(a.c, 1)
    else:
        a.joined, a.ldjoined = _ptr_rows(out, "out", h.shape, wide, dev)
    if pre is None:
        if normed is not None:
            raise ValueError("normed needs pre, the weight of the norm")
    else:
        if normed is None:
            normed = _new_like(h)
            a.normed, a.ldnormed = normed.data_ptr(), max(a.c, 1)
        else:
            a.normed, a.ldnormed = _ptr_rows(normed, "normed", h.shape, h.dtype, dev)
    _call("gspn_block_join_fwd", a, dt, dev)
    return out, normed


def gspn_block_join_bwd(h, gjoined, gnormed, joined, gate=None, residual=None, post=None, scale=None, pre=None,
                        eps: float = 1e-6, workspace=None) -> tuple:
    """Gradients of gspn_block_join_fwd for dL/djoined = gjoined (None: zero)
    and dL/dnormed = gnormed (with pre): (dh, dgate, dresidual, dpost, dscale,
    dpre), None for what was not given.  ``joined``: the forward's (read with
    pre)."""
    dt = _need_rows(h, "h")
    dev, c = h.get_device(), h.shape[-1]
    wide = _wide(h, residual)
    a = _join_args(h, gate, residual, post, scale, pre, eps, wide)
    if gjoined is not None:
        a.gjoined, a.ldgjoined = _ptr_rows(gjoined, "gjoined", h.shape, wide, dev)
    if pre is not None:
        if gnormed is None or joined is None:
            raise ValueError("with pre the backward needs gnormed and joined")
        a.gnormed, a.ldgnormed = _ptr_rows(gnormed, "gnormed", h.shape, h.dtype, dev)
        a.joined, a.ldjoined = _ptr_rows(joined, "joined", h.shape, wide, dev)
    elif gnormed is not None:
        raise ValueError("gnormed needs pre, the weight of the norm")
    dh = _new_like(h)
    a.dh, a.lddh = dh.data_ptr(), c
    dgate = dres = None
    if gate is not None:
        dgate = _new_like(h)
        a.dgate, a.lddgate = dgate.data_ptr(), c
    if residual is not None:
        dres = _new_like(h, wide)
        a.dresidual, a.lddres = dres.data_ptr(), c
    dpost, dscale, dpre = (None if t is None else _new_like(t) for t in (post, scale, pre))
    a.dpost, a.dscale, a.dpre = (None if t is None else t.data_ptr() for t in (dpost, dscale, dpre))
    ws = None
    if post is not None or scale is not None or pre is not None:
        ws = _workspace(a, workspace, _bytes("gspn_block_join_bwd_workspace_bytes", a.rows, c), h)
    _call("gspn_block_join_bwd", a, dt, dev)
    return dh, dgate, dres, dpost, dscale, dpre


# --------------------------------------------------------------------------------------------------- autograd

def _wants_grad(*tensors) -> bool:
    """Whether autograd will ask for a gradient; if not, nothing is kept for a backward."""
    return torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad for t in tensors)


def _no_tangents(*tensors) -> None:
    """Refuses forward-mode derivatives: the calls read a tensor's values alone, and an output without a tangent would
    be taken for one whose derivative is zero."""
    for t in tensors:
        if isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None:
            raise NotImplementedError("the sequence operators have no forward-mode derivative")


def _clear(x, cu):
    """With packed sequences, an output whose rows outside them are zero."""
    return None if cu is None or not isinstance(x, torch.Tensor) else x.new_zeros(x.shape)


def _grad_rows(g, like):
    """A gradient in its tensor's dtype, with contiguous columns."""
    _no_tangents(g)
    return g.to(like).contiguous()


class _CausalConv(torch.autograd.Function):
    """gspn_causal_conv_fwd as an autograd node whose backward is gspn_causal_conv_bwd."""

    @staticmethod
    def forward(ctx, silu, cu, nseq, x, weight, bias):
        y = gspn_causal_conv_fwd(x, weight, bias, silu, cu, nseq, out=_clear(x, cu))
        ctx.silu, ctx.nseq = silu, nseq
        ctx.save_for_backward(x, weight, bias, cu)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gy):
        x, weight, bias, cu = ctx.saved_tensors
        dx, dw, db = gspn_causal_conv_bwd(x, weight, bias, _grad_rows(gy, x.dtype), ctx.silu, cu, ctx.nseq)
        return None, None, None, dx, dw, db


def causal_conv(x, weight, bias=None, silu: bool = True, cu=None, nseq=None) -> torch.Tensor:
    """The short causal convolution as a differentiable op (no state); rows
    outside the sequences of ``cu`` are zero."""
    _no_tangents(x, weight, bias)
    if not _wants_grad(x, weight, bias):
        return gspn_causal_conv_fwd(x, weight, bias, silu, cu, nseq, out=_clear(x, cu))
    return _CausalConv.apply(bool(silu), cu, nseq, x, weight, bias)


class _SelectiveScan(torch.autograd.Function):
    """gspn_selective_scan_fwd, keeping its checkpoints, as an autograd node whose backward is
    gspn_selective_scan_bwd."""

    @staticmethod
    def forward(ctx, softplus, cu, nseq, x, dt, A, B, C, D, z, dt_bias):
        y, kept = gspn_selective_scan_fwd(x, dt, A, B, C, D, z, dt_bias, softplus, cu, nseq, checkpoints=True,
                                          out=_clear(x, cu))
        ctx.softplus, ctx.nseq = softplus, nseq
        ctx.save_for_backward(x, dt, A, B, C, D, z, dt_bias, cu, kept)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gy):
        x, dt, A, B, C, D, z, dt_bias, cu, kept = ctx.saved_tensors
        dx, ddt, dA, dB, dC, dD, dz, db = gspn_selective_scan_bwd(
            x, dt, A, B, C, _grad_rows(gy, x.dtype), D, z, dt_bias, ctx.softplus, cu, ctx.nseq, checkpoints=kept)
        return None, None, None, dx, ddt, dA, dB, dC, dD, dz, db


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus: bool = True, cu=None,
                   nseq=None) -> torch.Tensor:
    """The selective scan as a differentiable op (no state); rows outside the
    sequences of ``cu`` are zero.  The forward keeps its states before every
    8th row (n / 2 bytes an element of x) until the backward."""
    _no_tangents(x, dt, A, B, C, D, z, dt_bias)
    if not _wants_grad(x, dt, A, B, C, D, z, dt_bias):
        return gspn_selective_scan_fwd(x, dt, A, B, C, D, z, dt_bias, softplus, cu, nseq, out=_clear(x, cu))
    return _SelectiveScan.apply(bool(softplus), cu, nseq, x, dt, A, B, C, D, z, dt_bias)


class _BlockJoin(torch.autograd.Function):
    """gspn_block_join_fwd as an autograd node whose backward is gspn_block_join_bwd."""

    @staticmethod
    def forward(ctx, eps, h, gate, residual, post, scale, pre):
        joined, normed = gspn_block_join_fwd(h, gate, residual, post, scale, pre, eps)
        ctx.eps = eps
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(h, gate, residual, post, scale, pre, joined if pre is not None else None)
        return joined, normed

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gjoined, gnormed):
        h, gate, residual, post, scale, pre, joined = ctx.saved_tensors
        wide = h.dtype if residual is None else residual.dtype
        if gjoined is not None:
            gjoined = _grad_rows(gjoined, wide)
        if pre is not None:
            gnormed = _zeros_like(h) if gnormed is None \
                else _grad_rows(gnormed, h.dtype)
        dh, dgate, dres, dpost, dscale, dpre = gspn_block_join_bwd(h, gjoined, gnormed, joined, gate, residual, post,
                                                                   scale, pre, ctx.eps)
        return None, dh, dgate, dres, dpost, dscale, dpre


def block_join(h, gate=None, residual=None, post=None, scale=None, pre=None, eps: float = 1e-6) -> tuple:
    """The join of a block's output to the residual stream as a differentiable
    op: (joined, normed), normed None without pre."""
    _no_tangents(h, gate, residual, post, scale, pre)
    if not _wants_grad(h, gate, residual, post, scale, pre):
        return gspn_block_join_fwd(h, gate, residual, post, scale, pre, eps)
    return _BlockJoin.apply(float(eps), h, gate, residual, post, scale, pre)
