"""Thin ctypes binding of libgspn's attention operators (include/gspn_attention.h).

The norm and rotation of each head's queries and keys, and softmax attention
with grouped heads: prompts, prompts that continue a cache entry, single
tokens, gradients.  As in ``sequence``, whose rows, sequences and slots these
calls share: argument marshalling only, the current HIP stream, no
synchronisation, outputs and workspaces allocated by torch unless given, so
that every call can be captured in a HIP graph.

Rows.  q and its companions are [rows, heads, d] tensors with heads and d
contiguous (a row stride is taken as it is, so the slices of a projection's
output need no copy), or [batch, length, heads, d] tensors of evenly spaced
rows, whose batch entries are the sequences.

Caches.  ``state`` is a pair of pools (keys, values), [entries, capacity,
kv_heads, d] each, that a call reads and appends to in place; ``held`` (int32
[nseq]) says how many rows each sequence's entry holds.  It is left as it is:
a program adds the new rows' number itself.  A length that does not fit, like
a slot out of range or named twice, makes that sequence's output NaN and
leaves the pools alone.

Gradients have autograd forms (``head_rotary``, ``attention``), reverse mode
only, with ``sequence``'s rule for captured backwards.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import gspn as G
from . import sequence as S

GSPN_ATTENTION_MAX_HEAD = 128
GSPN_ROTARY_MAX_HEAD = 256
GSPN_ROTARY_MAX_AXES = 4

# Symbols declared in include/gspn_attention.h.
EXPORTS = ("gspn_head_rotary_fwd", "gspn_head_rotary_bwd_workspace_bytes", "gspn_head_rotary_bwd", "gspn_attention_fwd",
           "gspn_attention_step_workspace_bytes", "gspn_attention_step", "gspn_attention_bwd_workspace_bytes",
           "gspn_attention_bwd")

_i64, _vp = ctypes.c_int64, ctypes.c_void_p


class RotaryArgs(ctypes.Structure):
    _fields_ = S._fields("rows heads kv_heads d pairs axes interleaved") + [
        ("section", _i64 * GSPN_ROTARY_MAX_AXES), ("eps", ctypes.c_double)] + S._fields(
        "q* ldq k* ldk q_weight* k_weight* positions* ldpos freqs* q_out* ldqo k_out* ldko gq* ldgq gk* ldgk dq* lddq "
        "dk* lddk dq_weight* dk_weight* workspace* workspace_bytes")


class AttnArgs(ctypes.Structure):
    _fields_ = [("seq", S.Sequences)] + S._fields("kv_rows kv_cu* heads kv_heads d causal") + [
        ("scale", ctypes.c_double)] + S._fields(
        "q* ldq k* ldk v* ldv out* ldo lse* k_pool* v_pool* capacity held* gout* ldgo dq* lddq dk* lddk dv* lddv "
        "workspace* workspace_bytes")


_calls: dict = {}


def lib() -> ctypes.CDLL:
    """libgspn with the attention calls' argument types set."""
    h = G.lib()
    if not _calls:
        ready = {}
        for name in EXPORTS:
            f = getattr(h, name)
            if name.endswith("_bytes"):
                f.restype = _i64
                f.argtypes = [_i64] * {"gspn_head_rotary_bwd_workspace_bytes": 2,
                                       "gspn_attention_step_workspace_bytes": 5}.get(name, 6)
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


def _call(name: str, args: ctypes.Structure, dtype: int, index: int) -> None:
    if not _calls:
        lib()
    # the launches go to the tensors' device whatever the current one is
    if index == S._current_device():
        st = _calls[name](ctypes.byref(args), dtype, S._raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = _calls[name](ctypes.byref(args), dtype, S._raw_stream(index))
    if st:
        G._raise(st, name)


def _need_heads(x, name: str) -> tuple:
    """A [.., heads, d] tensor's shape, device index and storage type."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    shape, dev = x.shape, x.get_device()
    if len(shape) not in (3, 4):
        raise ValueError("%s must be [rows, heads, d] or [batch, length, heads, d], got %s" % (name, tuple(shape)))
    if dev < 0:
        raise ValueError("%s must live on a HIP device" % name)
    if shape[-1] < 1 or shape[-2] < 1:
        raise ValueError("%s must have at least one head of at least one element, got %s" % (name, tuple(shape)))
    return shape, dev, G._dtype_code(x)


def _heads_beside(x, shape, name: str) -> int:
    """The heads of a companion of rows of ``shape``."""
    if not isinstance(x, torch.Tensor) or x.dim() != len(shape):
        raise ValueError("%s must be a tensor of %d dimensions" % (name, len(shape)))
    return x.shape[-2]


def _out_rows(out, x, shape, dev: int, name: str) -> tuple:
    """Rows of x's shape to write to, new ones if not given: the tensor, its pointer and row stride."""
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
        return out, out.data_ptr(), shape[-1] * shape[-2]
    return (out, *S._ptr_rows(out, name, shape, x.dtype, dev, 2))


# ------------------------------------------------------------------------------------------------ head rotary

_Sections = _i64 * GSPN_ROTARY_MAX_AXES


def _rotary_args(shape, dev, q, positions, freqs, k, q_weight, k_weight, sections, interleaved, eps,
                 read: bool = True) -> RotaryArgs:
    """The arguments up to the outputs."""
    d, heads, lead, dtype = shape[-1], shape[-2], shape[:-2], q.dtype
    rows = lead[0] if len(lead) == 1 else lead[0] * lead[1]
    pairs = freqs.numel() if isinstance(freqs, torch.Tensor) else 0
    pfreqs = S._flat(freqs, "freqs", (pairs,), torch.float64, dev)
    if freqs is None:
        raise TypeError("freqs must be a torch.Tensor")
    sections = (pairs,) if sections is None else tuple(sections)
    axes = len(sections)
    if not 1 <= axes <= GSPN_ROTARY_MAX_AXES or sum(sections) != pairs or min(sections) < 0:
        raise ValueError("sections %s must share out %d pairs among 1 to %d axes" % (sections, pairs,
                                                                                      GSPN_ROTARY_MAX_AXES))
    if 2 * pairs > d:
        raise ValueError("%d pairs do not fit into heads of %d elements" % (pairs, d))
    if axes == 1 and isinstance(positions, torch.Tensor) and positions.dim() == len(lead):
        positions = positions.unsqueeze(-1)
    ppos, ldpos = S._ptr_rows(positions, "positions", (*lead, axes), torch.int32, dev)
    pqw = S._flat(q_weight, "q_weight", (d,), torch.float32, dev)
    pq = ldq = pk = ldk = kv_heads = 0
    pkw = None
    if read or pqw is not None:
        pq, ldq = S._ptr_rows(q, "q", shape, dtype, dev, 2)
    if k is not None:
        kv_heads = _heads_beside(k, shape, "k")
        pkw = S._flat(k_weight, "k_weight", (d,), torch.float32, dev)
        if read or pkw is not None:
            pk, ldk = S._ptr_rows(k, "k", (*lead, kv_heads, d), dtype, dev, 2)
    elif k_weight is not None:
        raise ValueError("k_weight needs k")
    return RotaryArgs(rows, heads, kv_heads, d, pairs, axes, 1 if interleaved else 0, _Sections(*sections), eps, pq, ldq, pk,
                      ldk, pqw, pkw, ppos, ldpos, pfreqs)


def gspn_head_rotary_fwd(q, positions, freqs, k=None, q_weight=None, k_weight=None, sections=None,
                         interleaved: bool = False, eps: float = 1e-6, out=None, out_k=None) -> tuple:
    """Each head of q [rows, heads, d] and k [rows, kv_heads, d], root mean
    square normalised where its weight (fp32 [d]) is given, its pairs of
    elements then turned by positions * freqs (float64, radians a position).
    Pair j is elements (j, pairs + j), or (2 j, 2 j + 1) with ``interleaved``;
    elements behind the pairs are not turned.  ``positions``: int32 [rows, axes]
    ([rows] for one axis); ``sections``: how many pairs, in order, turn by each
    axis (default: all by one).  Returns (q, k) turned, k None without k."""
    shape, dev, dt = _need_heads(q, "q")
    a = _rotary_args(shape, dev, q, positions, freqs, k, q_weight, k_weight, sections, interleaved, eps)
    out, a.q_out, a.ldqo = _out_rows(out, q, shape, dev, "out")
    if k is not None:
        out_k, a.k_out, a.ldko = _out_rows(out_k, k, k.shape, dev, "out_k")
    elif out_k is not None:
        raise ValueError("out_k needs k")
    _call("gspn_head_rotary_fwd", a, dt, dev)
    return out, out_k


def gspn_head_rotary_bwd(q, positions, freqs, gq, k=None, gk=None, q_weight=None, k_weight=None, sections=None,
                         interleaved: bool = False, eps: float = 1e-6, workspace=None) -> tuple:
    """Gradients of gspn_head_rotary_fwd for dL/dq_out = gq, dL/dk_out = gk:
    (dq, dk, dq_weight, dk_weight), None for what was not given.  q and k are
    read where they are normalised."""
    shape, dev, dt = _need_heads(q, "q")
    a = _rotary_args(shape, dev, q, positions, freqs, k, q_weight, k_weight, sections, interleaved, eps, read=False)
    a.gq, a.ldgq = S._ptr_rows(gq, "gq", shape, q.dtype, dev, 2)
    dq, a.dq, a.lddq = _out_rows(None, q, shape, dev, "dq")
    dk = None
    if k is not None:
        a.gk, a.ldgk = S._ptr_rows(gk, "gk", k.shape, q.dtype, dev, 2)
        dk, a.dk, a.lddk = _out_rows(None, k, k.shape, dev, "dk")
    elif gk is not None:
        raise ValueError("gk needs k")
    dqw, dkw = (None if w is None else S._new_like(w) for w in (q_weight, k_weight))
    a.dq_weight, a.dk_weight = (None if w is None else w.data_ptr() for w in (dqw, dkw))
    ws = None
    if dqw is not None or dkw is not None:
        ws = S._workspace(a, workspace, _bytes("gspn_head_rotary_bwd_workspace_bytes", a.rows, a.d), q)
    _call("gspn_head_rotary_bwd", a, dt, dev)
    return dq, dk, dqw, dkw


# -------------------------------------------------------------------------------------------------- attention

def _attn_args(shape, dev, q, k, v, causal, scale, cu, nseq, cu_k, state=None, slots=None) -> AttnArgs:
    """The arguments up to the output."""
    dtype, d, heads = q.dtype, shape[-1], shape[-2]
    kv_heads = _heads_beside(k, shape, "k")
    seq = S._sequences_of(shape[:-2], dev, cu, nseq, None if state is None else state[0], slots)
    scale = d ** -0.5 if scale is None else float(scale)
    if kv_heads < 1 or heads % kv_heads:
        raise ValueError("%d heads are not equal groups for %d of keys" % (heads, kv_heads))
    lead = k.shape[:-2]
    kv_rows = lead[0] if len(lead) == 1 else lead[0] * lead[1]
    kv_cu = None
    if cu_k is not None:
        if len(shape) != 3:
            raise ValueError("cu_k goes with [rows, heads, d] tensors")
        kv_cu = S._flat(cu_k, "cu_k", (seq.nseq + 1,), torch.int32, dev)
    elif len(lead) == 2 and lead[0] != shape[0]:
        raise ValueError("q holds %d sequences, k %d" % (shape[0], lead[0]))
    elif cu is not None:
        if kv_rows != seq.rows:
            raise ValueError("keys of other lengths than the queries' need cu_k")
    elif seq.nseq and kv_rows % seq.nseq:
        raise ValueError("%d rows of keys are not %d equal sequences" % (kv_rows, seq.nseq))
    kshape = (*lead, kv_heads, d)
    return AttnArgs(seq, kv_rows, kv_cu, heads, kv_heads, d, 1 if causal else 0, scale,
                    *S._ptr_rows(q, "q", shape, dtype, dev, 2), *S._ptr_rows(k, "k", kshape, dtype, dev, 2),
                    *S._ptr_rows(v, "v", kshape, dtype, dev, 2))


def _cache(a: AttnArgs, q, state, held) -> None:
    if a.kv_cu or a.kv_rows != a.seq.rows:
        raise ValueError("a cache takes one new key for every row of queries")
    dev = q.get_device()
    shape = (state[0].shape[0], state[0].shape[1], a.kv_heads, a.d)
    a.k_pool = S._flat(state[0], "state[0]", shape, q.dtype, dev)
    a.v_pool = S._flat(state[1], "state[1]", shape, q.dtype, dev)
    a.capacity = shape[1]
    a.held = S._flat(held, "held", (a.seq.nseq,), torch.int32, dev)


def _pools(state):
    if state is None:
        return None
    if not isinstance(state, (tuple, list)) or len(state) != 2:
        raise ValueError("state must be the pair of pools of keys and values")
    for p in state:
        if not isinstance(p, torch.Tensor) or p.dim() != 4:
            raise ValueError("state must hold [entries, capacity, kv_heads, d] pools")
    return tuple(state)


def gspn_attention_fwd(q, k, v, causal: bool = True, scale=None, cu=None, nseq=None, cu_k=None, state=None, slots=None,
                       held=None, lse=None, out=None):
    """Softmax attention within each sequence: q [rows, heads, d], k and v
    [kv_rows, kv_heads, d], kv_heads dividing heads; ``scale`` defaults to
    d ** -0.5.  ``causal``: the last row sees every key, each row before it one
    less.  ``cu_k``: the keys' own sequences, beside ``cu`` (or equal) ones of
    the queries; without it keys go with queries row by row, or in equal shares.
    A row that sees no key is zero.  ``state``, ``slots``, ``held``: the keys
    before these rows, from a cache that receives the new ones.  ``lse`` (True,
    or an fp32 [heads, rows] tensor): also the logarithms of the softmax's sums
    for gspn_attention_bwd; the call then returns (out, lse).  Rows outside the
    sequences of ``cu`` are left as they are in ``out``."""
    shape, dev, dt = _need_heads(q, "q")
    state = _pools(state)
    a = _attn_args(shape, dev, q, k, v, causal, scale, cu, nseq, cu_k, state, slots)
    if state is not None:
        _cache(a, q, state, held)
    elif held is not None:
        raise ValueError("held counts rows of a cache: pass state")
    out, a.out, a.ldo = _out_rows(out, q, shape, dev, "out")
    keep = lse is not None and lse is not False
    if keep:
        if lse is True:
            lse = q.new_empty((a.heads, a.seq.rows), dtype=torch.float32)
        a.lse = S._flat(lse, "lse", (a.heads, a.seq.rows), torch.float32, dev)
    _call("gspn_attention_fwd", a, dt, dev)
    return (out, lse) if keep else out


def gspn_attention_step(q, k, v, state, held, slots=None, scale=None, out=None, workspace=None) -> torch.Tensor:
    """One row per sequence (q [nseq, heads, d], k and v [nseq, kv_heads, d]):
    the new key and value go behind the ``held`` rows of the sequence's cache
    entry, and the row attends to all of them.  Padding rows (negative slot) are
    left as they are in ``out``."""
    shape, dev, dt = _need_heads(q, "q")
    if len(shape) != 3:
        raise ValueError("a step takes one row per sequence: q [nseq, heads, d]")
    state = _pools(state)
    if state is None or held is None:
        raise ValueError("a step continues a cache: pass state and held")
    n = shape[0]
    a = _attn_args(shape, dev, q, k, v, True, scale, None, n if n else None, None, state, slots)
    _cache(a, q, state, held)
    out, a.out, a.ldo = _out_rows(out, q, shape, dev, "out")
    if n:
        need = _bytes("gspn_attention_step_workspace_bytes", a.seq.nseq, a.heads, a.kv_heads, a.d, a.capacity)
        ws = S._workspace(a, workspace, need, q) if need > 0 else None
        _call("gspn_attention_step", a, dt, dev)
    return out


def gspn_attention_bwd(q, k, v, out, lse, gout, causal: bool = True, scale=None, cu=None, nseq=None, cu_k=None,
                       workspace=None) -> tuple:
    """Gradients of gspn_attention_fwd without a cache, for dL/dout = gout, from
    its ``out`` and ``lse``: (dq, dk, dv).  Rows outside the sequences have zero
    gradients."""
    shape, dev, dt = _need_heads(q, "q")
    a = _attn_args(shape, dev, q, k, v, causal, scale, cu, nseq, cu_k)
    a.out, a.ldo = S._ptr_rows(out, "out", shape, q.dtype, dev, 2)
    a.gout, a.ldgo = S._ptr_rows(gout, "gout", shape, q.dtype, dev, 2)
    if lse is None:
        raise ValueError("the backward needs the forward's lse")
    a.lse = S._flat(lse, "lse", (a.heads, a.seq.rows), torch.float32, dev)
    dq, a.dq, a.lddq = _out_rows(None, q, shape, dev, "dq")
    dk, a.dk, a.lddk = _out_rows(None, k, k.shape, dev, "dk")
    dv, a.dv, a.lddv = _out_rows(None, v, k.shape, dev, "dv")
    need = 0
    if a.seq.nseq:
        need = _bytes("gspn_attention_bwd_workspace_bytes", a.seq.rows, a.seq.nseq, a.heads, a.kv_rows, a.kv_heads, a.d)
    ws = S._workspace(a, workspace, need, q)
    _call("gspn_attention_bwd", a, dt, dev)
    return dq, dk, dv


# --------------------------------------------------------------------------------------------------- autograd

class _HeadRotary(torch.autograd.Function):
    """gspn_head_rotary_fwd as an autograd node whose backward is gspn_head_rotary_bwd."""

    @staticmethod
    def forward(ctx, sections, interleaved, eps, positions, freqs, q, k, q_weight, k_weight):
        out = gspn_head_rotary_fwd(q, positions, freqs, k, q_weight, k_weight, sections, interleaved, eps)
        ctx.sections, ctx.interleaved, ctx.eps = sections, interleaved, eps
        ctx.save_for_backward(positions, freqs, q, k, q_weight, k_weight)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gq, gk):
        positions, freqs, q, k, qw, kw = ctx.saved_tensors
        gq = S._grad_rows(gq, q.dtype)
        gk = None if k is None else S._grad_rows(gk, q.dtype)
        dq, dk, dqw, dkw = gspn_head_rotary_bwd(q, positions, freqs, gq, k, gk, qw, kw, ctx.sections, ctx.interleaved,
                                                ctx.eps)
        return None, None, None, None, None, dq, dk, dqw, dkw


def head_rotary(q, positions, freqs, k=None, q_weight=None, k_weight=None, sections=None, interleaved: bool = False,
                eps: float = 1e-6) -> tuple:
    """The norm and rotation of heads as a differentiable op (positions and
    freqs have no gradient): (q, k), k None without k."""
    S._no_tangents(q, k, q_weight, k_weight, freqs)
    if isinstance(freqs, torch.Tensor) and freqs.requires_grad and torch.is_grad_enabled():
        raise NotImplementedError("the rotation has no gradient for its frequencies")
    if not S._wants_grad(q, k, q_weight, k_weight):
        return gspn_head_rotary_fwd(q, positions, freqs, k, q_weight, k_weight, sections, interleaved, eps)
    sections = None if sections is None else tuple(sections)
    return _HeadRotary.apply(sections, bool(interleaved), float(eps), positions, freqs, q, k, q_weight, k_weight)


def _clear(q, cu):
    """With packed sequences, an output whose rows outside them are zero."""
    return None if cu is None or not isinstance(q, torch.Tensor) else q.new_zeros(q.shape)


class _Attention(torch.autograd.Function):
    """gspn_attention_fwd as an autograd node whose backward is gspn_attention_bwd."""

    @staticmethod
    def forward(ctx, causal, scale, cu, nseq, cu_k, q, k, v):
        out, lse = gspn_attention_fwd(q, k, v, causal, scale, cu, nseq, cu_k, lse=True, out=_clear(q, cu))
        ctx.causal, ctx.scale, ctx.nseq = causal, scale, nseq
        ctx.save_for_backward(q, k, v, out, lse, cu, cu_k)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gout):
        q, k, v, out, lse, cu, cu_k = ctx.saved_tensors
        dq, dk, dv = gspn_attention_bwd(q, k, v, out, lse, S._grad_rows(gout, q.dtype), ctx.causal, ctx.scale, cu,
                                        ctx.nseq, cu_k)
        return None, None, None, None, None, dq, dk, dv


def attention(q, k, v, causal: bool = True, scale=None, cu=None, nseq=None, cu_k=None) -> torch.Tensor:
    """Attention as a differentiable op (no cache); rows outside the sequences
    of ``cu`` are zero."""
    S._no_tangents(q, k, v)
    if not S._wants_grad(q, k, v):
        return gspn_attention_fwd(q, k, v, causal, scale, cu, nseq, cu_k, out=_clear(q, cu))
    return _Attention.apply(bool(causal), None if scale is None else float(scale), cu, nseq, cu_k, q, k, v)
