"""CPU tests of the attention operators' C ABI (include/gspn_attention.h): the library exports every declared symbol, the
binding's structs follow the header's, host-side validation rejects bad arguments before anything reaches a device, and
every launch's replay (libgspn_check.so) stays in its buffers.  No call into the real library passes validation with a
non-empty tensor, so nothing is launched."""
import ctypes
import os
import re

import pytest
import torch

from linear_spatial_propagation_gspn_amd import attention as A
from linear_spatial_propagation_gspn_amd import build as hipbuild
from linear_spatial_propagation_gspn_amd import sequence as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gspn_attention.h")
OK, NULLP, SHAPE, DIR, DTYPE, CHUNK, WCH, MISAL, ALIAS, UNSUP, HIP, WSPACE, LAYOUT = range(13)
F32, BF16 = 0, 1


def _header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


@pytest.fixture(scope="module")
def lib():
    return A.lib()


def test_library_exports_every_declared_symbol(lib):
    declared = set(re.findall(r"\b(gspn_[a-z0-9_]+)\s*\(", _header()))
    assert declared == set(A.EXPORTS)
    for name in declared:
        assert hasattr(lib, name), name


@pytest.mark.parametrize("name,struct", [("gspn_rotary_args", A.RotaryArgs), ("gspn_attn_args", A.AttnArgs)])
def test_structs_follow_the_header(name, struct):
    body = re.search(r"typedef struct \{([^}]*)\} %s;" % name, _header()).group(1)
    fields = []
    for line in body.split(";"):
        if not line.strip():
            continue
        m = re.match(r"\s*(const\s+)?(\w+)(\*?)\s+(.*)$", line.strip(), re.S)
        for f in m.group(4).split(","):
            kind = S.Sequences if m.group(2) == "gspn_sequences" else ctypes.c_void_p if m.group(3) else {
                "int64_t": ctypes.c_int64, "double": ctypes.c_double}[m.group(2)]
            f = f.strip()
            if f.endswith("[GSPN_ROTARY_MAX_AXES]"):
                f, kind = f.split("[")[0], kind * A.GSPN_ROTARY_MAX_AXES
            fields.append((f, kind))
    assert fields == [tuple(f) for f in struct._fields_]


def test_limits_follow_the_header():
    for name in ("GSPN_ATTENTION_MAX_HEAD", "GSPN_ROTARY_MAX_HEAD", "GSPN_ROTARY_MAX_AXES"):
        assert int(re.search(r"#define %s (\d+)" % name, _header()).group(1)) == getattr(A, name)


class Space:
    """Made-up device addresses, far apart; with a check library, registered there as buffers of the given size."""

    def __init__(self, chk=None):
        self.next, self.chk = 1 << 44, chk
        if chk:
            chk.gspn_check_reset()

    def __call__(self, name, nbytes):
        at = self.next
        self.next += 1 << 37
        if self.chk and nbytes:
            assert self.chk.gspn_check_add_buffer(name.encode(), at, nbytes) == 0
        return at


def rotary_args(sp, lib, dt=F32, rows=9, heads=3, kv_heads=2, d=20, sections=(4, 2), kind="fwd", ld=0, norm=True):
    es = 4 if dt == F32 else 2
    a = A.RotaryArgs()
    a.rows, a.heads, a.kv_heads, a.d, a.pairs, a.axes, a.eps = rows, heads, kv_heads, d, sum(sections), len(sections), 1e-6
    a.section[:len(sections)] = sections
    ldq, ldk = (ld or h * d for h in (heads, kv_heads))
    size = {"q": ((rows - 1) * ldq + heads * d) * es, "k": ((rows - 1) * ldk + kv_heads * d) * es}
    a.positions, a.ldpos = sp("positions", rows * a.axes * 4), a.axes
    a.freqs = sp("freqs", a.pairs * 8)
    for n in ("q", "k")[:2 if kv_heads else 1]:
        both = [n, n + "_out"] if kind == "fwd" else [n, "g" + n, "d" + n]
        for f in both:
            setattr(a, f, sp(f, size[n]))
            setattr(a, "ld" + f.replace("_out", "o"), ldq if n == "q" else ldk)
        if norm:
            setattr(a, n + "_weight", sp(n + "_weight", d * 4))
            if kind == "bwd":
                setattr(a, "d%s_weight" % n, sp("d%s_weight" % n, d * 4))
    if kind == "bwd":
        a.workspace_bytes = lib.gspn_head_rotary_bwd_workspace_bytes(rows, d)
        a.workspace = sp("workspace", a.workspace_bytes)
    return a


def attn_args(sp, lib, dt=F32, rows=40, nseq=2, kv_rows=None, heads=6, kv_heads=2, d=20, kind="fwd", cu=False, kv_cu=False,
              capacity=0, slots=0, held=True, ld=0, lse=True, causal=1):
    es = 4 if dt == F32 else 2
    a = A.AttnArgs()
    if kind == "step":
        rows, capacity = nseq, capacity or 50
    a.seq.rows, a.seq.nseq, a.kv_rows = rows, nseq, rows if kv_rows is None else kv_rows
    if cu:
        a.seq.cu = sp("cu", 4 * (nseq + 1))
    if kv_cu:
        a.kv_cu = sp("kv_cu", 4 * (nseq + 1))
    a.heads, a.kv_heads, a.d, a.causal, a.scale = heads, kv_heads, d, causal, 0.2
    ldq, ldk = (ld or h * d for h in (heads, kv_heads))
    qs = max(0, (rows - 1) * ldq + heads * d) * es
    ks = max(0, (a.kv_rows - 1) * ldk + kv_heads * d) * es
    for f, size, l in (("q", qs, ldq), ("k", ks, ldk), ("v", ks, ldk), ("out", qs, ldq)):
        setattr(a, f, sp(f, size))
        setattr(a, "ldo" if f == "out" else "ld" + f, l)
    if kind == "bwd" or (kind == "fwd" and lse):
        a.lse = sp("lse", heads * rows * 4)
    if capacity:
        a.capacity, a.seq.nslots = capacity, slots or nseq
        a.k_pool, a.v_pool = (sp(f, a.seq.nslots * capacity * kv_heads * d * es) for f in ("k_pool", "v_pool"))
        if slots:
            a.seq.slots = sp("slots", nseq * 4)
        if held:
            a.held = sp("held", nseq * 4)
    if kind == "bwd":
        for f, size, l in (("gout", qs, ldq), ("dq", qs, ldq), ("dk", ks, ldk), ("dv", ks, ldk)):
            setattr(a, f, sp(f, size))
            setattr(a, "ldgo" if f == "gout" else "ld" + f, l)
        a.workspace_bytes = lib.gspn_attention_bwd_workspace_bytes(rows, nseq, heads, a.kv_rows, kv_heads, d)
    if kind == "step":
        a.workspace_bytes = lib.gspn_attention_step_workspace_bytes(nseq, heads, kv_heads, d, capacity)
    if a.workspace_bytes:
        a.workspace = sp("workspace", a.workspace_bytes)
    return a


CALLS = {"rotary": (rotary_args, "gspn_head_rotary_"), "attn": (attn_args, "gspn_attention_")}


def refuse(lib, op, kind, want, dtype=F32, build=None, **change):
    """A call that is right but for ``change`` (field or field of seq -> value) returns ``want``."""
    make, prefix = CALLS[op]
    a = make(Space(), lib, kind=kind, **(build or {}))
    for f, v in change.items():
        v = v(a) if callable(v) else v
        if f.startswith("seq_"):
            setattr(a.seq, f[4:], v)
        elif f.startswith("section"):
            a.section[int(f[7:])] = v
        else:
            setattr(a, f, v)
    assert getattr(lib, prefix + kind)(ctypes.byref(a), dtype, None) == want, (op, kind, change)


def test_rotary_validation(lib):
    assert lib.gspn_head_rotary_fwd(None, F32, None) == NULLP
    for kind in ("fwd", "bwd"):
        refuse(lib, "rotary", kind, DTYPE, dtype=2)
        refuse(lib, "rotary", kind, SHAPE, rows=-1)
        refuse(lib, "rotary", kind, SHAPE, rows=(1 << 30) + 1)
        refuse(lib, "rotary", kind, SHAPE, heads=0)
        refuse(lib, "rotary", kind, SHAPE, kv_heads=-1)
        refuse(lib, "rotary", kind, SHAPE, d=0)
        refuse(lib, "rotary", kind, SHAPE, d=11)              # six pairs need twelve elements
        refuse(lib, "rotary", kind, UNSUP, d=257)
        refuse(lib, "rotary", kind, UNSUP, heads=4097)
        refuse(lib, "rotary", kind, UNSUP, axes=5)
        refuse(lib, "rotary", kind, SHAPE, axes=0)
        refuse(lib, "rotary", kind, SHAPE, axes=1)            # four of six pairs
        refuse(lib, "rotary", kind, SHAPE, section0=-4, section1=10)
        refuse(lib, "rotary", kind, SHAPE, pairs=-1)
        refuse(lib, "rotary", kind, SHAPE, eps=-1.0)
        refuse(lib, "rotary", kind, SHAPE, eps=float("inf"))
        refuse(lib, "rotary", kind, SHAPE, ldq=59)
        refuse(lib, "rotary", kind, SHAPE, ldpos=1)
        refuse(lib, "rotary", kind, UNSUP, ldk=(1 << 26) + 1)
        for f in ("q", "k", "positions", "freqs"):
            refuse(lib, "rotary", kind, NULLP, **{f: None})
        refuse(lib, "rotary", kind, MISAL, freqs=lambda a: a.freqs + 4)
        refuse(lib, "rotary", kind, MISAL, positions=lambda a: a.positions + 2)
        refuse(lib, "rotary", kind, MISAL, q_weight=lambda a: a.q_weight + 2)
        refuse(lib, "rotary", kind, MISAL, q=lambda a: a.q + 2)
        refuse(lib, "rotary", kind, MISAL, dtype=BF16, q=lambda a: a.q + 1)
    for f in ("q_out", "k_out"):
        refuse(lib, "rotary", "fwd", NULLP, **{f: None})
        refuse(lib, "rotary", "fwd", ALIAS, **{f: lambda a, f=f: getattr(a, f[0])})
    refuse(lib, "rotary", "fwd", ALIAS, k_out=lambda a: a.q_out + 8)
    for f in ("gq", "gk", "dq", "dk"):
        refuse(lib, "rotary", "bwd", NULLP, **{f: None})
    refuse(lib, "rotary", "bwd", NULLP, q_weight=None)        # its gradient without it
    refuse(lib, "rotary", "bwd", ALIAS, dq=lambda a: a.gq)
    refuse(lib, "rotary", "bwd", ALIAS, dk_weight=lambda a: a.dq_weight + 4)
    refuse(lib, "rotary", "bwd", WSPACE, workspace_bytes=lambda a: a.workspace_bytes - 1)
    refuse(lib, "rotary", "bwd", NULLP, workspace=None)
    refuse(lib, "rotary", "fwd", OK, rows=0, q=None, positions=None, q_out=None)
    assert lib.gspn_head_rotary_bwd_workspace_bytes(40, 257) == -1
    assert lib.gspn_head_rotary_bwd_workspace_bytes(-1, 4) == -1


def test_attention_validation(lib):
    assert lib.gspn_attention_fwd(None, F32, None) == NULLP
    for kind in ("fwd", "step", "bwd"):
        refuse(lib, "attn", kind, DTYPE, dtype=-1)
        refuse(lib, "attn", kind, SHAPE, heads=0)
        refuse(lib, "attn", kind, SHAPE, kv_heads=0)
        refuse(lib, "attn", kind, SHAPE, kv_heads=4)          # does not divide 6
        refuse(lib, "attn", kind, SHAPE, d=0)
        refuse(lib, "attn", kind, UNSUP, d=129)
        refuse(lib, "attn", kind, UNSUP, heads=4098, ldq=4098 * 20, ldo=4098 * 20)
        for bad in (float("nan"), float("inf"), 1e39):
            refuse(lib, "attn", kind, SHAPE, scale=bad)
        refuse(lib, "attn", kind, SHAPE, seq_rows=-1)
        refuse(lib, "attn", kind, SHAPE, seq_rows=(1 << 30) + 2)
        refuse(lib, "attn", kind, SHAPE, kv_rows=-1)
        refuse(lib, "attn", kind, SHAPE, kv_rows=(1 << 30) - 1)
        refuse(lib, "attn", kind, SHAPE, seq_resume=64)
        refuse(lib, "attn", kind, SHAPE, ldq=119)
        refuse(lib, "attn", kind, SHAPE, ldv=39)
        refuse(lib, "attn", kind, UNSUP, ldk=(1 << 26) + 1)
        for f in ("q", "k", "v", "out"):
            refuse(lib, "attn", kind, NULLP, **{f: None})
            refuse(lib, "attn", kind, MISAL, **{f: lambda a, f=f: getattr(a, f) + 2})
    for kind in ("fwd", "bwd"):
        refuse(lib, "attn", kind, SHAPE, kv_rows=41)          # not two equal sequences
        refuse(lib, "attn", kind, SHAPE, build=dict(cu=True), kv_rows=38)  # of other lengths, without offsets
        refuse(lib, "attn", kind, MISAL, build=dict(kv_cu=True), kv_cu=lambda a: a.kv_cu + 2)
        refuse(lib, "attn", kind, MISAL, build=dict(cu=True), seq_cu=2)
        refuse(lib, "attn", kind, SHAPE, seq_nseq=3)
        refuse(lib, "attn", kind, SHAPE, seq_slots=64)        # no cache
        refuse(lib, "attn", kind, SHAPE, held=64)
        # 2^32 lanes are a launch's most: workgroups of 128 rows of a head
        refuse(lib, "attn", kind, UNSUP, seq_rows=1 << 29, seq_nseq=1, kv_rows=1 << 29)
        refuse(lib, "attn", kind, UNSUP, seq_rows=1 << 23, seq_nseq=1 << 23, kv_rows=1 << 23)
    refuse(lib, "attn", "fwd", ALIAS, out=lambda a: a.q)
    refuse(lib, "attn", "fwd", ALIAS, lse=lambda a: a.out)
    cache = dict(rows=40, capacity=50, slots=5)
    refuse(lib, "attn", "fwd", NULLP, build=cache, v_pool=None)
    refuse(lib, "attn", "fwd", NULLP, build=cache, k_pool=None)
    refuse(lib, "attn", "fwd", SHAPE, build=cache, capacity=0)
    refuse(lib, "attn", "fwd", SHAPE, build=cache, kv_rows=38)
    refuse(lib, "attn", "fwd", SHAPE, build=cache, kv_cu=64)
    refuse(lib, "attn", "fwd", SHAPE, build=dict(rows=40, capacity=50), seq_nslots=1)
    refuse(lib, "attn", "fwd", UNSUP, build=cache, capacity=1 << 30, seq_nslots=1 << 20)
    refuse(lib, "attn", "fwd", ALIAS, build=cache, k_pool=lambda a: a.v_pool)
    refuse(lib, "attn", "fwd", ALIAS, build=cache, k_pool=lambda a: a.k)
    refuse(lib, "attn", "fwd", MISAL, build=cache, held=lambda a: a.held + 2)
    for f in ("k_pool", "v_pool", "held"):
        refuse(lib, "attn", "step", NULLP, **{f: None})
    refuse(lib, "attn", "step", SHAPE, lse=64)
    refuse(lib, "attn", "step", SHAPE, seq_rows=4)
    refuse(lib, "attn", "step", SHAPE, seq_cu=64)
    refuse(lib, "attn", "step", SHAPE, kv_cu=64)
    big = dict(capacity=5000)
    refuse(lib, "attn", "step", WSPACE, build=big, workspace_bytes=lambda a: a.workspace_bytes - 1)
    refuse(lib, "attn", "step", NULLP, build=big, workspace=None)
    refuse(lib, "attn", "step", MISAL, build=big, workspace=lambda a: a.workspace + 8)
    refuse(lib, "attn", "step", ALIAS, build=big, workspace=lambda a: a.k_pool)
    refuse(lib, "attn", "bwd", UNSUP, k_pool=64, v_pool=64)
    for f in ("lse", "gout", "dq", "dk", "dv", "workspace"):
        refuse(lib, "attn", "bwd", NULLP, **{f: None})
    refuse(lib, "attn", "bwd", WSPACE, workspace_bytes=lambda a: a.workspace_bytes - 1)
    refuse(lib, "attn", "bwd", ALIAS, dq=lambda a: a.gout)
    refuse(lib, "attn", "bwd", ALIAS, dk=lambda a: a.dv + 4)
    refuse(lib, "attn", "bwd", ALIAS, dv=lambda a: a.out)
    # nothing to do: no pointer is looked at
    refuse(lib, "attn", "fwd", OK, seq_rows=0, seq_nseq=0, kv_rows=0, q=None, k=None, v=None, out=None)
    refuse(lib, "attn", "fwd", OK, seq_rows=0, q=None, k=None)
    refuse(lib, "attn", "bwd", OK, seq_rows=0, kv_rows=0, q=None, dk=None)
    assert lib.gspn_attention_bwd_workspace_bytes(40, 2, 6, 40, 4, 20) == -1
    assert lib.gspn_attention_step_workspace_bytes(40, 6, 2, 129, 20) == -1
    assert lib.gspn_attention_step_workspace_bytes(64, 8, 8, 64, 128) == 0  # one run each


def test_python_refusals():
    x, w = torch.zeros(4, 2, 8), torch.zeros(8)
    pos, freqs = torch.zeros(4, 1, dtype=torch.int32), torch.zeros(4, dtype=torch.float64)
    pools, held = (torch.zeros(4, 9, 2, 8), torch.zeros(4, 9, 2, 8)), torch.zeros(4, dtype=torch.int32)
    for call in (lambda: A.gspn_head_rotary_fwd(x, pos, freqs), lambda: A.gspn_head_rotary_bwd(x, pos, freqs, x),
                 lambda: A.gspn_attention_fwd(x, x, x), lambda: A.gspn_attention_step(x, x, x, pools, held),
                 lambda: A.gspn_attention_bwd(x, x, x, x, None, x), lambda: A.attention(x, x, x),
                 lambda: A.head_rotary(x, pos, freqs, q_weight=w)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        A.gspn_attention_fwd([1.0], x, x)
    with pytest.raises(ValueError):
        A.gspn_attention_fwd(torch.zeros(4, 8), x, x)


def test_forward_mode_is_refused():
    from torch.autograd import forward_ad
    x, pos, freqs = torch.zeros(4, 2, 8), torch.zeros(4, 1, dtype=torch.int32), torch.zeros(4, dtype=torch.float64)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        with pytest.raises(NotImplementedError):
            A.attention(x, dual, x)
        with pytest.raises(NotImplementedError):
            A.head_rotary(dual, pos, freqs)
    with pytest.raises(NotImplementedError):
        A.head_rotary(x, pos, freqs.requires_grad_())


# ------------------------------------------------------------------------------------------- launch replays

@pytest.fixture(scope="module")
def chk():
    newest = max(os.path.getmtime(os.path.join(hipbuild.CSRC, f)) for f in os.listdir(hipbuild.CSRC))
    if not os.path.exists(hipbuild.CHECK_LIB) or os.path.getmtime(hipbuild.CHECK_LIB) < newest:
        hipbuild.build_check()
    h = ctypes.CDLL(hipbuild.CHECK_LIB)
    h.gspn_check_add_buffer.argtypes = [ctypes.c_char_p, ctypes.c_uint64, ctypes.c_uint64]
    for f in ("violations", "accesses", "launches", "report"):
        getattr(h, "gspn_check_" + f).restype = ctypes.c_int64
    h.gspn_check_report.argtypes = [ctypes.c_char_p, ctypes.c_int64]
    for name in A.EXPORTS:
        if not name.endswith("_bytes"):
            getattr(h, name).argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]
    return h


def replay(chk, lib, op, kind, dt=F32, **kw):
    make, prefix = CALLS[op]
    a = make(Space(chk), lib, dt=dt, kind=kind, **kw)
    assert getattr(chk, prefix + kind)(ctypes.byref(a), dt, None) == OK
    buf = ctypes.create_string_buffer(1 << 16)
    chk.gspn_check_report(buf, 1 << 16)
    text = buf.value.decode()
    assert chk.gspn_check_violations() == 0, text
    return [line.split()[1].strip("(").split("<")[0] for line in text.splitlines() if line.startswith("launch ")]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("d", [1, 20, 64, 72, 96, 128])
@pytest.mark.parametrize("ld", [0, 900])
def test_launches_stay_in_their_buffers(chk, lib, dt, d, ld):
    for cu in (False, True):
        for rows, nseq in ((40, 2), (1, 1), (1200, 3)):
            kw = dict(d=d, ld=ld, rows=rows, nseq=nseq, cu=cu)
            assert replay(chk, lib, "attn", "fwd", dt, **kw) == ["attn_fwd_kernel"]
            assert replay(chk, lib, "attn", "fwd", dt, capacity=1300, slots=5, **kw) == ["attn_fwd_kernel"]
            clear = ["reduce_parts_kernel"] * (2 if cu else 0)
            parts = ["attn_parts_kernel"] * (rows == 1200)  # rows enough to be cut
            assert replay(chk, lib, "attn", "bwd", dt, **kw) == clear + ["attn_dq_kernel", "attn_dkv_kernel"] + parts
            assert replay(chk, lib, "attn", "bwd", dt, kv_rows=60, kv_cu=True, **kw)[-2 - len(parts):] == [
                "attn_dq_kernel", "attn_dkv_kernel"] + parts
    assert replay(chk, lib, "attn", "step", dt, d=d, ld=ld, nseq=3, slots=5) == ["attn_step_kernel"]
    assert replay(chk, lib, "attn", "step", dt, d=d, ld=ld, nseq=3, capacity=5000) == ["attn_step_kernel",
                                                                                       "attn_step_join_kernel"]
    for sections in ((d // 2,), (d // 4, 0, d // 4)):
        kw = dict(d=d, sections=sections, ld=ld)
        assert replay(chk, lib, "rotary", "fwd", dt, **kw) == ["rotary_fwd_kernel"]
        assert replay(chk, lib, "rotary", "bwd", dt, **kw) == ["rotary_bwd_kernel", "reduce_parts_kernel"]
        assert replay(chk, lib, "rotary", "bwd", dt, norm=False, kv_heads=0, **kw) == ["rotary_bwd_kernel"]


def test_the_replay_sees_an_overrun(chk, lib):
    """An entry one row short is reported."""
    sp = Space(chk)
    a = attn_args(sp, lib, rows=40)
    a.capacity, a.seq.nslots = 50, 2
    a.k_pool, a.v_pool = sp("k_pool", 2 * 50 * 40 * 4), sp("v_pool", (2 * 50 - 1) * 40 * 4)
    assert chk.gspn_attention_fwd(ctypes.byref(a), F32, None) == OK
    assert chk.gspn_check_violations() > 0
