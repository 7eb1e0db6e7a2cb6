"""CPU tests of the sequence operators' C ABI (include/gspn_sequence.h): the
library exports every declared symbol, the binding's structs follow the
header's, host-side validation rejects bad arguments before anything reaches a
device, and every launch's replay (libgspn_check.so) stays in its buffers.  No
call into the real library passes validation with a non-empty tensor, so
nothing is launched."""
import ctypes
import os
import re

import pytest
import torch

from linear_spatial_propagation_gspn_amd import build as hipbuild
from linear_spatial_propagation_gspn_amd import gspn as G
from linear_spatial_propagation_gspn_amd import sequence as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gspn_sequence.h")
OK, NULLP, SHAPE, DIR, DTYPE, CHUNK, WCH, MISAL, ALIAS, UNSUP, HIP, WSPACE, LAYOUT = range(13)
F32, BF16 = 0, 1


def _header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


@pytest.fixture(scope="module")
def lib():
    return S.lib()


def test_library_exports_every_declared_symbol(lib):
    declared = set(re.findall(r"\b(gspn_[a-z0-9_]+)\s*\(", _header()))
    assert declared == set(S.EXPORTS)
    for name in declared:
        assert hasattr(lib, name), name


@pytest.mark.parametrize("name,struct", [("gspn_sequences", S.Sequences), ("gspn_conv_args", S.ConvArgs),
                                         ("gspn_selscan_args", S.SelscanArgs), ("gspn_join_args", S.JoinArgs)])
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
            fields.append((f.strip(), kind))
    assert fields == [tuple(f) for f in struct._fields_]


def test_limits_follow_the_header():
    for name in ("GSPN_CONV_MIN_WIDTH", "GSPN_CONV_MAX_WIDTH", "GSPN_SCAN_MAX_STATE", "GSPN_JOIN_MAX_CHANNELS",
                 "GSPN_SCAN_CHECKPOINT_ROWS"):
        assert int(re.search(r"#define %s (\d+)" % name, _header()).group(1)) == getattr(S, name)


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


def seq(sp, rows, nseq, cu=False, slots=0, resume=False, pool=False):
    s = S.Sequences()
    s.rows, s.nseq = rows, nseq
    if cu:
        s.cu = sp("cu", 4 * (nseq + 1))
    if pool:
        s.nslots = slots or nseq
    if slots:
        s.slots = sp("slots", 4 * nseq)
    if resume:
        s.resume = sp("resume", nseq)
    return s


def conv_args(sp, lib, dt=F32, rows=40, nseq=2, c=24, width=4, kind="fwd", pool=False, ld=0, **kw):
    es = 4 if dt == F32 else 2
    a = S.ConvArgs()
    a.seq = seq(sp, rows, nseq, pool=pool, **kw)
    ld = ld or c
    size = ((rows - 1) * ld + c) * es
    a.c, a.width, a.silu = c, width, 1
    a.x, a.ldx = sp("x", size), ld
    a.weight, a.bias = sp("weight", c * width * 4), sp("bias", c * 4)
    if kind == "bwd":
        a.gy, a.ldgy = sp("gy", size), ld
        a.dx, a.lddx = sp("dx", size), ld
        a.dweight, a.dbias = sp("dweight", c * width * 4), sp("dbias", c * 4)
        a.workspace_bytes = lib.gspn_causal_conv_bwd_workspace_bytes(rows, nseq, c, width)
        a.workspace = sp("workspace", a.workspace_bytes)
    else:
        a.y, a.ldy = sp("y", size), ld
    if pool:
        a.state = sp("state", a.seq.nslots * (width - 1) * c * es)
    return a


def scan_args(sp, lib, dt=F32, rows=40, nseq=2, c=24, groups=2, n=16, kind="fwd", pool=False, ld=0, gate=True,
              keep=False, **kw):
    es = 4 if dt == F32 else 2
    a = S.SelscanArgs()
    a.seq = seq(sp, rows, nseq, pool=pool, **kw)
    cu = 1 if kw.get("cu") else 0
    ld = ld or c
    size = ((rows - 1) * ld + c) * es
    bc = ((rows - 1) * (ld + 100) + groups * n) * es
    a.channels, a.groups, a.n, a.softplus = c, groups, n, 1
    a.x, a.ldx = sp("x", size), ld
    a.dt, a.lddt = sp("dt", size), ld
    if gate:
        a.z, a.ldz = sp("z", size), ld
    a.B, a.ldb = sp("B", bc), ld + 100
    a.C, a.ldc = sp("C", bc), ld + 100
    a.A, a.D, a.dt_bias = sp("A", c * n * 4), sp("D", c * 4), sp("dt_bias", c * 4)
    kept = lib.gspn_selective_scan_checkpoint_bytes(rows, nseq, c, n, cu)
    if keep or kind == "bwd":
        a.checkpoints = sp("checkpoints", kept)
    if kind == "bwd":
        a.gy, a.ldgy = sp("gy", size), ld
        a.dx, a.lddx = sp("dx", size), ld
        a.ddt, a.ldddt = sp("ddt", size), ld
        if gate:
            a.dz, a.lddz = sp("dz", size), ld
        a.dB, a.dC = sp("dB", rows * groups * n * es), sp("dC", rows * groups * n * es)
        a.dA, a.dD, a.ddt_bias = sp("dA", c * n * 4), sp("dD", c * 4), sp("ddt_bias", c * 4)
        a.workspace_bytes = lib.gspn_selective_scan_bwd_workspace_bytes(rows, nseq, c, groups, n, cu)
    else:
        a.out, a.ldo = sp("out", size), ld
        a.workspace_bytes = lib.gspn_selective_scan_workspace_bytes(rows, nseq, c, groups, n, cu)
    if a.workspace_bytes:
        a.workspace = sp("workspace", a.workspace_bytes)
    if pool:
        a.state = sp("state", a.seq.nslots * c * n * 4)
    return a


def join_args(sp, lib, dt=F32, rdt=F32, rows=9, c=40, kind="fwd", parts="grosp", ld=0):
    es, rs = (4 if d == F32 else 2 for d in (dt, rdt))
    a = S.JoinArgs()
    ld = ld or c
    size = lambda e: ((rows - 1) * ld + c) * e  # noqa: E731
    a.rows, a.c, a.residual_dtype, a.eps = rows, c, rdt, 1e-6
    a.h, a.ldh = sp("h", size(es)), ld
    if "g" in parts:
        a.gate, a.ldgate = sp("gate", size(es)), ld
    if "r" in parts and kind == "fwd":
        a.residual, a.ldres = sp("residual", size(rs)), ld
    for letter, f in (("o", "post"), ("s", "scale"), ("p", "pre")):
        if letter in parts:
            setattr(a, f, sp(f, c * 4))
            if kind == "bwd":
                setattr(a, "d" + f, sp("d" + f, c * 4))
    a.joined, a.ldjoined = sp("joined", size(rs)), ld
    if kind == "fwd":
        if "p" in parts:
            a.normed, a.ldnormed = sp("normed", size(es)), ld
        return a
    a.gjoined, a.ldgjoined = sp("gjoined", size(rs)), ld
    if "p" in parts:
        a.gnormed, a.ldgnormed = sp("gnormed", size(es)), ld
    a.dh, a.lddh = sp("dh", size(es)), ld
    if "g" in parts:
        a.dgate, a.lddgate = sp("dgate", size(es)), ld
    if "r" in parts:
        a.dresidual, a.lddres = sp("dresidual", size(rs)), ld
    a.workspace_bytes = lib.gspn_block_join_bwd_workspace_bytes(rows, c)
    a.workspace = sp("workspace", a.workspace_bytes)
    return a


CALLS = {"conv": (conv_args, "gspn_causal_conv_"), "scan": (scan_args, "gspn_selective_scan_"),
         "join": (join_args, "gspn_block_join_")}


def refuse(lib, op, kind, want, dtype=F32, build=None, **change):
    """A call that is right but for ``change`` (field or field of seq -> value) returns ``want``."""
    make, prefix = CALLS[op]
    a = make(Space(), lib, kind=kind, **(build or {}))
    for f, v in change.items():
        v = v(a) if callable(v) else v
        if f.startswith("seq_"):
            setattr(a.seq, f[4:], v)
        else:
            setattr(a, f, v)
    assert getattr(lib, prefix + kind)(ctypes.byref(a), dtype, None) == want, (op, kind, change)


def test_conv_validation(lib):
    assert lib.gspn_causal_conv_fwd(None, F32, None) == NULLP
    refuse(lib, "conv", "fwd", DTYPE, dtype=2)
    for kind in ("fwd", "bwd"):
        refuse(lib, "conv", kind, SHAPE, c=-1)
        refuse(lib, "conv", kind, SHAPE, c=(1 << 19) + 1)
        refuse(lib, "conv", kind, UNSUP, width=1)
        refuse(lib, "conv", kind, UNSUP, width=5)
        refuse(lib, "conv", kind, SHAPE, seq_rows=-1)
        refuse(lib, "conv", kind, SHAPE, seq_rows=(1 << 31) - 1)  # with the sequences past 2^31 chunk ids
        refuse(lib, "conv", kind, UNSUP, seq_rows=1 << 24, seq_nseq=(1 << 23) + 1)
        refuse(lib, "conv", kind, SHAPE, seq_rows=(1 << 30) + 2)
        refuse(lib, "conv", kind, SHAPE, seq_nseq=3)          # does not divide 40 rows
        refuse(lib, "conv", kind, SHAPE, seq_nseq=0)          # rows without a sequence
        refuse(lib, "conv", kind, SHAPE, ldx=23)
        refuse(lib, "conv", kind, NULLP, x=None)
        refuse(lib, "conv", kind, NULLP, weight=None)
        refuse(lib, "conv", kind, MISAL, x=lambda a: a.x + 2)
        refuse(lib, "conv", kind, MISAL, weight=lambda a: a.weight + 1)
        refuse(lib, "conv", kind, MISAL, seq_cu=2)
        refuse(lib, "conv", kind, SHAPE, seq_resume=64)       # no pool to resume from
    refuse(lib, "conv", "fwd", NULLP, y=None)
    refuse(lib, "conv", "step", UNSUP, seq_rows=(1 << 16) + 1, seq_nseq=(1 << 16) + 1, seq_slots=64, seq_nslots=1 << 17)
    refuse(lib, "conv", "fwd", ALIAS, y=lambda a: a.x + 8)
    refuse(lib, "conv", "fwd", ALIAS, y=lambda a: a.weight)
    # column slices of one matrix: a slice that reaches into the other, or past its row's end into the next
    refuse(lib, "conv", "fwd", ALIAS, build=dict(ld=60), y=lambda a: a.x + 23 * 4)
    refuse(lib, "conv", "fwd", ALIAS, build=dict(ld=60), y=lambda a: a.x + 37 * 4)
    refuse(lib, "conv", "fwd", ALIAS, build=dict(ld=60), y=lambda a: a.x + 24 * 4, ldy=59)
    refuse(lib, "conv", "fwd", ALIAS, build=dict(pool=True), state=lambda a: a.y)
    refuse(lib, "conv", "fwd", SHAPE, build=dict(pool=True), seq_nslots=1)
    refuse(lib, "conv", "step", NULLP, build=dict(rows=2, pool=True), state=None)
    refuse(lib, "conv", "step", SHAPE, build=dict(rows=4, pool=True))
    refuse(lib, "conv", "step", SHAPE, build=dict(rows=2, pool=True, resume=True))
    refuse(lib, "conv", "step", SHAPE, build=dict(rows=2, pool=True, cu=True))
    refuse(lib, "conv", "bwd", UNSUP, state=64)
    refuse(lib, "conv", "bwd", WSPACE, workspace_bytes=lambda a: a.workspace_bytes - 1)
    refuse(lib, "conv", "bwd", NULLP, workspace=None)
    refuse(lib, "conv", "bwd", NULLP, dweight=None)
    refuse(lib, "conv", "bwd", ALIAS, dbias=lambda a: a.bias)
    refuse(lib, "conv", "bwd", ALIAS, dx=lambda a: a.gy)
    # nothing to do: no pointer is looked at
    refuse(lib, "conv", "fwd", OK, seq_rows=0, seq_nseq=0, x=None, y=None, weight=None)
    refuse(lib, "conv", "fwd", OK, c=0, ldx=0, x=None)
    assert lib.gspn_causal_conv_bwd_workspace_bytes(40, 2, 24, 5) == -1


def test_scan_validation(lib):
    assert lib.gspn_selective_scan_fwd(None, F32, None) == NULLP
    for kind in ("fwd", "bwd"):
        refuse(lib, "scan", kind, DTYPE, dtype=-1)
        refuse(lib, "scan", kind, UNSUP, n=17)
        refuse(lib, "scan", kind, SHAPE, n=0)
        refuse(lib, "scan", kind, SHAPE, groups=0)
        refuse(lib, "scan", kind, SHAPE, groups=5)
        refuse(lib, "scan", kind, UNSUP, channels=1 << 17, groups=1 << 17)
        refuse(lib, "scan", kind, SHAPE, seq_nseq=7)
        refuse(lib, "scan", kind, SHAPE, lddt=23)
        refuse(lib, "scan", kind, SHAPE, ldb=31)
        refuse(lib, "scan", kind, UNSUP, ldc=(1 << 26) + 1)
        for f in ("x", "dt", "B", "C", "A"):
            refuse(lib, "scan", kind, NULLP, **{f: None})
            refuse(lib, "scan", kind, MISAL, **{f: lambda a, f=f: getattr(a, f) + 2})
        refuse(lib, "scan", kind, MISAL, dt_bias=lambda a: a.dt_bias + 2)
    refuse(lib, "scan", "fwd", NULLP, out=None)
    refuse(lib, "scan", "fwd", ALIAS, out=lambda a: a.z)
    refuse(lib, "scan", "fwd", ALIAS, build=dict(keep=True), checkpoints=lambda a: a.out)
    refuse(lib, "scan", "fwd", WSPACE, build=dict(rows=400), workspace_bytes=lambda a: a.workspace_bytes - 1)
    refuse(lib, "scan", "fwd", NULLP, build=dict(rows=400), workspace=None)
    refuse(lib, "scan", "fwd", ALIAS, build=dict(rows=400, pool=True), state=lambda a: a.workspace)
    refuse(lib, "scan", "step", NULLP, build=dict(rows=2, pool=True), state=None)
    refuse(lib, "scan", "step", SHAPE, build=dict(rows=4, pool=True))
    refuse(lib, "scan", "bwd", UNSUP, state=64)
    refuse(lib, "scan", "bwd", NULLP, checkpoints=None)
    refuse(lib, "scan", "bwd", NULLP, dz=None)
    refuse(lib, "scan", "bwd", NULLP, dA=None)
    refuse(lib, "scan", "bwd", WSPACE, workspace_bytes=0)
    refuse(lib, "scan", "bwd", ALIAS, dB=lambda a: a.dC)
    refuse(lib, "scan", "bwd", ALIAS, ddt=lambda a: a.dx + 4)
    refuse(lib, "scan", "fwd", OK, seq_rows=0, seq_nseq=0, x=None, A=None)
    assert lib.gspn_selective_scan_workspace_bytes(40, 2, 24, 5, 16, 0) == -1
    assert lib.gspn_selective_scan_workspace_bytes(16, 1, 24, 1, 16, 1) == 0  # one chunk
    # states before rows 0, 8, .. 32 of each sequence; packed: room for any offsets
    assert lib.gspn_selective_scan_checkpoint_bytes(80, 2, 24, 16, 0) == 2 * 5 * 16 * 24 * 4
    assert lib.gspn_selective_scan_checkpoint_bytes(80, 2, 24, 16, 1) == (80 // 8 + 2) * 16 * 24 * 4


def test_join_validation(lib):
    assert lib.gspn_block_join_fwd(None, F32, None) == NULLP
    for kind in ("fwd", "bwd"):
        refuse(lib, "join", kind, DTYPE, dtype=2)
        refuse(lib, "join", kind, DTYPE, residual_dtype=BF16)  # narrower than the storage type
        refuse(lib, "join", kind, SHAPE, rows=-1)
        refuse(lib, "join", kind, SHAPE, eps=-1e-6)
        refuse(lib, "join", kind, SHAPE, eps=float("nan"))
        refuse(lib, "join", kind, UNSUP, c=16385)
        refuse(lib, "join", kind, SHAPE, ldgate=39)
        refuse(lib, "join", kind, NULLP, h=None)
        refuse(lib, "join", kind, NULLP, joined=None)
        refuse(lib, "join", kind, MISAL, pre=lambda a: a.pre + 2)
    refuse(lib, "join", "fwd", NULLP, normed=None)
    refuse(lib, "join", "fwd", ALIAS, joined=lambda a: a.residual)
    refuse(lib, "join", "bwd", NULLP, gnormed=None)
    refuse(lib, "join", "bwd", NULLP, post=None)   # dpost without it
    refuse(lib, "join", "bwd", NULLP, gate=None)
    refuse(lib, "join", "bwd", WSPACE, workspace_bytes=lambda a: a.workspace_bytes - 1)
    refuse(lib, "join", "bwd", ALIAS, dh=lambda a: a.gjoined)
    refuse(lib, "join", "bwd", ALIAS, dpre=lambda a: a.dscale)
    refuse(lib, "join", "fwd", OK, rows=0, h=None)


def test_python_refuses_host_tensors():
    x, w = torch.zeros(4, 8), torch.zeros(8, 4)
    A, bc = torch.zeros(8, 16), torch.zeros(4, 1, 16)
    for call in (lambda: S.gspn_causal_conv_fwd(x, w), lambda: S.gspn_causal_conv_step(x, w, None, torch.zeros(4, 3, 8)),
                 lambda: S.gspn_causal_conv_bwd(x, w, None, x), lambda: S.gspn_selective_scan_fwd(x, x, A, bc, bc),
                 lambda: S.gspn_block_join_fwd(x), lambda: S.gspn_block_join_bwd(x, x, None, None)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        S.gspn_causal_conv_fwd([1.0], w)


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
    for name in S.EXPORTS:
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
@pytest.mark.parametrize("c,ld", [(24, 0), (7, 0), (64, 200), (521, 530)])
def test_launches_stay_in_their_buffers(chk, lib, dt, c, ld):
    for cu in (False, True):
        for rows, nseq in ((40, 2), (1, 1), (1200, 3)):
            assert replay(chk, lib, "conv", "fwd", dt, c=c, ld=ld, rows=rows, nseq=nseq, cu=cu, pool=True,
                          resume=True, slots=5) == ["conv_fwd_kernel"]
            assert replay(chk, lib, "conv", "bwd", dt, c=c, ld=ld, rows=rows, nseq=nseq, cu=cu) == [
                "conv_bwd_kernel", "reduce_parts_kernel"]
            for n in (1, 3, 16):
                names = replay(chk, lib, "scan", "fwd", dt, c=c, ld=ld, groups=1, n=n, rows=rows, nseq=nseq, cu=cu,
                               pool=True, slots=5, resume=True, keep=True)
                # whole sequences; cut into more chunks than a walk joins
                whole = ["selscan_kernel" if n == 1 else "selscan_quad_kernel"]
                assert names in (whole, ["selscan_kernel"] * 2,
                                 ["selscan_kernel", "selscan_join_kernel", "selscan_kernel"]), names
                assert (len(names) == 3) == (rows == 1200), names
                names = replay(chk, lib, "scan", "bwd", dt, c=c, ld=ld, groups=1, n=n, rows=rows, nseq=nseq, cu=cu)
                assert names[-3:] == ["selscan_bwd_kernel", "selscan_bc_kernel", "reduce_parts_kernel"], names
    assert replay(chk, lib, "conv", "step", dt, c=c, ld=ld, rows=3, nseq=3, pool=True, slots=5) == ["conv_step_kernel"]
    assert replay(chk, lib, "scan", "step", dt, c=c, ld=ld, groups=1, rows=3, nseq=3, pool=True, slots=5) == [
        "selscan_step_kernel"]
    for rdt in (F32, dt):
        for parts in ("grosp", "", "rp", "os"):
            assert replay(chk, lib, "join", "fwd", dt, rdt=rdt, c=c, ld=ld, parts=parts) == ["join_fwd_kernel"]
            names = replay(chk, lib, "join", "bwd", dt, rdt=rdt, c=c, ld=ld, parts=parts)
            assert names == ["join_bwd_kernel", "reduce_parts_kernel"][:2 if parts else 1]


def test_the_replay_sees_an_overrun(chk, lib):
    """A kept-states buffer one value short is reported."""
    sp = Space(chk)
    a = scan_args(sp, lib, keep=False)
    a.checkpoints = sp("checkpoints", lib.gspn_selective_scan_checkpoint_bytes(40, 2, 24, 16, 0) - 4)
    assert chk.gspn_selective_scan_fwd(ctypes.byref(a), F32, None) == OK
    assert chk.gspn_check_violations() > 0
