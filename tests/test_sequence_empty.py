"""CPU tests of sequence calls whose rows no sequence covers, through the C ABI: a backward gives zero gradients to rows
outside every sequence, also where there is no sequence at all."""
import ctypes

import pytest

from test_sequence_abi import (BF16, CALLS, F32, NULLP, OK, ALIAS, SHAPE, Space, chk, lib, refuse, replay)  # noqa: F401


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("op", ["conv", "scan"])
def test_rows_without_a_sequence_are_cleared(chk, lib, op, dt):  # noqa: F811
    """One launch that writes every gradient, replayed within its buffers; no workspace and no checkpoints."""
    make, prefix = CALLS[op]
    for rows in (1, 40):
        a = make(Space(chk), lib, dt=dt, kind="bwd", rows=rows, nseq=1, cu=True)
        a.seq.nseq = 0
        a.workspace, a.workspace_bytes = None, 0
        if op == "scan":
            a.checkpoints = None
        assert getattr(chk, prefix + "bwd")(ctypes.byref(a), dt, None) == OK
        buf = ctypes.create_string_buffer(1 << 16)
        chk.gspn_check_report(buf, 1 << 16)
        text = buf.value.decode()
        assert chk.gspn_check_violations() == 0, text
        assert chk.gspn_check_launches() == 1 and "reduce_parts_kernel" in text, text


@pytest.mark.parametrize("op", ["conv", "scan"])
def test_a_call_without_a_sequence_is_still_checked(lib, op):  # noqa: F811
    build = dict(cu=True)
    refuse(lib, op, "bwd", NULLP, build=build, seq_nseq=0, dx=None)
    refuse(lib, op, "bwd", ALIAS, build=build, seq_nseq=0, dx=lambda a: a.gy)
    refuse(lib, op, "bwd", SHAPE, build=build, seq_nseq=0, lddx=23)
    refuse(lib, op, "bwd", SHAPE, seq_nseq=0)  # rows, no sequence and no offsets
    # nothing to write: no pointer is looked at
    refuse(lib, op, "bwd", OK, build=build, seq_nseq=0, seq_rows=0, dx=None, x=None)
    refuse(lib, op, "fwd", OK, build=build, seq_nseq=0, x=None)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("cu,nseq", [(False, 2), (True, 2), (True, 0)])
def test_rows_without_a_channel_have_sums_over_none(chk, lib, cu, nseq, dt):  # noqa: F811
    """dB and dC [rows][groups][n] are sums over the channels: with none of them they are zero, and written."""
    make, prefix = CALLS["scan"]
    a = make(Space(chk), lib, dt=dt, kind="bwd", rows=40, nseq=2, cu=cu)
    a.seq.nseq, a.channels = nseq, 0
    for f in ("x", "dt", "z", "gy", "dx", "ddt", "dz", "A", "D", "dt_bias", "dA", "dD", "ddt_bias", "checkpoints", "workspace"):
        setattr(a, f, None)
    a.workspace_bytes = 0
    assert chk.gspn_selective_scan_bwd(ctypes.byref(a), dt, None) == OK
    buf = ctypes.create_string_buffer(1 << 16)
    chk.gspn_check_report(buf, 1 << 16)
    text = buf.value.decode()
    assert chk.gspn_check_violations() == 0, text
    assert chk.gspn_check_launches() == 1 and "reduce_parts_kernel" in text, text
    a.dB = None
    assert lib.gspn_selective_scan_bwd(ctypes.byref(a), dt, None) == NULLP
    a.seq.rows = 0
    assert lib.gspn_selective_scan_bwd(ctypes.byref(a), dt, None) == OK
