"""CPU tests of the attention operators' launches: that few rows are spread over the device as their comments say, and
that workspaces hold what such a launch writes (host replays, libgspn_check.so)."""
import ctypes
import re

import pytest

from test_attention_abi import BF16, F32, OK, Space, chk, lib, rotary_args  # noqa: F401 (fixtures)


def grids(chk, lib, dt, kind, **kw):
    """{kernel: workgroups} of one call, whose every access is inside its buffers."""
    a = rotary_args(Space(chk), lib, dt=dt, kind=kind, **kw)
    assert getattr(chk, "gspn_head_rotary_" + kind)(ctypes.byref(a), dt, None) == OK
    buf = ctypes.create_string_buffer(1 << 16)
    chk.gspn_check_report(buf, 1 << 16)
    text = buf.value.decode()
    assert chk.gspn_check_violations() == 0, text
    return {m.group(1): int(m.group(2)) for m in re.finditer(r"launch \(?(\w+).*grid=(\d+)", text)}


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("heads,kv_heads,d", [(32, 8, 128), (16, 16, 72), (5, 1, 80), (1, 0, 64), (64, 64, 256)])
def test_a_rotations_gradient_has_the_waves_of_its_forward(chk, lib, dt, norm, heads, kv_heads, d):
    """Waves share a row's heads in the backward as in the forward: at least half as many, up to the 1024 workgroups that a
    backward walks its rows with, and none without a row's share."""
    for rows in (1, 3, 4, 64, 65, 500, 1023, 1500, 2047, 2048, 2049, 9001):
        kw = dict(rows=rows, heads=heads, kv_heads=kv_heads, d=d, sections=(d // 2,), norm=norm)
        fwd = grids(chk, lib, dt, "fwd", **kw)["rotary_fwd_kernel"]
        assert min(fwd, 1024) <= 2 * grids(chk, lib, dt, "bwd", **kw)["rotary_bwd_kernel"] <= 2 * min(fwd, 1024), rows
