"""CPU tests of what bench.py's counter summaries are tied to: the sources and flags that a measured kernel is built
from, and nothing that another operator brings."""
import os
import shutil

import pytest

import bench
from linear_spatial_propagation_gspn_amd import build as hipbuild

KERNELS = sorted(bench.KERNEL_SOURCES) + [None]


@pytest.fixture
def sources(tmp_path, monkeypatch):
    """A copy of the package's sources, which the digests are taken from."""
    package = tmp_path / "package"
    shutil.copytree(bench.CSRC, package / "csrc")
    shutil.copy(os.path.join(os.path.dirname(bench.CSRC), "build.py"), package / "build.py")
    monkeypatch.setattr(bench, "CSRC", str(package / "csrc"))
    return package


@pytest.mark.parametrize("kernel", KERNELS)
def test_other_operators_leave_a_digest_alone(sources, kernel):
    before = bench.kernel_sources_digest(kernel)
    build = sources / "build.py"
    build.write_text(build.read_text().replace('"head_rotary.hip", ', '"head_rotary.hip", "another.hip", '))
    for name in bench.TOKEN_ROW_SOURCES:
        with open(sources / "csrc" / name, "a") as f:
            f.write("// changed\n")
    assert bench.kernel_sources_digest(kernel) == before


@pytest.mark.parametrize("kernel", KERNELS)
def test_own_sources_and_flags_change_a_digest(sources, kernel, monkeypatch):
    before = bench.kernel_sources_digest(kernel)
    monkeypatch.setattr(hipbuild, "DEVICE", hipbuild.DEVICE + ["-ffast-math"])
    flags = bench.kernel_sources_digest(kernel)
    monkeypatch.undo()
    monkeypatch.setattr(bench, "CSRC", str(sources / "csrc"))
    assert flags != before and bench.kernel_sources_digest(kernel) == before
    for name in (bench.KERNEL_SOURCES[kernel] if kernel else ["api.cpp", "scan.hip"]) + ["device.hpp"]:
        with open(sources / "csrc" / name, "a") as f:
            f.write("// changed\n")
        after = bench.kernel_sources_digest(kernel)
        assert after != before, name
        before = after


def test_the_two_kinds_of_sources_share_no_file():
    listed = {n for names in bench.KERNEL_SOURCES.values() for n in names} | {"device.hpp", "check.hpp", "launch.hpp"}
    assert not listed & set(bench.TOKEN_ROW_SOURCES)
    for name in bench.TOKEN_ROW_SOURCES:
        assert os.path.exists(os.path.join(bench.CSRC, name)), name
    # no source of a step includes a header of those operators
    headers = [n for n in bench.TOKEN_ROW_SOURCES if n.endswith(".hpp")]
    for name in sorted(os.listdir(bench.CSRC)):
        if name not in bench.TOKEN_ROW_SOURCES and name.endswith((".hip", ".hpp", ".cpp")):
            text = open(os.path.join(bench.CSRC, name)).read()
            assert not [h for h in headers if '"%s"' % h in text], name
