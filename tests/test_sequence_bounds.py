"""CPU tests of the bounds that the sequence operators' GPU results are held to: fp32 arithmetic by the definition
passes them, and results that are off by what a mistake would make them off by do not."""
import pytest
import torch

import sequence_bounds as Q
import sequence_cases as P
import sequence_differences as D
import sequence_reference as R
from test_sequence_abi import BF16 as BF16CODE, F32 as F32CODE, chk, lib, replay  # noqa: F401

F64, F32 = torch.float64, torch.float32


def rnd(g, *shape, by=1.0):
    return (torch.randn(shape, generator=g) * by).float()


def scan_inputs(g, rows, c, groups, n, gate=True):
    return [rnd(g, rows, c), rnd(g, rows, c, by=0.5), -torch.exp(rnd(g, c, n, by=0.7)), rnd(g, rows, groups, n),
            rnd(g, rows, groups, n), rnd(g, c), rnd(g, rows, c) if gate else None, rnd(g, c) - 2]


CASES = [(40, 6, 1, 16, True, [40]), (60, 12, 3, 5, False, [25, 0, 34, 1]), (130, 4, 2, 1, True, [100, 30])]


def within(got, ref, bound):
    return bool(((got.double() - ref).abs() <= bound * Q.U + 1e-37).all())


@pytest.mark.parametrize("rows,c,groups,n,gate,lengths", CASES)
def test_scan_bounds_hold_for_fp32_and_not_for_bf16(rows, c, groups, n, gate, lengths):
    g = torch.Generator().manual_seed(rows + n)
    args = scan_inputs(g, rows, c, groups, n, gate)
    gy = rnd(g, rows, c)
    seqs = R.spans(lengths)
    w = [None if t is None else t.double() for t in args]
    bounds = Q.scan_bounds(*w, True, seqs, gy.double(), 0, rows)
    ref, _ = R.scan_backward(*w, True, seqs, gy.double())
    got, _ = R.scan_backward(*args, True, seqs, gy)
    ref["out"], ref["states"] = R.scan(*w, True, seqs)[:2]
    got["out"], got["states"] = R.scan(*args, True, seqs)[:2]
    assert set(bounds) == set(ref)
    for name in ref:
        assert within(got[name], ref[name], bounds[name]), name
        assert not within(ref[name].bfloat16(), ref[name], bounds[name]), name  # half the width
        assert not within(ref[name] * (1 + 2.0 ** -9), ref[name], bounds[name]), name
        assert not within(torch.roll(ref[name], 1, 0), ref[name], bounds[name]), name


@pytest.mark.parametrize("c", [9, 515, 4093, 8199, 12001, 16384])
def test_norm_bound_rejects_a_lost_column(c):
    """Rows of ones with fp32 values: any one of their columns missing from the sum of squares, or one counted twice."""
    assert (Q.norm_count(c) + 4) * Q.U < 0.5 / c * 0.98


@pytest.mark.parametrize("case", P.PLANS, ids=P.name)
def test_cases_take_the_plans_they_are_for(chk, lib, case):  # noqa: F811
    dtype, c, groups, n, gate, lengths, packed, fwd, bwd = case
    dt = F32CODE if dtype == "f32" else BF16CODE
    rows, nseq = sum(lengths), len(lengths)
    kw = dict(c=c, groups=groups, n=n, rows=rows, nseq=nseq, cu=packed, gate=gate, ld=max(c, groups * n))

    def chunk(ids):  # the rows of a chunk, from the number of their ids
        for s in range(4, 31):
            if ids == ((rows >> s) + nseq if packed else nseq * max(1, (rows // nseq + (1 << s) - 1) >> s)):
                return 1 << s

    names = replay(chk, lib, "scan", "fwd", dt, keep=True, **kw)
    floats = lib.gspn_selective_scan_workspace_bytes(rows, nseq, c, groups, n, int(packed)) // 4
    if fwd in ("quad", "lane"):
        assert names == ["selscan_quad_kernel" if fwd == "quad" else "selscan_kernel"] and floats == 0
    else:
        joined = ["selscan_join_kernel"] * (max(lengths) > 4 * fwd)
        assert names == ["selscan_kernel", *joined, "selscan_kernel"]
        assert chunk(floats // ((n + 1) * c)) == fwd
    names = replay(chk, lib, "scan", "bwd", dt, **kw)
    floats = lib.gspn_selective_scan_bwd_workspace_bytes(rows, nseq, c, groups, n, int(packed)) // 4
    ids = (floats - P.backward_blocks(c, groups, n) * rows * 2 * groups * n) // ((2 * n + 3) * c)
    cut = "selscan_bwd_local_kernel" in names
    assert cut == bool(bwd)
    if cut:
        assert chunk(ids) == bwd
    else:
        assert chunk(ids) >= max(lengths) > 8  # one chunk a sequence, of several tiles


@pytest.mark.parametrize("op", D.OPS)
def test_differences_accept_the_gradient_and_reject_others(op):
    """The definition in fp32, with its own gradient, passes; zero, negated and doubled gradients are rejected by the
    comparison itself."""
    g = torch.Generator().manual_seed(61)
    ts, _, ref = D.case(op, g)
    gy = rnd(g, *ts[0].shape)
    for i, t in enumerate(ts):
        leaf = t.clone().requires_grad_()
        grad, = torch.autograd.grad(ref(*ts[:i], leaf, *ts[i + 1:])[0], leaf, gy)
        D.compare(ts, gy, i, grad, lambda *a: ref(*a)[0], ref)
        for wrong in (0 * grad, -grad, 2 * grad):
            with pytest.raises(AssertionError):
                D.compare(ts, gy, i, wrong, lambda *a: ref(*a)[0], ref)
