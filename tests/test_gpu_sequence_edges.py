"""The sequence operators on the GPU where calls and values are at their edges: nothing to sum over, values at the ends
of their type's range."""
import math

import pytest
import torch

import sequence_reference as R
from linear_spatial_propagation_gspn_amd import sequence as S
from test_gpu_sequence import (BF16, DEV, F32, _gpu, _say, check, cu_of, dev, gate_count, gen, on_gpu, ref_args, rnd,  # noqa: F401
                               run_bwd, run_fwd, scan_case, wide)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------------ nothing to sum

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,c,n", [(1, 1, 1), (40, 70, 16), (3000, 5, 3)])
def test_rows_without_a_sequence_get_zero_gradients(dtype, rows, c, n):
    """The C calls themselves (the binding answers such a call without one): every gradient is written."""
    none = torch.zeros(1, dtype=torch.int32, device=DEV)
    code = 0 if dtype == F32 else 1
    g = gen(1)
    k = on_gpu(scan_case(g, rows, c, 1, n, dtype))
    seq = S._sequences(k["x"], none, None)
    wide_dx = torch.full((rows, c + 3), 7.0, dtype=dtype, device=DEV)
    full = lambda like: torch.full(like.shape, 7.0, dtype=like.dtype, device=DEV)  # noqa: E731

    w, b = dev(rnd(g, c, 4)), dev(rnd(g, c))
    a = S._conv_args(k["x"], w, b, True, seq)
    a.gy, a.ldgy = k["x"].data_ptr(), c
    outs = [wide_dx[:, :c], full(w), full(b)]
    a.dx, a.lddx = outs[0].data_ptr(), c + 3
    a.dweight, a.dbias = outs[1].data_ptr(), outs[2].data_ptr()
    S._call("gspn_causal_conv_bwd", a, code, 0)
    assert all((t == 0).all() for t in outs) and (wide_dx[:, c:] == 7.0).all()

    a = S._scan_args(k["x"], k["dt"], k["A"], k["B"], k["C"], k["D"], k["z"], k["dt_bias"], True, seq)
    a.gy, a.ldgy = k["x"].data_ptr(), c
    wide_dx.fill_(7.0)
    outs = {"dx": wide_dx[:, :c], "ddt": full(k["x"]), "dz": full(k["x"]), "dB": full(k["B"]), "dC": full(k["C"]),
            "dA": full(k["A"]), "dD": full(k["D"]), "ddt_bias": full(k["D"])}
    for name, t in outs.items():
        setattr(a, name, t.data_ptr())
    a.lddx, a.ldddt, a.lddz = c + 3, c, c
    S._call("gspn_selective_scan_bwd", a, code, 0)
    for name, t in outs.items():
        assert (t == 0).all(), name
    assert (wide_dx[:, c:] == 7.0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kw", [{}, {"nseq": 2}, {"cu": [1, 5]}, {"cu": [0]}])
def test_rows_without_a_channel_have_zero_sums(dtype, kw):
    kw = {n: cu_of([b - a for a, b in zip(v, v[1:])], v[0]) if n == "cu" else v for n, v in kw.items()}
    x, A = torch.empty(6, 0, dtype=dtype, device=DEV), torch.empty(0, 5, device=DEV)
    bc = torch.randn(6, 3, 5, device=DEV).to(dtype)
    assert S.gspn_selective_scan_fwd(x, x, A, bc, bc, **kw).shape == (6, 0)
    grads = S.gspn_selective_scan_bwd(x, x, A, bc, bc, x, **kw)
    for t, shape in zip(grads[:5], ((6, 0), (6, 0), (0, 5), (6, 3, 5), (6, 3, 5))):
        assert t.shape == shape and (t == 0).all()
    leaf = bc.clone().requires_grad_()
    S.selective_scan(x, x, A, leaf, leaf, **kw).sum().backward()
    assert (leaf.grad == 0).all()


def test_gradients_of_an_empty_batch():
    """No rows: the sums over them are zero, also for a gradient whose strides are those of an expanded scalar."""
    x, bc = (torch.empty(0, *s, device=DEV, requires_grad=True) for s in ((12,), (1, 4)))
    w, A, pre = (torch.randn(*s, device=DEV).requires_grad_() for s in ((12, 4), (12, 4), (12,)))
    for f, leaves in ((lambda: S.causal_conv(x, w), (x, w)), (lambda: S.selective_scan(x, x, A, bc, bc), (x, A, bc)),
                      (lambda: S.block_join(x, x, x, pre=pre)[1], (x, pre))):
        for t, g in zip(leaves, torch.autograd.grad(f().sum(), leaves)):
            assert g.shape == t.shape and (g == 0).all()


# ------------------------------------------------------------------------------------------ gates far from zero

GATES = [-60.0, -86.5, -87.0, -87.25, -88.0, -89.5, -95.0, -104.0, -110.0, -200.0, -1000.0, -1e6, -1e20, -1e30, -3e38,
         0.0, 1.0, 60.0, 88.0, 200.0, 1e20, 3e38]


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gates_far_from_zero(dtype):
    """silu and its slope over the whole range of the type: what a gate of the type's lowest value closes stays closed
    (its silu is -0).  Roundings: the gate's argument (2 |v|) and 8, as everywhere, of what is not yet zero.  bf16's
    form takes a logistic below the normal numbers of fp32 as zero: there all of silu may be lost."""
    c = len(GATES)
    v = torch.tensor([GATES, GATES[::-1]]).to(dtype)
    v[0, 14], v[1, 7] = torch.finfo(dtype).min, torch.finfo(dtype).min
    one, gy = torch.ones(2, c, dtype=dtype), torch.ones(2, c, dtype=dtype)
    w, s, ds = wide(v), R.silu(wide(v)), R.dsilu(wide(v))
    count = 2 * w.abs().clamp(max=110) + 8
    slope, size = R.dsilu_scale(w), s.abs()
    if dtype != F32:
        lost = torch.sigmoid(w) < 2.0 ** -126
        size, slope = torch.where(lost, size / (count * R.U), size), torch.where(lost, slope / (count * R.U), slope)

    taps = torch.tensor([0.0, 1.0]).expand(c, 2).contiguous()  # the pre-activation is the row itself
    check(S.gspn_causal_conv_fwd(dev(v), dev(taps)), s, size, count, "convolution")
    pool = torch.zeros(2, 1, c, dtype=dtype, device=DEV)
    check(S.gspn_causal_conv_step(dev(v), dev(taps), None, pool), s, size, count, "convolution's step")
    dx = S.gspn_causal_conv_bwd(dev(v), dev(taps), None, dev(gy), nseq=2)[0]
    check(dx, ds, slope, 2 * count + 8, "convolution's dx")

    for n in (1, 16):  # x = 1, B = 0, D = 1: the gate's value is the row
        k = dict(x=dev(one), dt=dev(one), A=-torch.ones(c, n, device=DEV), B=torch.zeros(2, 1, n, dtype=dtype, device=DEV),
                 C=torch.ones(2, 1, n, dtype=dtype, device=DEV), D=torch.ones(c, device=DEV), z=dev(v), dt_bias=None)
        for kw in ({}, {"nseq": 2}):
            check(run_fwd(k, **kw), s, size, count + 2, "scan")
            got = run_bwd(k, dev(gy), **kw)
            check(got["dx"], s, size, count + 4, "scan's dx")
            check(got["dz"], ds, slope, 2 * count + 10, "scan's dz")
        pool = torch.zeros(2, c, n, device=DEV)
        y = S.gspn_selective_scan_step(k["x"], k["dt"], k["A"], k["B"], k["C"], pool, k["D"], k["z"])
        check(y, s, size, count + 2, "scan's step")

    joined = S.gspn_block_join_fwd(dev(one), dev(v))[0]
    check(joined, s, size, count + 2, "join")
    dh, dgate = S.gspn_block_join_bwd(dev(one), dev(gy), None, None, dev(v))[:2]
    check(dh, s, size, count + 2, "join's dh")
    check(dgate, ds, slope, 2 * count + 8, "join's dgate")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_gate_of_minus_infinity_is_what_the_formula_says(dtype):
    """-Inf times a logistic of 0: NaN, in that element alone, whichever storage type."""
    c = 8
    one = torch.ones(1, c, dtype=dtype, device=DEV)
    v = one.clone()
    v[0, 3] = -math.inf
    taps = torch.tensor([0.0, 1.0], device=DEV).expand(c, 2).contiguous()
    k = dict(x=one, dt=one, A=-torch.ones(c, 1, device=DEV), B=torch.zeros(1, 1, 1, dtype=dtype, device=DEV),
             C=torch.ones(1, 1, 1, dtype=dtype, device=DEV), D=torch.ones(c, device=DEV), z=v, dt_bias=None)
    for y in (S.gspn_causal_conv_fwd(v, taps), run_fwd(k), S.gspn_block_join_fwd(one, v)[0]):
        assert torch.isnan(y[0, 3]) and torch.isfinite(y[0, torch.arange(c) != 3]).all()


# ------------------------------------------------------------------------------- decays at the end of the range

FORGET = [-torch.finfo(F32).max, -3e38, -2.4e38, -1e30]


@pytest.mark.parametrize("n", [16, 8, 5, 1])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lengths", [[37, 1, 0, 16, 17, 2], [150, 1, 16, 0, 65], [18, 18, 18], [5]])
def test_scan_with_decay_rates_at_the_end_of_the_range(lengths, dtype, n):
    """A so low that A log2 e passes fp32: a step of the scan forgets everything (e^(d A) = 0), a skipped row (d = 0)
    nothing, and the rows that a kernel computes past a sequence's end are not seen.  A state is then that of the last
    row that was not skipped: a product of three factors, no decay's roundings in it."""
    g = gen(n + len(lengths))
    c, rows = len(FORGET), sum(lengths)
    seqs = R.spans(lengths)
    k = scan_case(g, rows, c, 1, n, dtype)
    k["A"] = torch.tensor(FORGET)[:, None].expand(c, n).contiguous()
    gy = rnd(g, rows, c, dtype=dtype)
    equal = len(set(lengths)) == 1
    kw = {"nseq": len(lengths)} if equal else {"cu": cu_of(lengths)}

    def count(args):
        return R.scan_roundings(args[0], args[1], torch.zeros_like(args[2]), args[7], True, seqs)

    def lowest(o):  # -Inf forgets no more than the lowest number does
        o = dict(o, A=o["A"].clone())
        o["A"][0] = -math.inf
        return o

    args = ref_args(k)
    ref, mag = R.scan_backward(*args, True, seqs, wide(gy))
    got, low = run_bwd(on_gpu(k), dev(gy), **kw), run_bwd(lowest(on_gpu(k)), dev(gy), **kw)
    both = 2 * (count(args) + 2 * gate_count(k)) + 16
    for name, more in {"dx": n, "ddt": n, "dz": n, "dB": c, "dC": c, "dA": rows, "dD": rows, "dbias": rows + n}.items():
        check(got[name], ref[name], mag[name], both + more, name)
        assert torch.equal(got[name], low[name]), name

    k["dt"][rows // 2:rows // 2 + 9:2] = -math.inf
    k["dt"][rows - 1] = -math.inf
    args = ref_args(k)
    ry, _, last, sy, _ = R.scan(*args, True, seqs)
    state, other = (torch.zeros(len(lengths), c, n, device=DEV) for _ in range(2))
    out = run_fwd(on_gpu(k), state=state, **kw)
    check(out, ry, sy, count(args) + gate_count(k), "out")
    check(state, torch.stack(last), torch.stack(last).abs(), count(args), "state")
    assert torch.equal(run_fwd(lowest(on_gpu(k)), state=other, **kw), out) and torch.equal(other, state)

    h0 = torch.randn(rows, c, n, generator=g)  # and a token that continues a state, or skips
    pool, o = dev(h0.clone()), lowest(on_gpu(k))
    S.gspn_selective_scan_step(o["x"], o["dt"], o["A"], o["B"], o["C"], pool, o["D"], o["z"], o["dt_bias"])
    last = R.scan(*args, True, R.spans([1] * rows), list(wide(h0)))[2]
    check(pool, torch.stack(last), torch.stack(last).abs(), count(args), "state after a token")


@pytest.mark.parametrize("n", [16, 5, 1])
@pytest.mark.parametrize("lengths", [[240], [48], [64]])  # joined by its own launch; by its chunks
def test_scan_growth_of_a_subnormal_state(lengths, n):
    """16 rows that multiply by e^192 lie past fp32 also for a state below its normal numbers: the rows one by one
    overflow, and so do the chunks.  Forward with the state 1.2e-40 before those rows; the same against the row order."""
    rows, = lengths
    c = 8
    k = dict(x=torch.zeros(rows, c), dt=torch.full((rows, c), 0.01), A=torch.ones(c, n), B=torch.ones(rows, 1, n),
             C=torch.ones(rows, 1, n), D=None, z=None, dt_bias=None)
    k["dt"][15], k["dt"][16:32] = 12.0, 12.0
    k["x"][15, ::2] = 1e-41
    cu = cu_of(lengths + [1] * 40, 0)  # packed with tokens, so that it is cut
    pad = lambda t: torch.cat([t, torch.zeros(40, *t.shape[1:])])  # noqa: E731
    o = on_gpu({m: pad(t) if t is not None and t.shape[0] == rows else t for m, t in k.items()})
    state = torch.zeros(41, c, n, device=DEV)
    out = run_fwd(o, softplus=False, cu=cu, state=state)
    assert (state[0, ::2] == math.inf).all() and (state[0, 1::2] == 0).all()
    assert (out[31:rows, ::2] == math.inf).all() and (out[:rows, 1::2] == 0).all()
    gy = torch.zeros(rows + 40, c, device=DEV)
    gy[32, ::2] = 1e-40  # dL/dh before row 16: e^192 times that
    got = run_bwd(o, gy, softplus=False, cu=cu)
    assert (got["dx"][:16, ::2] == math.inf).all() and (got["dx"][:32, 1::2] == 0).all()


@pytest.mark.parametrize("n", [16, 5, 1])
@pytest.mark.parametrize("lengths", [[240], [48], [64]])
def test_scan_steps_whose_sum_passes_the_range(lengths, n):
    """Steps of 3e38 with A = 0 leave a state as it is, row by row and therefore chunk by chunk, whose sum of steps is
    past fp32; with A < 0 they forget it.  x is zero in those rows, so that nothing else overflows."""
    rows, = lengths
    c = 8
    k = dict(x=torch.zeros(rows, c), dt=torch.full((rows, c), 3e38), A=torch.zeros(c, n), B=torch.ones(rows, 1, n),
             C=torch.ones(rows, 1, n), D=None, z=None, dt_bias=None)
    k["dt"][0], k["x"][0] = 1.0, 2.0
    k["A"][1::2] = -1.0
    pad = lambda t: torch.cat([t, torch.zeros(40, *t.shape[1:])])  # noqa: E731
    o = on_gpu({m: pad(t) if t is not None and t.shape[0] == rows else t for m, t in k.items()})
    cu = cu_of(lengths + [1] * 40, 0)
    state = torch.zeros(41, c, n, device=DEV)
    out = run_fwd(o, softplus=False, cu=cu, state=state)
    assert (state[0, ::2] == 2).all() and (state[0, 1::2] == 0).all()
    assert (out[:rows, ::2] == 2 * n).all() and (out[1:rows, 1::2] == 0).all()
    gy = torch.zeros(rows + 40, c, device=DEV)
    gy[rows - 1] = 1.0
    got = run_bwd(o, gy, softplus=False, cu=cu)
    # row 0: d = 1, x = 2, and dL/dh = C = 1 in the channels that forget nothing
    assert (got["dx"][0, ::2] == n).all() and (got["dx"][0, 1::2] == 0).all()
    assert (got["dB"][0] == 2 * c // 2).all()
