"""The sequence operators on the GPU against their 64-bit references.

Tolerances are counted, not chosen: fp32 roundings on a result's way (U =
2^-24 each) times the magnitude of the terms it is made of, plus half a step
of the type it is stored in.  The counts stand at each comparison."""
import math
import sys

import pytest
import torch

import sequence_reference as R
from linear_spatial_propagation_gspn_amd import gspn as G
from linear_spatial_propagation_gspn_amd import sequence as S

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    S.lib()
    yield
    torch.cuda.synchronize()


@pytest.fixture(autouse=True)
def _say(request):
    print("case:", request.node.name, flush=True)
    sys.stdout.flush()
    yield
    torch.cuda.synchronize()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rnd(g, *shape, dtype=F32, by=1.0):
    return (torch.randn(shape, generator=g) * by).to(dtype)


def wide(t):
    return None if t is None else t.detach().cpu().double()


def dev(t):
    return None if t is None else t.to(DEV)


def strided(t):
    """t's values as the right part of wider rows."""
    big = torch.full((*t.shape[:-1], t.shape[-1] * 2 + 3), 7.0, dtype=t.dtype, device=DEV)
    view = big[..., t.shape[-1] + 3:]
    view.copy_(t)
    return view


def strided_bc(b, c):
    """B and C as slices of one projection's rows."""
    rows, g, n = b.shape
    big = torch.full((rows, 2 * g * n + 5), 7.0, dtype=b.dtype, device=DEV)
    big[:, 5:5 + g * n] = b.reshape(rows, -1).to(DEV)
    big[:, 5 + g * n:] = c.reshape(rows, -1).to(DEV)
    return big[:, 5:5 + g * n].unflatten(1, (g, n)), big[:, 5 + g * n:].unflatten(1, (g, n))


def check(got, ref, scale, roundings, what, rows=None):
    """|got - ref| <= half a step of got's type of ref + roundings U scale, element by element."""
    half = R.half_step(got.dtype) if got.dtype != F32 else 0.0
    got = wide(got)
    if rows is not None:
        got, ref, scale = got[rows], ref[rows], scale[rows]
    assert got.shape == ref.shape, what
    bound = half * ref.abs() * (1 + 2.0 ** -8) + roundings * R.U * scale + 1e-37
    off = (got - ref).abs()
    assert torch.isfinite(got).all(), what
    assert (off <= bound).all(), "%s: worst %.3g of its bound" % (what, float((off / bound).max()))


def cu_of(lengths, first=0):
    return torch.tensor([a for a, _ in R.spans(lengths, first)] + [first + sum(lengths)], dtype=torch.int32, device=DEV)


def inside(seqs):
    return [t for lo, hi in seqs for t in range(lo, hi)]


# ------------------------------------------------------------------------------------------------ causal conv

# p: width products and sums.  silu: the gate's argument product (|p| roundings), the exponential, sum, reciprocal and
# product (6), and a slope of at most 1.1 for p's own error.  (bf16's half step covers its gate's extra |p| U.)
def conv_count(width, pre, act=True):
    return 1.1 * (width + 2) + (2 * float(pre[torch.isfinite(pre)].abs().max()) + 8 if act else 0)


CONV_SEQS = [([1], 0), ([5], 0), ([64], 0), ([3, 1, 0, 2], 0), ([70, 0, 1, 9, 33], 2), ([1] * 70, 0)]


@pytest.mark.parametrize("lengths,first", CONV_SEQS)
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("dtype,c,act,view", [(F32, 1, True, False), (F32, 68, True, True), (BF16, 520, True, False),
                                              (BF16, 77, False, True), (BF16, 64, True, False)])
def test_conv_forward_and_backward(dtype, c, act, view, width, lengths, first):
    g = gen(width * 1000 + c)
    seqs = R.spans(lengths, first)
    rows = first + sum(lengths) + (3 if first else 0)  # rows before and behind the sequences
    x, gy = rnd(g, rows, c, dtype=dtype), rnd(g, rows, c, dtype=dtype)
    w, b = rnd(g, c, width, by=0.7), rnd(g, c, by=0.5)
    y, pre, scale, _ = R.conv(wide(x), wide(w), wide(b), act, seqs)
    (rdx, rdw, rdb), (mx, mw, mb) = R.conv_backward(wide(x), wide(w), wide(b), act, seqs, wide(gy))
    xd, gd = (strided(x), strided(gy)) if view else (dev(x), dev(gy))
    out = torch.full((rows, c), 3.0, dtype=dtype, device=DEV)
    S.gspn_causal_conv_fwd(xd, dev(w), dev(b), act, cu_of(lengths, first), out=out)
    dx, dw, db = S.gspn_causal_conv_bwd(xd, dev(w), dev(b), gd, act, cu_of(lengths, first))
    at = inside(seqs)
    n = conv_count(width, pre, act)
    check(out, y, scale + y.abs(), n, "y", at)
    others = [t for t in range(rows) if t not in set(at)]
    assert (out[others] == 3.0).all() and (dx[others] == 0).all()
    # e = gy silu'(p): silu' has the gate's roundings twice and 4 products; then width terms a row, `rows` a sum
    check(dx, rdx, mx, 2 * n + 8 + width, "dx", at)
    check(dw, rdw, mw, 2 * n + 8 + rows, "dweight")
    check(db, rdb, mb, 2 * n + 8 + rows, "dbias")


def test_conv_equal_lengths_and_batch_form():
    g = gen(5)
    x, w = rnd(g, 3, 21, 40), rnd(g, 40, 4)
    flat = x.reshape(63, 40)
    y, pre, scale, _ = R.conv(wide(flat), wide(w), torch.zeros(40, dtype=torch.float64), True, R.spans([21] * 3))
    got = S.gspn_causal_conv_fwd(dev(x), dev(w))
    check(got.view(63, 40), y, scale + y.abs(), conv_count(4, pre), "y")
    assert torch.equal(S.gspn_causal_conv_fwd(dev(flat), dev(w), nseq=3), got.view(63, 40))
    both = torch.cat([x, x], 2).to(DEV)  # the halves of a projection's rows
    assert torch.equal(S.gspn_causal_conv_fwd(both[..., 40:], dev(w)), got)


@pytest.mark.parametrize("dtype,c", [(F32, 12), (BF16, 136), (BF16, 9)])
@pytest.mark.parametrize("width", [2, 4])
def test_conv_pool(dtype, c, width):
    """Prompts that continue their entry or start anew, empty ones, padding, a repeated and an impossible index; then
    the same rows one token at a time."""
    g = gen(11)
    lengths = [5, 0, 1, 2, 0, 40, 3, 4]
    slots = [4, 7, 0, -1, 2, 5, 5, 99]  # 5 twice: the later sequence is in error; 99: out of range
    resume = [True, True, False, True, False, True, True, True]
    pool = rnd(g, 9, width - 1, c, dtype=dtype)
    x, w, b = rnd(g, sum(lengths), c, dtype=dtype), rnd(g, c, width), rnd(g, c)
    seqs = R.spans(lengths)
    heads = [wide(pool[s]) * r if 0 <= s < 9 else torch.zeros(width - 1, c, dtype=torch.float64)
             for s, r in zip(slots, resume)]
    y, pre, scale, tails = R.conv(wide(x), wide(w), wide(b), True, seqs, heads)
    state = dev(pool.clone())
    out = S.gspn_causal_conv_fwd(dev(x), dev(w), dev(b), cu=cu_of(lengths), state=state,
                                 slots=torch.tensor(slots, dtype=torch.int32, device=DEV),
                                 resume=torch.tensor(resume, device=DEV))
    good = inside(seqs[:6])
    check(out, y, scale + y.abs(), conv_count(width, pre), "y", good)
    assert torch.isnan(out[seqs[6][0]:]).all()
    want = wide(pool.clone())
    for i in (0, 1, 2, 4, 5):
        want[slots[i]] = tails[i]
    assert torch.equal(wide(state), want)  # the entry's rows are copies

    # one token at a time gives what the prompt gave, bit for bit
    xs = rnd(g, 6, 3, c, dtype=dtype)
    whole = S.gspn_causal_conv_fwd(dev(xs.transpose(0, 1).contiguous()), dev(w), dev(b))
    st = torch.zeros(3, width - 1, c, dtype=dtype, device=DEV)
    for t in range(6):
        assert torch.equal(S.gspn_causal_conv_step(dev(xs[t]), dev(w), dev(b), st), whole[:, t])


def test_conv_step_padding_and_bad_slots():
    c = 24
    pool = torch.arange(4 * 3 * c, dtype=F32, device=DEV).view(4, 3, c)
    keep = pool.clone()
    x, w = torch.randn(5, c, device=DEV), torch.randn(c, 4, device=DEV)
    out = torch.full((5, c), 2.0, device=DEV)
    S.gspn_causal_conv_step(x, w, None, pool, torch.tensor([2, -1, 2, 4, 0], dtype=torch.int32, device=DEV), out=out)
    assert (out[1] == 2.0).all() and torch.isnan(out[2]).all() and torch.isnan(out[3]).all()
    assert torch.isfinite(out[[0, 4]]).all()
    for s, i in ((2, 0), (0, 4)):
        assert torch.equal(pool[s], torch.cat([keep[s, 1:], x[i:i + 1]]))
    assert torch.equal(pool[[1, 3]], keep[[1, 3]])


# --------------------------------------------------------------------------------------------- selective scan

def scan_case(g, rows, c, groups, n, dtype, gate=True, skip=True, bias=True, spread=0.5):
    return dict(x=rnd(g, rows, c, dtype=dtype), dt=rnd(g, rows, c, dtype=dtype, by=spread),
                A=-torch.exp(rnd(g, c, n, by=0.7)), B=rnd(g, rows, groups, n, dtype=dtype),
                C=rnd(g, rows, groups, n, dtype=dtype), D=rnd(g, c) if skip else None,
                z=rnd(g, rows, c, dtype=dtype) if gate else None, dt_bias=rnd(g, c) - 2 if bias else None)


def ref_args(k):
    c = k["x"].shape[1]
    zero = torch.zeros(c, dtype=torch.float64)
    return [wide(k["x"]), wide(k["dt"]), wide(k["A"]), wide(k["B"]), wide(k["C"]),
            zero if k["D"] is None else wide(k["D"]), wide(k["z"]), zero if k["dt_bias"] is None else wide(k["dt_bias"])]


def on_gpu(k, view=False):
    o = {n: dev(t) for n, t in k.items()}
    if view:
        for n in ("x", "dt", "z"):
            if k[n] is not None:
                o[n] = strided(k[n])
        o["B"], o["C"] = strided_bc(k["B"], k["C"])
    return o


def run_fwd(o, **more):
    return S.gspn_selective_scan_fwd(o["x"], o["dt"], o["A"], o["B"], o["C"], o["D"], o["z"], o["dt_bias"], **more)


def run_bwd(o, gy, **more):
    r = S.gspn_selective_scan_bwd(o["x"], o["dt"], o["A"], o["B"], o["C"], gy, o["D"], o["z"], o["dt_bias"], **more)
    return dict(zip(("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias"), r))


# the gate adds its argument's product (2 |z|) and 8 roundings
def gate_count(k):
    return 2 * float(k["z"].float().abs().max()) + 8 if k["z"] is not None else 0


SCAN_CASES = [
    # dtype, channels, groups, n, gate, D, bias, softplus, view, lengths, first
    (F32, 64, 1, 16, True, True, True, True, False, [40], 0),
    (F32, 1, 1, 1, True, True, True, True, False, [1], 0),
    (F32, 70, 1, 16, True, True, True, True, True, [37, 1, 0, 16, 17, 2], 3),
    (BF16, 128, 1, 16, True, True, True, True, False, [100, 31], 0),
    (BF16, 130, 2, 16, False, True, False, True, True, [33, 15], 1),
    (BF16, 96, 4, 8, True, False, True, True, False, [20, 50, 1], 0),
    (F32, 36, 3, 5, True, True, True, False, True, [18, 18], 0),
    (BF16, 66, 1, 3, True, True, True, True, True, [65], 0),
    (BF16, 300, 2, 1, False, False, True, True, False, [35, 8], 0),
    (F32, 520, 4, 1, True, True, True, True, True, [49], 2),
    (F32, 24, 24, 4, True, True, True, True, False, [19], 0),
    (BF16, 17, 1, 13, True, True, True, True, True, [5, 0, 0, 16], 0),
    (F32, 8, 1, 2, False, True, True, False, False, [16, 16, 16], 0),
    (F32, 4, 2, 16, True, True, True, True, False, [1] * 70, 0),
    # batches that are cut into chunks: sequences that the chunks join by themselves, and longer ones
    (F32, 70, 1, 16, True, True, True, True, False, [50, 64, 16, 17, 0, 33, 1], 1),
    (BF16, 64, 1, 16, True, True, True, True, True, [150, 1, 16, 0, 65], 0),
    (BF16, 40, 2, 8, False, True, True, True, False, [200, 48], 3),
    (F32, 12, 1, 4, True, False, True, True, True, [3, 190, 64], 0),
    (BF16, 33, 1, 11, True, True, False, True, False, [64, 120, 7], 0),
    (F32, 66, 2, 1, True, True, True, True, False, [130, 80], 2),
    (BF16, 20, 1, 6, True, True, True, False, True, [1] * 100 + [90], 0),
]


@pytest.mark.parametrize("case", SCAN_CASES)
def test_scan_forward_and_backward(case):
    dtype, c, groups, n, gate, skip, bias, softplus, view, lengths, first = case
    g = gen(c * 100 + n)
    seqs = R.spans(lengths, first)
    rows = first + sum(lengths) + (2 if first else 0)
    k = scan_case(g, rows, c, groups, n, dtype, gate, skip, bias)
    if not softplus:
        k["dt"] = k["dt"].abs() * 0.2
        k["dt_bias"] = None if k["dt_bias"] is None else k["dt_bias"].abs() * 0.1
    gy = rnd(g, rows, c, dtype=dtype)
    args = ref_args(k)
    ry, _, _, sy, _ = R.scan(*args, softplus, seqs)
    ref, mag = R.scan_backward(*args, softplus, seqs, wide(gy))
    o = on_gpu(k, view)
    gd = strided(gy) if view else dev(gy)
    out = torch.full((rows, c), 3.0, dtype=dtype, device=DEV)
    cu = cu_of(lengths, first)
    _, kept = run_fwd(o, softplus=softplus, cu=cu, checkpoints=True, out=out)
    got = run_bwd(o, gd, softplus=softplus, cu=cu, checkpoints=kept)
    again = run_bwd(o, gd, softplus=softplus, cu=cu)  # running the forward again itself
    at = inside(seqs)
    others = [t for t in range(rows) if t not in set(at)]
    count = R.scan_roundings(args[0], args[1], args[2], args[7], softplus, seqs)
    check(out, ry, sy, count + gate_count(k), "out", at)
    assert (out[others] == 3.0).all()
    # a gradient passes a state's way twice (forward states, then back), both gates, and its own sum: n states,
    # the group's channels, or the rows
    both = 2 * (count + 2 * gate_count(k)) + 16
    sums = {"dx": n, "ddt": n, "dz": n, "dB": c // groups, "dC": c // groups, "dA": rows, "dD": rows, "dbias": rows + n}
    for name, more in sums.items():
        if got[name] is None:
            assert (name, gate, skip, bias) in (("dz", False, skip, bias), ("dD", gate, False, bias),
                                                ("dbias", gate, skip, False))
            continue
        assert torch.equal(got[name], again[name]), name  # fixed order: the same bits
        per_row = name in ("dx", "ddt", "dz", "dB", "dC")
        check(got[name], ref[name], mag[name], both + more, name, at if per_row else None)
        if per_row:
            assert (got[name][others] == 0).all(), name


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scan_many_chunks(dtype):
    """A sequence long enough that its chunks' states are joined by the second launch, equal lengths against packed."""
    g = gen(3)
    k = scan_case(g, 700, 66, 1, 16, dtype)
    args = ref_args(k)
    ry, _, last, sy, ms = R.scan(*args, True, [(0, 350), (350, 700)])
    state = torch.zeros(2, 66, 16, device=DEV)
    out = run_fwd(on_gpu(k), nseq=2, state=state)
    count = R.scan_roundings(args[0], args[1], args[2], args[7], True, [(0, 350)])
    check(out, ry, sy, count + gate_count(k), "out")
    check(state, torch.stack(last), torch.stack([ms[349], ms[699]]), count, "state")
    packed = torch.zeros(2, 66, 16, device=DEV)
    assert torch.equal(run_fwd(on_gpu(k), cu=cu_of([350, 350]), state=packed), out)
    assert torch.equal(packed, state)
    batch = {n: t.view(2, 350, *t.shape[1:]) if n in ("x", "dt", "z", "B", "C") else t for n, t in on_gpu(k).items()}
    assert torch.equal(run_fwd(batch).view(700, 66), out)


@pytest.mark.parametrize("long", [50, 220])
@pytest.mark.parametrize("dtype,n", [(F32, 16), (BF16, 16), (F32, 1), (BF16, 6), (F32, 8), (BF16, 4)])
def test_scan_pool(dtype, n, long):
    g = gen(17)
    c, lengths = 72, [long, 0, 1, 4, 0, 18, 3, 2]
    slots = [4, 7, 0, -1, 2, 5, 5, 99]
    resume = [True, True, False, True, False, True, True, True]
    k = scan_case(g, sum(lengths), c, 1, n, dtype)
    pool = rnd(g, 9, c, n)
    seqs = R.spans(lengths)
    zero = torch.zeros(c, n, dtype=torch.float64)
    h0 = [wide(pool[s]) * r if 0 <= s < 9 else zero for s, r in zip(slots, resume)]
    args = ref_args(k)
    ry, _, last, sy, _ = R.scan(*args, True, seqs, h0)
    mag = R.scan(*[a.abs() if i in (0, 3, 4) else a for i, a in enumerate(args)], True, seqs, [h.abs() for h in h0])[2]
    state = dev(pool.clone())
    out = run_fwd(on_gpu(k), cu=cu_of(lengths), state=state,
                  slots=torch.tensor(slots, dtype=torch.int32, device=DEV), resume=torch.tensor(resume, device=DEV))
    count = R.scan_roundings(args[0], args[1], args[2], args[7], True, seqs)
    check(out, ry, sy, count + gate_count(k), "out", inside(seqs[:6]))
    assert torch.isnan(out[seqs[6][0]:]).all()
    for e in range(9):
        if e in (4, 7, 0, 2, 5):
            i = slots.index(e)
            check(state[e], last[i], mag[i], count, "entry %d" % e)
        else:
            assert torch.equal(state[e].cpu(), pool[e])
    assert torch.equal(state[7].cpu(), pool[7]) and (state[2] == 0).all()  # the empty sequences


@pytest.mark.parametrize("dtype,n,groups", [(F32, 16, 1), (BF16, 16, 2), (F32, 1, 2), (BF16, 8, 1), (F32, 7, 1),
                                            (BF16, 4, 1), (BF16, 12, 3)])
def test_scan_steps_follow_the_prompt(dtype, n, groups):
    """A prompt in two parts, then tokens one by one, against the whole sequence at once."""
    g = gen(23)
    s, length, c = 3, 30, 78
    k = scan_case(g, s * length, c, groups, n, dtype)
    args = ref_args(k)
    seqs = R.spans([length] * s)
    ry, _, last, sy, ms = R.scan(*args, True, seqs)
    o = on_gpu(k, True)
    rows = lambda lo, hi: torch.cat([torch.arange(i * length + lo, i * length + hi) for i in range(s)]).to(DEV)  # noqa: E731
    take = lambda r: {m: t[r] if m in ("x", "dt", "z", "B", "C") else t for m, t in o.items()}  # noqa: E731
    state = torch.full((5, c, n), 9.0, device=DEV)
    slots = torch.tensor([3, 0, 4], dtype=torch.int32, device=DEV)
    parts = [run_fwd(take(rows(0, 17)), nseq=s, state=state, slots=slots).view(s, 17, c)]
    parts.append(run_fwd(take(rows(17, 22)), nseq=s, state=state, slots=slots,
                         resume=torch.ones(s, dtype=torch.bool, device=DEV)).view(s, 5, c))
    for t in range(22, length):
        p = take(rows(t, t + 1))
        parts.append(S.gspn_selective_scan_step(p["x"], p["dt"], p["A"], p["B"], p["C"], state, p["D"], p["z"],
                                                p["dt_bias"], slots=slots).view(s, 1, c))
    count = R.scan_roundings(args[0], args[1], args[2], args[7], True, seqs)
    check(torch.cat(parts, 1).view(s * length, c), ry, sy, count + gate_count(k), "out")
    check(state[[3, 0, 4]], torch.stack(last), torch.stack([ms[hi - 1] for _, hi in seqs]), count, "state")
    assert (state[[1, 2]] == 9.0).all()


def test_scan_step_padding_and_bad_slots():
    c, n = 40, 16
    g = gen(2)
    k = on_gpu(scan_case(g, 5, c, 1, n, F32))
    pool = torch.randn(4, c, n, device=DEV)
    keep = pool.clone()
    out = torch.full((5, c), 2.0, device=DEV)
    S.gspn_selective_scan_step(k["x"], k["dt"], k["A"], k["B"], k["C"], pool, k["D"], k["z"], k["dt_bias"],
                               slots=torch.tensor([2, -1, 2, 4, 0], dtype=torch.int32, device=DEV), out=out)
    assert (out[1] == 2.0).all() and torch.isnan(out[2]).all() and torch.isnan(out[3]).all()
    assert torch.isfinite(out[[0, 4]]).all()
    assert torch.equal(pool[[1, 3]], keep[[1, 3]]) and not torch.equal(pool[2], keep[2])


def test_scan_skipped_rows_and_extremes():
    """dt = -Inf passes a row over; a huge step forgets the state; neither leaves a NaN behind, forward or backward."""
    g = gen(29)
    k = scan_case(g, 40, 8, 1, 16, F32)
    k["dt"][3:20] = -math.inf
    k["dt"][25] = 300.0
    seqs = [(0, 40)]
    args = ref_args(k)
    ry, _, _, sy, _ = R.scan(*args, True, seqs)
    o = on_gpu(k)
    out, kept = run_fwd(o, checkpoints=True)
    # roundings: as ever but for the step of 300, whose decays are zero (e^-300) on both sides
    finite = args[1].clone()
    finite[25] = 0.0
    count = R.scan_roundings(args[0], finite, args[2], args[7], True, seqs)
    check(out, ry, sy, count + gate_count(k), "out")
    got = run_bwd(o, torch.ones(40, 8, device=DEV), checkpoints=kept)
    for name, t in got.items():
        assert torch.isfinite(t).all(), name
    assert (got["ddt"][3:20] == 0).all()


def test_scan_nan_stays_in_its_channel_and_sequence():
    g = gen(31)
    k = scan_case(g, 60, 20, 1, 16, F32)
    k["x"][5, 7] = math.nan
    k["dt"][10, 3] = math.inf
    out = run_fwd(on_gpu(k), cu=cu_of([30, 30])).cpu()
    bad = torch.zeros(60, 20, dtype=torch.bool)
    bad[5:30, 7] = True
    bad[10:30, 3] = True
    assert torch.isfinite(out[~bad]).all()
    assert torch.isnan(out[5:30, 7]).all()


@pytest.mark.parametrize("n", [16, 5, 1])
def test_scan_growth_past_the_range_of_a_chunk(n):
    """A > 0: 16 rows of step 6 multiply a state by up to e^96, past fp32.  States that are zero stay zero, and a
    small one that the rows one by one keep in range is what they make it; the same against the row order."""
    g = gen(37)
    lengths = [209, 33]  # one joined by its own launch, one by its chunks
    seqs = R.spans(lengths, 0)
    k = scan_case(g, 242, 12, 1, n, F32, gate=False, skip=False, bias=False)
    k["A"] = 1.0 - 0.2 * torch.rand(12, n, generator=g)
    k["dt"] = torch.full((242, 12), 6.0)
    gy = torch.zeros(242, 12)
    x = torch.zeros(242, 12)
    for begin, end in seqs:
        k["dt"][begin:begin + 16] = 0.01
        x[end - 18] = 1e-30 * k["x"][end - 18]  # the last row of the last whole chunk but one
        gy[begin + 32] = 1e-30
    k["x"] = x
    args = ref_args(k)
    ry, _, last, sy, ms = R.scan(*args, False, seqs)
    ref, mag = R.scan_backward(*args, False, seqs, wide(gy))
    assert all(float(t.abs().max()) < 1e30 for t in ref.values() if t is not None)
    o = on_gpu(k)
    state = torch.zeros(2, 12, n, device=DEV)
    out = run_fwd(o, softplus=False, cu=cu_of(lengths), state=state)
    count = R.scan_roundings(args[0], args[1], args[2], args[7], False, seqs)
    check(out, ry, sy, count, "out")
    check(state, torch.stack(last), torch.stack([ms[208], ms[241]]), count, "state")
    got = run_bwd(o, dev(gy), softplus=False, cu=cu_of(lengths))
    for name, more in {"dx": n, "ddt": n, "dB": 12, "dC": 12, "dA": 242}.items():
        check(got[name], ref[name], mag[name], 2 * count + 16 + more, name)


@pytest.mark.parametrize("long", [0, 300])
def test_scan_of_more_sequences_than_a_grid_is_wide(long):
    """70000 sequences of one row, which is then D x + sum_n C d x B, and behind them, packed, one that is cut."""
    g = gen(39)
    many, c, n = 70000, 4, 2
    rows = many + long
    k = scan_case(g, rows, c, 1, n, F32, gate=False)
    o = on_gpu(k)
    kw = {"cu": cu_of([1] * many + [long])} if long else {"nseq": many}
    out = run_fwd(o, **kw)
    gy = rnd(g, rows, c)
    got = run_bwd(o, dev(gy), **kw)
    args = ref_args(k)
    x, d = args[0][:many], torch.nn.functional.softplus(args[1][:many] + args[7])
    terms = args[4][:many, 0, None, :] * (d * x)[..., None] * args[3][:many, 0, None, :]
    skip = args[5] * x
    # d: an exponential, a logarithm and their sum; then products and a sum of n + 1 terms
    count = R.scan_roundings(args[0][:1], args[1][:many], args[2], args[7], True, [(0, 1)]) + 2 * n + 16
    check(out[:many], terms.sum(-1) + skip, terms.abs().sum(-1) + skip.abs(), count, "out")
    ddx = (args[4][:many, 0, None, :] * args[3][:many, 0, None, :]).sum(-1) * d + args[5]
    mag = (args[4][:many, 0, None, :] * args[3][:many, 0, None, :]).abs().sum(-1) * d + args[5].abs()
    check(got["dx"][:many], wide(gy)[:many] * ddx, wide(gy)[:many].abs() * mag, count, "dx")
    if long:
        tail = [t[many:] if t is not None and t.shape[0] == rows else t for t in args]
        ry, _, _, sy, _ = R.scan(*tail, True, [(0, long)])
        ref, m = R.scan_backward(*tail, True, [(0, long)], wide(gy)[many:])
        count = R.scan_roundings(tail[0], tail[1], tail[2], tail[7], True, [(0, long)])
        check(out[many:], ry, sy, count, "out of the last")
        check(got["dx"][many:], ref["dx"], m["dx"], 2 * count + 16 + n, "dx of the last")


# ------------------------------------------------------------------------------------------------- block join

JOIN_PARTS = ["grosp", "r", "rp", "os", "gp", "o", "", "rsp", "go"]
JOIN_SIZES = [(F32, F32, 1, 3), (F32, F32, 96, 5), (BF16, F32, 192, 9), (BF16, BF16, 513, 3), (BF16, F32, 1152, 70),
              (F32, F32, 1001, 4), (BF16, BF16, 1032, 2), (BF16, F32, 2304, 5), (F32, F32, 4097, 2),
              (BF16, BF16, 5000, 3), (BF16, F32, 16384, 2), (F32, F32, 12001, 2)]


@pytest.mark.parametrize("parts", JOIN_PARTS)
@pytest.mark.parametrize("dtype,rt,c,rows", JOIN_SIZES)
def test_join_forward_and_backward(dtype, rt, c, rows, parts):
    g = gen(c + rows)
    rt = rt if "r" in parts else dtype
    h = rnd(g, rows, c, dtype=dtype)
    k = dict(gate=rnd(g, rows, c, dtype=dtype) if "g" in parts else None,
             residual=rnd(g, rows, c, dtype=rt, by=2.0) if "r" in parts else None,
             post=rnd(g, c, by=0.3) + 1 if "o" in parts else None, scale=rnd(g, c) if "s" in parts else None,
             pre=rnd(g, c, by=0.3) + 1 if "p" in parts else None)
    gj, gn = rnd(g, rows, c, dtype=rt), rnd(g, rows, c, dtype=dtype) if "p" in parts else None
    eps = 1e-5
    kd = {n: dev(t) for n, t in k.items()}
    joined, normed = S.gspn_block_join_fwd(dev(h), **kd, eps=eps)
    stored = wide(joined)
    kw = {n: wide(t) for n, t in k.items()}
    rj, rn, mj = R.join(wide(h), **kw, eps=eps, store=lambda v: stored)
    # the norm's root: a sum of c squares (a tree, but c covers any order) halved by the root, and 4; gate: 2 |z| + 8;
    # three products and the sum
    norm = c / 2 + 4
    gate = 2 * float(k["gate"].float().abs().max()) + 8 if "g" in parts else 0
    count = ("o" in parts) * norm + gate + 6
    check(joined, rj, mj, count, "joined")
    if "p" in parts:
        check(normed, rn, rn.abs(), norm + 4, "normed")
    grads = S.gspn_block_join_bwd(dev(h), dev(gj), dev(gn), joined, **kd, eps=eps)
    got = dict(zip(("dh", "dgate", "dresidual", "dpost", "dscale", "dpre"), grads))
    ref, mag = R.join_backward(wide(h), **kw, eps=eps, joined=stored, gjoined=wide(gj), gnormed=wide(gn))
    # back through up to two norms, each with its root (cubed: 3 times) and a sum over the channels
    back = 2 * (3 * norm + c + 8) + 2 * gate + 8
    assert {n for n, t in got.items() if t is not None} == set(ref)
    for name in ref:
        check(got[name], ref[name], mag[name], back + (rows if name in ("dpost", "dscale", "dpre") else 0), name)


@pytest.mark.parametrize("parts", ["grosp", "rp"])
@pytest.mark.parametrize("dtype,rt", [(F32, F32), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("c", [2, 7, 8, 9, 12, 17, 67, 511, 515, 1023, 4093, 8190, 8199])
def test_join_rows_of_any_width(c, dtype, rt, parts):
    """Widths around the lanes' eight and four columns, the wave's 512 and the workgroups' 4096 and 8192."""
    test_join_forward_and_backward(dtype, rt, c, 3, parts)


@pytest.mark.parametrize("c", [5, 9, 64, 130, 515, 5003, 8201])
def test_join_writes_its_rows_alone(c):
    """Outputs as columns of wider rows whose other columns hold 7: they still do, and the values are the plain call's
    (within the roundings of another order, as in the strided test)."""
    g = gen(44)
    h, gate, res = (rnd(g, 4, c, dtype=BF16) for _ in range(3))
    w = [rnd(g, c, by=0.3) + 1 for _ in range(3)]
    out, normed = strided(torch.zeros_like(h)), strided(torch.zeros_like(h))
    for v in (out, normed):
        v.fill_(0)
    a = S.gspn_block_join_fwd(dev(h), dev(gate), dev(res), *map(dev, w))
    S.gspn_block_join_fwd(dev(h), dev(gate), dev(res), *map(dev, w), out=out, normed=normed)
    steps = torch.finfo(BF16).eps + c * R.U
    for v, ref in ((out, a[0]), (normed, a[1])):
        whole = v._base if v._base is not None else v
        assert (whole[:, :c + 3] == 7.0).all()
        # joined: the gated term's rounding and the sum's, of terms not larger than |ref| + |res|; normed: that times
        # pre / rms, which is below 2 for rows of such sums
        assert (v.float() - ref.float()).abs().le((ref.float().abs() + dev(res).float().abs()) * 2 * steps).all()


@pytest.mark.parametrize("c", [96, 2050])
def test_join_strided_rows_and_one_sided_gradients(c):
    g = gen(41)
    h, gate, res = (rnd(g, 6, c, dtype=BF16) for _ in range(3))
    pre = rnd(g, c)
    a = S.gspn_block_join_fwd(dev(h), dev(gate), dev(res), pre=dev(pre))
    b = S.gspn_block_join_fwd(strided(h), strided(gate), strided(res), pre=dev(pre), out=strided(torch.zeros_like(h)),
                              normed=strided(torch.zeros_like(h)))
    # the strided rows' alignment may take the element form, which adds a row's squares in another order: the root's
    # c / 2 roundings and then a step of bf16
    assert torch.equal(a[0], b[0])
    assert (a[1].float() - b[1].float()).abs().le(a[1].float().abs() * (torch.finfo(BF16).eps + c * R.U)).all()
    only = S.gspn_block_join_bwd(dev(h), None, dev(gate), a[0], dev(gate), dev(res), pre=dev(pre))
    zero = S.gspn_block_join_bwd(dev(h), torch.zeros_like(a[0]), dev(gate), a[0], dev(gate), dev(res), pre=dev(pre))
    for x, y in zip(only, zero):
        assert (x is None and y is None) or torch.equal(x, y)


@pytest.mark.parametrize("c", [96, 1032, 5000, 33])
def test_join_without_a_norm_keeps_infinities_out_of_dh(c):
    g = gen(43)
    h, scale, gj = rnd(g, 3, c), rnd(g, c), rnd(g, 3, c)
    h[0, 1], h[1, 0], h[2, c - 1] = math.inf, -math.inf, math.nan
    dh = S.gspn_block_join_bwd(dev(h), dev(gj), None, None, residual=dev(gj), scale=dev(scale))[0]
    assert torch.equal(dh.cpu(), gj * scale)


def test_join_zero_rows_and_row_of_zeros():
    c = 64
    h = torch.zeros(2, c, device=DEV)
    post, pre = torch.ones(c, device=DEV), torch.ones(c, device=DEV)
    j, n = S.gspn_block_join_fwd(h, post=post, pre=pre)
    assert (j == 0).all() and (n == 0).all()
    grads = S.gspn_block_join_bwd(h, torch.ones_like(h), torch.ones_like(h), j, post=post, pre=pre)
    assert all(torch.isfinite(t).all() for t in grads if t is not None)
    e = torch.empty(0, c, device=DEV)
    j, n = S.gspn_block_join_fwd(e, post=post, pre=pre)
    assert j.shape == (0, c) and n.shape == (0, c)
    grads = S.gspn_block_join_bwd(e, e, e, e, post=post, pre=pre)
    assert (grads[3] == 0).all() and (grads[5] == 0).all()  # sums over no rows


# -------------------------------------------------------------------------------------- empty calls, far strides

def test_empty_calls():
    c, n = 32, 16
    w, A = torch.randn(c, 4, device=DEV), -torch.rand(c, n, device=DEV)
    x, bc = torch.empty(0, c, device=DEV), torch.empty(0, 1, n, device=DEV)
    none = torch.zeros(1, dtype=torch.int32, device=DEV)  # no sequence
    for kw in ({"cu": none}, {"nseq": 1}, {"cu": torch.zeros(4, dtype=torch.int32, device=DEV)}):
        assert S.gspn_causal_conv_fwd(x, w, **kw).shape == (0, c)
        dx, dw, _ = S.gspn_causal_conv_bwd(x, w, None, x, **kw)
        assert dx.shape == (0, c) and (dw == 0).all()
        assert S.gspn_selective_scan_fwd(x, x, A, bc, bc, **kw).shape == (0, c)
        grads = S.gspn_selective_scan_bwd(x, x, A, bc, bc, x, **kw)
        assert (grads[2] == 0).all()
    pool = torch.ones(2, c, n, device=DEV)
    S.gspn_selective_scan_fwd(x, x, A, bc, bc, cu=torch.zeros(3, dtype=torch.int32, device=DEV), state=pool,
                              resume=torch.tensor([True, False], device=DEV))
    assert (pool[0] == 1).all() and (pool[1] == 0).all()
    assert S.gspn_causal_conv_step(x, w, None, torch.ones(1, 3, c, device=DEV)).shape == (0, c)
    assert S.gspn_selective_scan_step(x, x, A, bc, bc, pool).shape == (0, c)


def test_rows_beyond_32_bits():
    """The widest row stride, 2^26 elements: the last of 70 rows lies past 2^32 elements."""
    ld, c, rows = 1 << 26, 16, 70
    big = torch.empty((rows - 1) * ld + 1024, dtype=BF16, device=DEV)
    g = gen(6)
    far = lambda at: torch.as_strided(big, (rows, c), (ld, 1), at)  # noqa: E731
    k = scan_case(g, rows, c, 1, 8, BF16)
    w = dev(rnd(g, c, 4))
    x, dt, z = far(0), far(64), far(128)
    for t, v in ((x, k["x"]), (dt, k["dt"]), (z, k["z"])):
        t.copy_(v)
    near = on_gpu(k)
    assert torch.equal(S.gspn_causal_conv_fwd(x, w, out=far(256)), S.gspn_causal_conv_fwd(near["x"], w))
    for a, b in zip(S.gspn_causal_conv_bwd(x, w, None, z)[:2], S.gspn_causal_conv_bwd(near["x"], w, None, near["z"])):
        assert torch.equal(a, b)
    o = dict(near, x=x, dt=dt, z=z)
    out, kept = run_fwd(o, checkpoints=True, out=far(512))
    assert torch.equal(out, run_fwd(near))
    for a, b in zip(run_bwd(o, x, checkpoints=kept).values(), run_bwd(near, near["x"]).values()):
        assert torch.equal(a, b)
    pre = dev(rnd(g, c))
    far_join, near_join = (S.gspn_block_join_fwd(a, b, d, pre=pre) for a, b, d in
                           ((x, z, dt), (near["x"], near["z"], near["dt"])))
    assert all(torch.equal(a, b) for a, b in zip(far_join, near_join))
    with pytest.raises(G.GspnError):
        S.gspn_causal_conv_fwd(torch.as_strided(big, (2, c), (ld + 1, 1)), w)


# ------------------------------------------------------------------------------------- autograd, streams, graphs

def leaves(*ts):
    return [None if t is None else t.detach().clone().requires_grad_() for t in ts]


@pytest.mark.parametrize("packed", [False, True])
def test_autograd_forms_give_the_backward_calls(packed):
    g = gen(50)
    cu = cu_of([9, 14], 1) if packed else None
    kw = {"cu": cu} if packed else {"nseq": 2}
    rows = 24
    k = on_gpu(scan_case(g, rows, 40, 1, 16, BF16))
    w, b, gy = dev(rnd(g, 40, 4)), dev(rnd(g, 40)), dev(rnd(g, rows, 40, dtype=BF16))
    x, wl, bl = leaves(k["x"], w, b)
    y = S.causal_conv(x, wl, bl, **kw)
    for got, ref in zip(torch.autograd.grad(y, [x, wl, bl], gy), S.gspn_causal_conv_bwd(k["x"], w, b, gy, **kw)):
        assert torch.equal(got, ref)
    names = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")
    ls = leaves(*(k[n] for n in names))
    y = S.selective_scan(*ls, **kw)
    ref = run_bwd(k, gy, **kw)
    for n, got in zip(("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias"), torch.autograd.grad(y, ls, gy)):
        assert torch.equal(got, ref[n]), n
    if packed:
        assert (y[0] == 0).all()
    h, gate, res, pre = leaves(k["x"], k["z"], k["dt"].float(), dev(rnd(g, 40)))
    j, n = S.block_join(h, gate, res, pre=pre)
    got = torch.autograd.grad([j, n], [h, gate, res, pre], [gy.float(), gy])
    ref = S.gspn_block_join_bwd(h, gy.float(), gy, j.detach(), gate, res, pre=pre)
    for a, b in zip(got, (ref[0], ref[1], ref[2], ref[5])):
        assert torch.equal(a, b)
    # only one of the two outputs used
    got = torch.autograd.grad(S.block_join(h, gate, res, pre=pre)[1].float().sum(), [res])[0]
    ref = S.gspn_block_join_bwd(h, None, torch.ones_like(gy), j.detach(), gate, res, pre=pre)[2]
    assert torch.equal(got, ref)


@pytest.mark.parametrize("packed", [False, True])
def test_autograd_forms_without_a_gradient(packed):
    """No leaf, or no gradients wanted: the same values, and nothing kept for a backward."""
    g = gen(51)
    kw = {"cu": cu_of([9, 14], 1)} if packed else {"nseq": 2}
    k = on_gpu(scan_case(g, 24, 40, 1, 16, BF16))
    w, pre = dev(rnd(g, 40, 4)), dev(rnd(g, 40))
    names = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")
    calls = [(lambda x, w: S.causal_conv(x, w, **kw), (k["x"], w)),
             (lambda *a: S.selective_scan(*a, **kw), [k[n] for n in names]),
             (lambda h, p: S.block_join(h, pre=p)[0], (k["x"], pre)), (lambda h, p: S.block_join(h, pre=p)[1], (k["x"], pre))]
    for f, ts in calls:
        ref = f(*leaves(*ts))
        assert ref.grad_fn is not None
        plain = f(*ts)
        with torch.no_grad():
            off = f(*leaves(*ts))
        for y in (plain, off):
            assert y.grad_fn is None and torch.equal(y, ref)


@pytest.mark.parametrize("op", ["conv", "scan", "join"])
def test_gradients_by_differences(op):
    """The fp32 gradient along a direction against a central difference of the fp32 forward.  With a step h the
    difference carries h^2 of the third derivative (values of order one here) and the forward's own error over h: for
    sums of 2000 values of 100 U that is 100 U sqrt(2000) / h.  At h = 2^-6 both are below 2e-2 of the slope's scale."""
    g = gen(60)
    k = on_gpu(scan_case(g, 50, 40, 1, 16, F32))
    gy = dev(rnd(g, 50, 40))
    if op == "conv":
        ts = [k["x"], dev(rnd(g, 40, 4)), dev(rnd(g, 40))]
        f = lambda *a: S.causal_conv(*a)  # noqa: E731
    elif op == "scan":
        ts = [k[n] for n in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")]
        f = lambda *a: S.selective_scan(*a)  # noqa: E731
    else:
        ts = [k["x"], k["z"], k["dt"], dev(rnd(g, 40)), dev(rnd(g, 40)), dev(rnd(g, 40))]
        f = lambda *a: sum(S.block_join(*a))  # noqa: E731
    ls = leaves(*ts)
    grads = torch.autograd.grad(f(*ls), ls, gy)
    h = 2.0 ** -6
    for i, t in enumerate(ts):
        v = torch.randn(t.shape, generator=g).to(DEV)
        v *= 1.0 / v.norm()
        at = lambda s: float((f(*ts[:i], t + s * v, *ts[i + 1:]).double() * gy.double()).sum())  # noqa: E731
        slope = (at(h) - at(-h)) / (2 * h)
        assert abs(slope - float((grads[i].double() * v.double()).sum())) <= 2e-2 * max(1.0, float(grads[i].norm())), i


def test_another_stream_and_two_at_once():
    g = gen(70)
    k = on_gpu(scan_case(g, 300, 64, 1, 16, BF16))
    k2 = on_gpu(scan_case(g, 300, 64, 1, 16, BF16))
    ref, ref2 = run_fwd(k), run_fwd(k2)
    gy = torch.ones_like(ref)
    gref = run_bwd(k, gy)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(a):
        y = run_fwd(k)
        gr = run_bwd(k, gy)
    with torch.cuda.stream(b):
        y2 = run_fwd(k2)
    torch.cuda.synchronize()
    assert torch.equal(y, ref) and torch.equal(y2, ref2)
    for n in gref:
        assert torch.equal(gr[n], gref[n]), n


def test_graphs_replay_what_eager_gives():
    """A decoding step and a training step, each captured; replays with new inputs and eager work between them."""
    g = gen(80)
    c, n, s = 64, 16, 4
    k = on_gpu(scan_case(g, s, c, 1, n, BF16))
    w, b = dev(rnd(g, c, 4)), dev(rnd(g, c))
    pre = dev(rnd(g, c))
    res = dev(rnd(g, s, c))
    conv0, scan0 = dev(rnd(g, s, 3, c, dtype=BF16)), dev(rnd(g, s, c, n))
    slots = torch.tensor([3, 1, 0, 2], dtype=torch.int32, device=DEV)

    def step(x, conv, state):
        u = S.gspn_causal_conv_step(x, w, b, conv, slots)
        y = S.gspn_selective_scan_step(u, k["dt"], k["A"], k["B"], k["C"], state, k["D"], k["z"], k["dt_bias"],
                                       slots=slots)
        return S.gspn_block_join_fwd(y, residual=res, pre=pre)

    t = on_gpu(scan_case(g, 96, c, 1, n, BF16))
    gy = dev(rnd(g, 96, c, dtype=BF16))
    tl = leaves(*(t[m] for m in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")))
    wl, bl = leaves(w, b)

    def train(x):
        u = S.causal_conv(x, wl, bl, nseq=2)
        y = S.selective_scan(u, *tl[1:], nseq=2)
        j, _ = S.block_join(y, residual=x)
        return torch.autograd.grad(j, [wl, bl, *tl[1:]], gy)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    conv, state, x = conv0.clone(), scan0.clone(), k["x"].clone()
    xt = t["x"].clone()
    with torch.cuda.stream(side):
        step(x, conv, state)
        train(xt)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    decode, training = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(decode):
        out = step(x, conv, state)
    with torch.cuda.graph(training):
        grads = train(xt)
    conv.copy_(conv0)
    state.copy_(scan0)
    ec, es = conv0.clone(), scan0.clone()
    for i in range(4):
        x.copy_(rnd(g, s, c, dtype=BF16))
        xt.copy_(rnd(g, 96, c, dtype=BF16))
        decode.replay()
        training.replay()
        torch.cuda.synchronize()
        eager = step(x, ec, es)
        for a, r in zip(out, eager):
            assert torch.equal(a, r), i
        assert torch.equal(conv, ec) and torch.equal(state, es), i
        for a, r in zip(grads, train(xt)):
            assert torch.equal(a, r), i
        torch.cuda.synchronize()


# --------------------------------------------------------------------------------------- together, as they are used

def mixer(p, h, conv, scan, join, residual):
    """A state space block: norm'd input h -> projection -> convolution -> scan -> projection -> join."""
    c, n = p["A"].shape
    rank = p["dtw"].shape[0]
    both = h @ p["inw"]
    u = conv(both[..., :c])
    dbc = u @ p["xw"]
    dt = dbc[..., :rank] @ p["dtw"]
    B, C = dbc[..., rank:rank + n].unflatten(-1, (1, n)), dbc[..., rank + n:].unflatten(-1, (1, n))
    y = scan(u, dt, B, C, both[..., c:])
    return join(y @ p["outw"], residual)


def mixer_params(g, m=48, c=96, n=16, rank=6):
    return {"inw": rnd(g, m, 2 * c, by=m ** -0.5), "cw": rnd(g, c, 4, by=0.5), "cb": rnd(g, c, by=0.1),
            "xw": rnd(g, c, rank + 2 * n, by=c ** -0.5), "dtw": rnd(g, rank, c, by=rank ** -0.5),
            "dtb": rnd(g, c) - 2, "A": -torch.exp(rnd(g, c, n, by=0.5)), "D": rnd(g, c),
            "outw": rnd(g, c, m, by=c ** -0.5), "post": rnd(g, m, by=0.1) + 1, "scale": rnd(g, m, by=0.1) + 0.5,
            "pre": rnd(g, m, by=0.1) + 1}


def test_block_prompt_then_tokens_and_its_gradients():
    g = gen(90)
    p = {k: dev(v) for k, v in mixer_params(g).items()}
    s, length, m = 3, 40, 48
    h0, res0 = dev(rnd(g, s, length, m)), dev(rnd(g, s, length, m))

    def whole(p, h, res):
        return mixer(p, h, lambda u: S.causal_conv(u, p["cw"], p["cb"]),
                     lambda u, dt, B, C, z: S.selective_scan(u, dt, p["A"], B, C, p["D"], z, p["dtb"]),
                     lambda y, r: S.block_join(y, None, r, p["post"], p["scale"], p["pre"]), res)

    def plain(p, h, res):  # the same block in float64, by definition
        def conv(u):
            pad = torch.nn.functional.pad(u, (0, 0, 3, 0))
            return R.silu(sum(pad[:, j:j + length] * p["cw"][:, j] for j in range(4)) + p["cb"])

        def scan(u, dt, B, C, z):
            d = torch.nn.functional.softplus(dt + p["dtb"], threshold=700.0)
            hs, ys = torch.zeros(s, *p["A"].shape, dtype=u.dtype), []
            for t in range(length):
                hs = torch.exp(d[:, t, :, None] * p["A"]) * hs + (d[:, t] * u[:, t])[..., None] * B[:, t]
                ys.append((hs * C[:, t]).sum(-1) + p["D"] * u[:, t])
            return torch.stack(ys, 1) * R.silu(z)

        def join(y, r):
            rms = lambda v: torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6)  # noqa: E731
            o = r + p["scale"] * (y / rms(y) * p["post"])
            return o, o / rms(o) * p["pre"]

        return mixer(p, h, conv, scan, join, res)

    lp = {k: v.clone().requires_grad_() for k, v in p.items()}
    lh, lr = leaves(h0, res0)
    joined, normed = whole(lp, lh, lr)
    pd = {k: wide(v).requires_grad_() for k, v in p.items()}
    hd, rd = wide(h0).requires_grad_(), wide(res0).requires_grad_()
    dj, dn = plain(pd, hd, rd)
    # five chained products of up to 96 terms, the scan over 40 rows and two norms of 48: below 2^12 roundings of
    # values of order one along any way, and what passes several ways adds up like their number's root
    tol = 2 ** 12 * R.U
    for a, b in ((joined, dj), (normed, dn)):
        assert (wide(a) - b.detach()).norm() <= tol * b.detach().norm()
    gj, gn = dev(rnd(g, s, length, m)), dev(rnd(g, s, length, m))
    names = sorted(lp)
    got = torch.autograd.grad([joined, normed], [lp[k] for k in names] + [lh, lr], [gj, gn])
    ref = torch.autograd.grad([dj, dn], [pd[k] for k in names] + [hd, rd], [wide(gj), wide(gn)])
    for k, a, b in zip(names + ["h", "residual"], got, ref):
        assert (wide(a) - b).norm() <= 4 * tol * b.norm(), k

    # serving: a prompt into the pools, then token by token
    conv, state = torch.zeros(5, 3, 96, device=DEV), torch.zeros(5, 96, 16, device=DEV)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device=DEV)
    cut = 31
    outs = [mixer(p, h0[:, :cut], lambda u: S.gspn_causal_conv_fwd(u, p["cw"], p["cb"], state=conv, slots=slots),
                  lambda u, dt, B, C, z: S.gspn_selective_scan_fwd(u, dt, p["A"], B, C, p["D"], z, p["dtb"],
                                                                   state=state, slots=slots),
                  lambda y, r: S.gspn_block_join_fwd(y, None, r, p["post"], p["scale"], p["pre"]),
                  res0[:, :cut].contiguous())[1]]  # rows evenly spaced over the batch
    for t in range(cut, length):
        outs.append(mixer(p, h0[:, t], lambda u: S.gspn_causal_conv_step(u, p["cw"], p["cb"], conv, slots),
                          lambda u, dt, B, C, z: S.gspn_selective_scan_step(u, dt, p["A"], B, C, state, p["D"], z,
                                                                            p["dtb"], slots=slots),
                          lambda y, r: S.gspn_block_join_fwd(y, None, r, p["post"], p["scale"], p["pre"]),
                          res0[:, t])[1][:, None])
    assert (wide(torch.cat(outs, 1)) - dn.detach()).norm() <= tol * dn.detach().norm()


# ------------------------------------------------------------------------------------------------ refusals

def test_refusals_on_the_device():
    """Arguments refused by the binding (ValueError, TypeError) or the library (GspnError), nothing launched."""
    c, n = 32, 16
    x, w = torch.randn(8, c, device=DEV), torch.randn(c, 4, device=DEV)
    A, bc = -torch.rand(c, n, device=DEV), torch.randn(8, 1, n, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    cases = [
        (TypeError, lambda: S.gspn_causal_conv_fwd(x.half(), w)),
        (TypeError, lambda: S.gspn_causal_conv_fwd(x, w.bfloat16())),
        (ValueError, lambda: S.gspn_causal_conv_fwd(x, w[:, :, None])),
        (ValueError, lambda: S.gspn_causal_conv_fwd(x.t(), w)),
        (ValueError, lambda: S.gspn_causal_conv_fwd(x[None, None], w)),
        (ValueError, lambda: S.gspn_causal_conv_fwd(x, w, nseq=3)),
        (ValueError, lambda: S.gspn_causal_conv_fwd(x, w, cu=torch.zeros(2, **i32), nseq=2)),
        (TypeError, lambda: S.gspn_causal_conv_fwd(x, w, cu=torch.zeros(2, dtype=torch.int64, device=DEV))),
        (ValueError, lambda: S.gspn_causal_conv_fwd(x, w, cu=torch.zeros(2, dtype=torch.int32))),
        (ValueError, lambda: S.gspn_causal_conv_fwd(x, w, slots=torch.zeros(1, **i32))),
        (ValueError, lambda: S.gspn_causal_conv_fwd(x, w, nseq=2, state=torch.zeros(1, 3, c, device=DEV))),
        (ValueError, lambda: S.gspn_causal_conv_fwd(x, w, state=torch.zeros(1, 4, c, device=DEV))),
        (ValueError, lambda: S.gspn_causal_conv_step(x, w, None, None)),
        (ValueError, lambda: S.gspn_causal_conv_fwd(x[:1].expand(8, c), w)),
        (G.GspnError, lambda: S.gspn_causal_conv_fwd(x, torch.randn(c, 5, device=DEV))),
        (G.GspnError, lambda: S.gspn_causal_conv_fwd(x, w, out=x)),
        (ValueError, lambda: S.gspn_selective_scan_fwd(x, x, A, bc[:, 0], bc)),
        (ValueError, lambda: S.gspn_selective_scan_fwd(x, x, A, bc.expand(8, 3, n), bc)),
        (ValueError, lambda: S.gspn_selective_scan_fwd(x, x[:4], A, bc, bc)),
        (ValueError, lambda: S.gspn_selective_scan_fwd(x, x, A[:4], bc, bc)),
        (TypeError, lambda: S.gspn_selective_scan_fwd(x, x.bfloat16(), A, bc, bc)),
        (ValueError, lambda: S.gspn_selective_scan_bwd(x, x, A, bc, bc, x, checkpoints=torch.zeros(3, device=DEV))),
        (G.GspnError, lambda: S.gspn_selective_scan_fwd(x, x, -torch.rand(c, 17, device=DEV),
                                                        *[torch.randn(8, 1, 17, device=DEV)] * 2)),
        (G.GspnError, lambda: S.gspn_selective_scan_fwd(x, x, A, bc, bc, out=x)),
        (G.GspnError, lambda: S.gspn_selective_scan_bwd(x, x, A, bc, bc, x,
                                                        workspace=torch.empty(64, dtype=torch.uint8, device=DEV))),
        (TypeError, lambda: S.gspn_block_join_fwd(x, residual=x.half())),
        (TypeError, lambda: S.gspn_block_join_fwd(x, residual=x.bfloat16())),
        (ValueError, lambda: S.gspn_block_join_fwd(x, normed=x)),
        (ValueError, lambda: S.gspn_block_join_fwd(x, pre=w[0])),
        (ValueError, lambda: S.gspn_block_join_bwd(x, x, x, x)),
        (ValueError, lambda: S.gspn_block_join_bwd(x, x, None, x, pre=torch.ones(c, device=DEV))),
        (G.GspnError, lambda: S.gspn_block_join_fwd(x, out=x)),
        (G.GspnError, lambda: S.gspn_block_join_fwd(x, eps=-1.0)),
        (G.GspnError, lambda: S.gspn_block_join_fwd(torch.zeros(1, 16385, device=DEV))),
    ]
    for i, (error, call) in enumerate(cases):
        with pytest.raises(error):
            call()
            print("case %d was not refused" % i, flush=True)
