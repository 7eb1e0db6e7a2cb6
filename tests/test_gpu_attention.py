"""The attention operators on the GPU against their 64-bit definitions (attention_reference), element by element within
the bounds that stand there, plus half a step of the type that a result is stored in."""
import math
import sys

import pytest
import torch

import attention_reference as R
from linear_spatial_propagation_gspn_amd import attention as A
from linear_spatial_propagation_gspn_amd import sequence as S

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    A.lib()
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
    rows, h, d = t.shape
    big = torch.full((rows, 2 * h * d + 3), 7.0, dtype=t.dtype, device=DEV)
    view = big[:, h * d + 3:].unflatten(1, (h, d))
    view.copy_(t)
    return view


def cu_of(lengths, first=0):
    return torch.tensor([a for a, _ in R.spans(lengths, first)] + [first + sum(lengths)], dtype=torch.int32, device=DEV)


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def check(got, ref, what, rows=None, store=True):
    """|got - value| <= half a step of got's type + the bound, element by element; infinities where the value has them."""
    value, bound = ref
    half = R.half_step(got.dtype) if store else 0.0
    got = wide(got)
    if rows is not None:
        got, value, bound = got[rows], value[rows], bound[rows]
    assert got.shape == value.shape, what
    inf = torch.isinf(value)
    assert torch.equal(got[inf], value[inf]), what
    got, value, bound = got[~inf], value[~inf], bound[~inf]
    most = half * value.abs() * (1 + 2.0 ** -7) + 1.01 * R.U * bound + 1e-37
    off = (got - value).abs()
    assert torch.isfinite(got).all(), what
    assert (off <= most).all(), "%s: worst %.3g of its bound" % (what, float((off / most).max()))


def inside(seqs):
    return [t for lo, hi in seqs for t in range(lo, hi)]


def check_lse(got, ref, rows):
    check(got[:, rows], (ref[0][:, rows], ref[1][:, rows]), "lse", store=False)


# ------------------------------------------------------------------------------------------------ head rotary

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,heads,kv_heads,d,sections,view", [
    (1, 1, 1, 2, (1,), False), (7, 3, 2, 16, (8,), True), (65, 5, 1, 80, (6, 14, 14), False), (33, 2, 2, 27, (3, 4), True),
    (130, 4, 0, 128, (64,), False), (9, 2, 1, 256, (30, 0, 60, 38), True), (21, 17, 3, 1, (0,), False),
    (40, 9, 2, 62, (31,), False), (5, 2, 2, 200, (11,), False), (11, 5, 2, 72, (36,), True), (6, 3, 1, 96, (18, 6), False),
    (4, 2, 2, 64, (32,), True), (3, 1, 1, 252, (126,), False), (70, 6, 6, 24, (6,), True)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [True, False])
def test_rotary(dtype, rows, heads, kv_heads, d, sections, view, interleaved, norm):
    g = gen(rows + d)
    pairs = sum(sections)
    freqs = 10000.0 ** -torch.rand(pairs, generator=g, dtype=torch.float64)
    pos = torch.randint(-3000, 1000000, (rows, len(sections)), generator=g, dtype=torch.int32)
    args, kw, refs = {}, {}, {}
    for n, h in (("q", heads), ("k", kv_heads)):
        if not h:
            continue
        x, go = rnd(g, rows, h, d, dtype=dtype), rnd(g, rows, h, d, dtype=dtype)
        w = 1 + rnd(g, d, by=0.2) if norm else None
        refs[n] = R.rotary(wide(x), wide(w), pos, freqs, sections, interleaved, 1e-6, wide(go))
        kw[n] = strided(x) if view else dev(x)
        kw["g" + n] = strided(go) if view else dev(go)
        kw[n + "_weight"] = dev(w)
    q, gq = kw.pop("q"), kw.pop("gq")
    gk = kw.pop("gk", None)
    more = dict(kw, sections=sections, interleaved=interleaved)
    y, yk = A.gspn_head_rotary_fwd(q, dev(pos), dev(freqs), **more)
    dq, dk, dqw, dkw = A.gspn_head_rotary_bwd(q, dev(pos), dev(freqs), gq, gk=gk, **more)
    for n, got in (("q", (y, dq, dqw)), ("k", (yk, dk, dkw))):
        if n not in refs:
            assert got == (None, None, None)
            continue
        for part, t in zip(("y", "dx", "dw"), got):
            if part in refs[n]:
                check(t, refs[n][part], n + part)
            else:
                assert t is None
    again = A.gspn_head_rotary_bwd(q, dev(pos), dev(freqs), gq, gk=gk, **more)
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dqw, dkw), again) if a is not None)


def test_rotary_batch_form_outputs_and_many_rows():
    g = gen(1)
    q, k = rnd(g, 3, 11, 4, 32, dtype=BF16), rnd(g, 3, 11, 2, 32, dtype=BF16)
    pos, freqs = torch.arange(11, dtype=torch.int32).expand(3, 11).contiguous(), torch.rand(16, dtype=torch.float64)
    y, yk = A.gspn_head_rotary_fwd(dev(q), dev(pos), dev(freqs), dev(k))
    flat = A.gspn_head_rotary_fwd(dev(q).view(33, 4, 32), dev(pos).view(33, 1), dev(freqs), dev(k).view(33, 2, 32))
    assert torch.equal(y.view(33, 4, 32), flat[0]) and torch.equal(yk.view(33, 2, 32), flat[1])
    both = torch.full((33, 6 * 32), 5.0, dtype=BF16, device=DEV)  # the outputs as slices of one matrix
    out, out_k = both[:, :128].unflatten(1, (4, 32)), both[:, 128:].unflatten(1, (2, 32))
    A.gspn_head_rotary_fwd(dev(q).view(33, 4, 32), dev(pos).view(33), dev(freqs), dev(k).view(33, 2, 32), out=out,
                           out_k=out_k)
    assert torch.equal(out, flat[0]) and torch.equal(out_k, flat[1])
    # more rows than the backward has waves
    rows = 9001
    x, go, w = rnd(g, rows, 1, 8), rnd(g, rows, 1, 8), 1 + rnd(g, 8, by=0.1)
    p = torch.arange(rows, dtype=torch.int32)[:, None]
    f = torch.rand(3, generator=g, dtype=torch.float64)
    ref = R.rotary(wide(x), wide(w), p, f, (3,), False, 1e-6, wide(go))
    dq, _, dw, _ = A.gspn_head_rotary_bwd(dev(x), dev(p), dev(f), dev(go), q_weight=dev(w))
    check(dq, ref["dx"], "dx")
    check(dw, ref["dw"], "dw")
    none = A.gspn_head_rotary_bwd(dev(x)[:0], dev(p)[:0], dev(f), dev(go)[:0], q_weight=dev(w))
    assert none[0].shape == (0, 1, 8) and (none[2] == 0).all()


def test_rotary_far_positions_and_values_at_the_ends():
    """Angles of 2^31 positions keep their place in the turn; a NaN or an infinity stays in its own head."""
    pos = ints([[2 ** 31 - 1], [-2 ** 31], [0]])
    freqs = torch.tensor([1.0, 0.7310585786300049, 1e-9], dtype=torch.float64, device=DEV)
    x = torch.randn(3, 2, 6, device=DEV)
    ref = R.rotary(wide(x), None, pos.cpu(), freqs.cpu(), (3,), False, 0.0)
    y, _ = A.gspn_head_rotary_fwd(x, pos, freqs)
    value, bound = ref["y"]
    # the angle itself, up to 2^31 radians in 64 bits: three roundings of 2^-53 of it
    check(y, (value, bound + 2.0 ** 31 * 3 * 2.0 ** -53 / R.U * R.size(wide(x), torch.zeros(3, 3), False)), "y")
    w = torch.ones(6, device=DEV)
    z = x.clone()
    z[1, 0, 2], z[2, 1, 0] = math.nan, math.inf
    out, _ = A.gspn_head_rotary_fwd(z, pos, freqs, q_weight=w)
    plain, _ = A.gspn_head_rotary_fwd(x, pos, freqs, q_weight=w)
    keep = torch.ones(3, 2, dtype=torch.bool)
    keep[1, 0] = keep[2, 1] = False
    assert torch.equal(out[keep], plain[keep]) and torch.isnan(out[1, 0]).any()


# -------------------------------------------------------------------------------------------------- attention

SHAPES = [  # lengths of queries, of keys (None: the same), rows before the first
    ([1], None, 0), ([31], None, 0), ([128], None, 0), ([129], None, 0), ([65, 0, 1, 200], None, 3),
    ([40, 7, 0, 130], [9, 30, 20, 131], 0), ([300], [64], 0), ([5, 3, 0], [0, 4, 0], 2), ([1] * 70, None, 0)]
HEADS = [(F32, 2, 1, 64, True), (F32, 1, 1, 1, False), (F32, 4, 2, 100, False), (BF16, 3, 3, 128, True),
         (BF16, 6, 2, 72, False), (BF16, 2, 1, 33, True), (BF16, 4, 4, 64, False), (F32, 2, 2, 80, True),
         (BF16, 2, 1, 80, False), (BF16, 2, 2, 79, True), (BF16, 1, 1, 90, False), (BF16, 2, 2, 112, False)]


@pytest.mark.parametrize("lengths,keys,first", SHAPES)
@pytest.mark.parametrize("dtype,heads,kv_heads,d,view", HEADS)
@pytest.mark.parametrize("causal", [True, False])
def test_attention(dtype, heads, kv_heads, d, view, causal, lengths, keys, first):
    g = gen(d * 100 + len(lengths))
    qs = R.spans(lengths, first)
    ks = qs if keys is None else R.spans(keys, first)
    behind = 3 if first else 0  # rows behind the sequences too
    rows, krows = first + sum(lengths) + behind, (first + sum(lengths if keys is None else keys) + behind)
    q, go = rnd(g, rows, heads, d, dtype=dtype), rnd(g, rows, heads, d, dtype=dtype)
    k, v = rnd(g, krows, kv_heads, d, dtype=dtype), rnd(g, krows, kv_heads, d, dtype=dtype)
    ref = R.attention(*map(wide, (q, k, v)), qs, ks, d ** -0.5, causal, dtype == BF16, wide(go))
    at, kat = inside(qs), inside(ks)
    outside = sorted(set(range(rows)) - set(at))
    koutside = sorted(set(range(krows)) - set(kat))
    for t, o in ((q, outside), (go, outside), (k, koutside), (v, koutside)):
        t[o] = math.nan  # what lies outside counts for nothing
    qd, kd, vd, gd = (strided(t) if view else dev(t) for t in (q, k, v, go))
    kw = dict(causal=causal, cu=cu_of(lengths, first), cu_k=None if keys is None else cu_of(keys, first))
    out = torch.full((rows, heads, d), 3.0, dtype=dtype, device=DEV)
    _, lse = A.gspn_attention_fwd(qd, kd, vd, lse=True, out=out, **kw)
    check(out, ref["out"], "out", at)
    check_lse(lse, ref["lse"], at)
    assert (out[outside] == 3.0).all()
    dq, dk, dv = A.gspn_attention_bwd(qd, kd, vd, out, lse, gd, **kw)
    check(dq, ref["dq"], "dq")
    check(dk, ref["dk"], "dk")
    check(dv, ref["dv"], "dv")
    assert (dq[outside] == 0).all() and (dk[koutside] == 0).all() and (dv[koutside] == 0).all()
    again = A.gspn_attention_bwd(qd, kd, vd, out, lse, gd, **kw)
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dv), again))


@pytest.mark.parametrize("dtype,heads,kv_heads,d", [(BF16, 2, 1, 128), (BF16, 1, 1, 72), (BF16, 3, 1, 64), (BF16, 1, 1, 90),
                                                    (F32, 1, 1, 96)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_long(dtype, heads, kv_heads, d, causal):
    """Many tiles, and keys enough that rows are not cut into parts."""
    g = gen(d)
    lengths = [1500, 64, 701]
    seqs = R.spans(lengths)
    rows = sum(lengths)
    q, go = rnd(g, rows, heads, d, dtype=dtype), rnd(g, rows, heads, d, dtype=dtype)
    k, v = rnd(g, rows, kv_heads, d, dtype=dtype), rnd(g, rows, kv_heads, d, dtype=dtype)
    ref = R.attention(*map(wide, (q, k, v)), seqs, seqs, d ** -0.5, causal, dtype == BF16, wide(go))
    cu = cu_of(lengths)
    out, lse = A.gspn_attention_fwd(dev(q), dev(k), dev(v), causal=causal, cu=cu, lse=True)
    check(out, ref["out"], "out")
    check_lse(lse, ref["lse"], list(range(rows)))
    for n, t in zip(("dq", "dk", "dv"), A.gspn_attention_bwd(dev(q), dev(k), dev(v), out, lse, dev(go), causal=causal, cu=cu)):
        check(t, ref[n], n)


@pytest.mark.parametrize("d", [72, 128])
def test_attention_many_workgroups(d):
    """More rows of keys than two workgroups a CU hold: sums of their own, no parts.  Every sequence is the same, and so
    must its results be."""
    g = gen(d)
    n, t, h = 24, 200, 8
    one = [rnd(g, t, h, d, dtype=BF16) for _ in range(4)]
    q, k, v, go = (x.to(DEV).repeat(n, 1, 1) for x in one)
    out, lse = A.gspn_attention_fwd(q, k, v, nseq=n, lse=True)
    res = (out, *A.gspn_attention_bwd(q, k, v, out, lse, go, nseq=n))
    seqs = [(0, t)]
    ref = R.attention(*map(wide, one[:3]), seqs, seqs, d ** -0.5, True, True, wide(one[3]))
    for name, x in zip(("out", "dq", "dk", "dv"), res):
        x = x.view(n, t, h, d)
        assert (x == x[:1]).all(), name
        check(x[0], ref[name], name)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 1e-30, 3.0])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attention_scales(dtype, scale):
    g = gen(4)
    q, k, v, go = (rnd(g, 150, 2, 24, dtype=dtype) for _ in range(4))
    seqs = [(0, 150)]
    ref = R.attention(*map(wide, (q, k, v)), seqs, seqs, scale, True, dtype == BF16, wide(go))
    out, lse = A.gspn_attention_fwd(dev(q), dev(k), dev(v), scale=scale, lse=True)
    check(out, ref["out"], "out")
    check_lse(lse, ref["lse"], list(range(150)))
    grads = A.gspn_attention_bwd(dev(q), dev(k), dev(v), out, lse, dev(go), scale=scale)
    for n, t in zip(("dq", "dk", "dv"), grads):
        check(t, ref[n], n)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attention_growing_scores(dtype):
    """Scores that grow along the keys, far past the point where the sums are scaled anew, and shrink."""
    n, d = 400, 16
    q = torch.ones(n, 1, d, dtype=dtype)
    ramp = torch.linspace(-200, 200, n)
    for values in (ramp, ramp.flip(0)):
        k = (values[:, None, None] / d).expand(n, 1, d).to(dtype).contiguous()
        v, go = rnd(gen(1), n, 1, d, dtype=dtype), rnd(gen(2), n, 1, d, dtype=dtype)
        seqs = [(0, n)]
        ref = R.attention(*map(wide, (q, k, v)), seqs, seqs, 1.0, True, dtype == BF16, wide(go))
        out, lse = A.gspn_attention_fwd(dev(q), dev(k), dev(v), scale=1.0, lse=True)
        check(out, ref["out"], "out")
        for m, t in zip(("dq", "dk", "dv"), A.gspn_attention_bwd(dev(q), dev(k), dev(v), out, lse, dev(go), scale=1.0)):
            check(t, ref[m], m)


def test_attention_batch_form_and_equal_lengths():
    g = gen(9)
    q, k, v = rnd(g, 3, 50, 4, 32, dtype=BF16), rnd(g, 3, 20, 2, 32, dtype=BF16), rnd(g, 3, 20, 2, 32, dtype=BF16)
    a = A.gspn_attention_fwd(dev(q), dev(k), dev(v), causal=False)
    flat = (dev(q).view(150, 4, 32), dev(k).view(60, 2, 32), dev(v).view(60, 2, 32))
    b = A.gspn_attention_fwd(*flat, causal=False, nseq=3)
    c = A.gspn_attention_fwd(*flat, causal=False, cu=cu_of([50] * 3), cu_k=cu_of([20] * 3))
    e = A.gspn_attention_fwd(*flat, causal=False, nseq=3, cu_k=cu_of([20] * 3))
    assert torch.equal(a.view(150, 4, 32), b) and torch.equal(b, c) and torch.equal(b, e)
    leaves = [t.to(DEV).requires_grad_() for t in (q, k, v)]
    A.attention(*leaves, causal=False).sum().backward()
    assert all(t.grad.shape == t.shape for t in leaves)


def test_attention_without_sequences_rows_or_keys():
    x = torch.randn(5, 2, 8, device=DEV)
    none = x[:0]
    assert A.gspn_attention_fwd(none, none, none).shape == (0, 2, 8)
    out, lse = A.gspn_attention_fwd(x, none, none, causal=False, lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    dq, dk, dv = A.gspn_attention_bwd(x, none, none, out, lse, x, causal=False)
    assert (dq == 0).all() and dk.shape == none.shape
    cu = ints([0])  # no sequence: nothing is written, and every gradient is zero
    keep = torch.full_like(x, 3.0)
    A.gspn_attention_fwd(x, x, x, cu=cu, out=keep)
    assert (keep == 3.0).all()
    lse = torch.zeros(2, 5, device=DEV)
    assert all((t == 0).all() for t in A.gspn_attention_bwd(x, x, x, keep, lse, x, cu=cu))
    # keys whose queries are all in other sequences
    q = torch.randn(4, 2, 8, device=DEV)
    kw = dict(causal=False, cu=cu_of([0, 4]), cu_k=cu_of([3, 2]))
    out, lse = A.gspn_attention_fwd(q, x, x, lse=True, **kw)
    dq, dk, dv = A.gspn_attention_bwd(q, x, x, out, lse, q, **kw)
    assert (dk[:3] == 0).all() and (dv[:3] == 0).all() and (dv[3:] != 0).any()


@pytest.mark.parametrize("dtype,heads,kv_heads,d", [(F32, 4, 2, 20), (BF16, 6, 2, 72), (BF16, 2, 2, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_cache(dtype, heads, kv_heads, d, causal):
    """Prompts behind the rows that their entry holds, fresh ones, padding, repeated and impossible slots, lengths that do
    not fit; what lies behind an entry's rows and in other entries counts for nothing and stays as it is."""
    g = gen(11)
    lengths = [5, 0, 33, 2, 140, 3, 4, 6, 7]
    slots = [4, 7, 0, -1, 2, 2, 99, 5, 6]
    held = [9, 4, 0, 7, 150, 0, 0, -1, 294]  # 7 rows behind 294 do not fit into 300
    fine = [0, 1, 2, 3, 4]
    cap = 300
    rows = sum(lengths)
    q, k, v = rnd(g, rows, heads, d, dtype=dtype), rnd(g, rows, kv_heads, d, dtype=dtype), rnd(g, rows, kv_heads, d,
                                                                                              dtype=dtype)
    pools = [torch.full((9, cap, kv_heads, d), math.nan, dtype=dtype) for _ in range(2)]
    for i in fine:
        if slots[i] >= 0:
            for p in pools:
                p[slots[i], :held[i]] = rnd(g, held[i], kv_heads, d, dtype=dtype)
    state = tuple(dev(p) for p in pools)
    heldd = ints(held)
    out = torch.full((rows, heads, d), 3.0, dtype=dtype, device=DEV)
    _, lse = A.gspn_attention_fwd(dev(q), dev(k), dev(v), causal=causal, cu=cu_of(lengths), state=state, slots=ints(slots),
                                  held=heldd, lse=True, out=out)
    assert torch.equal(heldd, ints(held))
    want = [p.clone() for p in pools]
    for i, (a, b) in enumerate(R.spans(lengths)):
        if i not in fine:
            assert torch.isnan(out[a:b]).all() and torch.isnan(lse[:, a:b]).all(), i
            continue
        old = [p[slots[i], :held[i]] if slots[i] >= 0 else p[0, :0] for p in pools]
        kk, vv = (torch.cat([o, t[a:b]]) for o, t in zip(old, (k, v)))
        if slots[i] >= 0:
            for p, t in zip(want, (k, v)):
                p[slots[i], held[i]:held[i] + b - a] = t[a:b]
        ref = R.attention(wide(q[a:b]), wide(kk), wide(vv), [(0, b - a)], [(0, len(kk))], d ** -0.5, causal, dtype == BF16)
        check(out[a:b], ref["out"], "out %d" % i)
        check_lse(lse[:, a:b], ref["lse"], list(range(b - a)))
    for p, w in zip(state, want):
        assert torch.equal(torch.nan_to_num(p.cpu().float(), 12345.0), torch.nan_to_num(w.float(), 12345.0))


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 32)])
@pytest.mark.parametrize("slots", [None, [1, -1, 0]])
def test_attention_cache_unaligned_rows(dtype, d, slots):
    """New rows at odd addresses beside whole chunks in the entries: those of padding are read where they are."""
    g = gen(77 + d)
    n, length, heads, kv_heads = 3, 150, 4, 2
    wide_rows = rnd(g, n * length, 2 * kv_heads * d + 3, dtype=dtype)
    rows = dev(wide_rows)
    at = lambda t, i: t[:, 1 + i * kv_heads * d:1 + (i + 1) * kv_heads * d].unflatten(-1, (kv_heads, d))
    q = rnd(g, n * length, heads, d, dtype=dtype)
    state = tuple(torch.full((n, length + 5, kv_heads, d), math.nan, dtype=dtype, device=DEV) for _ in range(2))
    out = A.gspn_attention_fwd(dev(q), at(rows, 0), at(rows, 1), nseq=n, state=state, slots=slots and ints(slots))
    spans = [(i * length, (i + 1) * length) for i in range(n)]
    ref = R.attention(wide(q), wide(at(wide_rows, 0)), wide(at(wide_rows, 1)), spans, spans, d ** -0.5, True, dtype == BF16)
    check(out, ref["out"], "out")
    for i, p in enumerate(state):
        for b, e in enumerate(range(n) if slots is None else slots):
            if e >= 0:
                assert torch.equal(p[e, :length], at(rows, i)[spans[b][0]:spans[b][1]])


@pytest.mark.parametrize("dtype,heads,kv_heads,d", [(BF16, 4, 2, 128), (BF16, 2, 2, 80), (F32, 3, 1, 32), (BF16, 2, 1, 30)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_cache_seams(dtype, heads, kv_heads, d, causal):
    """Entries that end before, at and behind a tile's end, and new rows that begin there."""
    g = gen(78 + d)
    held = [0, 1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200]
    lengths = [1, 64, 33, 1, 130, 1, 65, 2, 1, 64, 128, 57]
    n, cap, rows = len(held), 330, sum(lengths)
    q, k, v = (rnd(g, rows, h, d, dtype=dtype) for h in (heads, kv_heads, kv_heads))
    pools = [torch.full((n, cap, kv_heads, d), math.nan, dtype=dtype) for _ in range(2)]
    for i in range(n):
        for p in pools:
            p[i, :held[i]] = rnd(g, held[i], kv_heads, d, dtype=dtype)
    state = tuple(dev(p) for p in pools)
    out = A.gspn_attention_fwd(dev(q), dev(k), dev(v), causal=causal, cu=cu_of(lengths), state=state, held=ints(held))
    for i, (a, b) in enumerate(R.spans(lengths)):
        for p, t, s in zip(pools, (k, v), state):
            p[i, held[i]:held[i] + b - a] = t[a:b]
            assert torch.equal(torch.nan_to_num(s[i].cpu().float(), 12345.0), torch.nan_to_num(p[i].float(), 12345.0)), i
        kk, vv = (wide(p[i, :held[i] + b - a]) for p in pools)
        ref = R.attention(wide(q[a:b]), kk, vv, [(0, b - a)], [(0, len(kk))], d ** -0.5, causal, dtype == BF16)
        check(out[a:b], ref["out"], "out %d" % i)


@pytest.mark.parametrize("dtype,heads,kv_heads,d", [(F32, 4, 2, 20), (F32, 3, 1, 128), (BF16, 8, 2, 72), (BF16, 40, 1, 128),
                                                    (BF16, 2, 2, 33), (F32, 2, 2, 96)])
@pytest.mark.parametrize("cap", [1, 40, 2500])
def test_step(dtype, heads, kv_heads, d, cap):
    """Single tokens over entries of every fill, padding, repeated and impossible slots, entries that are full."""
    g = gen(cap + d)
    slots = [2, -1, 0, 5, 2, 99, 3, 1, 4]
    held = [0, 3, cap // 2, cap - 1, 0, 0, cap, -1, min(cap - 1, 33)]
    fine = [0, 2, 3, 8]
    n = len(slots)
    q, k, v = (rnd(g, n, h, d, dtype=dtype) for h in (heads, kv_heads, kv_heads))
    pools = [torch.full((7, cap, kv_heads, d), math.nan, dtype=dtype) for _ in range(2)]
    for i in fine:
        for p in pools:
            p[slots[i], :held[i]] = rnd(g, held[i], kv_heads, d, dtype=dtype)
    state = tuple(dev(p) for p in pools)
    out = torch.full((n, heads, d), 3.0, dtype=dtype, device=DEV)
    A.gspn_attention_step(strided(q), strided(k), strided(v), state, ints(held), slots=ints(slots), out=out)
    want = [p.clone() for p in pools]
    for i in range(n):
        if slots[i] == -1:
            assert (out[i] == 3.0).all()
        elif i not in fine:
            assert torch.isnan(out[i]).all(), i
        else:
            for p, t in zip(want, (k, v)):
                p[slots[i], held[i]] = t[i]
            kk, vv = (wide(p[slots[i], :held[i] + 1]) for p in want)
            ref = R.attention(wide(q[i:i + 1]), kk, vv, [(0, 1)], [(0, len(kk))], d ** -0.5, True, dtype == BF16)
            check(out[i:i + 1], ref["out"], "out %d" % i)
    for p, w in zip(state, want):
        assert torch.equal(torch.nan_to_num(p.cpu().float(), 12345.0), torch.nan_to_num(w.float(), 12345.0))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_steps_continue_a_prompt(dtype):
    """A layer as it serves and as it trains: heads normalised and rotated, a prompt into the cache, then tokens one at a
    time, against the whole sequence at once and its gradients."""
    g = gen(21)
    n, t, hq, hk, d = 3, 40, 6, 2, 64
    x = rnd(g, n, t, (hq + 2 * hk) * d, dtype=dtype).to(DEV)
    q, k, v = (s.unflatten(2, (-1, d)) for s in x.split([hq * d, hk * d, hk * d], 2))
    wq, wk = (1 + rnd(g, d, by=0.1).to(DEV) for _ in range(2))
    freqs = (10000.0 ** -(torch.arange(d // 2, dtype=torch.float64) / (d // 2))).to(DEV)
    pos = torch.arange(t, dtype=torch.int32, device=DEV).expand(n, t).contiguous()
    qr, kr = A.gspn_head_rotary_fwd(q, pos, freqs, k, wq, wk)
    whole, lse = A.gspn_attention_fwd(qr, kr, v, lse=True)
    state = tuple(torch.full((n, t, hk, d), math.nan, dtype=dtype, device=DEV) for _ in range(2))
    held = torch.zeros(n, dtype=torch.int32, device=DEV)
    cut = 25
    part = A.gspn_attention_fwd(qr[:, :cut].contiguous(), kr[:, :cut].contiguous(), v[:, :cut].contiguous(), state=state,
                                held=held)
    held += cut
    outs = [part]
    for i in range(cut, t):
        qi, ki = A.gspn_head_rotary_fwd(q[:, i], pos[:, i].contiguous(), freqs, k[:, i], wq, wk)
        assert torch.equal(ki, kr[:, i])
        outs.append(A.gspn_attention_step(qi, ki, v[:, i], state, held)[:, None])
        held += 1
    assert torch.equal(state[0], kr) and torch.equal(state[1], v)
    seqs = R.spans([t] * n)
    flat = [wide(z).reshape(n * t, -1, d) for z in (qr, kr, v)]
    ref = R.attention(*flat, seqs, seqs, d ** -0.5, True, dtype == BF16)
    for got in (whole, torch.cat(outs, 1)):
        check(got.reshape(n * t, hq, d), ref["out"], "out")


# ------------------------------------------------------------------------------------- autograd, graphs, streams

def layer(x, wq, wk, pos, freqs, hq, hk, d, cu):
    q, k, v = (s.unflatten(1, (-1, d)) for s in x.split([hq * d, hk * d, hk * d], 1))
    q, k = A.head_rotary(q, pos, freqs, k, wq, wk, sections=(10, 22), interleaved=True)
    return A.attention(q, k, v, cu=cu)


def test_layer_gradients_against_the_definition():
    g = gen(30)
    lengths, hq, hk, d = [50, 0, 77], 4, 2, 64
    rows = sum(lengths)
    x, go = rnd(g, rows, (hq + 2 * hk) * d), rnd(g, rows, hq, d)
    wq, wk = 1 + rnd(g, d, by=0.1), 1 + rnd(g, d, by=0.1)
    pos = torch.randint(0, 60, (rows, 2), generator=g, dtype=torch.int32)
    freqs = torch.rand(32, generator=g, dtype=torch.float64)
    leaves = [t.to(DEV).requires_grad_() for t in (x, wq, wk)]
    y = layer(*leaves, dev(pos), dev(freqs), hq, hk, d, cu_of(lengths))
    grads = torch.autograd.grad(y, leaves, dev(go))
    wl = [t.double().requires_grad_() for t in (x, wq, wk)]
    q, k, v = (s.unflatten(1, (-1, d)) for s in wl[0].split([hq * d, hk * d, hk * d], 1))
    t = R.angles(pos, freqs, (10, 22))
    q, k = (R.turn(z / torch.sqrt((z * z).mean(-1, keepdim=True) + 1e-6) * w, t, True) for z, w in ((q, wl[1]), (k, wl[2])))
    outs = []
    for a, b in R.spans(lengths):
        s = torch.einsum("ihd,jhd->hij", q[a:b], k[a:b].repeat_interleave(hq // hk, 1)) * d ** -0.5
        p = torch.softmax(s.masked_fill(~R.visible(b - a, b - a, True), -math.inf), -1)
        outs.append(torch.einsum("hij,jhd->ihd", p, v[a:b].repeat_interleave(hq // hk, 1)))
    ref = torch.cat(outs)
    want = torch.autograd.grad(ref, wl, go.double())
    # two operators one after the other, some 77 + 64 roundings each way: 2^10 of the largest value's own
    for got, w in zip((y, *grads), (ref.detach(), *want)):
        assert (wide(got) - w).abs().max() <= 2 ** 10 * R.U * w.abs().max()


def test_gradients_against_differences():
    """fp32 gradients of out's projection on a fixed tensor against central differences of the kernel's own forward, along
    directions half of which is the gradient's own."""
    g = gen(31)
    n, hq, hk, d = 90, 2, 1, 32
    ts = [rnd(g, n, h, d) for h in (hq, hk, hk)]
    go = rnd(g, n, hq, d)
    ref = R.attention(*map(wide, ts), [(0, n)], [(0, n)], d ** -0.5, True, False, wide(go))
    out, lse = A.gspn_attention_fwd(*map(dev, ts), lse=True)
    grads = A.gspn_attention_bwd(*map(dev, ts), out, lse, dev(go))
    for i, name in enumerate(("dq", "dk", "dv")):
        exact = ref[name][0]
        r = torch.randn(ts[i].shape, generator=g, dtype=torch.float64)
        u = exact / exact.norm() + r / r.norm()
        u = (u / u.norm()).float()
        step = 2.0 ** -4 / float(u.abs().max())

        def value(sign, f):
            at = list(ts)
            at[i] = ts[i] + sign * step * u
            return float((f(at) * go.double()).sum())

        def own(at):
            return wide(A.gspn_attention_fwd(*map(dev, at)))

        def true(at):
            return R.attention(*map(wide, at), [(0, n)], [(0, n)], d ** -0.5, True)["out"][0]

        fd = (value(1, own) - value(-1, own)) / (2 * step)
        slope = float((exact * u.double()).sum())
        truncation = abs((value(1, true) - value(-1, true)) / (2 * step) - slope)
        rounding = float((go.double().abs() * (ref["out"][1] + ref["out"][0].abs())).sum()) * 1.1 * R.U / step
        got = float((wide(grads[i]) * u.double()).sum())
        bound = truncation + rounding + 2 ** 12 * R.U * float(exact.norm())
        assert abs(got - fd) <= bound, (name, got, fd, bound)
        for wrong in (0.0, -got, 2 * got):
            assert abs(wrong - fd) > 4 * bound, (name, wrong, fd, bound)


def test_graphs_replay_with_new_inputs():
    g = gen(40)
    lengths, hq, hk, d, cap = [70, 3, 130], 4, 2, 72, 300
    rows = sum(lengths)
    q, k, v, go = (rnd(g, rows, h, d, dtype=BF16).to(DEV) for h in (hq, hk, hk, hq))
    w = torch.ones(d, device=DEV)
    pos, freqs = torch.arange(rows, dtype=torch.int32, device=DEV)[:, None], torch.rand(36, dtype=torch.float64, device=DEV)
    cu, held = cu_of(lengths), ints([5, 0, 40])
    state = tuple(rnd(g, 3, cap, hk, d, dtype=BF16).to(DEV) for _ in range(2))

    def work():
        qr, kr = A.gspn_head_rotary_fwd(q, pos, freqs, k, w, w)
        out, lse = A.gspn_attention_fwd(qr, kr, v, cu=cu, lse=True)
        dqr, dkr, dv = A.gspn_attention_bwd(qr, kr, v, out, lse, go, cu=cu)
        back = A.gspn_head_rotary_bwd(q, pos, freqs, dqr, k, dkr, w, w)
        served = A.gspn_attention_fwd(qr, kr, v, cu=cu, state=state, held=held)
        step = A.gspn_attention_step(qr[:3], kr[:3], v[:3], state, held + 130)
        return (out, dv, *back, served, step)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work()
    for i in range(4):
        q.copy_(rnd(gen(50 + i), rows, hq, d, dtype=BF16))
        v.copy_(rnd(gen(60 + i), rows, hk, d, dtype=BF16))
        held.copy_(ints([i, 7 * i, 0]))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        want = work()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_calls_on_two_streams_at_once():
    g = gen(41)
    sets = [[rnd(g, 600, 4, 64, dtype=BF16).to(DEV) for _ in range(3)] for _ in range(2)]
    pools = [tuple(rnd(g, 8, 3000, 4, 64, dtype=BF16).to(DEV) for _ in range(2)) for _ in range(2)]
    held = ints([2990 - 100 * i for i in range(8)])
    want = [(A.gspn_attention_fwd(*s), A.gspn_attention_step(*(t[:8] for t in s), p, held)) for s, p in zip(sets, pools)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for st, s, p in zip(streams, sets, pools):
            with torch.cuda.stream(st):
                got.append((A.gspn_attention_fwd(*s), A.gspn_attention_step(*(t[:8] for t in s), p, held)))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for w, h in zip(want, got) for a, b in zip(w, h))


def test_rows_and_entries_far_into_memory():
    """Offsets past 32 bits: rows two gibibytes apart, and entries behind four gibibytes of others."""
    d, hk = 64, 2
    ld = 1 << 21
    big = torch.zeros(1030, ld, dtype=BF16, device=DEV)  # 4.3 GB
    g = gen(42)
    q = rnd(g, 1030, hk, d, dtype=BF16)
    view = big[:, 64:64 + hk * d].unflatten(1, (hk, d))
    view.copy_(q)
    assert torch.equal(A.gspn_attention_fwd(view, view, view), A.gspn_attention_fwd(dev(q), dev(q), dev(q)))
    pos, freqs = torch.arange(1030, dtype=torch.int32, device=DEV), torch.ones(32, dtype=torch.float64, device=DEV)
    assert torch.equal(A.gspn_head_rotary_fwd(view, pos, freqs)[0], A.gspn_head_rotary_fwd(dev(q), pos, freqs)[0])
    del big, view
    cap = 1 << 19
    pools = tuple(torch.zeros(40, cap, hk, d, dtype=BF16, device=DEV) for _ in range(2))  # 5.4 GB each
    small = tuple(torch.zeros(1, 64, hk, d, dtype=BF16, device=DEV) for _ in range(2))
    x = dev(q)[:30]
    a = A.gspn_attention_fwd(x, x, x, state=pools, slots=ints([39]), held=ints([0]))
    b = A.gspn_attention_fwd(x, x, x, state=small, held=ints([0]))
    assert torch.equal(a, b) and torch.equal(pools[0][39, :30], x) and not pools[0][:39].any()
    y = dev(q)[30:31]
    a = A.gspn_attention_step(y, y, y, pools, ints([30]), slots=ints([39]))
    b = A.gspn_attention_step(y, y, y, small, ints([30]))
    # the runs differ with the capacity: two orders of the same sum, within the step's half and a few roundings
    ref = R.attention(wide(y), wide(small[0][0, :31]), wide(small[1][0, :31]), [(0, 1)], [(0, 31)], d ** -0.5, True, True)
    check(a, ref["out"], "out")
    check(b, ref["out"], "out")
    last = A.gspn_attention_step(y, y, y, (pools[1].view(1, -1, hk, d), pools[0].view(1, -1, hk, d)),
                                 ints([40 * cap - 1]))
    assert torch.isfinite(last).all() and torch.equal(pools[1][39, cap - 1], y[0])
