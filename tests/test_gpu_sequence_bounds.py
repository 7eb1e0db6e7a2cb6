"""The sequence operators on the GPU, held to bounds that follow each element's own errors (sequence_bounds.py): the
plans that larger calls take, sums over many blocks of channels, norms whose energy sits in a row's last columns, and
gradients against differences along directions in which they are large."""
import pytest
import torch

import sequence_bounds as Q
import sequence_cases as P
import sequence_differences as D
import sequence_reference as R
from linear_spatial_propagation_gspn_amd import sequence as S
from test_gpu_sequence import (BF16, DEV, F32, _gpu, _say, check, cu_of, dev, gen, leaves, on_gpu, ref_args, rnd,  # noqa: F401
                               run_bwd, run_fwd, scan_case, strided, wide)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", P.PLANS, ids=P.name)
def test_scan_plans(case):
    dtype, c, groups, n, gate, lengths, packed, fwd, bwd = case
    dtype = F32 if dtype == "f32" else BF16
    g = gen(c + n + len(lengths))
    seqs, rows = R.spans(lengths), sum(lengths)
    k = scan_case(g, rows, c, groups, n, dtype, gate)
    gy = rnd(g, rows, c, dtype=dtype)
    kw = {"cu": cu_of(lengths)} if packed else {"nseq": len(lengths)}
    args = ref_args(k)
    chunk = max(fwd if isinstance(fwd, int) else 0, bwd)
    # a chunk's rows, then its sums over 16 runs of chunks and those 16, and over the lanes that share a channel
    depth = (bwd or max(lengths)) + (rows // (bwd or max(lengths)) + len(lengths)) // 16 + 24
    bound = Q.scan_bounds(*args, True, seqs, wide(gy), chunk, depth)
    ref, _ = R.scan_backward(*args, True, seqs, wide(gy))
    ry = R.scan(*args, True, seqs)[0]
    o = on_gpu(k)
    out, kept = run_fwd(o, checkpoints=True, **kw)
    got = run_bwd(o, dev(gy), checkpoints=kept, **kw)
    again = run_bwd(o, dev(gy), **kw)
    check(out, ry, bound["out"], 1, "out")
    for name, r in ref.items():
        check(got[name], r, bound[name], 1, name)
        assert torch.equal(got[name], again[name]), name

    # from a pool, every other sequence continuing its entry
    slots = torch.randperm(len(lengths) + 2, generator=g)[:len(lengths)]
    resume = torch.arange(len(lengths)) % 2 == 0
    pool = rnd(g, len(lengths) + 2, c, n)
    h0 = list(wide(pool)[slots] * resume[:, None, None])
    ry, hs, last, _, _ = R.scan(*args, True, seqs, h0)
    bound = Q.scan_bounds(*args, True, seqs, None, chunk, depth, h0)
    state = dev(pool.clone())
    out = run_fwd(o, state=state, slots=dev(slots.int()), resume=dev(resume), **kw)
    check(out, ry, bound["out"], 1, "out from a pool")
    for i, (lo, hi) in enumerate(seqs):
        zero = torch.zeros(c, n, dtype=torch.float64)
        check(state[slots[i]], last[i], bound["states"][hi - 1] if hi > lo else zero, 1, "entry of sequence %d" % i)
    others = [e for e in range(len(lengths) + 2) if e not in set(slots.tolist())]
    assert torch.equal(state[others].cpu(), pool[others])


@pytest.mark.parametrize("tail", [1, 3, 8])
@pytest.mark.parametrize("dtype,rt", [(F32, F32), (BF16, F32)])
@pytest.mark.parametrize("c", [1, 7, 9, 12, 64, 67, 511, 512, 515, 1001, 1024, 2305, 4093, 4096, 4099, 8190, 8192, 8199, 12001,
                               16384])
def test_join_with_its_energy_in_the_last_columns(c, dtype, rt, tail):
    """Rows whose last ``tail`` columns hold nearly all of the norms and sums: one of them dropped or taken twice moves
    every result by far more than the roundings that the sums can have."""
    g = gen(c + tail)
    rows, tail, eps = 3, min(tail, c), 1e-6
    shape = torch.full((c,), 2.0 ** -6)
    shape[c - tail:] = 2.0 ** 6
    h, gate = (rnd(g, rows, c) * shape).to(dtype), rnd(g, rows, c, dtype=dtype)
    res = rnd(g, rows, c) * shape
    post, scale, pre = (rnd(g, c, by=0.1) + 1 for _ in range(3))
    gj, gn = rnd(g, rows, c) * shape, (rnd(g, rows, c) * shape).to(dtype)
    k = dict(gate=gate, residual=res, post=post, scale=scale, pre=pre)
    kd = {n: dev(t) for n, t in k.items()}
    joined, normed = S.gspn_block_join_fwd(dev(h), **kd, eps=eps)
    stored = wide(joined)
    kw = {n: wide(t) for n, t in k.items()}
    rj, rn, mj = R.join(wide(h), **kw, eps=eps, store=lambda v: stored)
    norm, total = Q.norm_count(c), Q.sum_count(c)
    act = Q.exp_count(wide(gate))
    check(joined, rj, mj, norm + act + 6, "joined")
    check(normed, rn, rn.abs(), norm + 4, "normed")
    got = dict(zip(("dh", "dgate", "dresidual", "dpost", "dscale", "dpre"),
                   S.gspn_block_join_bwd(dev(h), dev(gj), dev(gn), joined, **kd, eps=eps)))
    ref, mag = R.join_backward(wide(h), **kw, eps=eps, joined=stored, gjoined=wide(gj), gnormed=wide(gn))
    # dL/djoined: a root cubed, a row's sum and 8 products; behind it the gate's two factors, and once more a norm
    do = 3 * norm + total + 8
    back = do + 2 * float(act.max()) + 16
    check(got["dresidual"], ref["dresidual"], mag["dresidual"], do, "dresidual")
    check(got["dpre"], ref["dpre"], mag["dpre"], norm + 4 + rows, "dpre")
    for name in ("dgate", "dscale", "dpost"):
        check(got[name], ref[name], mag[name], back + norm + rows, name)
    check(got["dh"], ref["dh"], mag["dh"], back + do, "dh")


@pytest.mark.parametrize("op", D.OPS)
def test_gradients_along_their_own_direction(op):
    g = gen(61)
    ts, f, ref = D.case(op, g)
    gy = rnd(g, *ts[0].shape)
    td = [dev(t) for t in ts]
    ls = leaves(*td)
    grads = torch.autograd.grad(f(S, *ls), ls, dev(gy))
    for i in range(len(ts)):
        D.compare(ts, gy, i, grads[i].cpu(), lambda *a: f(S, *map(dev, a)).cpu(), ref)
