"""Gradients of the sequence operators against central differences of their own fp32 forward, along directions in which
the slope is large: half of a direction is the 64-bit gradient's own, so that the slope is about |gradient| / sqrt(2)
and a gradient that is zero, negated or doubled misses it by as much.

What a difference may be off by is counted.  Truncation is measured in 64 bits, at the same points: the difference with
the same step against one 64 times smaller, whose own truncation is 4096 times less.  Rounding is the forward's bound
for each value, twice, over twice the step.  The gradient itself may carry 2^12 roundings of its own size."""
import torch

import sequence_bounds as Q
import sequence_reference as R

OPS = ["conv", "scan", "joined", "normed"]
ROWS, C, N, EPS = 50, 40, 16, 1e-6


def case(op, g):
    """(fp32 tensors, f(S, *tensors) of the library, its 64-bit definition with each value's bound in units of U)."""
    rnd = lambda *s, by=1.0: torch.randn(s, generator=g) * by  # noqa: E731
    seqs = [(0, ROWS)]
    if op == "conv":
        def ref(x, w, b):
            rows = torch.cat([torch.zeros_like(x[:3]), x])
            terms = [rows[j:j + ROWS] * w[:, j] for j in range(4)]
            pre = sum(terms) + b
            y = R.silu(pre)
            return y, 1.1 * 6 * (sum(t.abs() for t in terms) + b.abs()) + y.abs() * Q.exp_count(pre)
        return [rnd(ROWS, C), rnd(C, 4), rnd(C)], lambda S, *a: S.causal_conv(*a), ref
    if op == "scan":
        def ref(x, dt, A, B, Cc, D, z, bias):
            a = (x, dt, A, B, Cc, D, z, bias)
            with torch.no_grad():
                bound = Q.scan_bounds(*a, True, seqs, None, 16, 0)["out"]
            return R.scan(*a, True, seqs)[0], bound
        ts = [rnd(ROWS, C), rnd(ROWS, C, by=0.5), -torch.exp(rnd(C, N, by=0.7)), rnd(ROWS, 1, N), rnd(ROWS, 1, N), rnd(C),
              rnd(ROWS, C), rnd(C) - 2]
        return ts, lambda S, *a: S.selective_scan(*a), ref

    def ref(h, gate, res, post, scale, pre=None):
        j, n, mag = R.join(h, gate, res, post, scale, pre, EPS, lambda v: v)
        bj = mag * (Q.norm_count(C) + Q.exp_count(gate) + 6)
        if op == "joined":
            return j, bj
        # the norm of the joined rows: its own roundings, and what the rows carry, in the row and in the root, whose
        # mean(|j| bj) is at most rms(j) times the largest bj
        most = bj.amax(1, True)
        return n, n.abs() * (Q.norm_count(C) + 4) + (n / j).abs() * most * (1 + (n / pre).abs())

    ts = [rnd(ROWS, C), rnd(ROWS, C), rnd(ROWS, C), rnd(C), rnd(C)] + ([rnd(C)] if op == "normed" else [])
    if op == "joined":
        return ts, lambda S, *a: S.block_join(*a, eps=EPS)[0], ref
    return ts, lambda S, *a: S.block_join(*a, eps=EPS)[1], ref


def compare(ts, gy, i, grad, forward, ref):
    """grad of tensor i against the difference of ``forward``; and that 0, -1 and 2 times it would be seen."""
    wide = [t.double() for t in ts]
    leaf = wide[i].clone().requires_grad_()
    exact, = torch.autograd.grad(ref(*wide[:i], leaf, *wide[i + 1:])[0], leaf, gy.double())
    g = torch.Generator().manual_seed(100 + i)
    v = torch.randn(ts[i].shape, generator=g).double()
    v = exact / exact.norm() + v / v.norm()
    v = (v / v.norm()).float()
    step = 2.0 ** -4 / float(v.abs().max())

    def slope(f, h, widen):
        at = [ts[i] + s * h * v for s in (1.0, -1.0)]  # the same fp32 points for both
        ys = [f(*[t.double() if widen else t for t in (*ts[:i], p, *ts[i + 1:])]) for p in at]
        apart = (at[0].double() - at[1].double())  # what the points are apart, rounded as they are
        h2 = float((apart * v.double()).sum() / (v.double() ** 2).sum())
        return sum(s * float((y.double() * gy.double()).sum()) for s, y in zip((1.0, -1.0), ys)) / h2

    fd = slope(forward, step, False)
    exact_fd = slope(lambda *a: ref(*a)[0], step, True)
    truncation = abs(exact_fd - float((exact * v.double()).sum()))
    rounding = float((gy.double().abs() * ref(*wide)[1]).sum()) * 1.1 * R.U / step
    got = float((grad.double() * v.double()).sum())
    bound = truncation + rounding + 2 ** 12 * R.U * float(exact.norm())
    assert abs(got - fd) <= bound, (i, got, fd, bound)
    for wrong in (0.0, -got, 2 * got):
        assert abs(wrong - fd) > 4 * bound, (i, wrong, fd, bound)
