"""How far the scan's and the join's fp32 arithmetic may be from their 64-bit references, element by element.

Every result carries its own bound, in units of U = 2^-24 (half a step of fp32), propagated along the formulas: a
product adds its factors' relative errors and one rounding, a sum of k terms the terms' errors and at most as many
roundings of the sum of their magnitudes as its longest path has additions.  A state's error decays with the state, so
a bound is not the worst channel's times the number of rows."""
import torch

import sequence_reference as R

U = R.U


def exp_count(v):
    """Relative error of e^v: the argument's own rounding and its product with log2 e (1 each, and 0.22 for the
    constant), times the argument; the exponential's last place (2), a reciprocal's (2), and the sum and products
    around them (6)."""
    return 2.25 * v.abs() + 10


def scan_bounds(x, dt, A, B, C, D, z, bias, softplus, seqs, gy, chunk, depth, h0=None):
    """{name: bound} of scan and scan_backward for float64 tensors: out, states (after every row), dx, ddt, dz, dB, dC,
    dA, dD, dbias.  chunk: rows of a chunk of the passes (0: uncut), whose sum of step sizes has as many roundings;
    depth: additions on the longest way of a sum over rows."""
    c, n = A.shape
    groups, rows = B.shape[1], x.shape[0]
    per = c // groups
    v = dt + bias
    d = R.step_size(dt, bias, softplus).abs()
    ed = exp_count(v) if softplus else torch.ones_like(v)
    slope = torch.sigmoid(v) if softplus else torch.ones_like(v)
    es = exp_count(v)
    bb, cc = R.per_channel(B, c).abs(), R.per_channel(C, c).abs()
    gate = R.silu(z).abs() if z is not None else torch.ones_like(x)
    eg = exp_count(z) if z is not None else torch.zeros_like(x)
    da = d[..., None] * A.abs()
    a = torch.exp(R.step_size(dt, bias, softplus)[..., None] * A)
    # a decay: its exponent's error (the step's, two products and a constant; for a chunk's whole decay the sum's), the
    # exponential's last place and the product with it; the few roundings of a join spread over its 16 rows at least
    ea = da * (ed[..., None] + 4 + chunk) + 4
    u = (d * x.abs())[..., None] * bb
    eu = ed[..., None] + 2

    m, e = torch.zeros(rows, c, n, dtype=x.dtype), torch.zeros(rows, c, n, dtype=x.dtype)  # of states: size, error
    m1, e1 = m.clone(), e.clone()  # of the states before each row
    for i, (lo, hi) in enumerate(seqs):
        mh = torch.zeros(c, n, dtype=x.dtype) if h0 is None else h0[i].abs()
        eh = torch.zeros(c, n, dtype=x.dtype)
        for t in range(lo, hi):
            m1[t], e1[t] = mh, eh
            eh = a[t] * eh + a[t] * mh * ea[t] + u[t] * eu[t]
            mh = a[t] * mh + u[t]
            eh = eh + mh
            m[t], e[t] = mh, eh
    out = {"states": e}
    my = (cc * m).sum(-1) + (D * x).abs()
    ey = (cc * e).sum(-1) + (n + 2) * my
    out["out"] = gate * (ey + my * (eg + 1))
    if gy is None:
        return out

    gp = gy.abs() * gate
    egp = eg + 1
    g, ge = torch.zeros_like(m), torch.zeros_like(m)  # of dL/dh
    for lo, hi in seqs:
        mc, ec = torch.zeros(c, n, dtype=x.dtype), torch.zeros(c, n, dtype=x.dtype)
        for t in reversed(range(lo, hi)):
            own = cc[t] * gp[t][:, None]
            g[t] = mc + own
            ge[t] = ec + own * (egp[t][:, None] + 1) + g[t]
            mc = a[t] * g[t]
            ec = a[t] * ge[t] + mc * (ea[t] + 1)
    gb, egb = (g * bb).sum(-1), (ge * bb).sum(-1)
    egb = egb + (n + 1) * gb
    out["dx"] = d * egb + d * gb * (ed + 1) + D.abs() * gp * (egp + 1) + d * gb + D.abs() * gp
    gq = a * g * m1
    egq = a * ge * m1 + a * g * e1 + gq * (ea + 2)
    dd = (gq * A.abs()).sum(-1) + x.abs() * gb
    edd = (egq * A.abs()).sum(-1) + (gq * A.abs()).sum(-1) * (n + 5) + x.abs() * egb + dd
    out["ddt"] = slope * (edd + dd * (es + 1))
    out["dA"] = (d[..., None] * (egq + gq * (ed[..., None] + 1 + depth))).sum(0)
    out["dD"] = (gp * x.abs() * (egp + 1 + depth)).sum(0)
    out["dbias"] = (out["ddt"] + depth * slope * dd).sum(0)
    # over a wave's channels (6 steps), a block's four waves (2), and the blocks of 64 (256 with one state) one by one
    over = 8 + (per + 63) // 64
    fold = lambda t: t.reshape(rows, groups, per, n).sum(2)  # noqa: E731
    du = (d * x.abs())[..., None]
    out["dB"] = fold(ge * du + g * du * (ed[..., None] + 2 + over))
    out["dC"] = fold(gp[..., None] * (e + m * (egp[..., None] + 1 + over)))
    if z is not None:
        ds = gy.abs() * R.dsilu_scale(z)
        out["dz"] = ds * (ey + my * (2 * eg + 6))
    return out


def norm_count(c):
    """Relative error of 1 / rms over c columns: at most 16 of them on a lane, 6 steps over a wave, 16 waves one by
    one (squares have one sign), halved by the root; the mean's product, the root's last place and the sum with eps."""
    return (min(c, 16) + 6 + 16) / 2 + 4


def sum_count(c):
    """Additions on the longest way of a row's sum."""
    return min(c, 16) + 6 + 16
