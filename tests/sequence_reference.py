"""Plain 64-bit references of the sequence operators, and how far fp32
arithmetic may stray from them.

Every function takes float64 CPU tensors (the storage type's values widened)
and runs the operator's definition row by row.  The ``scale`` results are the
same sums with every term replaced by its magnitude: a sum computed in fp32
with k roundings on the way from its inputs is off by at most about k 2^-24
times that.  A result stored in a narrower type is off by half a step of that
type more (``torch.finfo(t).eps / 2`` of its value)."""
import torch

U = 2.0 ** -24  # half a step of fp32, relative


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def silu(v):
    return v * torch.sigmoid(v)


def dsilu(v):
    s = torch.sigmoid(v)
    return s * (1 + v * (1 - s))


def dsilu_scale(v):
    """silu' = s (1 + v (1 - s)) is a sum of two terms, of opposite signs for v < 0, that cancels at v = -1.278...: each
    rounding of the sum is relative to the terms, s (1 + |v| (1 - s)), and not to what is left of them."""
    s = torch.sigmoid(v)
    return s * (1 + v.abs() * (1 - s))


def spans(lengths, first=0):
    out, at = [], first
    for n in lengths:
        out.append((at, at + n))
        at += n
    return out


# ------------------------------------------------------------------------------------------------ causal conv

def conv(x, w, b, act, seqs, heads=None):
    """(y, pre-activation, its scale, the rows left behind): rows outside the sequences are NaN."""
    k = w.shape[1]
    y, pre, scale = (torch.full_like(x, float("nan")) for _ in range(3))
    tails = []
    for i, (lo, hi) in enumerate(seqs):
        head = torch.zeros(k - 1, x.shape[1], dtype=x.dtype) if heads is None else heads[i]
        rows = torch.cat([head, x[lo:hi]])
        tails.append(rows[hi - lo:])
        for t in range(lo, hi):
            win = rows[t - lo:t - lo + k]
            pre[t] = (win * w.t()).sum(0) + b
            scale[t] = (win.abs() * w.t().abs()).sum(0) + b.abs()
            y[t] = silu(pre[t]) if act else pre[t]
    return y, pre, scale, tails


def conv_backward(x, w, b, act, seqs, gy):
    """((dx, dw, db), the same sums' scales)."""
    k = w.shape[1]
    _, pre, scale, _ = conv(x, w, b, act, seqs)
    e = gy * (dsilu(pre) if act else 1.0)
    # silu' has a slope of at most 1/2: the pre-activation's error reaches e by that
    es = gy.abs() * ((dsilu_scale(pre) + 0.5 * scale) if act else 1.0)
    out = [torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(b)]
    mag = [torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(b)]
    for lo, hi in seqs:
        for t in range(lo, hi):
            out[2] += e[t]
            mag[2] += es[t]
            for j in range(k):
                s = t - (k - 1) + j  # the row under tap j
                if s >= lo:
                    out[0][s] += w[:, j] * e[t]
                    out[1][:, j] += e[t] * x[s]
                    mag[0][s] += w[:, j].abs() * es[t]
                    mag[1][:, j] += es[t] * x[s].abs()
    return out, mag


# --------------------------------------------------------------------------------------------- selective scan

def step_size(dt, bias, softplus):
    v = dt + bias
    return torch.nn.functional.softplus(v, threshold=700.0) if softplus else v


def per_channel(m, c):
    """B or C rows [rows, groups, n] -> [rows, channels, n]."""
    return m.repeat_interleave(c // m.shape[1], 1)


def scan(x, dt, A, B, C, D, z, bias, softplus, seqs, h0=None):
    """(out, states after every row, last states, scale of out, scale of the states)."""
    c, n = A.shape
    d = step_size(dt, bias, softplus)
    bb, cc = per_channel(B, c), per_channel(C, c)
    out, scale = (torch.full_like(x, float("nan")) for _ in range(2))
    hs = torch.full((x.shape[0], c, n), float("nan"), dtype=x.dtype)
    mags = hs.clone()
    last = []
    for i, (lo, hi) in enumerate(seqs):
        h = torch.zeros(c, n, dtype=x.dtype) if h0 is None else h0[i]
        m = h.abs()
        for t in range(lo, hi):
            a = torch.exp(d[t][:, None] * A)
            u = (d[t] * x[t])[:, None] * bb[t]
            h = a * h + u
            m = a * m + u.abs()
            hs[t], mags[t] = h, m
            y = (cc[t] * h).sum(1) + D * x[t]
            s = (cc[t].abs() * m).sum(1) + (D * x[t]).abs()
            if z is not None:
                y, s = y * silu(z[t]), s * silu(z[t]).abs()
            out[t], scale[t] = y, s
        last.append(h)
    return out, hs, last, scale, mags


def scan_backward(x, dt, A, B, C, D, z, bias, softplus, seqs, gy):
    """Gradients and their scales as dicts: dx ddt dz dB dC dA dD dbias."""
    c, n = A.shape
    g_ = B.shape[1]
    d = step_size(dt, bias, softplus)
    slope = torch.sigmoid(dt + bias) if softplus else torch.ones_like(dt)
    bb, cc = per_channel(B, c), per_channel(C, c)
    _, hs, _, _, mags = scan(x, dt, A, B, C, D, z, bias, softplus, seqs)

    def run(absolute):
        m = torch.abs if absolute else (lambda v: v)
        st = mags if absolute else hs
        gate = m(silu(z)) if z is not None else torch.ones_like(x)
        o = {k: torch.zeros_like(v) for k, v in (("dx", x), ("ddt", x), ("dB", B), ("dC", C), ("dA", A), ("dD", D),
                                                 ("dbias", D))}
        if z is not None:
            o["dz"] = torch.zeros_like(x)
        for lo, hi in seqs:
            carry = torch.zeros(c, n, dtype=x.dtype)
            for t in reversed(range(lo, hi)):
                gp = m(gy[t]) * gate[t]
                g = m(cc[t]) * gp[:, None] + carry
                a = torch.exp(d[t][:, None] * A)
                before = st[t - 1] if t > lo else torch.zeros(c, n, dtype=x.dtype)
                ah = a * before
                gb = (g * m(bb[t])).sum(1)
                dd = (g * ah * m(A)).sum(1) + m(x[t]) * gb
                o["dx"][t] = m(d[t]) * gb + m(D) * gp
                o["ddt"][t] = dd * slope[t]
                o["dA"] += g * ah * m(d[t])[:, None]
                o["dD"] += gp * m(x[t])
                o["dbias"] += o["ddt"][t]
                o["dB"][t] = (g * m(d[t] * x[t])[:, None]).reshape(g_, c // g_, n).sum(1)
                o["dC"][t] = (st[t] * gp[:, None]).reshape(g_, c // g_, n).sum(1)
                if z is not None:
                    y = (m(cc[t]) * st[t]).sum(1) + m(D) * m(x[t])
                    o["dz"][t] = m(gy[t]) * y * (dsilu_scale(z[t]) if absolute else dsilu(z[t]))
                carry = a * g
        return o

    return run(False), run(True)


def scan_roundings(x, dt, A, bias, softplus, seqs) -> float:
    """Roundings (in units of U, relative to the scales) on a state's way.

    The step size: e^-|v| carries 2|v| + 2 (its exponent's product, the
    exponential), the logarithm, sum and products some 6 more.  The decay
    e^(dA): |dA| times those of d, plus the products' 3, plus 2 of its own.  A
    row multiplies by one decay and adds one product (2 + 3): a state that has
    passed L rows has at most L of each, and the few of one row's output
    (n + 12) come on top."""
    v = (dt + bias).abs()
    v = v[torch.isfinite(v)]
    vmax = float(v.max()) if softplus and v.numel() else 0.0
    d = step_size(dt, bias, softplus)
    d = d[torch.isfinite(d)]
    da = float(d.max() * A.abs().max()) if d.numel() else 0.0
    rows = max([hi - lo for lo, hi in seqs] + [1])
    step = 2 * vmax + 8
    return rows * (7 + da * (step + 3)) + step + A.shape[1] + 12


# ------------------------------------------------------------------------------------------------- block join

def join(h, gate, residual, post, scale, pre, eps, store):
    """(joined, normed, scale of joined); ``store`` rounds the joined rows as they are stored."""
    rms = lambda v: torch.sqrt((v * v).mean(1, keepdim=True) + eps)  # noqa: E731
    q = h / rms(h) * post if post is not None else h
    if gate is not None:
        q = q * silu(gate)
    if scale is not None:
        q = q * scale
    mag = q.abs()
    if residual is not None:
        mag = mag + residual.abs()
        q = q + residual
    normed = None
    if pre is not None:
        o = store(q)
        normed = o / rms(o) * pre
    return q, normed, mag


def join_backward(h, gate, residual, post, scale, pre, eps, joined, gjoined, gnormed):
    """Gradients and scales as dicts, from the joined rows as stored."""
    mean = lambda v: v.mean(1, keepdim=True)  # noqa: E731

    def norm_back(v, w, g):  # d/dv of v / rms(v) * w, and the terms' magnitudes
        r = 1 / torch.sqrt(mean(v * v) + eps)
        gw = g * w
        return (r * (gw - v * r * r * mean(gw * v)),
                r * (gw.abs() + v.abs() * r * r * mean((gw * v).abs())), r)

    out, mag = {}, {}
    do = torch.zeros_like(h) if gjoined is None else gjoined.clone()
    dm = do.abs()
    if pre is not None:
        g, m, r = norm_back(joined, pre, gnormed)
        do, dm = do + g, dm + m
        out["dpre"], mag["dpre"] = (gnormed * joined * r).sum(0), (gnormed * joined * r).abs().sum(0)
    if residual is not None:
        out["dresidual"], mag["dresidual"] = do, dm
    r1 = 1 / torch.sqrt(mean(h * h) + eps)
    q = h * r1 * post if post is not None else h
    act = silu(gate) if gate is not None else torch.ones_like(h)
    if scale is not None:
        out["dscale"], mag["dscale"] = (do * q * act).sum(0), (dm * (q * act).abs()).sum(0)
        do, dm = do * scale, dm * scale.abs()
    if gate is not None:
        out["dgate"], mag["dgate"] = do * q * dsilu(gate), dm * q.abs() * dsilu_scale(gate)
    dq, qm = do * act, dm * act.abs()
    if post is not None:
        out["dpost"], mag["dpost"] = (dq * h * r1).sum(0), (qm * (h * r1).abs()).sum(0)
        out["dh"] = norm_back(h, post, dq)[0]
        gw = qm * post.abs()
        mag["dh"] = r1 * (gw + h.abs() * r1 * r1 * mean(gw * h.abs()))
    else:
        out["dh"], mag["dh"] = dq, qm
    return out, mag
