"""Definitions of the attention operators in 64 bits, with each result's bound in units of U = 2^-24 (half a step of
fp32) beside it: plain loops over sequences and heads, dense matrices within.

A bound follows the formulas.  A score has one rounding a product and a sum (d + 2) of the magnitudes it is made of, and
its exponent the roundings of its product with log2 e, of the maximum's and of their sum (4, times the larger of the
score and the maximum); the exponential ends within 2 units.  A sum over n keys has at most n additions on its way and
one more for each time it is scaled anew, which is counted as 4 with the factor's own roundings.  An exponential below
2^-126 is 0, and so may be a factor of a product: e^-88 / e^0 is, and a key that 300 rows see so has a dv whose sum of
300 such terms lacks 300 2^-126 |gout| at most.  bf16 kernels round the
numerators, and the scores' gradients, to bf16: 2^-8 of each."""
import torch

U = 2.0 ** -24
BF16 = 2.0 ** -8  # half a step of bf16
TINY = 2.0 ** -126 / U  # what an underflow loses


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def spans(lengths, first=0):
    out, at = [], first
    for n in lengths:
        out.append((at, at + n))
        at += n
    return out


def visible(nq, nk, causal):
    """[nq, nk] truth values: which keys a row sees."""
    if not causal:
        return torch.ones(nq, nk, dtype=torch.bool)
    return torch.arange(nk)[None, :] <= torch.arange(nq)[:, None] + (nk - nq)


def attend(q, k, v, scale, causal, narrow=False, gout=None):
    """One head of one sequence, float64 [n, d]: {name: (value, bound)} of out, lse and, with gout, dq, dk, dv.
    narrow: the kernels for bf16."""
    nq, d = q.shape
    nk = k.shape[0]
    see = visible(nq, nk, causal)
    some = see.any(1)
    s = scale * (q @ k.t())
    mag = abs(scale) * (q.abs() @ k.abs().t())
    hid = torch.where(see, s, -torch.inf)
    m = torch.where(some, hid.amax(1) if nk else torch.zeros(nq, dtype=q.dtype), 0.0)
    e = torch.where(see, torch.exp(s - m[:, None]), 0.0)
    total = e.sum(1)
    p = torch.where(some[:, None], e / total.clamp(min=1e-300)[:, None], 0.0)
    out = p @ v
    # relative errors of the numerators, and of their sum
    er = mag * (d + 2) + 4 * torch.maximum(s.abs(), m.abs()[:, None]) + 6
    es = (p * er).sum(1) + nk + 8
    r = BF16 / U if narrow else 0.0
    bound = (p * (er + es[:, None] + nk + 8 + r) + TINY * see) @ v.abs()
    lse = torch.where(some, m + torch.log(total.clamp(min=1e-300)), -torch.inf)
    res = {"out": (out, bound), "lse": (lse, es + 4 * (m.abs() + 1) + 4 * torch.where(some, lse, 0.0).abs())}
    if gout is None:
        return res
    g = gout
    dp = g @ v.t()
    delta = (g * out).sum(1)
    ds = p * (dp - delta[:, None])
    # p from the scores and lse; dp a sum of d; delta from the stored out, whose rounding counts for bf16
    ep = er + res["lse"][1][:, None] + 4
    edp = (g.abs() @ v.abs().t()) * (d + 1)
    edelta = (g.abs() * (bound + out.abs() * (r + d + 2))).sum(1)
    eds = ds.abs() * (ep + 2 + r) + p * (edp + edelta[:, None]) + TINY * see * (dp.abs() + delta.abs()[:, None] + 1)
    ads = ds.abs()
    c = abs(scale)
    res["dq"] = (scale * ds @ k, c * ((eds + ads * (nk + 4)) @ k.abs()))
    res["dk"] = (scale * ds.t() @ q, c * ((eds + ads * (nq + 4)).t() @ q.abs()))
    res["dv"] = (p.t() @ g, (p * (ep + nq + 4 + r) + TINY * see).t() @ g.abs())
    return res


def attention(q, k, v, qseqs, kseqs, scale, causal, narrow=False, gout=None):
    """Packed rows [rows, heads, d] in float64: {name: (value, bound)}, zeros outside the sequences (lse: NaN)."""
    hq, hk = q.shape[1], k.shape[1]
    shapes = {"out": q.shape, "dq": q.shape, "dk": k.shape, "dv": v.shape}
    names = ["out"] + (["dq", "dk", "dv"] if gout is not None else [])
    res = {n: (torch.zeros(shapes[n], dtype=q.dtype), torch.zeros(shapes[n], dtype=q.dtype)) for n in names}
    res["lse"] = (torch.full((hq, q.shape[0]), torch.nan, dtype=q.dtype), torch.zeros(hq, q.shape[0], dtype=q.dtype))
    for (a, b), (c, e) in zip(qseqs, kseqs):
        for h in range(hq):
            j = h // (hq // hk)
            one = attend(q[a:b, h], k[c:e, j], v[c:e, j], scale, causal, narrow, None if gout is None else gout[a:b, h])
            for i in range(2):
                res["lse"][i][h, a:b] = one["lse"][i]
                for n in names:
                    rows, head = (slice(a, b), h) if n in ("out", "dq") else (slice(c, e), j)
                    res[n][i][rows, head] += one[n][i]
    for n in ("dk", "dv"):  # the heads of a group are added up in turn
        if n in res:
            res[n] = (res[n][0], res[n][1] + (hq // hk) * res[n][0].abs())
    return res


def turn(x, angle, interleaved, back=False):
    """Pairs of x's last dimension turned by angle [rows, pairs]."""
    pairs = angle.shape[1]
    cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    if back:
        sin = -sin
    y = x.clone()
    a, b = (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)) if interleaved else (slice(0, pairs), slice(pairs, 2 * pairs))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., a] * sin + x[..., b] * cos
    return y


def size(x, angle, interleaved):
    """|a| + |b| at both elements of each pair, |x| elsewhere: what a turn's result is made of."""
    pairs = angle.shape[1]
    y = x.abs()
    a, b = (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)) if interleaved else (slice(0, pairs), slice(pairs, 2 * pairs))
    both = y[..., a] + y[..., b]
    y[..., a] = both
    y[..., b] = both
    return y


def angles(positions, freqs, sections):
    along = torch.cat([positions[:, i:i + 1].expand(-1, n) for i, n in enumerate(sections)], 1)
    return along.double() * freqs


def rotary(x, weight, positions, freqs, sections, interleaved, eps, g=None):
    """One of q and k, float64 [rows, heads, d]: {name: (value, bound)} of y and, with g, dx and dw.  A norm has d
    squares and sums halved by the root and 6 around them; a sine or cosine is within 6 units, a turn adds 3."""
    t = angles(positions, freqs, sections)
    d = x.shape[-1]
    en = d / 2 + 6 if weight is not None else 0
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) if weight is not None else torch.ones_like(x[..., :1])
    w = weight if weight is not None else torch.ones(d, dtype=x.dtype)
    n = x * r
    res = {"y": (turn(n * w, t, interleaved), size(n * w, t, interleaved) * (en + 2 + 9))}
    if g is None:
        return res
    gt, gm = turn(g, t, interleaved, back=True), size(g, t, interleaved)
    if weight is None:
        res["dx"] = (gt, gm * 9)
        return res
    mean = (gt * w * n).mean(-1, keepdim=True)
    big = (gm * (w * n).abs()).mean(-1, keepdim=True)
    res["dx"] = (r * (gt * w - n * mean), r * (gm * w.abs() * (12 + en) + n.abs() * big * (12 + d + 3 * en)))
    terms = gm * n.abs()
    res["dw"] = ((gt * n).sum((0, 1)), (terms * (10 + en + x.shape[0] * x.shape[1])).sum((0, 1)))
    return res
