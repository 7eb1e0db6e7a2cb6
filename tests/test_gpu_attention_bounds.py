"""The attention operators on the GPU where their bounds are closer than attention_reference's, and where a call takes a
way of its own that test_gpu_attention.py does not: against the same 64-bit definitions, element by element."""
import math
import sys

import pytest
import torch

import attention_bounds as B
import attention_reference as R
from linear_spatial_propagation_gspn_amd import attention as A

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


def rnd(g, *shape, dtype=F32, by=1.0):
    return (torch.randn(shape, generator=g) * by).to(dtype)


def wide(t):
    return None if t is None else t.detach().cpu().double()


def dev(t):
    return None if t is None else t.to(DEV)


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def check(got, value, bound, what):
    """|got - value| <= half a step of got's type + the bound, element by element."""
    off = (wide(got) - value).abs()
    most = R.half_step(got.dtype) * value.abs() * (1 + 2.0 ** -7) + 1.01 * R.U * bound + 1e-37
    assert torch.isfinite(off).all(), what
    assert (off <= most).all(), "%s: worst %.3g of its bound" % (what, float((off / most).max()))


@pytest.mark.parametrize("heads,kv_heads,d,cap", [(8, 2, 128, 300), (4, 4, 72, 40), (40, 1, 64, 200), (6, 2, 33, 2500),
                                                  (8, 1, 96, 2500), (2, 1, 80, 700), (1, 1, 1, 9)])
def test_step_adds_no_error_of_bf16(heads, kv_heads, d, cap):
    """The numerators' rounding to bf16 does not reach a single token's result."""
    g = torch.Generator().manual_seed(cap + d)
    held = [cap - 1, cap // 2, 0, min(cap - 1, 33)]
    n = len(held)
    q, k, v = (rnd(g, n, h, d, dtype=BF16) for h in (heads, kv_heads, kv_heads))
    pools = [rnd(g, n, cap, kv_heads, d, dtype=BF16) for _ in range(2)]
    out = A.gspn_attention_step(dev(q), dev(k), dev(v), tuple(dev(p) for p in pools), ints(held))
    for i, m in enumerate(held):
        for h in range(heads):
            j = h // (heads // kv_heads)
            kk, vv = (torch.cat([wide(p[i, :m, j]), wide(t[i:i + 1, j])]) for p, t in zip(pools, (k, v)))
            check(out[i:i + 1, h], *B.step(wide(q[i:i + 1, h]), kk, vv, d ** -0.5), "out %d %d" % (i, h))


def test_rotation_of_a_unit_is_its_sine_and_cosine():
    """(1, 0) turned by t is (cos t, sin t), each within 1.35 U.  The angle is formed in 64 bits and rounded once, 2^-25 at
    most for an eighth of a turn: 0.44 U in a sine (slope up to 0.88 where the angle is above a half), 0.35 in a cosine.
    Sine: its last sum 0.5 U, the cubic's factor 0.19, cut series and coefficients 0.09; cosine: its last sum 0.5 U, the
    square's rounding 0.25, the factor before it 0.16, the rest 0.05."""
    g = torch.Generator().manual_seed(5)
    rows, pairs = 8192, 128
    pos = torch.randint(-1000, 1000, (rows,), generator=g, dtype=torch.int32)
    freqs = torch.rand(pairs, generator=g, dtype=torch.float64)
    q = torch.zeros(rows, 1, 2 * pairs)
    q[..., :pairs] = 1
    y, _ = A.gspn_head_rotary_fwd(dev(q), dev(pos), dev(freqs))
    y = wide(y)[:, 0]
    t = pos.double()[:, None] * freqs
    for name, got, want in (("cos", y[:, :pairs], torch.cos(t)), ("sin", y[:, pairs:], torch.sin(t))):
        assert float((got - want).abs().max()) <= 1.35 * R.U, name


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [0.0, 1e-42, -1e-40])
def test_scales_near_zero_weigh_alike(dtype, scale):
    """Scores of 1e36 and more times (next to) nothing: every key that a row sees has the same weight, but for
    exponents up to 3.4e38 1e-40 = 0.034."""
    g = torch.Generator().manual_seed(6)
    n, d = 70, 8
    q, k = (rnd(g, n, 1, d).to(dtype) * 2.0 ** 60 for _ in range(2))
    v, go = rnd(g, n, 1, d, dtype=dtype), rnd(g, n, 1, d, dtype=dtype)
    out, lse = A.gspn_attention_fwd(dev(q), dev(k), dev(v), scale=scale, lse=True)
    # the scale itself, rounded to a multiple of 2^-149, is off by 2^-150: times |score| log2 e, and the same in lse
    mag = wide(q[:, 0]).abs() @ wide(k[:, 0]).abs().t()
    assert float(mag.max()) < 3e38
    off = float(mag.max()) * 2.0 ** -149 * 2 / R.U
    ref = R.attend(wide(q[:, 0]), wide(k[:, 0]), wide(v[:, 0]), scale, True, dtype == BF16)
    p = R.attend(wide(q[:, 0]), wide(k[:, 0]), wide(v[:, 0].abs()), scale, True, dtype == BF16)["out"][0]
    check(out[:, 0], ref["out"][0], ref["out"][1] + off * p, "out")
    assert float((wide(lse[0]) - ref["lse"][0]).abs().max()) <= R.U * float(ref["lse"][1].max() + off + 4)
    step = A.gspn_attention_step(dev(q[-1:]), dev(k[-1:]), dev(v[-1:]), (dev(k[None]).contiguous(), dev(v[None]).contiguous()),
                                 ints([n - 1]), scale=scale)
    check(step[:, 0], ref["out"][0][-1:], (ref["out"][1] + off * p)[-1:], "step")
    grads = A.gspn_attention_bwd(dev(q), dev(k), dev(v), out, lse, dev(go), scale=scale)
    assert all(torch.isfinite(t).all() for t in grads)
    back = R.attend(wide(q[:, 0]), wide(k[:, 0]), wide(v[:, 0]), scale, True, dtype == BF16, wide(go[:, 0]))["dv"]
    pg = R.attend(wide(q[:, 0]), wide(k[:, 0]), wide(v[:, 0]), scale, True, dtype == BF16, wide(go[:, 0].abs()))["dv"][0]
    check(grads[2][:, 0], back[0], back[1] + 2 * off * pg, "dv")


def common(g, rows, heads, d, mean):
    """Rows about a common vector: <gout, v_j> - D is then far smaller than either."""
    sign = (torch.randint(0, 2, (heads, d), generator=g) * 2 - 1).float()
    return (mean * sign + torch.randn(rows, heads, d, generator=g)).to(BF16)


@pytest.mark.parametrize("nq,nk,causal", [(40, 40, True), (64, 64, True), (33, 50, False), (7, 64, False),
                                          (30, 70, True), (100, 90, True), (130, 141, True), (1, 33, True)])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_within_one_tile_take_their_sums_from_the_weights(nq, nk, causal, d):
    """D of a row that sees 64 keys or less does not carry the rounding of its bf16 out, whatever its neighbours see."""
    g = torch.Generator().manual_seed(nq * 7 + nk)
    heads, kv_heads, scale = 4, 2, d ** -0.5
    q, go = rnd(g, nq, heads, d, dtype=BF16), rnd(g, nq, heads, d, dtype=BF16)
    k, v = common(g, nk, kv_heads, d, 4.0), common(g, nk, kv_heads, d, 32.0)
    out, lse = A.gspn_attention_fwd(dev(q), dev(k), dev(v), causal=causal, scale=scale, cu=ints([0, nq]), cu_k=ints([0, nk]),
                                    lse=True)
    dq, dk, dv = A.gspn_attention_bwd(dev(q), dev(k), dev(v), out, lse, dev(go), causal=causal, scale=scale,
                                      cu=ints([0, nq]), cu_k=ints([0, nk]))
    near = R.visible(nq, nk, causal).sum(1) <= B.TILE
    want = {"dk": [0.0, 0.0], "dv": [0.0, 0.0]}
    for h in range(heads):
        one = B.gradients(*(wide(t) for t in (q[:, h], k[:, h // 2], v[:, h // 2])), scale, causal, wide(go[:, h]))
        check(dq[:, h][near], one["dq"][0][near], one["dq"][1][near], "dq %d" % h)
        for n in want:
            want[n] = [a + b for a, b in zip(want[n], one[n])]
            if h % 2:
                check({"dk": dk, "dv": dv}[n][:, h // 2], want[n][0], want[n][1] + 2 * want[n][0].abs(), n)
                want[n] = [0.0, 0.0]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,heads,kv_heads,d,sections", [(1, 2, 1, 64, (32,)), (70, 5, 3, 72, (18, 18)), (33, 2, 2, 27, (4,)),
                                                            (9, 1, 9, 128, (20, 12)), (600, 6, 2, 48, (24,))])
@pytest.mark.parametrize("which", ["q", "k"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_of_queries_or_keys_alone(dtype, rows, heads, kv_heads, d, sections, which, interleaved):
    g = torch.Generator().manual_seed(rows + d)
    pairs = sum(sections)
    freqs = 10000.0 ** -torch.rand(pairs, generator=g, dtype=torch.float64)
    pos = torch.randint(-3000, 100000, (rows, len(sections)), generator=g, dtype=torch.int32)
    x = {n: rnd(g, rows, h, d, dtype=dtype) for n, h in (("q", heads), ("k", kv_heads))}
    go = {n: rnd(g, rows, h, d, dtype=dtype) for n, h in (("q", heads), ("k", kv_heads))}
    w = 1 + rnd(g, d, by=0.2)
    kw = {which + "_weight": dev(w), "sections": sections, "interleaved": interleaved}
    y = A.gspn_head_rotary_fwd(dev(x["q"]), dev(pos), dev(freqs), dev(x["k"]), **kw)
    dq, dk, dqw, dkw = A.gspn_head_rotary_bwd(dev(x["q"]), dev(pos), dev(freqs), dev(go["q"]), dev(x["k"]), dev(go["k"]), **kw)
    leaves = {n: x[n].to(DEV).requires_grad_() for n in x}
    lw = w.to(DEV).requires_grad_()
    z = A.head_rotary(leaves["q"], dev(pos), dev(freqs), leaves["k"], **dict(kw, **{which + "_weight": lw}))
    auto = torch.autograd.grad(z, [leaves["q"], leaves["k"], lw], [dev(go["q"]), dev(go["k"])])
    got = {"q": (y[0], dq, dqw), "k": (y[1], dk, dkw)}
    for n in "qk":
        ref = R.rotary(wide(x[n]), wide(w) if n == which else None, pos, freqs, sections, interleaved, 1e-6, wide(go[n]))
        for part, t in zip(("y", "dx", "dw"), got[n]):
            if part in ref:
                check(t, *ref[part], n + part)
            else:
                assert t is None
    assert torch.equal(auto[0], dq) and torch.equal(auto[1], dk) and torch.equal(auto[2], dqw if which == "q" else dkw)
    assert torch.equal(z[0], y[0]) and torch.equal(z[1], y[1])
