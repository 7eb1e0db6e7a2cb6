"""Bounds of attention_reference for the places where a kernel for bf16 rounds less than its other forms do, in the same
units of U = 2^-24.

Single tokens: a numerator goes into the product with the values as two bf16 factors, itself rounded (2^-8 of it lost at
most) and what that lost rounded (2^-8 of that): 2^-16 of it in all.

Gradients of rows that see one tile of keys (64) or less: D = <gout, out> comes from the weights and <gout, v_j> in
fp32, not from the stored out.  A term of that sum of n is off by p's error times |<gout, v_j>|, and p times the
latter's; the sum adds n + 2 roundings."""
import torch

from attention_reference import BF16, TINY, U, attend, visible

TWO = 2.0 ** -16 / U
TILE = 64


def step(q, k, v, scale):
    """One head's single row over its keys, bf16 inputs in float64: (value, bound)."""
    value, bound = attend(q, k, v, scale, True)["out"]
    p = torch.softmax(scale * (q @ k.t()), -1)
    return value, bound + TWO * (p @ v.abs())


def gradients(q, k, v, scale, causal, gout):
    """One head of one sequence whose rows all see TILE keys or less, bf16 inputs in float64: {name: (value, bound)} of
    dq, dk, dv.  (A row that sees more may be there; its own bounds are the reference's.)"""
    ref = attend(q, k, v, scale, causal, True, gout)
    nq, d = q.shape
    nk = k.shape[0]
    see = visible(nq, nk, causal)
    count = see.sum(1)
    some = count > 0
    s = scale * (q @ k.t())
    mag = abs(scale) * (q.abs() @ k.abs().t())
    m = torch.where(see, s, -torch.inf).amax(1)
    m = torch.where(some, m, 0.0)
    e = torch.where(see, torch.exp(s - m[:, None]), 0.0)
    p = torch.where(some[:, None], e / e.sum(1, keepdim=True).clamp(min=1e-300), 0.0)
    er = mag * (d + 2) + 4 * torch.maximum(s.abs(), m.abs()[:, None]) + 6
    ep = er + ref["lse"][1][:, None] + 4
    dp = gout @ v.t()
    edp = (gout.abs() @ v.abs().t()) * (d + 1)
    delta = (p * dp).sum(1)
    near = (p * (dp.abs() * (ep + nk + 2) + edp)).sum(1)
    far = (gout.abs() * (ref["out"][1] + ref["out"][0].abs() * (BF16 / U + d + 2))).sum(1)
    edelta = torch.where(count <= TILE, near, far)
    ds = p * (dp - delta[:, None])
    eds = ds.abs() * (ep + 2 + BF16 / U) + p * (edp + edelta[:, None]) + TINY * see * (dp.abs() + delta.abs()[:, None] + 1)
    c = abs(scale)
    assert torch.allclose(scale * ds @ k, ref["dq"][0])
    return {"dq": (ref["dq"][0], c * ((eds + ds.abs() * (nk + 4)) @ k.abs())),
            "dk": (ref["dk"][0], c * ((eds + ds.abs() * (nq + 4)).t() @ q.abs())), "dv": ref["dv"]}
