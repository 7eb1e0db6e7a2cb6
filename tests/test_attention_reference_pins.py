"""The 64-bit definitions that the attention operators are held to, against torch's own (autograd, softmax) on the CPU."""
import math

import pytest
import torch

import attention_reference as R


@pytest.mark.parametrize("nq,nk,causal", [(7, 7, True), (5, 9, True), (9, 4, True), (6, 3, False), (1, 1, True),
                                          (4, 0, False), (0, 3, True)])
def test_attend(nq, nk, causal):
    g = torch.Generator().manual_seed(nq * 10 + nk)
    q, k, v, go = (torch.randn(n, 6, generator=g, dtype=torch.float64, requires_grad=True) for n in (nq, nk, nk, nq))
    see = R.visible(nq, nk, causal)
    for i in range(nq):  # the last row sees every key
        assert int(see[i].sum()) == (max(0, min(nk, i + 1 + nk - nq)) if causal else nk)
    res = R.attend(*(t.detach() for t in (q, k, v)), 0.3, causal, gout=go.detach())
    some = see.any(1)
    s = (0.3 * q @ k.t()).masked_fill(~see, -math.inf)[some]
    out = torch.softmax(s, -1) @ v
    assert torch.allclose(res["out"][0][some], out) and (res["out"][0][~some] == 0).all()
    assert torch.allclose(res["lse"][0][some], torch.logsumexp(s, -1)) and (res["lse"][0][~some] == -math.inf).all()
    grads = torch.autograd.grad(out, [q, k, v], go[some].detach()) if nq and nk else [torch.zeros_like(t) for t in (q, k, v)]
    for n, want in zip(("dq", "dk", "dv"), grads):
        assert torch.allclose(res[n][0], want), n
    for n in res:
        assert (res[n][1] >= 0).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_rotary(interleaved, norm):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(5, 2, 11, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(11, generator=g, dtype=torch.float64, requires_grad=True) if norm else None
    pos = torch.randint(-50, 50, (5, 2), generator=g, dtype=torch.int32)
    freqs = torch.rand(4, generator=g, dtype=torch.float64)
    go = torch.randn(5, 2, 11, generator=g, dtype=torch.float64)
    res = R.rotary(x.detach(), None if w is None else w.detach(), pos, freqs, (1, 3), interleaved, 1e-5, go)
    y = x
    if norm:
        y = x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + 1e-5) * w
    z = y.clone()
    for j in range(4):
        t = pos[:, 0 if j < 1 else 1].double() * freqs[j]
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, 4 + j)
        z[..., a] = y[..., a] * torch.cos(t)[:, None] - y[..., b] * torch.sin(t)[:, None]
        z[..., b] = y[..., a] * torch.sin(t)[:, None] + y[..., b] * torch.cos(t)[:, None]
    assert torch.allclose(res["y"][0], z)
    grads = torch.autograd.grad(z, [x] + ([w] if norm else []), go)
    assert torch.allclose(res["dx"][0], grads[0])
    if norm:
        assert torch.allclose(res["dw"][0], grads[1])
