"""CPU tests of the sequence operators' autograd forms.  The library's calls are replaced by stand-ins that compute
nothing: what is tested is which of autograd's questions reach them."""
import pytest
import torch
from torch.autograd import forward_ad

from linear_spatial_propagation_gspn_amd import sequence as S


@pytest.fixture(autouse=True)
def stand_ins(monkeypatch):
    like = torch.zeros_like
    maybe = lambda t: None if t is None else like(t)  # noqa: E731
    monkeypatch.setattr(S, "gspn_causal_conv_fwd", lambda x, *a, **k: like(x))
    monkeypatch.setattr(S, "gspn_causal_conv_bwd", lambda x, w, b, *a, **k: (like(x), like(w), maybe(b)))
    monkeypatch.setattr(S, "gspn_selective_scan_fwd", lambda x, *a, **k: (like(x), x.new_zeros(1))
                        if k.get("checkpoints") else like(x))
    monkeypatch.setattr(S, "gspn_selective_scan_bwd", lambda x, dt, A, B, C, gy, D, z, b, *a, **k: tuple(
        map(maybe, (x, dt, A, B, C, D, z, b))))
    monkeypatch.setattr(S, "gspn_block_join_fwd", lambda h, *a, **k: (like(h), like(h)))
    monkeypatch.setattr(S, "gspn_block_join_bwd", lambda h, gj, gn, j, gate, res, post, scale, pre, *a, **k: tuple(
        map(maybe, (h, gate, res, post, scale, pre))))


def calls():
    """(form, its tensors) of each operator."""
    x, w, v = torch.randn(6, 4), torch.randn(4, 3), torch.randn(4)
    bc = torch.randn(6, 1, 2)
    return {"conv": (S.causal_conv, [x, w, v]),
            "scan": (S.selective_scan, [x, x + 1, torch.randn(4, 2), bc, bc + 1, v, x - 1, v + 1]),
            "join": (lambda *a: S.block_join(*a)[0], [x, x + 1, x + 2, v, v + 1, v + 2]),
            "normed": (lambda *a: S.block_join(*a)[1], [x, x + 1, x + 2, v, v + 1, v + 2])}


@pytest.mark.parametrize("wants", [False, True])
@pytest.mark.parametrize("op", ["conv", "scan", "join", "normed"])
def test_forward_mode_is_refused_for_every_input(op, wants):
    """A tangent is not dropped, which torch would take for a derivative of zero: there is no forward-mode rule, and
    the call says so, whichever input carries the tangent and whether or not one asks for a gradient."""
    f, ts = calls()[op]
    for i in range(len(ts)):
        with forward_ad.dual_level():
            args = [t.clone().requires_grad_(wants and j == 0) for j, t in enumerate(ts)]
            args[i] = forward_ad.make_dual(args[i], torch.ones_like(ts[i]))
            with pytest.raises(NotImplementedError):
                f(*args)
            with torch.no_grad(), pytest.raises(NotImplementedError):
                f(*args)


@pytest.mark.parametrize("op", ["conv", "scan", "join", "normed"])
def test_a_gradient_with_a_tangent_is_refused(op):
    f, ts = calls()[op]
    leaf = ts[0].clone().requires_grad_()
    y = f(leaf, *ts[1:])
    with forward_ad.dual_level():
        gy = forward_ad.make_dual(torch.ones_like(y), torch.ones_like(y))
        with pytest.raises(NotImplementedError):
            torch.autograd.grad(y, leaf, gy)


@pytest.mark.parametrize("op", ["conv", "scan", "join", "normed"])
def test_plain_calls_stay_plain_at_a_dual_level(op):
    """Without a tangent nothing changes: no graph where no gradient is wanted, one where it is."""
    f, ts = calls()[op]
    with forward_ad.dual_level():
        assert f(*ts).grad_fn is None
        leaf = ts[0].clone().requires_grad_()
        y = f(leaf, *ts[1:])
        assert torch.equal(torch.autograd.grad(y, leaf, torch.ones_like(y))[0], torch.zeros_like(leaf))


@pytest.mark.parametrize("shape,tail,ld", [((0, 5), 1, 5), ((6, 0), 1, 1), ((2, 0, 5), 1, 5), ((0, 3, 4), 2, 12),
                                           ((6, 1, 0), 2, 1)])
def test_an_empty_tensor_has_rows_whatever_its_strides(monkeypatch, shape, tail, ld):
    """The gradient of an empty output's sum is an expanded scalar, all of whose strides are zero, and torch's
    contiguous() leaves it so."""
    monkeypatch.setattr(S, "_tensor", lambda *a: None)  # its device
    gy = torch.ones(()).expand(shape).contiguous()
    assert set(gy.stride()) == {0}
    assert S._rows(gy, "gy", gy.shape, gy.dtype, 0, tail) == ld
