"""The sequence operators on the GPU where calls and values are at their edges: nothing to sum over, values at the ends
of their type's range."""
import math

import pytest
import torch

import sequence_reference as R
from linear_spatial_propagation_gspn_amd import sequence as S
from test_gpu_sequence import (BF16, DEV, F32, _gpu, _say, check, cu_of, dev, gate_count, gen, on_gpu, ref_args, rnd,  # noqa: F401
                               run_bwd, run_fwd, scan_case, wide)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------------ nothing to sum

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,c,n", [(1, 1, 1), (40, 70, 16), (3000, 5, 3)])
def test_rows_without_a_sequence_get_zero_gradients(dtype, rows, c, n):
    """The C calls themselves (the binding answers such a call without one): every gradient is written."""
    none = torch.zeros(1, dtype=torch.int32, device=DEV)
    code = 0 if dtype == F32 else 1
    g = gen(1)
    k = on_gpu(scan_case(g, rows, c, 1, n, dtype))
    seq = S._sequences(k["x"], none, None)
    wide_dx = torch.full((rows, c + 3), 7.0, dtype=dtype, device=DEV)
    full = lambda like: torch.full(like.shape, 7.0, dtype=like.dtype, device=DEV)  # noqa: E731

    w, b = dev(rnd(g, c, 4)), dev(rnd(g, c))
    a = S._conv_args(k["x"], w, b, True, seq)
    a.gy, a.ldgy = k["x"].data_ptr(), c
    outs = [wide_dx[:, :c], full(w), full(b)]
    a.dx, a.lddx = outs[0].data_ptr(), c + 3
    a.dweight, a.dbias = outs[1].data_ptr(), outs[2].data_ptr()
    S._call("gspn_causal_conv_bwd", a, code, 0)
    assert all((t == 0).all() for t in outs) and (wide_dx[:, c:] == 7.0).all()

    a = S._scan_args(k["x"], k["dt"], k["A"], k["B"], k["C"], k["D"], k["z"], k["dt_bias"], True, seq)
    a.gy, a.ldgy = k["x"].data_ptr(), c
    wide_dx.fill_(7.0)
    outs = {"dx": wide_dx[:, :c], "ddt": full(k["x"]), "dz": full(k["x"]), "dB": full(k["B"]), "dC": full(k["C"]),
            "dA": full(k["A"]), "dD": full(k["D"]), "ddt_bias": full(k["D"])}
    for name, t in outs.items():
        setattr(a, name, t.data_ptr())
    a.lddx, a.ldddt, a.lddz = c + 3, c, c
    S._call("gspn_selective_scan_bwd", a, code, 0)
    for name, t in outs.items():
        assert (t == 0).all(), name
    assert (wide_dx[:, c:] == 7.0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kw", [{}, {"nseq": 2}, {"cu": [1, 5]}, {"cu": [0]}])
def test_rows_without_a_channel_have_zero_sums(dtype, kw):
    kw = {n: cu_of([b - a for a, b in zip(v, v[1:])], v[0]) if n == "cu" else v for n, v in kw.items()}
    x, A = torch.empty(6, 0, dtype=dtype, device=DEV), torch.empty(0, 5, device=DEV)
    bc = torch.randn(6, 3, 5, device=DEV).to(dtype)
    assert S.gspn_selective_scan_fwd(x, x, A, bc, bc, **kw).shape == (6, 0)
    grads = S.gspn_selective_scan_bwd(x, x, A, bc, bc, x, **kw)
    for t, shape in zip(grads[:5], ((6, 0), (6, 0), (0, 5), (6, 3, 5), (6, 3, 5))):
        assert t.shape == shape and (t == 0).all()
    leaf = bc.clone().requires_grad_()
    S.selective_scan(x, x, A, leaf, leaf, **kw).sum().backward()
    assert (leaf.grad == 0).all()


def test_gradients_of_an_empty_batch():
    """No rows: the sums over them are zero, also for a gradient whose strides are those of an expanded scalar."""
    x, bc = (torch.empty(0, *s, device=DEV, requires_grad=True) for s in ((12,), (1, 4)))
    w, A, pre = (torch.randn(*s, device=DEV).requires_grad_() for s in ((12, 4), (12, 4), (12,)))
    for f, leaves in ((lambda: S.causal_conv(x, w), (x, w)), (lambda: S.selective_scan(x, x, A, bc, bc), (x, A, bc)),
                      (lambda: S.block_join(x, x, x, pre=pre)[1], (x, pre))):
        for t, g in zip(leaves, torch.autograd.grad(f().sum(), leaves)):
            assert g.shape == t.shape and (g == 0).all()
