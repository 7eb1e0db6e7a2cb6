"""The sequence operators' 64-bit references pinned by checks independent of
their derivations: central differences of <gy, out> for every gradient, closed
forms, and torch's own float64 gradients of the same definition."""
import pytest
import torch

import sequence_reference as R

torch.set_default_dtype(torch.float32)
F64 = torch.float64


def rnd(*shape, seed=0, by=1.0):
    g = torch.Generator().manual_seed(hash((shape, seed)) % (1 << 31))
    return torch.randn(shape, generator=g, dtype=F64) * by


def differences(f, t, step=1e-5):
    """d f / d t by central differences (f: a number of t)."""
    out = torch.zeros_like(t)
    flat = t.view(-1)
    for i in range(flat.numel()):
        v = flat[i].item()
        flat[i] = v + step
        up = f()
        flat[i] = v - step
        down = f()
        flat[i] = v
        out.view(-1)[i] = (up - down) / (2 * step)
    return out


def close(a, b):
    # central differences with step 1e-5: truncation 1e-10 and cancellation 2^-53 / 1e-5 = 1e-11, times the values
    assert torch.allclose(a, b, rtol=1e-7, atol=1e-7 * max(1.0, float(b.abs().max()))), (a - b).abs().max()


@pytest.mark.parametrize("act", [True, False])
@pytest.mark.parametrize("width", [2, 3, 4])
def test_conv_gradients_by_differences(width, act):
    x, w, b, gy = rnd(9, 3), rnd(3, width), rnd(3), rnd(9, 3, seed=1)
    seqs = R.spans([4, 1, 0, 3], first=1)

    def f():
        y = R.conv(x, w, b, act, seqs)[0]
        return float(sum((gy[lo:hi] * y[lo:hi]).sum() for lo, hi in seqs))

    (dx, dw, db), _ = R.conv_backward(x, w, b, act, seqs, gy)
    for got, t in ((dx, x), (dw, w), (db, b)):
        close(got, differences(f, t))


def scan_inputs(rows=7, c=4, g=2, n=3, gate=True):
    A = -torch.exp(rnd(c, n, seed=3))
    return [rnd(rows, c), rnd(rows, c, seed=1), A, rnd(rows, g, n), rnd(rows, g, n, seed=1), rnd(c), rnd(rows, c, seed=2)
            if gate else None, rnd(c, seed=5)]


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("softplus", [True, False])
def test_scan_gradients_by_differences(softplus, gate):
    args = scan_inputs(gate=gate)
    gy = rnd(7, 4, seed=9)
    seqs = R.spans([3, 0, 1, 2])  # the last row is in no sequence

    def f():
        y = R.scan(*args, softplus, seqs)[0]
        return float(sum((gy[lo:hi] * y[lo:hi]).sum() for lo, hi in seqs))

    out, mag = R.scan_backward(*args, softplus, seqs, gy)
    names = ["dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias"]
    for name, t in zip(names, args):
        if t is not None:
            close(out[name], differences(f, t))
            assert (out[name].abs() <= mag[name] * (1 + 1e-12) + 1e-300).all(), name


def test_scan_closed_forms():
    # A = 0: the state is the running sum of d x B, and d = 1 where softplus is off
    x, dt = rnd(6, 2), torch.ones(6, 2, dtype=F64)
    one = torch.ones(6, 1, 1, dtype=F64)
    zero = torch.zeros(2, dtype=F64)
    y = R.scan(x, dt, torch.zeros(2, 1, dtype=F64), one, one, zero, None, zero, False, [(0, 6)])[0]
    assert torch.allclose(y, x.cumsum(0))
    # A = -ln 2 with d = 1 halves the state every row
    y = R.scan(torch.eye(6, 2, dtype=F64), dt, torch.full((2, 1), -0.6931471805599453, dtype=F64), one, one, zero, None,
               zero, False, [(0, 6)])[0]
    assert torch.allclose(y[:, 0], 0.5 ** torch.arange(6, dtype=F64))
    # a row skipped by dt = -Inf leaves the state
    d = dt.clone()
    d[2] = -float("inf")
    last = R.scan(x, d, -torch.ones(2, 1, dtype=F64), one, one, zero, None, zero, True, [(0, 3)])[2][0]
    assert torch.equal(last, R.scan(x, d, -torch.ones(2, 1, dtype=F64), one, one, zero, None, zero, True, [(0, 2)])[2][0])


@pytest.mark.parametrize("parts", ["grosp", "r", "p", "os", "gp", "rp", ""])
def test_join_gradients_by_differences(parts):
    h, gate, res = rnd(3, 5), rnd(3, 5, seed=1), rnd(3, 5, seed=2)
    post, scale, pre = rnd(5, seed=3), rnd(5, seed=4), rnd(5, seed=5)
    gj, gn = rnd(3, 5, seed=6), rnd(3, 5, seed=7)
    given = dict(gate=gate if "g" in parts else None, residual=res if "r" in parts else None,
                 post=post if "o" in parts else None, scale=scale if "s" in parts else None,
                 pre=pre if "p" in parts else None)

    def f():
        o, n, _ = R.join(h, **given, eps=1e-3, store=lambda v: v)
        return float((o * gj).sum() + ((n * gn).sum() if n is not None else 0.0))

    joined = R.join(h, **given, eps=1e-3, store=lambda v: v)[0]
    out, _ = R.join_backward(h, **given, eps=1e-3, joined=joined, gjoined=gj, gnormed=gn)
    for name, t in [("dh", h)] + [("d" + k, v) for k, v in given.items() if v is not None]:
        close(out[name], differences(f, t))
