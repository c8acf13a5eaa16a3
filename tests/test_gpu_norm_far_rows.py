"""Layer norm's gradients of rows far from zero, against the float64 formula on the rows
themselves (their own mean, not the fp32 number the forward hands on), and the mean of rows
that hold an infinity.

u = 2^-24. With h = (s - mean) rstd and the mean handed on off by its rounding, every h of a
row is off by the same c, which is what the mean of those h is. Per element of h, as the
kernels form it: the difference and its product with rstd 2 u, rstd itself 60 u (the bound
the forward is tested with), c's own sum 40 u of the mean of |h + c| (at most 1 + |c|), its
subtraction u. |c| stays below 1/16 here, so (62 + 1) u (|h| + 1) + 43 u: 110 u (|h| + 1).
Rows whose mean lies within 8 spreads of zero keep c: 2^-24 of 8, with rstd's rounding 9 u.
Together less than 130 u (|h| + 1).
"""
import math

import pytest
import torch

import mixture_experts_layer_gate_amd as moe

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8
BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = math.inf, math.nan


def _say(msg):
    print(msg, flush=True)


def _formula(dy, s, w, eps=1e-5):
    z, up = s.double(), dy.double()
    mu = z.mean(1, keepdim=True)
    rs = 1 / torch.sqrt(((z - mu) ** 2).mean(1, keepdim=True) + eps)
    h, g = (z - mu) * rs, up * w.double()
    mg, mgh = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    return rs * (g - mg - h * mgh), h, g, rs


def _check(dy, s, w, dx, dw, db, half):
    T = s.shape[0]
    rx, h, g, rs = _formula(dy, s, w)
    up, e = dy.double(), h.abs() + 1
    # dh's part of dx: 130 u e mean|g h| + |h| mean(|g| 130 u e); rstd 60 u; the operations as near zero
    mg, mge = g.abs().mean(1, keepdim=True), (g.abs() * e).mean(1, keepdim=True)
    bound = rs * U * (70 * g.abs() + 110 * mg + 260 * e * mge) + (half + 2 * U) * rx.abs()
    bad = ((dx.double() - rx).abs() / bound).max()
    _say(f"  dx at {float(bad):.3f} of its bound")
    assert float(bad) <= 1
    rows = -(-T // 256) + 64
    bad = ((dw.double() - (up * h).sum(0)).abs() / ((rows + 134) * U * (up.abs() * e).sum(0))).max()
    _say(f"  dweight at {float(bad):.3f} of its bound")
    assert float(bad) <= 1
    assert bool(((db.double() - up.sum(0)).abs() <= rows * U * up.abs().sum(0)).all())


# one row, rows to waves and to workgroups, short batches and long ones, rows over 8192 columns
SHAPES = [(1, 64), (333, 1048), (333, 256), (37, 7168), (600, 4096), (1030, 520), (1100, 1032), (1030, 4104), (1500, 7168),
          (2500, 2048), (70, 8200), (300, 12296), (1100, 16384)]


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("offset", [3.0, 1e2, 1e4, 1e6, -3e7])
def test_gradients_of_rows_far_from_zero(offset, T, d):
    gen = torch.Generator(device="cuda").manual_seed(T + d)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x = (rn(T, d).double() * max(1.0, abs(offset) * 2.0 ** -20) + offset).float()
    dy, w = rn(T, d), 1 + 0.2 * rn(d)
    dims, opts = moe.Dims(T, d, 64, 1, 1, F32), moe.NormOptions("layer", 1e-5)
    _say(f"{T} x {d} around {offset}")
    _, s, mean, rstd = moe.norm_forward(dims, opts, x, w, keep=True)
    dx, dw, db = moe.norm_backward(dims, opts, dy, s, w, rstd, mean=mean, want_dbias=True)
    _check(dy, x, w, dx, dw, db, U)
    # the weight's gradient alone, the bias' alone, and in place: the same bits
    only = moe.norm_backward(dims, opts, dy, s, w, rstd, mean=mean)
    assert torch.equal(only[0], dx) and torch.equal(only[1], dw)
    only = moe.norm_backward(dims, opts, dy, s, w, rstd, mean=mean, want_dweight=False, want_dbias=True)
    assert torch.equal(only[0], dx) and torch.equal(only[2], db)
    for k in range(2):
        t = [dy.clone(), s.clone()]
        got = moe.norm_backward(dims, opts, t[0], t[1], w, rstd, mean=mean, dx=t[k], want_dbias=True)
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw) and torch.equal(got[2], db)


@pytest.mark.parametrize("T,d", [(64, 256), (333, 1048), (700, 7168), (1500, 1032), (70, 8200), (520, 16384)])
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_gradients_of_batches_with_some_far_rows(dt, T, d):
    """Every third row far from zero (bf16: one value but for a few elements one step apart), rows of zeros and of one
    value among ordinary ones; without a weight."""
    gen = torch.Generator(device="cuda").manual_seed(T + d)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x = rn(T, d) + 0.5 * rn(T, 1)
    if dt is F32:
        x[::3] += 1e5
    else:
        x[::3] = 1024.0
        x[::3, ::97] = 1032.0
    x[1] = 0.0
    x[2 % T] = 3.0
    x, dy = x.to(dt), rn(T, d).to(dt)
    dims, opts = moe.Dims(T, d, 64, 1, 1, dt), moe.NormOptions("layer", 1e-5)
    _say(f"{T} x {d} {dt}, some rows far from zero")
    _, s, mean, rstd = moe.norm_forward(dims, opts, x, keep=True)
    dx, dw, db = moe.norm_backward(dims, opts, dy, s, None, rstd, mean=mean, want_dbias=True)
    _check(dy, x, torch.ones(d, device="cuda"), dx, dw, db, BF if dt is BF16 else U)

@pytest.mark.parametrize("d", [256, 1032, 7168, 8200])
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_mean_of_rows_that_are_not_finite(dt, d):
    """An infinity (or several of a sign) is the row's mean; both signs, or a NaN, make it NaN; other rows keep theirs."""
    T = 7
    gen = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randn((T, d), generator=gen, device="cuda").to(dt)
    dims, opts = moe.Dims(T, d, 64, 1, 1, dt), moe.NormOptions("layer", 1e-5)
    _, _, m0, r0 = moe.norm_forward(dims, opts, x, keep=True)
    z = x.clone()
    z[1, d // 2] = INF
    z[2, 0] = -INF
    z[3, 3] = z[3, d - 1] = INF
    z[4, 3], z[4, d - 1] = INF, -INF
    z[5, 1] = NAN
    y, _, mean, rstd = moe.norm_forward(dims, opts, z, keep=True)
    assert mean[1:4].tolist() == [INF, -INF, INF] and bool(torch.isnan(mean[4:6]).all())
    assert bool(torch.isnan(rstd[1:6]).all()) and bool(torch.isnan(y[1:6]).all())
    assert torch.equal(mean[[0, 6]], m0[[0, 6]]) and torch.equal(rstd[[0, 6]], r0[[0, 6]])
    # gradients: those rows, and no other
    dy = torch.ones((T, d), device="cuda").to(dt)
    a = moe.norm_backward(dims, opts, dy, x, None, r0, mean=m0)
    b = moe.norm_backward(dims, opts, dy, z, None, rstd, mean=mean)
    assert bool(torch.isnan(b[0][1:6]).all()) and torch.equal(a[0][[0, 6]], b[0][[0, 6]])


@pytest.mark.parametrize("T,d", [(40, 256), (333, 1048), (700, 7168), (1100, 256), (1500, 1032), (300, 12296)])
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_infinite_gradients_of_far_rows(dt, T, d):
    """An infinite dy times h is an infinity of dweight's column, in rows far from zero as in others, and reaches no other
    column of it and no other row of dx."""
    gen = torch.Generator(device="cuda").manual_seed(T + d)
    x = torch.randn((T, d), generator=gen, device="cuda")
    x[::2] += 300.0
    x, dy = x.to(dt), torch.randn((T, d), generator=gen, device="cuda").to(dt)
    dims, opts = moe.Dims(T, d, 64, 1, 1, dt), moe.NormOptions("layer", 1e-5)
    _, s, mean, rstd = moe.norm_forward(dims, opts, x, keep=True)
    dx0, dw0, db0 = moe.norm_backward(dims, opts, dy, s, None, rstd, mean=mean, want_dbias=True)
    # (where h is off zero by more than the row's rounding)
    h = (x.double() - x.double().mean(1, keepdim=True)) * rstd.double()[:, None]
    z, want = dy.clone(), dw0.clone()
    for t, c in ((4, 7), (5, 20), (T - 2, d - 3), (T // 4 * 2, d // 2)):
        c = c + int(h[t, c:c + 2].abs().argmax())
        assert float(h[t, c].abs()) > 1e-3
        z[t, c] = INF
        want[c] = INF * float(h[t, c])
    dx, dw, db = moe.norm_backward(dims, opts, z, s, None, rstd, mean=mean, want_dbias=True)
    assert torch.equal(dw, want)
    assert torch.equal(db, torch.where(torch.isinf(want), torch.full_like(db0, INF), db0))
    rows = torch.isfinite(z).all(1)
    assert torch.equal(dx[rows], dx0[rows]) and not bool(torch.isfinite(dx[~rows]).any())
