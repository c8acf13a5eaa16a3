"""The norm in front of the layer and its gradients, the gradients' 2-norm and the
AdamW update with states in 32 or 8 bits, through the C ABI, against the float64
oracle (oracle/train_oracle.py).

Tolerances. u = 2^-24 is fp32's half step, BF = 2^-8 bf16's. A row's sum is a
chain of at most 16 terms in a thread, 6 levels in a wave and 16 waves: 40 u of
the terms' absolute sum, with the mean's division. Each further operation adds
its u. Weight gradients add (rows of a part + 64) u of their terms' absolute sum.
Codes and scales of 8-bit states must be equal to the definition's on the moments
as fp32 forms them (one rounding after each operation).
"""
import math
import sys

import numpy as np
import pytest
import torch

import mixture_experts_layer_gate_amd as moe
from oracle import router_oracle as ro
from oracle import train_oracle as to

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8
INF, NAN = math.inf, math.nan
BF16, F32 = torch.bfloat16, torch.float32


def _say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _guarded(shape, dtype, pad=64):
    """A contiguous tensor inside a larger buffer of sentinels, and a check that those are left alone."""
    n = int(np.prod(shape))
    buf = torch.full((n + 2 * pad,), 77, dtype=dtype, device="cuda")

    def check():
        assert bool((buf[:pad] == 77).all()) and bool((buf[pad + n:] == 77).all())
    return buf[pad:pad + n].view(shape), check


# -------------------------------------------------------------------- norm ----
def _norm_inputs(T, d, dt, wt, seed, offset=0.5):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x = rn(T, d) + offset * rn(T, 1)
    x[:, ::max(1, d // 7)] *= 20.0
    return x.to(dt), rn(T, d).to(dt), (1 + 0.2 * rn(d)).to(wt), (0.2 * rn(d)).to(wt)


def _check_norm(s, w, b, kind, eps, y, mean, rstd, half):
    """y, mean and rstd of rows s against the oracle's."""
    ry, rm, rr = to.norm(s, w, b, kind, eps)
    a, e = np.abs(s).mean(1), np.abs(s - rm[:, None])
    if kind == "layer":
        assert (np.abs(mean - rm) <= 40 * U * a).all()
    # var: 40 u of its own terms, u from each difference's rounding twice, and the mean's error, squared
    var_rel = 44 * U + ((40 * U * a) * rr) ** 2
    assert (np.abs(rstd - rr) <= (var_rel / 2 + 4 * U) * rr).all()
    wabs = 1.0 if w is None else np.abs(w)[None, :]
    bound = wabs * rr[:, None] * ((40 * U * a[:, None] if kind == "layer" else 0.0) + (30 * U + var_rel[:, None]) * e)
    assert (np.abs(y - ry) <= bound + (half + 2 * U) * np.abs(ry) + 2 * U * (0 if b is None else np.abs(b)[None, :])).all()


SHAPES = [(1, 8), (3, 64), (5, 520), (7, 1032), (4, 1048), (9, 4104), (6, 6144), (5, 7168), (3, 8200), (2, 16384),
          (1029, 256), (513, 1032), (40, 2048)]


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_norm_forward(dt, kind, T, d):
    half = BF if dt is BF16 else U
    dims = moe.Dims(T, d, 64, 8, 2, dt)
    for wt, residual, weight, bias in ((F32, True, True, True), (BF16, False, True, False), (BF16, True, True, True),
                                       (F32, False, False, False), (F32, True, False, True)):
        _say(f"norm {kind} {dt} {T} x {d}: weights {wt}, residual {residual}, weight {weight}, bias {bias}")
        bias = bias and kind == "layer"
        x, r, w, b = _norm_inputs(T, d, dt, wt, T + d)
        y, cy = _guarded((T, d), dt)
        s, cs = _guarded((T, d), dt)
        rstd, cr = _guarded((T,), F32)
        opts = moe.NormOptions(kind, 1e-5, wt)
        got = moe.norm_forward(dims, opts, x, w if weight else None, b if bias else None, residual=r if residual else None,
                               sum=s if residual else None, y=y, rstd=rstd, keep=True)
        torch.cuda.synchronize()
        for c in (cy, cs, cr):
            c()
        if residual:
            assert torch.equal(got[1], (x.float() + r.float()).to(dt))
        else:
            assert got[1] is x
        assert (got[2] is None) == (kind == "rms")
        _check_norm(_np(got[1]), _np(w) if weight else None, _np(b) if bias else None, kind, 1e-5, _np(y), _np(got[2]),
                    _np(rstd), half)


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_norm_backward(dt, kind, T, d):
    half = BF if dt is BF16 else U
    dims = moe.Dims(T, d, 64, 8, 2, dt)
    layer = kind == "layer"
    for wt, add, weight in ((F32, True, True), (BF16, False, True), (F32, True, False)):
        _say(f"norm gradients {kind} {dt} {T} x {d}: weights {wt}, dx_in {add}, weight {weight}")
        x, r, w, _ = _norm_inputs(T, d, dt, wt, T + d)
        dy, dx_in = (torch.randn((T, d), device="cuda") * 0.01).to(dt), (r.float() * 0.01).to(dt)
        opts = moe.NormOptions(kind, 1e-5, wt)
        _, s, mean, rstd = moe.norm_forward(dims, opts, x, w if weight else None, keep=True)
        dx, cx = _guarded((T, d), dt)
        dw, cw = _guarded((d,), F32)
        db, cb = _guarded((d,), F32)
        out = moe.norm_backward(dims, opts, dy, s, w if weight else None, rstd, mean=mean, dx_in=dx_in if add else None,
                                dx=dx, dweight=dw, dbias=db if layer else None)
        torch.cuda.synchronize()
        for c in (cx, cw, cb):
            c()
        assert out[0] is dx and out[1] is dw and out[2] is (db if layer else None)
        ny, ns, nw = _np(dy), _np(s), _np(w) if weight else np.ones(d)
        nm, nr = _np(mean) if layer else np.zeros(T), _np(rstd)
        rx, rw, rb, aw, ab = to.norm_backward(ny, ns, nw, kind, nm, nr, _np(dx_in) if add else None)
        rows = -(-T // 256) + 64  # (at least 256 parts where there are so many rows)
        assert (np.abs(_np(dw) - rw) <= (rows + 4) * U * aw).all()
        if layer:
            assert (np.abs(_np(db) - rb) <= rows * U * ab).all()
        h, g = np.abs((ns - nm[:, None]) * nr[:, None]), np.abs(ny * nw)
        mg, mgh = g.mean(1, keepdims=True), (g * h).mean(1, keepdims=True)
        bound = nr[:, None] * U * (4 * g + 50 * h * mgh + (46 * mg if layer else 0)) + (half + 2 * U) * np.abs(rx)
        bound += 2 * U * (np.abs(_np(dx_in)) if add else 0)
        assert (np.abs(_np(dx) - rx) <= bound).all()
        # what is not wanted changes nothing else
        a = moe.norm_backward(dims, opts, dy, s, w if weight else None, rstd, mean=mean, dx_in=dx_in if add else None,
                              want_dweight=False)
        assert torch.equal(a[0], dx) and a[1] is None and a[2] is None
        if layer:
            a = moe.norm_backward(dims, opts, dy, s, w if weight else None, rstd, mean=mean, want_dweight=False,
                                  want_dbias=True)
            assert torch.equal(a[2], db) and a[1] is None


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_gradient_by_differences(kind):
    """fp32, along a random direction: f(x + h v) - f(x - h v) over 2 h, h = 2^-9. Its curvature leaves about h^2 = 4e-6
    of the gradient's size, fp32's rounding of y (2^-24 of sqrt(T d) random terms) over h another 2^-15."""
    T, d = 64, 520
    dims, opts = moe.Dims(T, d, 64, 8, 2, F32), moe.NormOptions(kind, 1e-5, F32)
    x, v, w, b = _norm_inputs(T, d, F32, F32, 3)
    dy = torch.randn((T, d), device="cuda")
    _, s, mean, rstd = moe.norm_forward(dims, opts, x, w, b if kind == "layer" else None, keep=True)
    dx, dw, _ = moe.norm_backward(dims, opts, dy, s, w, rstd, mean=mean)
    h = 2.0 ** -9

    def f(xx, ww):
        y = moe.norm_forward(dims, opts, xx, ww, b if kind == "layer" else None)[0]
        return float((y.double() * dy.double()).sum())
    num = (f(x + h * v, w) - f(x - h * v, w)) / (2 * h)
    ref = float((dx.double() * v.double()).sum())
    assert abs(num - ref) <= 1e-3 * float(dx.double().norm() * v.double().norm()) / math.sqrt(T)
    vw = torch.randn(d, device="cuda")
    num = (f(x, w + h * vw) - f(x, w - h * vw)) / (2 * h)
    ref = float((dw.double() * vw.double()).sum())
    assert abs(num - ref) <= 1e-3 * float(dw.double().norm() * vw.double().norm()) / math.sqrt(d)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [256, 1032, 7168])
def test_norm_rows_of_every_size(d, dt, kind, rng):
    """Rows from 2^-120 to 2^127 in one batch, zero rows, rows of one value: each as if alone."""
    sizes = [-120, -70, -30, 0, 20, 60, 63, 64, 65, 100, 126]
    base = (rng.random((len(sizes), d)) - 0.5).astype(np.float64)
    x = torch.from_numpy(base * 2.0 ** np.array(sizes)[:, None]).to(dt).cuda()
    x = torch.cat([x, torch.zeros((1, d), dtype=dt, device="cuda"), torch.full((1, d), 3.0, dtype=dt, device="cuda")])
    T = x.shape[0]
    dims, opts = moe.Dims(T, d, 64, 8, 2, dt), moe.NormOptions(kind, 1e-5, F32)
    y, _, mean, rstd = moe.norm_forward(dims, opts, x, keep=True)
    assert bool(torch.isfinite(y).all())
    _check_norm(_np(x), None, None, kind, 1e-5, _np(y), _np(mean), _np(rstd), BF if dt is BF16 else U)
    # gradients: ordinary numbers where dy is of the row's size
    dy = (torch.randn((T, d), device="cuda").double() * torch.clamp(1 / rstd.double(), 1e-30, 1e30)[:, None]).to(dt)
    dx, _, _ = moe.norm_backward(dims, opts, dy, x, None, rstd, mean=mean, want_dweight=False)
    ny, ns, nm, nr = _np(dy), _np(x), _np(mean) if kind == "layer" else np.zeros(T), _np(rstd)
    rx, _, _, _, _ = to.norm_backward(ny, ns, None, kind, nm, nr)
    h, g = np.abs((ns - nm[:, None]) * nr[:, None]), np.abs(ny)
    bound = nr[:, None] * U * (4 * g + 50 * h * (g * h).mean(1, keepdims=True) + 46 * g.mean(1, keepdims=True))
    bound = bound + (BF if dt is BF16 else 2 * U) * np.abs(rx)
    assert (np.abs(_np(dx) - rx) <= bound + 2.0 ** -126)[:-2].all()


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("d", [256, 1032, 7168])
def test_norm_non_finite_rows_stay_their_own(d, value, kind):
    """A NaN or infinity takes its own row (and its column of dweight) as the formula does, and no other row."""
    T = 9
    x, _, w, _ = _norm_inputs(T, d, F32, F32, 5)
    dims, opts = moe.Dims(T, d, 64, 8, 2, F32), moe.NormOptions(kind, 1e-5, F32)
    y0, _, m0, r0 = moe.norm_forward(dims, opts, x, w, keep=True)
    z = x.clone()
    z[4, d // 2] = value
    y, s, m, r = moe.norm_forward(dims, opts, z, w, keep=True)
    rest = [t for t in range(T) if t != 4]
    assert torch.equal(y[rest], y0[rest]) and torch.equal(r[rest], r0[rest])
    if kind == "layer" or value != value:
        assert bool(torch.isnan(y[4]).all())
    else:  # 1 / sqrt(inf) = 0: zeros, and NaN where the infinity is
        want = torch.zeros(d, device="cuda")
        want[d // 2] = NAN
        assert torch.equal(torch.isnan(y[4]), torch.isnan(want)) and bool((y[4].nan_to_num() == 0).all())
    dy = torch.ones((T, d), device="cuda")
    dx0, _, _ = moe.norm_backward(dims, opts, dy, x, w, r0, mean=m0)
    dx, dw, _ = moe.norm_backward(dims, opts, dy, s, w, r, mean=m)
    assert torch.equal(dx[rest], dx0[rest]) and bool(torch.isnan(dx[4]).any()) and bool(torch.isnan(dw[d // 2]))


@pytest.mark.parametrize("d", [64, 1032, 7168, 16384])
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_norm_in_place(dt, d):
    """sum over x or residual, y over the other; dx over dy, s or dx_in: the same bits."""
    T = 33
    dims, opts = moe.Dims(T, d, 64, 8, 2, dt), moe.NormOptions("layer", 1e-5, F32)
    x, r, w, b = _norm_inputs(T, d, dt, F32, 8)
    y, s, m, q = moe.norm_forward(dims, opts, x, w, b, residual=r, keep=True)
    for first in (True, False):
        a, c = x.clone(), r.clone()
        moe.norm_forward(dims, opts, a, w, b, residual=c, sum=a if first else c, y=c if first else a)
        assert torch.equal(a if first else c, s) and torch.equal(c if first else a, y)
    a = s.clone()
    moe.norm_forward(dims, opts, a, w, b, y=a)
    assert torch.equal(a, y)
    dy, di = torch.randn((T, d), device="cuda").to(dt), torch.randn((T, d), device="cuda").to(dt)
    want = moe.norm_backward(dims, opts, dy, s, w, q, mean=m, dx_in=di, want_dbias=True)
    for k in range(3):
        t = [dy.clone(), s.clone(), di.clone()]
        got = moe.norm_backward(dims, opts, t[0], t[1], w, q, mean=m, dx_in=t[2], dx=t[k], want_dbias=True)
        assert all(torch.equal(p, c) for p, c in zip(got, want))


def test_norm_empty_batch_and_many_rows():
    d = 64
    for kind in ("rms", "layer"):
        opts, e = moe.NormOptions(kind), moe.Dims(0, d, 64, 8, 2)
        x, f = torch.zeros((0, d), dtype=BF16, device="cuda"), torch.zeros(0, device="cuda")
        assert moe.norm_forward(e, opts, x, keep=True)[0].shape == (0, d)
        dw = torch.full((d,), 5.0, device="cuda")
        db = torch.full((d,), 5.0, device="cuda") if kind == "layer" else None
        moe.norm_backward(e, opts, x, x, None, f, mean=f if kind == "layer" else None, dweight=dw, dbias=db)
        assert not dw.any() and (db is None or not db.any())
    # more rows than one pass of the grid covers
    d, T = 8, 2 ** 23 + 7
    x = torch.randn((T, d), device="cuda").to(BF16)
    dims, opts = moe.Dims(T, d, 64, 1, 1), moe.NormOptions("rms", 1e-6)
    y, _, _, rstd = moe.norm_forward(dims, opts, x, keep=True)
    want = torch.rsqrt(x.double().pow(2).mean(1) + 1e-6)
    assert float((rstd.double() / want - 1).abs().max()) <= 40 * U
    assert float((y.double() - x.double() * want[:, None]).abs().max()) <= (BF + 50 * U) * 3
    dx, dw, _ = moe.norm_backward(dims, opts, y, x, None, rstd)
    h = x.double() * rstd.double()[:, None]
    t = y.double() * h
    assert bool(((dw.double() - t.sum(0)).abs() <= (T / 512 + 64) * U * t.abs().sum(0)).all())
    ref = rstd.double()[:, None] * (y.double() - h * t.mean(1, keepdim=True))
    mag = rstd.double()[:, None] * (y.double().abs() + h.abs() * t.abs().mean(1, keepdim=True))
    assert bool(((dx.double() - ref).abs() <= BF * ref.abs() + 50 * U * mag).all())


# --------------------------------------------------------------- 2-norm -------
def _ragged(sizes, dtypes, seed, shift=0):
    """Tensors of the sizes, of alternating types, `shift` elements past a 16-byte boundary."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        dt = dtypes[i % len(dtypes)]
        buf = torch.randn(n + shift, generator=gen, device="cuda").to(dt)
        out.append(buf[shift:])
    return out


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("sizes", [[1], [7, 0, 8191], [8192, 8193, 3], [100003], [5] * 119, [5] * 120 + [9000], [17] * 300,
                                   [30000000, 1]], ids=lambda s: f"{len(s)}x{s[0]}")
def test_grad_norm(sizes, shift):
    gs = _ragged(sizes, (F32, BF16), 3, shift)
    total = math.sqrt(math.fsum(float(g.double().pow(2).sum()) for g in gs))
    for scale, most in ((1.0, INF), (0.25, 0.5), (-2.0, 1e-3), (2.0 ** -70, 1.0)):
        out, chk = _guarded((2,), F32)
        assert moe.grad_norm(gs, scale, most, out=out) is out
        chk()
        n = abs(scale) * total
        f = scale * min(1.0, most / (n + 1e-6))
        # sums in double: the outputs' own rounding
        assert abs(float(out[0]) - n) <= 1.01 * U * n and abs(float(out[1]) - f) <= 1.01 * U * abs(f)
        assert torch.equal(moe.grad_norm(moe.GradList(gs), scale, most), out)


def test_grad_norm_of_extremes():
    big = [torch.full((9000,), 3e38, device="cuda"), torch.full((5,), 1e-30, device="cuda")]
    out = moe.grad_norm(big, 2.0 ** -60, 1.0)
    n = 3e38 * math.sqrt(9000) * 2.0 ** -60
    assert abs(float(out[0]) / n - 1) < 1e-6
    # the factor, 3.5e-41, lies below 2^-126, where fp32's step is 2^-149: half of one
    assert abs(float(out[1]) - 2.0 ** -60 / n) <= 2.0 ** -150
    tiny = [torch.full((100,), 2.0 ** -140, device="cuda")]
    assert float(moe.grad_norm(tiny)[0]) == 10 * 2.0 ** -140
    assert moe.grad_norm([torch.zeros(3, device="cuda"), torch.zeros(0, device="cuda")], 1.0, 2.0).tolist() == [0.0, 1.0]
    assert moe.grad_norm([torch.zeros(0, device="cuda")], 0.5).tolist() == [0.0, 0.5]
    for v in (INF, -INF, NAN):
        for dt in (F32, BF16):
            g = torch.zeros(20000, device="cuda", dtype=dt)
            g[12345] = v
            out = moe.grad_norm([torch.ones(3, device="cuda"), g], 1.0, 1.0)
            assert not math.isfinite(float(out[0])) and math.isnan(float(out[1]))
    assert moe.grad_norm([torch.ones(4, device="cuda")], 1.0, 0.0).tolist() == [2.0, 0.0]


# ---------------------------------------------------------------- AdamW -------
ODD = [1, 7, 8, 127, 128, 129, 1000, 2048, 2049, 8192, 8193, 20000, 3]


def _snapshot(st):
    c = lambda ts: None if ts is None else [None if t is None else t.clone() for t in ts]  # noqa: E731
    return {n: c(getattr(st, n)) for n in ("params", "m", "v", "m_scale", "v_scale", "master")}


def _bases(sizes):
    out, at = [], 0
    for n in sizes:
        out.append(at)
        at += -(-n // 128) * 128
    return out


def _check_step(st, was, grads, opts, lr, step, gs, seed, off):
    """Every output of one step against the oracle, from the state before it."""
    sizes = [p.numel() for p in st.params]
    flat = lambda t: _np(t).reshape(-1)  # noqa: E731
    for i, (n, base) in enumerate(zip(sizes, _bases(sizes))):
        if n == 0:
            continue
        g = grads[i].float().cpu().numpy()
        u = to.numbers(n, base, seed, off) if st.bits == 8 or opts.stochastic else None
        if st.bits == 8:
            m0 = to.decode(was["m"][i].cpu().numpy(), was["m_scale"][i].cpu().numpy(), 3)
            r0 = to.decode(was["v"][i].cpu().numpy(), was["v_scale"][i].cpu().numpy(), 4).astype(np.float32)
            v0 = (r0 * r0).astype(np.float64)
        else:
            m0, v0 = _np(was["m"][i]), _np(was["v"][i])
        m1, v1 = to.adam_moments(g.astype(np.float64), gs, m0, v0, opts.beta1, opts.beta2)
        tm = np.abs(opts.beta1 * m0) + np.abs((1 - opts.beta1) * gs * g)
        if st.bits == 32:
            assert (np.abs(_np(st.m[i]) - m1) <= 4 * U * tm + 2.0 ** -149).all()
            assert (np.abs(_np(st.v[i]) - v1) <= 6 * U * v1 + 2.0 ** -148).all()
        else:
            mf, vf = to.adam_moments(g, gs, m0, v0, opts.beta1, opts.beta2, np.float32)
            for x, code, scale, fr in ((mf, st.m[i], st.m_scale[i], 3), (np.sqrt(vf), st.v[i], st.v_scale[i], 4)):
                c, e = to.encode(x, u, fr)
                np.testing.assert_array_equal(scale.cpu().numpy(), e)
                np.testing.assert_array_equal(code.cpu().numpy(), c)
        master = was["master"][i] if was["master"] is not None else None
        w0 = flat(was["params"][i] if master is None else master)
        w1 = to.adam_update(w0, m1, v1, lr, step, opts.beta1, opts.beta2, opts.eps, opts.weight_decay)
        den = np.sqrt(v1 / (1 - opts.beta2 ** step)) + opts.eps
        up = lr / (1 - opts.beta1 ** step) / den
        bound = up * (4 * U * tm + 12 * U * np.abs(m1)) + 4 * U * lr * opts.weight_decay * np.abs(w0)
        bound = bound + 2 * U * (np.abs(w0) + np.abs(w1))
        got = flat(st.params[i])
        if master is not None:
            assert (np.abs(flat(st.master[i]) - w1) <= bound).all()
            assert torch.equal(st.params[i], st.master[i].to(BF16))
        elif st.params[i].dtype is BF16:
            # to nearest: half a step of bf16 (2^-8 of the value); at random: less than a whole one
            assert (np.abs(got - w1) <= bound + (2 if opts.stochastic else 1) * BF * np.maximum(np.abs(w1), 2.0 ** -126)).all()
        else:
            assert (np.abs(got - w1) <= bound).all()


def _params(sizes, dtypes, seed, shift=0):
    return [(t.float() * 0.1).to(t.dtype) if not shift else t.mul_(0.1) for t in _ragged(sizes, dtypes, seed, shift)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pd,gd,master,stochastic", [
    ((F32,), (F32,), False, False), ((BF16,), (BF16,), False, False), ((BF16,), (F32,), True, False),
    ((BF16,), (F32,), False, True), ((F32, BF16), (BF16, F32, F32), True, False), ((BF16, F32, BF16), (F32,), False, True)])
def test_adam_steps(pd, gd, master, stochastic, bits):
    """Odd sizes, types mixed in one list, from the zero state on, with zero gradients, tiny and large ones."""
    _say(f"adam {bits} bits, params {pd}, grads {gd}, master {master}, stochastic {stochastic}")
    ps = _params(ODD, pd, 1)
    st = moe.adam_state(ps, bits, master)
    for step, lr, wd, b2, gs in ((1, 1e-3, 0.0, 0.999, None), (2, 1e-2, 0.1, 0.999, 0.5), (3, 3e-4, 0.1, 0.95, 1.0)):
        grads = _ragged(ODD, gd, 10 + step)
        for i, g in enumerate(grads):
            g.mul_(10.0 ** (-(i % 5) * 2))
            if i % 4 == step % 4:
                g[: g.numel() // 2] = 0
        opts = moe.AdamOptions(beta2=b2, weight_decay=wd, stochastic=stochastic)
        rng = torch.tensor([5 + (9 << 40), (3 << 33) + step], device="cuda")
        was = _snapshot(st)
        kept = [g.clone() for g in grads]
        assert moe.adam_step(opts, st, grads, lr=lr, step=step, rng=rng if bits == 8 or stochastic else None,
                             gscale=None if gs is None else torch.tensor([gs], device="cuda")) is st
        torch.cuda.synchronize()
        _check_step(st, was, grads, opts, lr, step, gs or 1.0, 5 + (9 << 40), (3 << 33) + step)
        assert all(torch.equal(a, b) for a, b in zip(grads, kept))


@pytest.mark.parametrize("bits", [32, 8])
def test_adam_leaves_the_neighbours_alone(bits):
    """Sentinels around every buffer, odd sizes, off the wide loads' alignment too: the same bits as aligned."""
    for shift in (0, 1):
        sizes = [5, 129, 2047, 8199]
        kind = F32 if bits == 32 else torch.uint8
        bufs, checks = [], []

        def make(n, dt, fill):
            t, c = _guarded((n + shift,), dt)
            t[:shift] = 77
            t[shift:] = fill.to(dt)
            checks.append(c)
            bufs.append(t)
            return t[shift:]
        ps = [make(n, BF16, torch.linspace(-1, 1, n, device="cuda")) for n in sizes]
        m, v = ([make(n, kind, torch.zeros(n, device="cuda")) for n in sizes] for _ in range(2))
        ms = vs = None
        if bits == 8:
            ms, vs = ([make(-(-n // 128), kind, torch.zeros(-(-n // 128), device="cuda")) for n in sizes] for _ in range(2))
        st = moe.AdamState(ps, m, v, ms, vs)
        grads = [torch.sin(torch.arange(n, device="cuda").float()) for n in sizes]
        rng = torch.tensor([1, 2], device="cuda")
        for k in (1, 2, 3):
            moe.adam_step(moe.AdamOptions(stochastic=True), st, grads, lr=1e-2, step=k, rng=rng)
        torch.cuda.synchronize()
        for c in checks:
            c()
        assert all(bool((b[:shift] == 77).all()) for b in bufs)
        now = [t.clone() for t in ps + m + v] + (([t.clone() for t in ms + vs]) if bits == 8 else [])
        if shift == 0:
            first = now
    assert all(torch.equal(a, b) for a, b in zip(first, now))


@pytest.mark.parametrize("bits", [32, 8])
def test_adam_list_is_its_tensors(bits):
    """A list longer than one launch holds: with 32-bit states each tensor as alone; with 8-bit ones as the whole
    list's numbering has it."""
    sizes = [(37 * i) % 300 + 1 for i in range(95)]
    ps = _params(sizes, (F32, BF16), 4)
    grads = _ragged(sizes, (BF16, F32, F32), 5)
    st = moe.adam_state([p.clone() for p in ps], bits)
    rng = torch.tensor([11, 12], device="cuda")
    opts = moe.AdamOptions(weight_decay=0.01)
    for k in (1, 2):
        was = _snapshot(st)
        moe.adam_step(opts, st, grads, lr=1e-3, step=k, rng=rng)
        _check_step(st, was, grads, opts, 1e-3, k, 1.0, 11, 12)
    if bits == 32:
        for i in (0, 39, 40, 94):
            one = moe.adam_state([ps[i].clone()])
            for k in (1, 2):
                moe.adam_step(opts, one, [grads[i]], lr=1e-3, step=k)
            assert torch.equal(one.params[0], st.params[i]) and torch.equal(one.v[0], st.v[i])


def test_adam_without_a_finite_factor_is_no_step():
    for bits in (32, 8):
        st = moe.adam_state(_params(ODD, (BF16, F32), 2), bits, True)
        rng = torch.tensor([1, 2], device="cuda")
        g = _ragged(ODD, (F32,), 3)
        moe.adam_step(moe.AdamOptions(), st, g, lr=1e-3, step=1, rng=rng)
        was = _snapshot(st)
        g[4][3] = INF
        norm = moe.grad_norm(g, 1.0, 1.0)
        for f in (norm[1:], torch.tensor([INF], device="cuda"), torch.tensor([-INF], device="cuda")):
            moe.adam_step(moe.AdamOptions(), st, g, lr=1e-3, step=2, rng=rng, gscale=f)
            now = _snapshot(st)
            for n in was:
                assert was[n] is None or all(a is None or torch.equal(a, b) for a, b in zip(was[n], now[n]))


@pytest.mark.parametrize("value", [NAN, INF, 3e38])
def test_adam_non_finite_gradients(value):
    """They go where the formula sends them: the element's own weight and states; with 8 bits its 128 elements, whose
    scale bytes say so from then on."""
    n = 1000
    p = torch.ones(n, device="cuda")
    g = torch.ones(n, device="cuda")
    g[300] = value
    st = moe.adam_state([p.clone()])
    moe.adam_step(moe.AdamOptions(), st, [g], lr=1e-2, step=1)
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[300] = True
    if value == 3e38:  # x^2 passes fp32's range: the step is 0
        assert bool(torch.isfinite(st.params[0]).all()) and float(st.params[0][300]) == 1.0
        assert torch.equal(torch.isinf(st.v[0]), bad)
    else:
        assert torch.equal(torch.isnan(st.params[0]), bad)
    rng = torch.tensor([1, 2], device="cuda")
    st = moe.adam_state([p.clone()], 8)
    for k in (1, 2):
        moe.adam_step(moe.AdamOptions(), st, [g], lr=1e-2, step=k, rng=rng)
        g = torch.ones(n, device="cuda")
    blk = torch.zeros(n, dtype=torch.bool, device="cuda")
    blk[256:384] = True
    m, r = moe.adam_state_values(st, dtype=F32)
    assert st.v_scale[0].tolist()[2] == 255 and torch.equal(torch.isnan(r[0]), blk)
    assert not st.v[0][256:384].any()
    # (m itself holds 3e38 and swamps its neighbours)
    assert torch.equal(torch.isnan(m[0]), blk if value != 3e38 else torch.zeros_like(blk))
    assert torch.equal(torch.isnan(st.params[0]) & ~blk, torch.zeros_like(blk))


def test_stochastic_rounding_of_weights():
    """bf16 weights are the fp32 weights' bits plus the element's number, cut: those weights from a step with master."""
    n = 5000
    p = _params([n], (BF16,), 6)[0]
    g = _ragged([n], (F32,), 7)
    rng = torch.tensor([21, 22], device="cuda")
    a, b = moe.adam_state([p.clone()], 32, True), moe.adam_state([p.clone()])
    moe.adam_step(moe.AdamOptions(), a, g, lr=1e-3, step=1)
    moe.adam_step(moe.AdamOptions(stochastic=True), b, g, lr=1e-3, step=1, rng=rng)
    u = to.numbers(n, 0, 21, 22)
    bits = a.master[0].cpu().numpy().view(np.uint32).astype(np.int64) + u
    want = ((bits >> 16) & 0xFFFF).astype(np.uint16)
    np.testing.assert_array_equal(b.params[0].view(torch.int16).cpu().numpy().view(np.uint16), want)
    # the mean over draws is the weight: 256 draws, each off by less than a step of 2^-7
    total = torch.zeros(n, dtype=torch.float64, device="cuda")
    for k in range(256):
        c = moe.adam_state([p.clone()])
        moe.adam_step(moe.AdamOptions(stochastic=True), c, g, lr=1e-3, step=1, rng=torch.tensor([21, 100 + k], device="cuda"))
        total += c.params[0].double()
    w = a.master[0].double()
    # standard deviation at most half a step over 16; all elements' average, 5 sigma
    err = (total / 256 - w) / (2.0 ** -7 * w.abs())
    assert float(err.mean().abs()) < 5 * 0.5 / 16 / math.sqrt(n)


def test_states_of_8_bits_follow_the_moments():
    """Gradients of a fixed sign and size: after 400 steps the first moment and the root of the second stand at their
    limits, on average over the elements (rounded to nearest, the second moment would stop where a step of 0.1% is less
    than half a code: 3%)."""
    n = 1 << 16
    size = torch.exp(torch.randn(n, device="cuda"))
    st = moe.adam_state([torch.zeros(n, device="cuda")], 8)
    opts, b2 = moe.AdamOptions(beta2=0.99), 0.99
    for k in range(1, 401):
        moe.adam_step(opts, st, [size], lr=0.0, step=k, rng=torch.tensor([3, k], device="cuda"))
    m, r = moe.adam_state_values(st, dtype=F32)
    # a code is off by at most 1/8 and 1/16 of the value; the moment averages 10 (100) of them
    assert abs(float((m[0] / size).mean()) - 1.0) < 0.01
    assert abs(float((r[0] ** 2 / size ** 2).mean()) - (1 - b2 ** 400)) < 0.02


def test_state_values():
    """Every code under several scales, both types, against the definition."""
    code = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(5)[:1279]
    scale = torch.tensor([1, 1, 127, 127, 200, 254, 60, 60, 255, 100], dtype=torch.uint8, device="cuda")
    st = moe.AdamState([torch.zeros(1279, device="cuda")], [code], [code.clone()], [scale], [scale.clone()])
    for dt in (F32, BF16):
        m, r = moe.adam_state_values(st, dtype=dt)
        for got, fr in ((m[0], 3), (r[0], 4)):
            want = to.decode(code.cpu().numpy(), scale.cpu().numpy(), fr)
            want = torch.from_numpy(want).float().to(dt)
            assert torch.equal(got.cpu().nan_to_num(7.0), want.nan_to_num(7.0))
            assert bool((torch.isnan(got.cpu()) == torch.isnan(want)).all())
    buf = torch.full((1281,), 9.0, device="cuda")
    moe.adam_state_values(st, m=[buf[1:1280]], r=[torch.empty(1279, device="cuda")])
    assert float(buf[0]) == 9.0 and float(buf[1280]) == 9.0


def test_against_torch_over_steps():
    """Twenty steps beside torch's AdamW in float64: fp32 weights drift by their own rounding, u a step and weight."""
    n, lr, wd = 3001, 1e-2, 0.05
    w0 = torch.randn(n, device="cuda")
    p = torch.nn.Parameter(w0.double().clone())
    opt = torch.optim.AdamW([p], lr=lr, betas=(0.9, 0.99), eps=1e-6, weight_decay=wd, foreach=False, fused=False)
    st = moe.adam_state([w0.clone()])
    for k in range(1, 21):
        g = torch.randn(n, device="cuda") * (0.1 + torch.rand(n, device="cuda"))
        p.grad = g.double()
        opt.step()
        moe.adam_step(moe.AdamOptions(beta2=0.99, eps=1e-6, weight_decay=wd), st, [g], lr=lr, step=k)
    # moments carry up to 20 * 4 u of their terms' size; a step is at most lr * 3 here
    err = (st.params[0].double() - p.detach()).abs()
    assert bool((err <= 20 * 2 * U * (w0.abs().double() + 1) + 20 * lr * 100 * U * 10).all())


# ------------------------------------------------------ streams and graphs ----
def _block_inputs(T, d, f, E, k, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    t = {"x": rn(T, d).to(BF16), "delta": (0.5 * rn(T, d)).to(BF16), "dout": rn(T, d).to(BF16),
         "rng": torch.tensor([seed + 5, 3], dtype=torch.int64, device="cuda"),
         "opt_rng": torch.tensor([seed + 6, 4], dtype=torch.int64, device="cuda"),
         "lr_step": torch.tensor([1e-3, 1.0], dtype=torch.float64, device="cuda")}
    params = [(1 + 0.1 * rn(d)), (rn(E, d) / math.sqrt(d)).to(BF16), 0.1 * rn(E), (rn(E, f, d) / math.sqrt(d)).to(BF16),
              (rn(E, f, d) / math.sqrt(d)).to(BF16), (rn(E, d, f) / math.sqrt(f)).to(BF16)]
    return moe.Dims(T, d, f, E, k, BF16), t, params


NORM, ROUTE = moe.NormOptions("rms", 1e-6, F32), moe.RouteOptions("sigmoid", 4, 2, "top2", True, 2.5)


def _block_step(dims, t, st, opts, p=0.25):
    """A block's training step as a program runs it: norm of the residual stream, scored router, experts, combine with
    dropout into the stream; their gradients; the gradients' norm; the update."""
    nw, wg, bias, w1, w3, w2 = st.params
    y, s, _, rstd = moe.norm_forward(dims, NORM, t["x"], nw, residual=t["delta"], keep=True)
    logits, idx, w = moe.route_scored(dims, ROUTE, y, wg, bias)
    counts, offsets, perm, inv = moe.permute(dims, idx)
    rows = moe.grouped_ffn(dims, y, perm, counts, offsets, w1, w3, w2)
    out = moe.combine_dropout(dims, p, t["rng"], rows, inv, w, s)
    dy = moe.dropout_backward(dims, p, t["rng"], t["dout"])
    r = {"topk_idx": idx, "topk_w": w, "counts": counts, "offsets": offsets, "perm": perm, "inv_perm": inv}
    g = moe.experts_backward(dims, y, w1, w3, w2, r, dy)
    dl = moe.route_select_backward(dims, ROUTE, logits, idx, w, g["dtopk_w"])
    dyn, dwg, db = moe.gate_backward(dims, y, wg, dl, g["dx"])
    ds, dnw, _ = moe.norm_backward(dims, NORM, dyn, s, nw, rstd, dx_in=t["dout"])
    grads = [dnw, dwg, db, g["dw1"], g["dw3"], g["dw2"]]
    norm = moe.grad_norm(grads, 1.0, 1.0)
    moe.adam_step(opts, st, grads, lr_step=t["lr_step"], gscale=norm[1:], rng=t["opt_rng"])
    return {"out": out, "ds": ds, "idx": idx, "norm": norm, "grads": grads}


@pytest.mark.parametrize("bits", [32, 8])
def test_block_training_step(bits):
    """All of it against float64 differentiation of the plain definition, the choice and the keep decisions fixed; the
    update against the formula on the gradients that came out. Bars: the layer's 2e-2 normwise (its bf16 roundings),
    which the norm's gradients inherit."""
    T, d, f, E, k, p = 130, 256, 256, 8, 2, 0.25
    dims, t, params = _block_inputs(T, d, f, E, k, 1)
    st = moe.adam_state([q.clone() for q in params], bits, True)
    opts = moe.AdamOptions(weight_decay=0.1)
    was = _snapshot(st)
    got = _block_step(dims, t, st, opts)
    torch.cuda.synchronize()
    leaf = [q.double().cpu().requires_grad_(True) for q in params]
    nw, wg, bias, w1, w3, w2 = leaf
    s = (t["x"].float() + t["delta"].float()).to(BF16).double().cpu().requires_grad_(True)
    y = s / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-6) * nw
    idx = got["idx"].long().cpu()
    sc = torch.sigmoid(y @ wg.t() + bias).gather(1, idx)
    w = 2.5 * sc / sc.sum(1, keepdim=True)
    keep = torch.from_numpy(ro.keep_mask(T * d, 6, 3, p).reshape(T, d))
    rows = []
    for i in range(T):
        acc = 0.0
        for j in range(k):
            e = int(idx[i, j])
            g, u = w1[e] @ y[i], w3[e] @ y[i]
            acc = acc + w[i, j] * (w2[e] @ (g * torch.sigmoid(g) * u))
        rows.append(acc)
    q = torch.stack(rows)
    out = s + torch.where(keep, q / (1 - p), torch.zeros_like(q))
    want = torch.autograd.grad((out * t["dout"].double().cpu()).sum(), [s] + leaf)
    assert float((got["out"].double().cpu() - out.detach()).abs().max() / out.detach().abs().max()) < 2e-2
    for name, a, b in zip(("ds", "dnorm", "dwg", "dbias", "dw1", "dw3", "dw2"), [got["ds"]] + got["grads"], want):
        err = float((a.double().cpu() - b).norm() / b.norm())
        _say(f"  {name} {err:.2e}")
        assert err < 2e-2, name
    n, fac = to.grad_norm([_np(g) for g in got["grads"]], 1.0, 1.0)
    assert abs(float(got["norm"][0]) / n - 1) < 2 * U and abs(float(got["norm"][1]) / fac - 1) < 2 * U
    if bits == 32:
        _check_step(st, was, [g.reshape(-1) for g in got["grads"]], opts, 1e-3, 1, float(got["norm"][1]), 7, 4)
    assert all(torch.equal(a, m.to(BF16)) for a, m in zip(st.params, st.master) if m is not None)


@pytest.mark.parametrize("bits", [32, 8])
def test_block_step_in_a_graph(bits):
    """Captured once, replayed over several steps with its owner's inputs, draws and schedule, against eager steps."""
    dims, t, params = _block_inputs(130, 256, 256, 8, 2, 7)
    opts = moe.AdamOptions(weight_decay=0.1, stochastic=True)
    a, b = moe.adam_state([q.clone() for q in params], bits), moe.adam_state([q.clone() for q in params], bits)
    zero = _snapshot(a)

    def reset(st, snap):
        for n, ts in snap.items():
            if ts is not None:
                for q, z in zip(getattr(st, n), ts):
                    if q is not None:
                        q.copy_(z)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _block_step(dims, t, a, opts)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _block_step(dims, t, a, opts)
    reset(a, zero)
    for it in range(4):
        _, u, _ = _block_inputs(130, 256, 256, 8, 2, 100 + it)
        u["lr_step"][0] = 1e-3 / (1 + it)
        u["lr_step"][1] = 1.0 + it
        for n in t:
            t[n].copy_(u[n])
        graph.replay()
        torch.cuda.synchronize()
        kept = [v.clone() for v in (got["out"], got["ds"], got["norm"])]
        want = _block_step(dims, u, b, opts)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(kept, (want["out"], want["ds"], want["norm"])))
        now, ref = _snapshot(a), _snapshot(b)
        for n in now:
            assert now[n] is None or all(x is None or torch.equal(x, y) for x, y in zip(now[n], ref[n])), (it, n)


def test_lr_and_step_on_the_host_or_the_device():
    """The same bits, from the first step to a far one."""
    for step in (1, 2, 10, 1000, 123457, 2 ** 40):
        st = [moe.adam_state(_params(ODD, (F32,), 2)) for _ in range(2)]
        g = _ragged(ODD, (F32,), 3)
        opts = moe.AdamOptions(weight_decay=0.1)
        moe.adam_step(opts, st[0], g, lr=2.7e-4, step=step)
        moe.adam_step(opts, st[1], g, lr_step=torch.tensor([2.7e-4, step], dtype=torch.float64, device="cuda"))
        assert all(torch.equal(a, b) for a, b in zip(st[0].params, st[1].params))
        ref = to.adam_update(_np(_params(ODD, (F32,), 2)[-2]), *to.adam_moments(_np(g[-2]), 1.0, np.zeros(20000), np.zeros(
            20000), 0.9, 0.999), 2.7e-4, step, 0.9, 0.999, 1e-8, 0.1)
        np.testing.assert_allclose(_np(st[0].params[-2]), ref, rtol=0, atol=40 * U)


def test_streams():
    """Calls on a stream of the caller's, and two steps at once on two streams, each with its own buffers."""
    dims, t, params = _block_inputs(130, 256, 256, 8, 2, 11)
    opts = moe.AdamOptions(stochastic=True)
    want = moe.adam_state([q.clone() for q in params], 8)
    ref = _block_step(dims, t, want, opts)
    torch.cuda.synchronize()
    s, r = torch.cuda.Stream(), torch.cuda.Stream()
    sts = [moe.adam_state([q.clone() for q in params], 8) for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for stream, st in zip((s, r), sts):
        with torch.cuda.stream(stream):
            got.append(_block_step(dims, t, st, opts))
    torch.cuda.synchronize()
    for g, st in zip(got, sts):
        assert torch.equal(g["out"], ref["out"]) and torch.equal(g["ds"], ref["ds"]) and torch.equal(g["norm"], ref["norm"])
        assert all(torch.equal(a, b) for a, b in zip(st.params + st.m + st.v, want.params + want.m + want.v))
    y, z, _, q = moe.norm_forward(dims, NORM, t["x"], params[0], residual=t["delta"], keep=True, stream=s)
    dx, dw, _ = moe.norm_backward(dims, NORM, t["dout"], z, params[0], q, stream=s)
    n = moe.grad_norm([dw], stream=s)
    st = moe.adam_state([params[0].clone()])
    s.wait_stream(torch.cuda.current_stream())
    moe.adam_step(moe.AdamOptions(), st, [dw], lr=1e-3, step=1, gscale=n[1:], stream=s)
    s.synchronize()
    a = moe.norm_forward(dims, NORM, t["x"], params[0], residual=t["delta"], keep=True)
    b = moe.norm_backward(dims, NORM, t["dout"], a[1], params[0], a[3])
    assert torch.equal(a[0], y) and torch.equal(b[0], dx) and torch.equal(b[1], dw)
    two = moe.adam_state([params[0].clone()])
    moe.adam_step(moe.AdamOptions(), two, [dw], lr=1e-3, step=1, gscale=moe.grad_norm([dw])[1:])
    assert torch.equal(two.params[0], st.params[0])


def test_gpu_refusals():
    dims, opts = moe.Dims(4, 64, 64, 8, 2), moe.NormOptions()
    x = torch.zeros((4, 64), dtype=BF16, device="cuda")
    f = torch.zeros(4, device="cuda")
    with pytest.raises(ValueError, match="dtype"):
        moe.norm_forward(dims, opts, x.float())
    with pytest.raises(ValueError, match="shape"):
        moe.norm_forward(dims, opts, x, torch.zeros(32, device="cuda"))
    with pytest.raises(ValueError, match="dtype"):
        moe.norm_forward(dims, opts, x, torch.zeros(64, dtype=BF16, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        moe.norm_forward(dims, opts, torch.zeros((64, 4), dtype=BF16, device="cuda").t())
    with pytest.raises(ValueError, match="is on cpu"):
        moe.norm_forward(dims, opts, x, torch.zeros(64))
    with pytest.raises(ValueError, match="residual"):
        moe.norm_forward(dims, opts, x, sum=x)
    with pytest.raises(moe.MoeError):
        moe.norm_forward(dims, opts, x, bias=torch.zeros(64, device="cuda"))        # an RMS norm has none
    with pytest.raises(moe.MoeError):
        moe.norm_forward(dims, opts, x, residual=x, sum=x, y=x)
    with pytest.raises(moe.MoeError):
        moe.norm_forward(dims, moe.NormOptions(eps=0.0), x)
    with pytest.raises(moe.MoeError):
        moe.norm_forward(moe.Dims(4, 60, 64, 8, 2), opts, torch.zeros((4, 60), dtype=BF16, device="cuda"))
    with pytest.raises(moe.MoeError):
        moe.norm_backward(dims, moe.NormOptions("layer"), x, x, None, f)            # a layer norm's mean is missing
    with pytest.raises(moe.MoeError):
        moe.norm_backward(dims, opts, x, x, None, f, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    g = [torch.zeros(8, device="cuda")]
    with pytest.raises(moe.MoeError):
        moe.grad_norm(g, math.inf)
    with pytest.raises(moe.MoeError):
        moe.grad_norm(g, 1.0, -1.0)
    with pytest.raises(moe.MoeError):
        moe.grad_norm([torch.zeros(1 << 20, device="cuda")], ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="is on cpu"):
        moe.grad_norm(g + [torch.zeros(4)])
    st = moe.adam_state([torch.zeros(8, device="cuda")])
    o = moe.AdamOptions()
    with pytest.raises(moe.MoeError):
        moe.adam_step(o, st, [torch.zeros(9, device="cuda")], lr=1e-3, step=1)
    with pytest.raises(moe.MoeError):
        moe.adam_step(o, st, g, lr=1e-3, step=0)
    with pytest.raises(moe.MoeError):
        moe.adam_step(moe.AdamOptions(beta2=1.0), st, g, lr=1e-3, step=1)
    with pytest.raises(moe.MoeError):
        moe.adam_step(o, st, [st.m[0]], lr=1e-3, step=1)
    with pytest.raises(ValueError, match="lr_step"):
        moe.adam_step(o, st, g, lr_step=torch.zeros(2, device="cuda"))
    with pytest.raises(ValueError, match="gscale"):
        moe.adam_step(o, st, g, lr=1e-3, step=1, gscale=torch.zeros(2, device="cuda"))
    with pytest.raises(ValueError, match="is on cpu"):
        moe.adam_step(o, st, [torch.zeros(8)], lr=1e-3, step=1)
