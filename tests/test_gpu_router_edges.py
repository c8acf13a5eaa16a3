"""Inputs at the edge of what the scored router's calls accept, against the float64
oracle (oracle/router_oracle.py) and the formulas: keys made of biases that cancel,
weights below fp32's normal range, gradients that are not finite or of extreme
size, infinities in the gate's operands, terms that cancel. Index arrays must be
equal; u = 2^-24 is fp32's half step, 2^-8 bf16's, and each test derives its bound
from them.
"""
import math
import sys

import numpy as np
import pytest
import torch

import mixture_experts_layer_gate_amd as moe
from oracle import router_oracle as ro

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
INF, NAN = math.inf, math.nan


def _say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def _opts(spec):
    return moe.RouteOptions(spec.score, spec.groups, spec.topk_groups, spec.group_rule, spec.renormalise, spec.scale)


def _gpu(*arrays):
    return [None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]


# ---------------------------------------------------------------- selection ----
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,per,kept", [(4, 2, 2), (4, 2, 1), (4, 2, 3), (8, 4, 4), (16, 2, 6), (64, 2, 20), (8, 32, 4)])
def test_group_keys_of_biases_that_cancel(groups, per, kept, score, rng):
    """Top-2 group keys 1e-5 to 1e-3 apart, those of one group in four made of biases of +-1000 (or +-2^20) that
    cancel: such a key is inexact in fp32 by far more than its neighbours', wherever it ranks."""
    T, E, k = 512, groups * per, min(4, kept * per)
    _say(f"cancelling biases: {groups} groups of {per}, {kept} kept, {score}")
    for rep in range(6):
        l = (10.0 ** (-5 + rep // 2) * rng.standard_normal((T, E))).astype(np.float32)
        b = np.zeros(E, np.float32)
        for g in rng.permutation(groups)[:max(1, groups // 4)]:
            at = g * per + rng.permutation(per)[:2]
            big = 1000.0 if rep % 2 == 0 else 2.0 ** 20
            b[g * per:(g + 1) * per] = -2.0 * big
            b[at] = big, -big
        spec = ro.RouteSpec(score, groups, kept, "top2", True, 1.0)
        tl, tb = _gpu(l, b)
        idx, w = moe.route_select(moe.Dims(T, 64, 64, E, k), _opts(spec), tl, tb)
        want_i, want_w = ro.select(l, b, k, spec)
        np.testing.assert_array_equal(idx.cpu().numpy(), want_i)
        # each weight a ratio of exponentials of differences below 1: (1 + 32) u
        np.testing.assert_allclose(w.cpu().numpy(), want_w, rtol=33 * U)


@pytest.mark.parametrize("scale", [1.0, 2.0 ** 20])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_weights_below_the_normal_range(score, renorm, scale, rng):
    """Scores from 2^-110 down to nothing: within 2^-126 of a score (its weight within that times the scale), and
    where such a weight has become 0 its gradient is 0 too."""
    T, E, k = 40, 16, 4
    l = -(76.0 + rng.random((T, E)) * 40.0).astype(np.float32)
    if score == "softmax" or renorm:
        l[:, 0] = 0.0  # the scores, or their quotients by the largest, are as small as before
    spec = ro.RouteSpec(score, renormalise=renorm, scale=scale)
    tl, = _gpu(l)
    dims = moe.Dims(T, 64, 64, E, k)
    idx, w = moe.route_select(dims, _opts(spec), tl)
    want_i, want_w = ro.select(l, None, k, spec)
    np.testing.assert_array_equal(idx.cpu().numpy(), want_i)
    w32 = w.cpu().numpy()
    # (spread + 32) u, the spread of the logits up to 116; a quotient is by a sum of at least 0.5
    np.testing.assert_allclose(w32, want_w, rtol=148 * U, atol=2.0 * scale * 2.0 ** -126)
    dl = moe.route_select_backward(dims, _opts(spec), tl, idx, w, torch.ones_like(w).cumsum(1)).cpu().numpy()
    assert np.isfinite(dl).all()
    if not (score == "softmax" and not renorm):  # (whose every logit takes part in the sum)
        assert not np.take_along_axis(dl, want_i, axis=1)[w32 == 0].any()


# ---------------------------------------------------------------- gradients ----
@pytest.mark.parametrize("E", [6, 70, 300])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_non_finite_gradients_of_the_losses_show(value, score, renorm, E, rng):
    """A z loss whose gradient is NaN or infinite gives that to every expert of the rows it covers, so that an
    overflow is seen; the rows outside every sequence keep the selection's gradient alone."""
    T, k = 9, 2
    l = (1.0 + 0.1 * rng.standard_normal((T, E))).astype(np.float32)  # log-sum-exp above 0, no share below 1e-3
    spec = ro.RouteSpec(score, renormalise=renorm)
    tl, tseq = _gpu(l, np.array([0, 4, 7], np.int32))
    dims, opts = moe.Dims(T, 64, 64, E, k), _opts(spec)
    idx, w = moe.route_select(dims, opts, tl)
    _, load = moe.balance_loss(dims, opts, tl, idx, tseq)
    dw = torch.ones((T, k), device="cuda").cumsum(1)
    up = torch.tensor([0.5, value], device="cuda")
    got = moe.route_select_backward(dims, opts, tl, idx, w, dw, up, load, tseq).cpu()
    alone = moe.route_select_backward(dims, opts, tl, idx, w, dw).cpu()
    assert torch.equal(got[7:], alone[7:])
    assert bool(torch.isnan(got[:7]).all() if value != value else (got[:7] == value).all())
    # the balance loss's: NaN, by the formula (inf - inf)
    up = torch.tensor([value, 0.5], device="cuda")
    got = moe.route_select_backward(dims, opts, tl, idx, w, dw, up, load, tseq).cpu()
    assert bool(torch.isnan(got[:7]).all()) and torch.equal(got[7:], alone[7:])


@pytest.mark.parametrize("E", [8, 90, 600])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("value", [NAN, INF])
def test_masked_experts_get_no_gradient_whatever_comes_in(value, score, renorm, E, rng):
    """Logits of -inf or NaN: gradient 0 there, also where dtopk_w or dlosses are not finite."""
    T, k = 6, 3
    l = rng.standard_normal((T, E)).astype(np.float32)
    dead = rng.random((T, E)) < 0.4
    dead[:, :k] = False  # three experts of every row are in the choice
    l[dead] = np.where(rng.random((T, E)) < 0.5, -INF, NAN)[dead]
    tl, = _gpu(l)
    dims, opts = moe.Dims(T, 64, 64, E, k), moe.RouteOptions(score, renormalise=renorm)
    idx, w = moe.route_select(dims, opts, tl)
    _, load = moe.balance_loss(dims, opts, tl, idx)
    dw = torch.ones((T, k), device="cuda")
    for up in ([value, 0.0], [0.0, value], [value, value]):
        up = torch.tensor(up, device="cuda")
        got = moe.route_select_backward(dims, opts, tl, idx, w, dw, up, load).cpu().numpy()
        assert not got[dead].any()
        got = moe.route_select_backward(dims, opts, tl, None, None, None, up, load).cpu().numpy()
        assert not got[dead].any()
    got = moe.route_select_backward(dims, opts, tl, idx, w, value * dw).cpu().numpy()
    assert not got[dead].any() and not np.isfinite(got).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("scale,k", [(2.0 ** -147, 4)] + [
    (scale, k) for scale in (2.0 ** -140, -(2.0 ** -130), 2.0 ** 100, 2.0 ** 127) for k in (4, 128)])
def test_gradient_of_weights_of_any_scale(scale, score, k):
    """k equal experts share the scale exactly; dw is scaled so that the gradients w_j (dw_j - mean dw) are
    ordinary numbers, while 1 / scale is not one where the scale is below 2^-128."""
    T, E = 5, 300
    w_one, unit = scale / k, 2.0 ** -math.frexp(scale / k)[1]
    unit = min(max(unit, 2.0 ** -100), 2.0 ** 100)
    l = np.full((T, E), -3.0, np.float32)
    l[:, :k] = 0.5
    tl, = _gpu(l)
    dims, opts = moe.Dims(T, 64, 64, E, k), moe.RouteOptions(score, renormalise=True, scale=scale)
    idx, w = moe.route_select(dims, opts, tl)
    # softmax: the scale over k, exactly. Sigmoid: s (scale / (k s)), where k s is exact and the quotient and the
    # product round once each: 2 u of the weight, or half a step of 2^-149 each below the normal range
    off = 0.0 if score == "softmax" else 2 * U * (1 + U) * abs(w_one) + 2.0 ** -149
    w64 = w.cpu().double().numpy()
    assert idx.tolist() == [list(range(k))] * T and (np.abs(w64 - w_one) <= off).all()
    dw = unit * (np.arange(T)[:, None] + np.arange(k)[None, :] % 5).astype(np.float32)
    got = moe.route_select_backward(dims, opts, tl, idx, w, _gpu(dw)[0]).cpu().double().numpy()
    d64 = dw.astype(np.float64)
    want = w64 * ((w64 / scale)[:, None, :] * (d64[:, :, None] - d64[:, None, :])).sum(axis=2)
    if score == "sigmoid":
        want = want / (1.0 + math.exp(0.5))
    # k terms, each a difference below 5 unit, times the weight and 1 - s: (k + 16) u of the largest
    assert (np.abs(got[:, :k] - want) <= (k + 16) * U * 5 * unit * abs(w_one) + 2.0 ** -149).all()
    assert not got[:, k:].any()


@pytest.mark.parametrize("E", [60, 600])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("power", [120, -110])
def test_gradient_of_the_balance_loss_is_linear_in_its_own(power, score, E, rng):
    """A dlosses[0] of 2^120 or 2^-110, whose product with E leaves fp32's range or whose quotient by the rows'
    square loses bits below 2^-126: the gradient of dlosses[0] = 1 times that, bit for bit but for denormals."""
    T, k = 5000, 1
    l = rng.standard_normal((T, E)).astype(np.float32)
    tl, = _gpu(l)
    dims, opts = moe.Dims(T, 64, 64, E, k), moe.RouteOptions(score)
    idx, w = moe.route_select(dims, opts, tl)
    _, load = moe.balance_loss(dims, opts, tl, idx)

    def grad(up):
        up = torch.tensor([up, 0.0], device="cuda")
        return moe.route_select_backward(dims, opts, tl, None, None, None, up, load).double()
    one, far = grad(1.0), grad(2.0 ** power) * 2.0 ** -power
    # powers of two commute with rounding; a sum of E terms and two products below 2^-126 are off by 2^-149 each
    assert bool(((far - one).abs() <= (E + 8) * 2.0 ** (-149 - power)).all() if power < 0 else torch.equal(far, one))


BF = 2.0 ** -8


def _agree(got, want, tol):
    """NaN and infinities (of the same sign) in the same places, the finite rest within tol. A value past the
    output type's range is an infinity of it: bf16's ends at 3.396e38, where its largest number 3.3895e38 (255 steps
    of 2^120) and half a step more round up, fp32's at 3.403e38."""
    got, near = got.double().cpu(), want.to(got.dtype).double()
    assert torch.equal(torch.isnan(got), torch.isnan(near))
    inf = torch.isinf(near)
    assert torch.equal(got[inf], near[inf])
    fin = torch.isfinite(near)
    assert bool(((got - want).abs()[fin] <= tol[fin]).all())


@pytest.mark.parametrize("with_in", [True, False])
@pytest.mark.parametrize("shape", [(40, 64, 6), (700, 264, 20), (33, 136, 65), (900, 520, 130), (1300, 2056, 70)],
                         ids=lambda s: "T{}_d{}_E{}".format(*s))
def test_gate_backward_of_infinities_in_x_and_wg(shape, with_in, rng):
    """x and Wg holding infinities, NaN and values whose products overflow go where the formula sends them,
    whatever bits of dlogits meet them (1, -1, 0, all 24 bits, denormals); everything else keeps its bounds."""
    T, d, E = shape
    _say(f"gate_backward, infinities in x and wg: {shape} dx_in={with_in}")
    bf = torch.bfloat16
    x = rng.standard_normal((T, d)).astype(np.float32)
    wg = rng.standard_normal((E, d)).astype(np.float32)
    dl = (rng.standard_normal((T, E)) * 10.0 ** rng.uniform(-6, 2, (T, E))).astype(np.float32)
    values = [INF, -INF, NAN, 3.0e38, -3.0e38]
    # one special value to a column, so that no two of them cancel
    for c, v in zip(rng.permutation(d)[:20], values * 4):
        t = int(rng.integers(T))
        x[t, c] = v
        dl[t, :4] = 1.0, -1.0, 0.0, 2.0 ** -140
        dl[t, 4:6] = 16777215.0, -16777215.0 * 2.0 ** -40
    for c, v in zip(rng.permutation(d)[:20], values * 4):
        e = int(rng.integers(E))
        wg[e, c] = v
        dl[rng.permutation(T)[:4], e] = 1.0, -1.0, 0.0, 2.0 ** -140
    x, wg, dl = (torch.from_numpy(v).cuda() for v in (x, wg, dl))
    x, wg = x.to(bf), wg.to(bf)
    dx_in = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).cuda().to(bf) if with_in else None
    if with_in:
        dx_in[T // 2, 3] = INF
    X, W, D = (v.double().cpu() for v in (x, wg, dl))
    I = torch.zeros((T, d), dtype=torch.float64) if dx_in is None else dx_in.double().cpu()
    dx, dwg, _ = moe.gate_backward(moe.Dims(T, d, 64, E, 1), x, wg, dl, dx_in, dx=dx_in)
    # fp32 sums of exact products; dx from dlogits within 2^-16 of each term (test_gate_backward's bounds). The
    # planes of dlogits are bf16, whose smallest step is 2^-133: a dlogits of fewer bits than that (2^-140, a
    # denormal) is off by half of it at most, 2^-134 times the x or Wg beside it
    step = 2.0 ** -134
    _agree(dwg, D.t() @ X, (T + 8) * U * (D.abs().t() @ X.abs()) + step * X.abs().sum(0))
    want = I + D @ W
    _agree(dx, want, BF * want.abs() + (2.0 ** -16 * (1 + BF) + (E + 8) * U) * (D.abs() @ W.abs()) + 4 * U * I.abs()
           + (1 + BF) * step * W.abs().sum(0))


@pytest.mark.parametrize("shape", [(40, 64, 8), (200, 264, 70), (700, 520, 130)], ids=lambda s: "T{}_d{}_E{}".format(*s))
def test_gate_backward_of_terms_that_cancel(shape, rng):
    """Experts in pairs of the same Wg whose logit gradients nearly cancel: dx within 2^-16 of each term, as the
    header has it (in the mean far less), and exact where dlogits has 16 bits; dWg's sums from all 24 bits."""
    T, d, E = shape
    _say(f"gate_backward, cancelling terms: {shape}")
    bf = torch.bfloat16
    x = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).cuda().to(bf)
    wg = rng.standard_normal((E // 2, d)).astype(np.float32).repeat(2, axis=0)
    wg = torch.from_numpy(wg).cuda().to(bf)
    a = rng.standard_normal((T, E // 2)).astype(np.float32)
    for part in (2.0 ** -12, 2.0 ** -20):
        b = (-a * (1.0 + part * rng.standard_normal(a.shape))).astype(np.float32)
        dl = torch.from_numpy(np.stack([a, b], axis=2).reshape(T, E)).cuda()
        dx, dwg, _ = moe.gate_backward(moe.Dims(T, d, 64, E, 1), x, wg, dl)
        X, W, D = (v.double().cpu() for v in (x, wg, dl))
        want, mag = D @ W, D.abs() @ W.abs()
        _agree(dx, want, BF * want.abs() + (2.0 ** -16 * (1 + BF) + (E + 8) * U) * mag)
        _agree(dwg, D.t() @ X, (T + 8) * U * (D.abs().t() @ X.abs()))
    # dlogits of 16 bits, and every pair equal and opposite: nothing is left
    b = torch.from_numpy(a).cuda()
    b = (b.view(torch.int32) & ~0xFF).view(torch.float32)
    dl = torch.stack([b, -b], dim=2).reshape(T, E).contiguous()
    dx, _, _ = moe.gate_backward(moe.Dims(T, d, 64, E, 1), x, wg, dl)
    want, mag = torch.zeros((T, d), dtype=torch.float64), dl.double().cpu().abs() @ W.abs()
    _agree(dx, want, (E + 8) * U * mag)
