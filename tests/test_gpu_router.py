"""Scored router, balance losses, their gradients, gate gradients and dropout
beside the combine, through the C ABI, against the float64 oracle
(oracle/router_oracle.py).

Tolerances. u = 2^-24 is fp32's half step. A score or share is a few fp32
operations on exp of a difference of logits: the difference's own rounding is
worth u |difference| <= u R relatively (R the row's spread of finite logits, at
most 104 before exp is 0), and the exponential, sums over a wave (6 levels and
up to 16 terms in a lane) and the division another 32 u at most; REL(R) = (R +
32) u. Sums add (terms) u. bf16 outputs add 2^-8 of the value. Index arrays,
loads and keep decisions must be equal.
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
BF = 2.0 ** -8
INF, NAN = math.inf, math.nan


def _say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def _spread(logits):
    f = logits[np.isfinite(logits) & (np.abs(logits) < 1e30)]
    return min(104.0, float(f.max() - f.min())) if f.size else 0.0


def _rel(logits):
    return (_spread(logits) + 32) * U


def _guarded(shape, dtype, pad=64):
    """A contiguous tensor inside a larger buffer of sentinels, and a check that those are left alone."""
    n = int(np.prod(shape))
    buf = torch.full((n + 2 * pad,), 77, dtype=dtype, device="cuda")

    def check():
        assert bool((buf[:pad] == 77).all()) and bool((buf[pad + n:] == 77).all())
    return buf[pad:pad + n].view(shape), check


def _opts(spec):
    return moe.RouteOptions(spec.score, spec.groups, spec.topk_groups, spec.group_rule, spec.renormalise, spec.scale)


def _logits(rng, T, E, kind):
    l = (1.25 * rng.standard_normal((T, E))).astype(np.float32)
    if kind == "masked":
        l[rng.random((T, E)) < 0.2] = -INF
        l[rng.random((T, E)) < 0.05] = NAN
        l[rng.random((T, E)) < 0.05] = np.finfo(np.float32).min
        l[rng.random((T, E)) < 0.02] = INF
        l[0] = -INF
        if T > 2:
            l[1] = NAN
            l[2] = np.finfo(np.float32).min
        if T > 3:
            l[3] = -INF
            l[3, E // 2] = -4.0
    if kind == "tied":
        l = np.round(l)
    if kind == "large":
        l *= 40.0
    if kind == "negative":
        l = l - 300.0
    return l.astype(np.float32)


SELECT = [
    # T, E, k, score, groups, kept, rule, renorm, scale, bias, logits
    (1, 256, 8, "sigmoid", 8, 4, "top2", True, 2.5, "small", "plain"),
    (1, 1, 1, "softmax", 1, 1, "max", True, 1.0, None, "plain"),
    (3, 2, 2, "sigmoid", 1, 1, "max", False, 1.0, None, "plain"),
    (256, 8, 2, "softmax", 1, 1, "max", True, 1.0, None, "plain"),
    (257, 256, 8, "sigmoid", 8, 4, "top2", True, 2.5, "small", "plain"),
    (130, 256, 8, "softmax", 8, 3, "max", False, 16.0, "small", "plain"),
    (65, 250, 6, "softmax", 1, 1, "max", False, 16.0, "masked", "plain"),
    (64, 160, 6, "softmax", 8, 3, "max", True, 1.0, None, "masked"),
    (64, 96, 5, "sigmoid", 4, 2, "top2", True, 2.5, "masked", "masked"),
    (40, 60, 4, "sigmoid", 1, 1, "max", True, 1.0, "small", "tied"),
    (40, 64, 8, "softmax", 16, 5, "top2", True, 1.0, None, "tied"),
    (33, 65, 7, "sigmoid", 5, 2, "top2", False, 1.0, "small", "large"),
    (33, 129, 8, "softmax", 1, 1, "max", True, 1.0, "small", "large"),
    (20, 72, 8, "sigmoid", 1, 1, "max", True, 1.0, None, "negative"),
    (20, 72, 8, "sigmoid", 9, 4, "max", True, 1.0, "small", "negative"),
    (7, 300, 9, "softmax", 4, 3, "top2", True, 1.0, "small", "plain"),
    (5, 513, 40, "sigmoid", 1, 1, "max", False, 1.0, "small", "plain"),
    (4, 1024, 1024, "softmax", 1, 1, "max", True, 1.0, None, "plain"),
    (4, 1024, 8, "sigmoid", 64, 7, "top2", True, 2.5, "small", "masked"),
    (9, 64, 3, "sigmoid", 64, 5, "top2", True, 1.0, "small", "plain"),
    (70, 256, 12, "softmax", 1, 1, "max", True, 1.0, "inf", "plain"),
    (70, 128, 8, "sigmoid", 1, 1, "max", True, 0.0, "small", "plain"),
    (50, 40, 8, "softmax", 1, 1, "max", True, 1.0, None, "tied"),
    (50, 200, 8, "softmax", 4, 4, "max", True, 1.0, None, "masked"),
    (300, 16, 4, "softmax", 1, 1, "max", False, 1.0, None, "plain"),
    (300, 30, 6, "sigmoid", 3, 2, "top2", True, 1.0, "masked", "plain"),
    (90, 128, 8, "sigmoid", 8, 3, "max", True, 1.0, "big", "plain"),
    (90, 200, 5, "softmax", 1, 1, "max", False, 1.0, "big", "plain"),
    (64, 256, 8, "softmax", 2, 1, "top2", True, 1.0, "small", "plain"),
    (64, 99, 3, "sigmoid", 33, 20, "max", True, 1.0, "small", "plain"),
]


def _bias(rng, E, kind):
    if kind is None:
        return None
    b = (0.05 * rng.standard_normal(E)).astype(np.float32)
    if kind == "masked":
        b[rng.permutation(E)[:max(1, E // 10)]] = -INF
        b[rng.integers(E)] = NAN
    if kind == "inf":
        b[rng.permutation(E)[:3]] = INF
    if kind == "big":  # fp32 keys would round to steps of 2^-14 (or 2^-4 above 2^20)
        b = (1000.0 + 0.01 * rng.standard_normal(E)).astype(np.float32)
        b[:2] += 2.0 ** 20
    return b


@pytest.mark.parametrize("case", SELECT, ids=lambda c: "T{}_E{}_k{}_{}_g{}-{}{}_n{:d}_b{}_{}".format(
    c[0], c[1], c[2], c[3], c[4], c[5], c[6], c[7], c[9], c[10]))
def test_select(case, rng):
    T, E, k, score, groups, kept, rule, renorm, scale, bkind, lkind = case
    _say(f"select {case}")
    spec = ro.RouteSpec(score, groups, kept, rule, renorm, scale)
    l, b = _logits(rng, T, E, lkind), _bias(rng, E, bkind)
    idx, check_i = _guarded((T, k), torch.int32)
    w, check_w = _guarded((T, k), torch.float32)
    dims = moe.Dims(T, 64, 64, E, k)
    moe.route_select(dims, _opts(spec), torch.from_numpy(l).cuda(), None if b is None else torch.from_numpy(b).cuda(),
                     topk_idx=idx, topk_w=w)
    torch.cuda.synchronize()
    check_i()
    check_w()
    want_i, want_w = ro.select(l, b, k, spec)
    np.testing.assert_array_equal(idx.cpu().numpy(), want_i)
    # below fp32's normal range a weight has only absolute precision
    np.testing.assert_allclose(w.cpu().numpy(), want_w, rtol=_rel(l), atol=abs(scale) * 2.0 ** -126)


def test_select_many_near_ties(rng):
    """Keys a few 1e-9 apart, far inside fp32's resolution of a score: the order is the float64 one."""
    T, E, k = 64, 256, 8
    l = rng.standard_normal((T, E)).astype(np.float32)
    s = 1.0 / (1.0 + np.exp(-l.astype(np.float64)))
    # a bias that brings expert e of row 0 near 0.9, up to 3e-9 (fp32 steps there are 6e-8)
    b = (0.9 - s[0] + 3e-9 * rng.standard_normal(E)).astype(np.float32)
    l[:] = l[0]
    spec = ro.RouteSpec("sigmoid", 8, 4, "top2", True, 2.5)
    idx, _ = moe.route_select(moe.Dims(T, 64, 64, E, k), _opts(spec), torch.from_numpy(l).cuda(),
                              torch.from_numpy(b).cuda())
    want, _ = ro.select(l[:1], b, k, spec)
    np.testing.assert_array_equal(idx.cpu().numpy(), np.repeat(want, T, axis=0))
    for groups, kept in ((1, 1), (8, 5)):
        spec = ro.RouteSpec("softmax", groups, kept, "max", True, 1.0)
        z = np.exp(l[0].astype(np.float64))
        b = (0.9 - z / z.sum() + 3e-9 * rng.standard_normal(E)).astype(np.float32)
        idx, _ = moe.route_select(moe.Dims(T, 64, 64, E, k), _opts(spec), torch.from_numpy(l).cuda(),
                                  torch.from_numpy(b).cuda())
        want, _ = ro.select(l[:1], b, k, spec)
        np.testing.assert_array_equal(idx.cpu().numpy(), np.repeat(want, T, axis=0))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 8])
@pytest.mark.parametrize("E", [64, 120, 256, 1024])
@pytest.mark.parametrize("kind", ["one small class", "few values", "one value", "opposite biases"])
def test_select_rows_with_many_candidates(kind, E, groups, score, rng):
    """Rows whose largest keys do not stand out by residues of the expert, are equal, or come from biases that cancel."""
    T, k = 24, 8
    l, b = rng.standard_normal((T, E)).astype(np.float32), None
    if kind == "one small class":
        for t in range(T):
            l[t, t % 8::8] = -30.0 - t
        l[::3, :] += 25.0 * (np.arange(E) < 3)  # fewer far above than are chosen
    elif kind == "few values":
        l = np.round(2.0 * l) / 2.0
    elif kind == "one value":
        l[:] = 0.25
        l[1::2, E // 2] = 0.5
    else:
        b = np.where(np.arange(E) % 2 == 0, 300.0, -300.0).astype(np.float32)
        b += (1e-3 * rng.integers(0, 2, E)).astype(np.float32)
        l *= 1e-3
    for bias in (b, np.zeros(E, np.float32) if b is None else -b):
        spec = ro.RouteSpec(score, groups, max(1, groups // 2), "top2" if groups > 1 else "max", True, 1.0)
        idx, w = moe.route_select(moe.Dims(T, 64, 64, E, k), _opts(spec), torch.from_numpy(l).cuda(),
                                  None if bias is None else torch.from_numpy(bias).cuda())
        want_i, want_w = ro.select(l, bias, k, spec)
        np.testing.assert_array_equal(idx.cpu().numpy(), want_i)
        np.testing.assert_allclose(w.cpu().numpy(), want_w, rtol=_rel(l), atol=2.0 ** -126)


def test_select_large_batch_against_torch():
    """A batch of many workgroups: the choice and weights of every row against float64 sorts."""
    T, E, k = 20011, 250, 6
    gen = torch.Generator(device="cuda").manual_seed(3)
    l = torch.randn((T, E), generator=gen, device="cuda")
    b = 0.02 * torch.randn(E, generator=gen, device="cuda")
    idx, w = moe.route_select(moe.Dims(T, 64, 64, E, k), moe.RouteOptions("sigmoid", scale=2.0), l, b)
    s = 1.0 / (1.0 + torch.exp(-l.double()))
    want = torch.sort(s + b.double(), dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(idx.long(), want)
    sel = s.gather(1, want)
    torch.testing.assert_close(w.double(), 2.0 * sel / sel.sum(1, keepdim=True), rtol=48 * U, atol=0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [0, 1, 70])
def test_route_scored_logits_are_routes(dtype, T, rng):
    d, E, k = 136, 24, 3
    dims = moe.Dims(T, d, 64, E, k, dtype)
    x = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).cuda().to(dtype)
    wg = torch.from_numpy(rng.standard_normal((E, d)).astype(np.float32) / math.sqrt(d)).cuda().to(dtype)
    bias = torch.from_numpy(0.1 * rng.standard_normal(E).astype(np.float32)).cuda()
    bb = torch.from_numpy(0.05 * rng.standard_normal(E).astype(np.float32)).cuda()
    spec = ro.RouteSpec("sigmoid", 4, 2, "top2", True, 2.5)
    l, idx, w = moe.route_scored(dims, _opts(spec), x, wg, bias, bb)
    if T == 0:
        assert l.shape == (0, E) and idx.shape == (0, k)
        return
    ref, _, _ = moe.route(dims, x, wg, bias)
    assert torch.equal(l, ref)
    want_i, want_w = ro.select(l.cpu().numpy(), bb.cpu().numpy(), k, spec)
    np.testing.assert_array_equal(idx.cpu().numpy(), want_i)
    np.testing.assert_allclose(w.cpu().numpy(), want_w, rtol=_rel(l.cpu().numpy()))


def test_softmax_choice_is_routes(rng):
    """Softmax, renormalised, no bias: the plain router's choice, and its weights."""
    T, d, E, k = 300, 128, 16, 4
    dims = moe.Dims(T, d, 64, E, k)
    x = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).cuda().bfloat16()
    wg = torch.from_numpy(rng.standard_normal((E, d)).astype(np.float32) / math.sqrt(d)).cuda().bfloat16()
    _, i0, w0 = moe.route(dims, x, wg)
    _, i1, w1 = moe.route_scored(dims, moe.RouteOptions(), x, wg)
    assert torch.equal(i0, i1)
    torch.testing.assert_close(w0, w1, rtol=96 * U, atol=0)


GRAD = [
    # T, E, k, score, renorm, scale, offsets (None: one sequence), logits, with dw, with losses
    (1, 4, 1, "softmax", True, 1.0, None, "plain", True, True),
    (1, 256, 8, "sigmoid", True, 2.5, None, "plain", True, True),
    (33, 60, 4, "softmax", True, 1.0, [0, 10, 10, 33], "plain", True, True),
    (50, 16, 4, "softmax", False, 2.0, [0, 50], "plain", True, True),
    (50, 250, 6, "sigmoid", False, 2.5, [0, 7, 50], "plain", True, True),
    (48, 96, 5, "sigmoid", True, 2.5, [4, 20, 40], "masked", True, True),
    (48, 96, 5, "softmax", False, 1.0, [4, 20, 40], "masked", True, True),
    (48, 96, 5, "softmax", True, 1.0, [0, 48], "masked", True, False),
    (20, 72, 8, "sigmoid", True, 1.0, [0, 20], "negative", True, True),
    (40, 65, 7, "softmax", True, 1.0, [0, 0, 0], "plain", True, True),
    (17, 8, 8, "sigmoid", False, 1.0, [0, 5, 17], "plain", False, True),
    (5, 1024, 16, "softmax", False, 1.0, [0, 2, 5], "plain", True, True),
    (6, 400, 70, "sigmoid", True, 1.0, [0, 6], "plain", True, True),
    (90, 1, 1, "softmax", False, 1.0, [0, 90], "plain", True, True),
    (130, 128, 2, "sigmoid", True, 1.0, list(range(131)), "plain", True, True),
]


@pytest.mark.parametrize("case", GRAD, ids=lambda c: "T{}_E{}_k{}_{}_n{:d}_{}_{}".format(
    c[0], c[1], c[2], c[3], c[4], "one" if c[6] is None else len(c[6]) - 1, c[7]))
def test_losses_and_gradient(case, rng):
    T, E, k, score, renorm, scale, seqs, lkind, with_dw, with_losses = case
    _say(f"grad {case}")
    spec = ro.RouteSpec(score, renormalise=renorm, scale=scale)
    l = _logits(rng, T, E, lkind)
    idx, w = ro.select(l, None, k, spec)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    if lkind == "masked":
        dw[w == 0] = NAN  # a slot out of the choice passes nothing on
    w32 = w.astype(np.float32)
    up = np.array([0.8, 0.05], np.float32)
    offs = [0, T] if seqs is None else seqs
    dims, opts = moe.Dims(T, 64, 64, E, k), _opts(spec)
    tl, ti, tw, tdw, tup = (torch.from_numpy(np.ascontiguousarray(v)).cuda() for v in (l, idx, w32, dw, up))
    tseq = None if seqs is None else torch.tensor(seqs, dtype=torch.int32, device="cuda")
    load, check_f = _guarded((len(offs) - 1, E), torch.int32)
    losses, load = moe.balance_loss(dims, opts, tl, ti, tseq, load=load)
    dl, check_d = _guarded((T, E), torch.float32)
    moe.route_select_backward(dims, opts, tl, ti, tw, tdw if with_dw else None, tup if with_losses else None,
                              load if with_losses else None, tseq if with_losses else None, dlogits=dl)
    torch.cuda.synchronize()
    check_f()
    check_d()
    want_l, want_f = ro.balance_losses(l, idx, offs, spec)
    np.testing.assert_array_equal(load.cpu().numpy(), want_f)
    rel = _rel(l) + T * U
    # lse: its own rounding is u |lse|, twice in the square; cancelling logits leave an absolute error
    big = float(np.abs(l[np.isfinite(l)]).max()) if np.isfinite(l).any() else 0.0
    # the output is fp32: a mean square past its largest value (rows of the lowest or largest logit,
    # lse = 3.4e38, squared 1.2e77) is inf there, as rounding the exact value to fp32 gives
    with np.errstate(over="ignore"):
        want_l = want_l.astype(np.float32)
    np.testing.assert_allclose(losses.cpu().numpy(), want_l, rtol=4 * rel, atol=1e-30)
    want = ro.select_backward(l, idx, w32.astype(np.float64), dw if with_dw else None, spec,
                              up if with_losses else None, want_f if with_losses else None, offs)
    # magnitude of the terms each element is made of
    mag = np.zeros((T, E))
    S = len(offs) - 1
    filled = sum(offs[s + 1] > offs[s] for s in range(S))
    for t in range(T):
        c = ro._clean(l[t])
        s = np.array(ro.scores(c, score))
        p = np.array(ro.scores(c, "softmax"))
        if with_dw:
            on = [j for j in range(k) if w32[t, j] != 0]
            D = sum(abs(float(w32[t, j] * dw[t, j])) for j in on)
            for j in on:
                mag[t, idx[t, j]] += abs(w32[t, j]) * (abs(dw[t, j]) + (D / scale if renorm else 0))
            if score == "softmax" and not renorm:
                mag[t] += s * D
        if with_losses:
            sid = next((q for q in range(S) if offs[q] <= t < offs[q + 1]), None)
            if sid is not None and any(v is not None for v in c):
                n = offs[sid + 1] - offs[sid]
                g = up[0] * E / (k * n * n * filled) * want_f[sid]
                q = np.array(ro._shares(c, spec))
                mag[t] += q * (g + (q * g).sum()) + p * up[1] * 2 * (abs(ro._lse(c)) + min(big, 1e4)) / (offs[-1] - offs[0])
    got = dl.cpu().numpy()
    assert np.isfinite(got).all()
    err = np.abs(got - want)
    assert (err <= (2 * _rel(l) + (k + 16) * U) * mag + 1e-37).all(), float((err / (mag + 1e-37)).max() / U)


def test_gradient_of_shares_below_the_normal_range(rng):
    """Logits some hundreds apart: shares below 2^-126 may be off by up to that, times what multiplies them."""
    T, E, k = 30, 300, 3
    spec, offs = ro.RouteSpec("softmax"), [0, 4, 30]
    l = (50.0 * rng.standard_normal((T, E))).astype(np.float32)
    idx, w = ro.select(l, None, k, spec)
    up = np.array([0.8, 0.05], np.float32)
    dims = moe.Dims(T, 64, 64, E, k)
    tl, ti, tup = (torch.from_numpy(np.ascontiguousarray(v)).cuda() for v in (l, idx, up))
    seq = torch.tensor(offs, dtype=torch.int32, device="cuda")
    _, load = moe.balance_loss(dims, _opts(spec), tl, ti, seq)
    got = moe.route_select_backward(dims, _opts(spec), tl, None, None, None, tup, load, seq).cpu().numpy()
    _, f = ro.balance_losses(l, idx, offs, spec)
    want = ro.select_backward(l, idx, w, None, spec, up, f, offs)
    for t in range(T):
        s = 0 if t < offs[1] else 1
        n = offs[s + 1] - offs[s]
        p = np.array(ro.scores(ro._clean(l[t]), "softmax"))
        g = float(up[0]) * E / (k * n * n * 2) * f[s]
        z = 2 * float(up[1]) * (abs(ro._lse(ro._clean(l[t]))) + float(np.abs(l[t]).max())) / T
        factor = g + (p * g).sum() + z  # of a share
        tol = (2 * _rel(l) + (k + 16) * U) * p * factor + 2.0 ** -126 * (factor + 1)
        assert (np.abs(got[t] - want[t]) <= tol).all()


def test_backward_repeated_and_foreign_indices(rng):
    """Repeated entries add up, entries outside [0, E) are skipped; both stay in bounds."""
    T, E, k = 6, 40, 4
    l = rng.standard_normal((T, E)).astype(np.float32)
    idx = rng.integers(0, E, (T, k)).astype(np.int32)
    idx[:, 1] = idx[:, 0]
    idx[2, 3], idx[3, 2] = -7, E + 100
    w = rng.random((T, k)).astype(np.float32)
    w /= w.sum(1, keepdims=True)  # renormalised weights add up to the scale
    dw = rng.standard_normal((T, k)).astype(np.float32)
    for spec in (ro.RouteSpec("sigmoid", renormalise=True), ro.RouteSpec("softmax", renormalise=False)):
        got = moe.route_select_backward(moe.Dims(T, 64, 64, E, k), _opts(spec), *(torch.from_numpy(v).cuda() for v in (
            l, idx, w, dw))).cpu().numpy()
        want = ro.select_backward(l, idx, w.astype(np.float64), dw, spec)
        # |w| <= 1, |dw| <= 5: a few terms of at most 20
        np.testing.assert_allclose(got, want, rtol=0, atol=20 * 64 * U)
    losses, load = moe.balance_loss(moe.Dims(T, 64, 64, E, k), moe.RouteOptions(), torch.from_numpy(l).cuda(),
                                    torch.from_numpy(idx).cuda())
    assert int(load.sum()) == T * k - 2


def test_losses_alone(rng):
    """The losses' gradient without a selection's: the difference of the other two."""
    T, E, k = 77, 40, 3
    l, dims = torch.from_numpy(_logits(rng, T, E, "plain")).cuda(), moe.Dims(77, 64, 64, 40, 3)
    for opts in (moe.RouteOptions("sigmoid"), moe.RouteOptions(renormalise=False)):
        idx, w = moe.route_select(dims, opts, l)
        up = torch.tensor([0.5, 0.25], device="cuda")
        _, load = moe.balance_loss(dims, opts, l, idx)
        dw = torch.ones((T, k), device="cuda").cumsum(1)
        both = moe.route_select_backward(dims, opts, l, idx, w, dw, up, load)
        sel = moe.route_select_backward(dims, opts, l, idx, w, dw)
        alone = moe.route_select_backward(dims, opts, l, None, None, None, up, load)
        torch.testing.assert_close(both - sel, alone, rtol=0, atol=4 * 3 * U)  # elements below 3, two roundings


def test_an_expert_of_no_share_gets_no_gradient():
    """One row whose largest logit is the largest there is: the others' gradients are 0, not NaN."""
    l = torch.tensor([[INF, 0.0, -INF, 1.0]], device="cuda")
    dims, opts = moe.Dims(1, 64, 64, 4, 1), moe.RouteOptions()
    idx, w = moe.route_select(dims, opts, l)
    _, load = moe.balance_loss(dims, opts, l, idx)
    dl = moe.route_select_backward(dims, opts, l, idx, w, torch.ones((1, 1), device="cuda"),
                                   torch.tensor([1.0, 1.0], device="cuda"), load)
    assert idx.tolist() == [[0]] and dl[0, 1:].tolist() == [0, 0, 0] and float(dl[0, 0]) > 1e38


def test_losses_of_an_empty_batch():
    dims = moe.Dims(0, 64, 64, 12, 2)
    lg, ix = torch.empty((0, 12), device="cuda"), torch.empty((0, 2), dtype=torch.int32, device="cuda")
    losses, load = moe.balance_loss(dims, moe.RouteOptions(), lg, ix,
                                    torch.zeros(4, dtype=torch.int32, device="cuda"))
    assert not losses.any() and load.shape == (3, 12) and not load.any()


def test_many_sequences(rng):
    """More sequences than a wave has lanes, most of them empty, offsets past T clamped."""
    T, E, k = 200, 12, 3
    cuts = np.sort(rng.integers(0, T + 1, 300))
    offs = [0, *cuts.tolist(), T]
    spec = ro.RouteSpec("softmax", renormalise=False)
    l = _logits(rng, T, E, "plain")
    idx, w = ro.select(l, None, k, spec)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    up = np.array([1.0, 0.0], np.float32)
    dims, opts = moe.Dims(T, 64, 64, E, k), _opts(spec)
    given = torch.tensor(offs[:-1] + [T + 1000], dtype=torch.int32, device="cuda")
    tl, ti, tw, tdw, tup = (torch.from_numpy(np.ascontiguousarray(v)).cuda() for v in (
        l, idx, w.astype(np.float32), dw, up))
    losses, load = moe.balance_loss(dims, opts, tl, ti, given)
    got = moe.route_select_backward(dims, opts, tl, ti, tw, tdw, tup, load, given).cpu().numpy()
    want_l, want_f = ro.balance_losses(l, idx, offs, spec)
    np.testing.assert_array_equal(load.cpu().numpy(), want_f)
    np.testing.assert_allclose(losses.cpu().numpy(), want_l, rtol=4 * (_rel(l) + T * U))
    want = ro.select_backward(l, idx, w.astype(np.float32).astype(np.float64), dw, spec, up, want_f, offs)
    np.testing.assert_allclose(got, want, rtol=0, atol=40 * 64 * U)


GATE = [(1, 8, 1), (1, 256, 8), (3, 72, 5), (31, 128, 16), (33, 136, 33), (128, 256, 64), (129, 264, 65), (200, 1000, 96),
        (257, 392, 130), (520, 256, 256), (70, 128, 1024), (2049, 512, 24), (900, 2048, 200),
        (256, 512, 40), (257, 512, 40), (255, 1000, 64), (512, 264, 256), (513, 264, 256), (511, 136, 65),
        (1100, 8448, 520), (8300, 136, 3)]


@pytest.mark.parametrize("with_in", [True, False])
@pytest.mark.parametrize("shape", GATE, ids=lambda s: "T{}_d{}_E{}".format(*s))
def test_gate_backward(shape, with_in, rng):
    T, d, E = shape
    _say(f"gate_backward {shape} dx_in={with_in}")
    bf = torch.bfloat16
    x = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).cuda().to(bf)
    wg = torch.from_numpy(rng.standard_normal((E, d)).astype(np.float32)).cuda().to(bf)
    dl = torch.from_numpy((rng.standard_normal((T, E)) * 10.0 ** rng.uniform(-6, 2, (T, E))).astype(np.float32)).cuda()
    dx_in = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).cuda().to(bf) if with_in else None
    dx, c0 = _guarded((T, d), bf)
    dwg, c1 = _guarded((E, d), torch.float32)
    db, c2 = _guarded((E,), torch.float32)
    moe.gate_backward(moe.Dims(T, d, 64, E, 1), x, wg, dl, dx_in, dx=dx, dwg=dwg, dbias=db)
    torch.cuda.synchronize()
    c0()
    c1()
    c2()
    X, W, D = (v.double().cpu() for v in (x, wg, dl))
    I = torch.zeros((T, d), dtype=torch.float64) if dx_in is None else dx_in.double().cpu()
    # fp32 sums of exact products: (terms + a few) u of the sum of magnitudes
    want = D.t() @ X
    assert bool(((dwg.double().cpu() - want).abs() <= (T + 8) * U * (D.abs().t() @ X.abs())).all())
    assert bool(((db.double().cpu() - D.sum(0)).abs() <= (T + 8) * U * D.abs().sum(0) + 1e-45).all())
    want = I + D @ W
    tol = BF * want.abs() + (2.0 ** -16 * (1 + BF) + (E + 8) * U) * (D.abs() @ W.abs()) + 4 * U * I.abs()
    assert bool(((dx.double().cpu() - want).abs() <= tol).all())


def test_gate_backward_special_values(rng):
    """inf, NaN, the largest finite value and denormals of dlogits go where the formula sends them; dx may be dx_in."""
    T, d, E = 40, 64, 6
    bf = torch.bfloat16
    x = torch.ones((T, d), dtype=bf, device="cuda")
    wg = torch.ones((E, d), dtype=bf, device="cuda")
    dl = torch.zeros((T, E), device="cuda")
    big = torch.finfo(torch.float32).max
    dl[3, 0], dl[4, 1], dl[5, 2], dl[6, 3] = INF, NAN, big, 2.0 ** -100
    io = torch.ones((T, d), dtype=bf, device="cuda")
    dx, dwg, db = moe.gate_backward(moe.Dims(T, d, 64, E, 1), x, wg, dl, io, dx=io)
    assert dx.data_ptr() == io.data_ptr()
    assert bool(torch.isinf(dwg[0]).all()) and bool(torch.isnan(dwg[1]).all())
    assert bool((dwg[2] == big).all()) and bool((dwg[3] == 2.0 ** -100).all()) and not dwg[4:].any()
    assert bool(torch.isinf(dx[3]).all()) and bool(torch.isnan(dx[4]).all())
    keep = torch.ones(T, dtype=torch.bool)
    keep[3:6] = False
    assert bool((dx[keep.cuda()] == 1).all())
    assert math.isinf(float(db[0])) and math.isnan(float(db[1])) and float(db[2]) == big


def test_gate_backward_empty_batch():
    d, E = 64, 8
    x = torch.empty((0, d), dtype=torch.bfloat16, device="cuda")
    wg = torch.ones((E, d), dtype=torch.bfloat16, device="cuda")
    dx, dwg, db = moe.gate_backward(moe.Dims(0, d, 64, E, 1), x, wg, torch.empty((0, E), device="cuda"))
    assert dx.shape == (0, d) and not dwg.any() and not db.any()


DROP = [(1, 8, 1, 0.1, True), (1, 6144, 2, 0.1, True), (7, 1048, 4, 0.25, False), (130, 136, 3, 0.5, True),
        (64, 256, 6, 0.0, True), (64, 256, 2, 1.0, True), (64, 256, 2, 1.0, False), (9, 64, 8, 0.999, True),
        (300, 72, 1, 0.3, False)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", DROP, ids=lambda c: "T{}_d{}_k{}_p{}_r{:d}".format(*c))
def test_combine_dropout(case, dtype, rng):
    T, d, k, p, with_res = case
    _say(f"combine_dropout {case} {dtype}")
    seed, off = int(rng.integers(-2 ** 63, 2 ** 63 - 1)), int(rng.integers(-2 ** 63, 2 ** 63 - 1))
    r = torch.tensor([seed, off], dtype=torch.int64, device="cuda")
    mk = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda().to(dtype)  # noqa: E731
    y, res, dout = mk(T * k, d), (mk(T, d) if with_res else None), mk(T, d)
    inv = torch.from_numpy(rng.permutation(T * k).astype(np.int32)).cuda()
    w = torch.from_numpy(rng.random((T, k)).astype(np.float32)).cuda()
    dims = moe.Dims(T, d, 64, max(k, 8), k, dtype)
    out, c0 = _guarded((T, d), dtype)
    dy, c1 = _guarded((T, d), dtype)
    moe.combine_dropout(dims, p, r, y, inv, w, res, out=out)
    moe.dropout_backward(dims, p, r, dout, dy=dy)
    torch.cuda.synchronize()
    c0()
    c1()
    h = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    eps = BF if dtype == torch.bfloat16 else U
    want = ro.combine_dropout(h(y), inv.cpu().numpy(), h(w), h(res), seed, off, p)
    mag = ro.combine_dropout(np.abs(h(y)), inv.cpu().numpy(), h(w), None if res is None else np.abs(h(res)), seed, off, p)
    assert (np.abs(h(out) - want) <= eps * np.abs(want) + (k + 4) * U * mag).all()
    want = ro.dropout_backward(h(dout), seed, off, p)
    assert (np.abs(h(dy) - want) <= (eps + 2 * U) * np.abs(want)).all()
    assert ((h(dy) == 0) >= (want == 0)).all()
    # in place: residual stream and gradient
    if with_res:
        moe.combine_dropout(dims, p, r, y, inv, w, res, out=res)
        assert torch.equal(res, out)
    moe.dropout_backward(dims, p, r, dout, dy=dout)
    assert torch.equal(dout, dy)


def test_dropout_of_special_values():
    """A dropped inf or NaN leaves the residual; kept ones come through as they are."""
    T, d = 16, 64
    for dtype in (torch.bfloat16, torch.float32):
        dims = moe.Dims(T, d, 64, 8, 1, dtype)
        r = torch.tensor([11, 22], dtype=torch.int64, device="cuda")
        keep = torch.from_numpy(ro.keep_mask(T * d, 11, 22, 0.5).reshape(T, d)).cuda()
        for v in (INF, -INF, NAN):
            y = torch.full((T, d), v, dtype=dtype, device="cuda")
            inv = torch.arange(T, dtype=torch.int32, device="cuda")
            w = torch.ones((T, 1), device="cuda")
            out = moe.combine_dropout(dims, 0.5, r, y, inv, w, torch.ones((T, d), dtype=dtype, device="cuda"))
            assert bool((out[~keep] == 1).all())
            assert bool((torch.isnan(out[keep]) if v != v else out[keep] == v).all())
            dy = moe.dropout_backward(dims, 0.5, r, y)
            assert not dy[~keep].any() and bool((torch.isnan(dy[keep]) if v != v else dy[keep] == v).all())


def test_dropout_rate_and_statistics():
    """Over 2^22 elements: the kept share within 5 standard deviations, and neighbours uncorrelated."""
    T, d, p = 1024, 4096, 0.1
    dims = moe.Dims(T, d, 64, 8, 1, torch.float32)
    r = torch.tensor([123456789, 0], dtype=torch.int64, device="cuda")
    keep = (moe.dropout_backward(dims, p, r, torch.ones((T, d), device="cuda")) != 0).double()
    n = T * d
    q = 1 - round(p * 65536) / 65536
    sd = math.sqrt(q * (1 - q) / n)
    assert abs(float(keep.mean()) - q) < 5 * sd
    z = keep.view(-1) - q
    for lag in (1, 7, 8, d):
        assert abs(float((z[:-lag] * z[lag:]).mean())) < 5 * q * (1 - q) / math.sqrt(n)


# ------------------------------------------------------------ used together ----
def _training_step(dims, opts, p, t, streams=None):
    """The router, the experts and their gradients as a training step runs them."""
    logits, idx, w = moe.route_scored(dims, opts, t["x"], t["wg"], t["bias"], t["bb"])
    counts, offsets, perm, inv = moe.permute(dims, idx, ws=t["ws"])
    y = moe.grouped_ffn(dims, t["x"], perm, counts, offsets, t["w1"], t["w3"], t["w2"], ws=t["ws"])
    out = moe.combine_dropout(dims, p, t["rng"], y, inv, w, t["x"])
    losses, load = moe.balance_loss(dims, opts, logits, idx, t["seq"])
    dy = moe.dropout_backward(dims, p, t["rng"], t["dout"])
    r = {"topk_idx": idx, "topk_w": w, "counts": counts, "offsets": offsets, "perm": perm, "inv_perm": inv}
    g = moe.experts_backward(dims, t["x"], t["w1"], t["w3"], t["w2"], r, dy, ws=t["bws"])
    dl = moe.route_select_backward(dims, opts, logits, idx, w, g["dtopk_w"], t["dlosses"], load, t["seq"])
    dx, dwg, dbias = moe.gate_backward(dims, t["x"], t["wg"], dl, g["dx"])
    return {"logits": logits, "idx": idx, "w": w, "out": out, "losses": losses, "load": load, "dl": dl, "dx": dx,
            "dwg": dwg, "dbias": dbias, "dw1": g["dw1"], "dw3": g["dw3"], "dw2": g["dw2"], "dtopk_w": g["dtopk_w"]}


def _step_inputs(T, d, f, E, k, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    t = {"x": rn(T, d).to(bf), "wg": (rn(E, d) / math.sqrt(d)).to(bf), "bias": 0.1 * rn(E), "bb": 0.05 * rn(E),
         "w1": (rn(E, f, d) / math.sqrt(d)).to(bf), "w3": (rn(E, f, d) / math.sqrt(d)).to(bf),
         "w2": (rn(E, d, f) / math.sqrt(f)).to(bf), "dout": rn(T, d).to(bf),
         "dlosses": torch.tensor([0.05, 0.01], device="cuda"),
         "seq": torch.tensor([0, T // 3, T // 3, T - 5], dtype=torch.int32, device="cuda"),
         "rng": torch.tensor([seed + 5, 3], dtype=torch.int64, device="cuda")}
    dims = moe.Dims(T, d, f, E, k, bf)
    t["ws"] = moe.make_workspace(dims)
    t["bws"] = torch.empty(moe.backward_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    return dims, t


SCORED = [moe.RouteOptions("sigmoid", 4, 2, "top2", True, 2.5), moe.RouteOptions("softmax", renormalise=False)]


@pytest.mark.parametrize("opts", SCORED, ids=["sigmoid_groups", "softmax_plain"])
def test_training_step_against_autograd(opts, rng):
    """The whole step against float64 differentiation of its plain definition, the choice and
    the keep decisions fixed. Bars: the layer's backward bar of 2e-2 normwise (its bf16
    roundings), which dx and the gate's gradients inherit through dtopk_w."""
    T, d, f, E, k, p = 150, 256, 256, 8, 2, 0.25
    dims, t = _step_inputs(T, d, f, E, k, 1)
    got = _training_step(dims, opts, p, t)
    torch.cuda.synchronize()
    c = {n: v.double().cpu() if v.is_floating_point() else v.cpu() for n, v in t.items() if n not in ("ws", "bws")}
    leaf = {n: c[n].clone().requires_grad_(True) for n in ("x", "wg", "bias", "w1", "w3", "w2")}
    idx = got["idx"].long().cpu()
    l = leaf["x"] @ leaf["wg"].t() + leaf["bias"]
    s = torch.sigmoid(l) if opts.score == "sigmoid" else torch.softmax(l, 1)
    w = s.gather(1, idx)
    w = opts.scale * (w / w.sum(1, keepdim=True) if opts.renormalise else w)
    keep = torch.from_numpy(ro.keep_mask(T * d, 6, 3, p).reshape(T, d))
    rows = []
    for i in range(T):
        acc = 0.0
        for j in range(k):
            e = int(idx[i, j])
            g, u = leaf["w1"][e] @ leaf["x"][i], leaf["w3"][e] @ leaf["x"][i]
            acc = acc + w[i, j] * (leaf["w2"][e] @ (g * torch.sigmoid(g) * u))
        rows.append(acc)
    s_out = torch.stack(rows)
    out = c["x"] + torch.where(keep, s_out / (1 - 0.25), torch.zeros_like(s_out))
    q = s / s.sum(1, keepdim=True)
    seq = c["seq"].tolist()
    bal = 0.0
    for a, b in zip(seq[:-1], seq[1:]):
        if b > a:
            fr = torch.bincount(idx[a:b].reshape(-1), minlength=E).double()
            bal = bal + E / (k * (b - a)) * (fr * q[a:b].mean(0)).sum() / 2
    z = (torch.logsumexp(l[seq[0]:seq[-1]], 1) ** 2).mean()
    f_ = (out * c["dout"]).sum() + 0.05 * bal + 0.01 * z
    grads = dict(zip(leaf, torch.autograd.grad(f_, list(leaf.values()))))
    assert float((got["out"].double().cpu() - out).abs().max() / out.abs().max()) < 2e-2
    np.testing.assert_allclose(got["losses"].cpu().numpy(), [float(bal.detach()), float(z.detach())], rtol=1e-4)
    for name, ref in (("dx", grads["x"]), ("dwg", grads["wg"]), ("dbias", grads["bias"]), ("dw1", grads["w1"]),
                      ("dw3", grads["w3"]), ("dw2", grads["w2"])):
        err = float((got[name].double().cpu() - ref).norm() / ref.norm())
        _say(f"  {name} {err:.2e}")
        assert err < 2e-2, name


def test_experts_backward_is_the_layers(rng):
    """With a zero gate the layer's backward is the experts' part alone: the same bits."""
    T, d, f, E, k = 200, 256, 512, 8, 2
    dims, t = _step_inputs(T, d, f, E, k, 2)
    out, r = moe.layer_forward(dims, t["x"], t["wg"], t["bias"], t["w1"], t["w3"], t["w2"], return_routing=True)
    zero = torch.zeros_like(t["wg"])
    for wt in (torch.float32, torch.bfloat16):
        a = moe.layer_backward(dims, t["x"], zero, t["w1"], t["w3"], t["w2"], r, t["dout"], want_dtopk_w=True,
                               wgrad_dtype=wt)
        b = moe.experts_backward(dims, t["x"], t["w1"], t["w3"], t["w2"], r, t["dout"], wgrad_dtype=wt)
        for n in ("dx", "dw1", "dw3", "dw2", "dtopk_w"):
            assert torch.equal(a[n], b[n]), n
    e = moe.Dims(0, d, f, E, k)
    r0 = {"topk_idx": r["topk_idx"][:0], "topk_w": r["topk_w"][:0], "counts": torch.zeros_like(r["counts"]),
          "offsets": torch.zeros_like(r["offsets"]), "perm": r["perm"][:0], "inv_perm": r["inv_perm"][:0]}
    g = moe.experts_backward(e, t["x"][:0], t["w1"], t["w3"], t["w2"], r0, t["dout"][:0])
    assert not g["dw1"].any() and not g["dw3"].any() and not g["dw2"].any()


def test_step_on_another_stream_and_twice_is_the_same(rng):
    dims, t = _step_inputs(190, 256, 256, 8, 2, 4)
    a = _training_step(dims, SCORED[0], 0.1, t)
    b = _training_step(dims, SCORED[0], 0.1, t)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c = _training_step(dims, SCORED[0], 0.1, t)
    s.synchronize()
    for n in a:
        assert torch.equal(a[n], b[n]) and torch.equal(a[n], c[n]), n
    # a stream given by hand, from the default stream
    l, idx, w = moe.route_scored(dims, SCORED[0], t["x"], t["wg"], t["bias"], t["bb"], stream=s)
    lo, ld = moe.balance_loss(dims, SCORED[0], l, idx, t["seq"], stream=s)
    dl = moe.route_select_backward(dims, SCORED[0], l, idx, w, a["dtopk_w"], t["dlosses"], ld, t["seq"], stream=s)
    dx, dwg, db = moe.gate_backward(dims, t["x"], t["wg"], dl, stream=s)
    dy = moe.dropout_backward(dims, 0.1, t["rng"], t["dout"], stream=s)
    s.synchronize()
    assert torch.equal(idx, a["idx"]) and torch.equal(lo, a["losses"]) and torch.equal(dl, a["dl"])
    assert torch.equal(dwg, a["dwg"]) and torch.equal(db, a["dbias"])
    assert torch.equal(dy, moe.dropout_backward(dims, 0.1, t["rng"], t["dout"]))


def test_step_in_a_graph(rng):
    """Captured once, replayed with other inputs and another draw each time, against the eager step."""
    dims, t = _step_inputs(170, 256, 256, 8, 2, 7)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _training_step(dims, SCORED[0], 0.2, t)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _training_step(dims, SCORED[0], 0.2, t)
    for it in range(4):
        _, u = _step_inputs(170, 256, 256, 8, 2, 100 + it)
        for n in t:
            if n not in ("ws", "bws"):
                t[n].copy_(u[n])
        graph.replay()
        torch.cuda.synchronize()
        kept = {n: v.clone() for n, v in got.items()}
        want = _training_step(dims, SCORED[0], 0.2, u)
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(kept[n], want[n]), (it, n)


def test_tensors_off_their_alignment(rng):
    """fp32 and int32 tensors that start one element past a 16-byte boundary: the same bits."""
    T, E, k = 37, 64, 8
    l, b = _logits(rng, T, E, "plain"), _bias(rng, E, "small")
    spec = ro.RouteSpec("sigmoid", 8, 4, "top2", True, 2.5)
    dims, opts = moe.Dims(T, 64, 64, E, k, torch.bfloat16), _opts(spec)

    def shifted(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        buf[1:].copy_(t.reshape(-1))
        return buf[1:].view(t.shape)

    def step(mv):
        tl, tb = mv(torch.from_numpy(l).cuda()), mv(torch.from_numpy(b).cuda())
        idx, w = mv(torch.zeros((T, k), dtype=torch.int32, device="cuda")), mv(torch.zeros((T, k), device="cuda"))
        moe.route_select(dims, opts, tl, tb, topk_idx=idx, topk_w=w)
        dw, up = mv(torch.ones((T, k), device="cuda").cumsum(1)), mv(torch.tensor([0.5, 0.25], device="cuda"))
        seq = mv(torch.tensor([0, 9, T], dtype=torch.int32, device="cuda"))
        load = mv(torch.zeros((2, E), dtype=torch.int32, device="cuda"))
        losses, _ = moe.balance_loss(dims, opts, tl, idx, seq, load=load, losses=mv(torch.zeros(2, device="cuda")))
        dl = moe.route_select_backward(dims, opts, tl, idx, w, dw, up, load, seq,
                                       dlogits=mv(torch.zeros((T, E), device="cuda")))
        x = torch.ones((T, 64), dtype=torch.bfloat16, device="cuda")
        wg = torch.ones((E, 64), dtype=torch.bfloat16, device="cuda")
        _, dwg, db = moe.gate_backward(dims, x, wg, dl, dbias=mv(torch.zeros(E, device="cuda")))
        return idx, w, losses, load, dl, dwg, db
    for a, c in zip(step(lambda t: t), step(shifted)):
        assert torch.equal(a, c)


def test_more_tokens_than_one_launch_holds():
    """Batches that take several launches: selection (2^25 tokens each) and the combine (2^23 workgroups each)."""
    T = 2 ** 25 + 5
    gen = torch.Generator(device="cuda").manual_seed(9)
    l = torch.randn((T, 2), generator=gen, device="cuda")
    dims = moe.Dims(T, 64, 64, 2, 1)
    idx, w = moe.route_select(dims, moe.RouteOptions(), l)
    assert torch.equal(idx[:, 0], (l[:, 1] > l[:, 0]).int()) and bool((w == 1).all())
    losses, load = moe.balance_loss(dims, moe.RouteOptions(), l, idx)
    assert torch.equal(load[0].long(), torch.bincount(idx[:, 0].long(), minlength=2))
    # p of the chosen expert minus 1 for it, plus p for the other, on every row
    dl = moe.route_select_backward(dims, moe.RouteOptions(renormalise=False), l, idx, torch.softmax(l, 1).gather(
        1, idx.long()), torch.ones((T, 1), device="cuda"))
    p = torch.softmax(l, 1)
    torch.testing.assert_close(dl.gather(1, idx.long())[:, 0], (p[:, 0] * p[:, 1]), rtol=0, atol=64 * U)
    del l, dl, p, idx, w
    T = 2 ** 23 + 3
    dims = moe.Dims(T, 8, 64, 8, 1)
    y = torch.randn((T, 8), generator=gen, device="cuda").bfloat16()
    r = torch.tensor([3, 4], dtype=torch.int64, device="cuda")
    out = moe.combine_dropout(dims, 0.5, r, y, torch.arange(T, dtype=torch.int32, device="cuda"),
                              torch.ones((T, 1), device="cuda"))
    assert torch.equal(out, moe.dropout_backward(dims, 0.5, r, y))


def test_two_steps_at_once(rng):
    """Two steps on two streams at the same time, each with its own buffers: each as when alone."""
    a, b = _step_inputs(300, 256, 256, 8, 2, 11), _step_inputs(210, 256, 256, 8, 2, 12)
    want = [_training_step(a[0], SCORED[0], 0.1, a[1]), _training_step(b[0], SCORED[1], 0.3, b[1])]
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(3):
        got = []
        with torch.cuda.stream(s):
            got.append(_training_step(a[0], SCORED[0], 0.1, a[1]))
        with torch.cuda.stream(t):
            got.append(_training_step(b[0], SCORED[1], 0.3, b[1]))
    torch.cuda.synchronize()
    for x, y in zip(want, got):
        for n in x:
            assert torch.equal(x[n], y[n]), n


def test_gpu_refusals():
    dims = moe.Dims(4, 64, 64, 8, 2)
    l = torch.zeros((4, 8), device="cuda")
    o = moe.RouteOptions()
    with pytest.raises(ValueError, match="dtype"):
        moe.route_select(dims, o, l.double())
    with pytest.raises(ValueError, match="shape"):
        moe.route_select(dims, o, l[:3])
    with pytest.raises(ValueError, match="contiguous"):
        moe.route_select(dims, o, torch.zeros((8, 4), device="cuda").t())
    with pytest.raises(ValueError, match="is on cpu"):
        moe.route_select(dims, o, l, torch.zeros(8))
    with pytest.raises(moe.MoeError):
        moe.route_select(dims, moe.RouteOptions(groups=3), l)
    with pytest.raises(moe.MoeError):
        moe.route_select(dims, moe.RouteOptions(scale=INF), l)
    i = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    w = torch.zeros((4, 2), device="cuda")
    with pytest.raises(ValueError, match="load"):
        moe.route_select_backward(dims, o, l, i, w, w, dlosses=torch.zeros(2, device="cuda"))
    with pytest.raises(ValueError, match="offsets"):
        moe.balance_loss(dims, o, l, i, torch.zeros(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(moe.MoeError):
        moe.balance_loss(dims, o, l, i, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    f = moe.Dims(4, 64, 64, 8, 2, torch.float32)
    x = torch.zeros((4, 64), device="cuda")
    with pytest.raises(moe.MoeError):
        moe.gate_backward(f, x, torch.zeros((8, 64), device="cuda"), l)
    with pytest.raises(moe.MoeError):
        moe.dropout_backward(f, 1.5, torch.zeros(2, dtype=torch.int64, device="cuda"), x)
    with pytest.raises(ValueError, match="dtype"):
        moe.dropout_backward(f, 0.5, torch.zeros(2, dtype=torch.int32, device="cuda"), x)
