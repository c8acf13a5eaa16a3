"""The scored router's oracle against independent statements of it (brute force,
closed forms, automatic and finite differences, published generator outputs),
and the refusals of the new entry points. Host-only: no call reaches a launch."""
import copy
import ctypes
import itertools
import math
import os
import pickle

import numpy as np
import pytest
import torch

import mixture_experts_layer_gate_amd as moe
from mixture_experts_layer_gate_amd import api
from oracle import router_oracle as ro

built = pytest.mark.skipif(not os.path.exists(moe.library_path()), reason="HIP library not built")
needs_no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="host-only validation test")
A = 0x10000  # 16-byte aligned placeholder, never dereferenced


# ------------------------------------------------------------------ oracle ----
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,topk_groups,rule", [(1, 1, "max"), (4, 2, "max"), (4, 2, "top2"), (4, 3, "top2")])
def test_selection_by_brute_force(rng, score, groups, topk_groups, rule):
    """Every kept set of groups and every set of k experts compared by hand on dyadic-free random rows."""
    T, E, k = 12, 12, 3
    logits = rng.standard_normal((T, E)).astype(np.float32)
    bias = (0.2 * rng.standard_normal(E)).astype(np.float32)
    spec = ro.RouteSpec(score, groups, topk_groups, rule, True, 1.5)
    idx, w = ro.select(logits, bias, k, spec)
    per = E // groups
    for t in range(T):
        z = logits[t].astype(np.float64)
        s = 1 / (1 + np.exp(-z)) if score == "sigmoid" else np.exp(z) / np.exp(z).sum()
        c = s + bias

        def group_key(g):
            m = np.sort(c[g * per:(g + 1) * per])[::-1]
            return m[0] + m[1] if rule == "top2" else m[0]
        best_groups = max(itertools.combinations(range(groups), topk_groups), key=lambda q: sum(map(group_key, q)))
        pool = [e for g in best_groups for e in range(g * per, (g + 1) * per)]
        best = max(itertools.combinations(pool, k), key=lambda q: sum(c[e] for e in q))
        assert set(idx[t]) == set(best)
        assert all(c[idx[t, j]] >= c[idx[t, j + 1]] for j in range(k - 1))
        np.testing.assert_allclose(w[t], 1.5 * s[idx[t]] / s[idx[t]].sum(), rtol=1e-12)


def test_selection_ties_and_masks():
    inf, nan = math.inf, math.nan
    # equal keys: lower expert; saturated sigmoids: the larger logit first
    idx, _ = ro.select(np.array([[1.0, 1.0, 0.0, 1.0]]), None, 3, ro.RouteSpec("sigmoid"))
    assert idx.tolist() == [[0, 1, 3]]
    idx, _ = ro.select(np.array([[80.0, 90.0, 70.0]]), None, 3, ro.RouteSpec("sigmoid"))
    assert idx.tolist() == [[1, 0, 2]]
    # masked logits and biases; what is left over comes in ascending order with weight 0
    idx, w = ro.select(np.array([[nan, 3.0, -inf, 1.0, 2.0]]), np.array([0, 0, 0, -inf, 0.0]), 4, ro.RouteSpec())
    assert idx.tolist() == [[1, 4, 0, 2]] and w[0, 2:].tolist() == [0, 0]
    np.testing.assert_allclose(w[0, :2], np.exp([3, 2]) / np.exp([3, 2]).sum())
    idx, w = ro.select(np.full((1, 4), -inf), None, 2, ro.RouteSpec("sigmoid"))
    assert idx.tolist() == [[0, 1]] and not w.any()
    # a group with one expert left still counts; one with none comes last
    idx, _ = ro.select(np.array([[-inf, -inf, -inf, -5.0, 1.0, 1.0]]), np.array([0, 0, 0, 0, -inf, -inf]), 1,
                       ro.RouteSpec("sigmoid", 3, 1, "top2"))
    assert idx.tolist() == [[3]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradients_by_autograd_and_differences(rng, score, renorm):
    T, E, k, seqs = 9, 7, 3, [0, 4, 4, 9]
    logits = rng.standard_normal((T, E))
    dw = rng.standard_normal((T, k))
    up = np.array([0.7, -0.3])
    spec = ro.RouteSpec(score, renormalise=renorm, scale=1.75)
    idx, w = ro.select(logits, None, k, spec)
    losses, load = ro.balance_losses(logits, idx, seqs, spec)
    got = ro.select_backward(logits, idx, w, dw, spec, up, load, seqs)

    def total(l):
        s = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
        q = s / s.sum(1, keepdim=True)
        ws = s.gather(1, torch.from_numpy(idx.astype(np.int64)))
        ws = 1.75 * (ws / ws.sum(1, keepdim=True) if renorm else ws)
        bal = 0.0
        for a, b in ((0, 4), (4, 9)):
            f = torch.bincount(torch.from_numpy(idx[a:b].reshape(-1).astype(np.int64)), minlength=E).double()
            bal = bal + E / (k * (b - a)) * (f * q[a:b].mean(0)).sum() / 2
        z = (torch.logsumexp(l, 1) ** 2).mean()
        return (ws * torch.from_numpy(dw)).sum() + up[0] * bal + up[1] * z, bal, z
    l = torch.from_numpy(logits).requires_grad_(True)
    f, bal, z = total(l)
    np.testing.assert_allclose(losses, [float(bal), float(z)], rtol=1e-12)
    want, = torch.autograd.grad(f, l)
    np.testing.assert_allclose(got, want.numpy(), rtol=1e-10, atol=1e-13)
    # central differences along a random direction: error of order h^2 = 1e-10
    v, h = rng.standard_normal((T, E)), 1e-5
    num = (total(torch.from_numpy(logits + h * v))[0] - total(torch.from_numpy(logits - h * v))[0]) / (2 * h)
    assert abs(float(num) - float((got * v).sum())) < 1e-7


def test_generator_known_answers():
    """Outputs published with the generator (zeros, all ones, digits of pi)."""
    f = 0xFFFFFFFF
    assert ro.philox4x32([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert ro.philox4x32([f] * 4, [f] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert ro.philox4x32([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0]) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_keep_mask_rate_and_limits():
    assert ro.keep_mask(64, 1, 2, 0.0).all() and not ro.keep_mask(64, 1, 2, 1.0).any()
    m = ro.keep_mask(40000, 5, 9, 0.25)
    assert abs(m.mean() - 0.75) < 5 * math.sqrt(0.25 * 0.75 / 40000)
    assert (m == ro.keep_mask(40000, 5, 9, 0.25)).all() and (m != ro.keep_mask(40000, 5, 10, 0.25)).any()


# ---------------------------------------------------------------- refusals ----
def _dims(**kw):
    base = dict(T=64, d=128, f=256, E=8, k=2, dtype=1)
    base.update(kw)
    return api._Dims(base["T"], base["d"], base["f"], base["E"], base["k"], base["dtype"])


def _opts(**kw):
    base = dict(score=0, groups=1, topk_groups=1, group_rule=0, renormalise=1, scale=1.0)
    base.update(kw)
    return api._RouteOpts(*(base[n] for n in ("score", "groups", "topk_groups", "group_rule", "renormalise", "scale")))


BAD_OPTS = [dict(score=2), dict(score=-1), dict(group_rule=2), dict(renormalise=2), dict(groups=0), dict(groups=3),
            dict(groups=4, topk_groups=5), dict(groups=4, topk_groups=0), dict(scale=math.inf), dict(scale=math.nan)]


@built
@needs_no_gpu
@pytest.mark.parametrize("bad", BAD_OPTS)
def test_option_refusals(bad):
    lib, dm, op = moe.load_library(), _dims(), _opts(**bad)
    d, o = ctypes.byref(dm), ctypes.byref(op)
    assert lib.moe_route_select(d, o, A, None, A, A, None) == 1
    assert lib.moe_route_scored(d, o, A, A, None, None, A, A, A, None) == 1
    assert lib.moe_balance_loss(d, o, A, A, None, 1, A, A, A, 1 << 30, None) == 1
    assert lib.moe_route_select_backward(d, o, A, A, A, A, None, None, None, 1, A, None) == 1


@built
@needs_no_gpu
def test_pointer_and_shape_refusals():
    lib, op = moe.load_library(), _opts()
    o = ctypes.byref(op)

    def d(**kw):
        return ctypes.byref(_dims(**kw))
    too_few = _opts(groups=8, topk_groups=1)  # one expert per group, two wanted
    assert lib.moe_route_select(d(), ctypes.byref(too_few), A, None, A, A, None) == 1
    wide = _opts(groups=128, topk_groups=64)
    assert lib.moe_route_select(d(E=1024, k=2), ctypes.byref(wide), A, None, A, A, None) == 1
    for args in ((None, None, A, A), (A, A + 2, A, A), (A, None, None, A), (A, None, A, None)):
        assert lib.moe_route_select(d(), o, *args, None) == 1
    assert lib.moe_route_select(d(), None, A, None, A, A, None) == 1
    assert lib.moe_route_select(d(T=0), o, None, None, None, None, None) == 0
    assert lib.moe_route_select(d(k=9), o, A, None, A, A, None) == 1
    assert lib.moe_route_scored(d(d=100), o, A, A, None, None, A, A, A, None) == 2
    assert lib.moe_route_scored(d(), o, A + 8, A, None, None, A, A, A, None) == 1
    assert lib.moe_route_scored(d(), o, A, A, None, None, None, A, A, None) == 1
    # losses
    need = lib.moe_balance_workspace_bytes(d(), 3)
    assert need > 0 and lib.moe_balance_workspace_bytes(d(), 0) == 0 and lib.moe_balance_workspace_bytes(d(), 65536) == 0
    assert lib.moe_balance_loss(d(), o, A, A, None, 2, A, A, A, 1 << 30, None) == 1    # two sequences, no offsets
    assert lib.moe_balance_loss(d(), o, A, A, A, 0, A, A, A, 1 << 30, None) == 1
    assert lib.moe_balance_loss(d(), o, A, A, A, 65536, A, A, A, 1 << 40, None) == 2
    assert lib.moe_balance_loss(d(), o, A, A, A, 3, A, A, A, need - 1, None) == 3
    assert lib.moe_balance_loss(d(), o, A, A, A, 3, A, A, None, 0, None) == 3
    assert lib.moe_balance_loss(d(), o, A, A, A, 3, A, A, A + 64, 1 << 30, None) == 1
    assert lib.moe_balance_loss(d(), o, None, A, A, 3, A, A, A, 1 << 30, None) == 1
    # their gradient
    bwd = lib.moe_route_select_backward
    assert bwd(d(), o, A, None, A, A, None, None, None, 1, A, None) == 1               # dtopk_w without topk_idx
    assert bwd(d(), o, A, None, None, None, A, None, None, 1, A, None) == 1            # dlosses without load
    assert bwd(d(), o, A, None, None, None, A, A, None, 2, A, None) == 1
    assert bwd(d(), o, None, A, A, A, None, None, None, 1, A, None) == 1
    assert bwd(d(T=0), o, None, None, None, None, None, None, None, 1, None, None) == 0
    # gate gradients
    gate = lib.moe_gate_backward
    need = lib.moe_gate_backward_workspace_bytes(d())
    assert need > 0 and lib.moe_gate_backward_workspace_bytes(d(k=0)) == 0
    assert gate(d(), A, A, A, None, A, A, A, A, need - 1, None) == 3
    assert gate(d(), A, A, A, None, A, A, A, None, need, None) == 3
    assert gate(d(), A, A, A, None, A, A, A, A + 16, need, None) == 1
    assert gate(d(), A, A, A, A + 2, A, A, A, A, need, None) == 1
    assert gate(d(), A, A, A, None, None, A, A, A, need, None) == 1
    assert gate(d(dtype=0), A, A, A, None, A, A, A, A, need, None) == 2
    assert gate(d(d=100), A, A, A, None, A, A, A, A, 1 << 40, None) == 2
    assert gate(d(T=4194177, E=8), A, A, A, None, A, A, A, A, 1 << 50, None) == 2
    # dropout
    for p in (-0.1, 1.1, math.nan):
        assert lib.moe_combine_dropout(d(), p, A, A, A, A, None, A, None) == 1
        assert lib.moe_dropout_backward(d(), p, A, A, A, None) == 1
    assert lib.moe_combine_dropout(d(), 0.1, None, A, A, A, None, A, None) == 1
    assert lib.moe_combine_dropout(d(), 0.1, A + 4, A, A, A, None, A, None) == 1
    assert lib.moe_combine_dropout(d(), 0.1, A, A, A, A, A + 8, A, None) == 1
    assert lib.moe_combine_dropout(d(d=100), 0.1, A, A, A, A, None, A, None) == 2
    assert lib.moe_dropout_backward(d(d=100), 0.1, A, A, A, None) == 2
    assert lib.moe_dropout_backward(d(), 0.1, A, A, A + 2, None) == 1
    assert lib.moe_dropout_backward(d(T=0), 0.1, A, None, None, None) == 0
    # the experts' backward: the layer's limits
    ex = lib.moe_experts_backward
    a = [A] * 10
    assert ex(d(d=256), *a, None, None, 0, A, A, A, A, None, A, 1 << 40, None) == 1     # dtopk_w is required
    assert ex(d(d=256), *a, A, None, 7, A, A, A, A, A, A, 1 << 40, None) == 1
    assert ex(d(d=128), *a, A, None, 0, A, A, A, A, A, A, 1 << 40, None) == 2
    assert ex(d(d=256), *a, A, None, 0, A, A, A, A, A, A, 16, None) == 3


@built
def test_binding_refusals():
    dims = moe.Dims(4, 64, 64, 8, 2)
    with pytest.raises(ValueError, match="score"):
        moe.RouteOptions(score="tanh")
    with pytest.raises(ValueError, match="group_rule"):
        moe.RouteOptions(group_rule="mean")
    cpu = torch.zeros((4, 8))
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.route_select(dims, moe.RouteOptions(), cpu)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.balance_loss(dims, moe.RouteOptions(), cpu, cpu)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.dropout_backward(dims, 0.1, cpu, cpu)


@pytest.mark.parametrize("value", [moe.Dims(4, 64, 64, 8, 2), moe.RouteOptions("sigmoid", 4, 2, "top2", True, 2.5)])
def test_dims_and_options_are_copied_and_pickled_after_use(value):
    """Whatever a call keeps beside the fields stays behind, and the copy serves calls of its own."""
    fresh = pickle.dumps(value)
    value.ref()
    if isinstance(value, moe.Dims) and os.path.exists(moe.library_path()):
        assert moe.balance_workspace_bytes(value) > 0 and moe.gate_backward_workspace_bytes(value) > 0
    assert pickle.dumps(value) == fresh
    for other in (copy.copy(value), copy.deepcopy(value), pickle.loads(pickle.dumps(value))):
        assert other == value and hash(other) == hash(value)
        assert bytes(other.ref()._obj) == bytes(value.ref()._obj) and other.ref()._obj is not value.ref()._obj
