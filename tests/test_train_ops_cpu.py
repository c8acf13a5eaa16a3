"""The oracle of the norm, the gradients' 2-norm and the AdamW update against
independent statements of them (torch's own functions in float64, automatic and
finite differences, exhaustive rounding), and the refusals of the entry points.
Host-only: no call reaches a launch."""
import copy
import ctypes
import math
import os
import pickle

import numpy as np
import pytest
import torch

import mixture_experts_layer_gate_amd as moe
from mixture_experts_layer_gate_amd import api
from oracle import router_oracle as ro
from oracle import train_oracle as to

built = pytest.mark.skipif(not os.path.exists(moe.library_path()), reason="HIP library not built")
needs_no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="host-only validation test")
A = 0x10000  # 256-byte aligned placeholder, never dereferenced
BIG = 1 << 50


# ------------------------------------------------------------------ oracle ----
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_against_torch_and_differences(rng, kind):
    T, d, eps = 5, 24, 1e-3
    s, w, b, dy = (rng.standard_normal(n) for n in ((T, d), d, d, (T, d)))
    b = b if kind == "layer" else None
    y, mean, rstd = to.norm(s, w, b, kind, eps)

    def f(x, wt, bt):
        if kind == "layer":
            return torch.nn.functional.layer_norm(x, (d,), wt, bt, eps)
        return torch.nn.functional.rms_norm(x, (d,), wt, eps)
    ts, tw = (torch.from_numpy(a).requires_grad_(True) for a in (s, w))
    tb = torch.from_numpy(b).requires_grad_(True) if b is not None else None
    out = f(ts, tw, tb)
    np.testing.assert_allclose(y, out.detach().numpy(), rtol=1e-12, atol=1e-13)
    got = to.norm_backward(dy, s, w, kind, mean, rstd, dx_in=dy)
    want = torch.autograd.grad((out * torch.from_numpy(dy)).sum(), [ts, tw] + ([tb] if tb is not None else []))
    np.testing.assert_allclose(got[0], want[0].numpy() + dy, rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(got[1], want[1].numpy(), rtol=1e-10, atol=1e-12)
    if tb is not None:
        np.testing.assert_allclose(got[2], want[2].numpy(), rtol=1e-12)
    # central differences along a random direction: error of order h^2
    v, h = rng.standard_normal((T, d)), 1e-5
    num = sum(((to.norm(s + e * v, w, b, kind, eps)[0] * dy).sum() * e) for e in (h, -h)) / (2 * h * h)
    assert abs(num - ((got[0] - dy) * v).sum()) < 1e-6


def test_update_against_torch_over_steps(rng):
    """Eight steps of torch's AdamW in float64."""
    n, lr, b1, b2, eps, wd = 50, 3e-3, 0.9, 0.95, 1e-6, 0.1
    w = rng.standard_normal(n)
    p = torch.nn.Parameter(torch.from_numpy(w.copy()))
    opt = torch.optim.AdamW([p], lr=lr, betas=(b1, b2), eps=eps, weight_decay=wd)
    m, v = np.zeros(n), np.zeros(n)
    for t in range(1, 9):
        g = rng.standard_normal(n) * 10.0 ** rng.integers(-4, 2)
        p.grad = torch.from_numpy(g)
        opt.step()
        m, v = to.adam_moments(g, 1.0, m, v, b1, b2)
        w = to.adam_update(w, m, v, lr, t, b1, b2, eps, wd)
    np.testing.assert_allclose(w, p.detach().numpy(), rtol=1e-11)


def test_grad_norm_against_torch(rng):
    gs = [rng.standard_normal(n) for n in (1, 7, 300)]
    ps = [torch.nn.Parameter(torch.zeros(g.size, dtype=torch.float64)) for g in gs]
    for p, g in zip(ps, gs):
        p.grad = torch.from_numpy(g.copy())
    total = float(torch.nn.utils.clip_grad_norm_(ps, 0.5))
    n, f = to.grad_norm(gs, 1.0, 0.5)
    assert abs(n - total) < 1e-12 * total
    np.testing.assert_allclose(gs[2] * f, ps[2].grad.numpy(), rtol=1e-12)
    n, f = to.grad_norm([4.0 * g for g in gs], 0.25, 1e9)
    assert abs(n - total) < 1e-12 * total and f == 0.25


def test_numbers_are_those_of_the_dropout():
    """An element is kept where its number is at least the threshold."""
    seed, off = 0x123456789ABC, 0x7FFF00000003
    u = to.numbers(200, 64, seed, off)
    assert ((u >= 16384) == ro.keep_mask(264, seed, off, 0.25)[64:]).all()


@pytest.mark.parametrize("fraction", [3, 4])
def test_codes(fraction):
    """Ascending values, doubling by binade; decode inverts encode on the values themselves, whatever the number."""
    t = to.code_values(fraction)
    assert (np.diff(t) > 0).all() and t[0] == 0 and t[-1] == 2.0 - 2.0 ** -fraction
    k = 1 << fraction
    np.testing.assert_array_equal(t[2 * k:], 2 * t[k:-k])
    for e in (1, 100, 127, 190, 254):
        x = (t * 2.0 ** (e - 127)).astype(np.float32)
        x = x[x == t * 2.0 ** (e - 127)]  # (those that fp32 holds)
        x = np.concatenate([x[-to.BLOCK:], -x[-100:] if fraction == 3 else x[-100:]])
        for u in (0, 65535):
            c, s = to.encode(x, np.full(x.size, u), fraction)
            np.testing.assert_array_equal(to.decode(c, s, fraction), x.astype(np.float64))


@pytest.mark.parametrize("fraction", [3, 4])
def test_rounding_is_unbiased(rng, fraction):
    """Over all 65536 numbers the codes' mean is the value, to the number's own grid (2^-16 of a step); the root's
    least code is taken by what would else be 0."""
    x = (rng.standard_normal(to.BLOCK) * np.exp(rng.standard_normal(to.BLOCK))).astype(np.float32)
    if fraction == 4:
        x = np.abs(x)
    table = to.code_values(fraction)
    lo, hi = (to.decode(*to.encode(x, np.full(to.BLOCK, u), fraction), fraction) for u in (0, 65535))
    assert (np.abs(lo) <= np.abs(x)).all() and (np.abs(hi) >= np.abs(x) * (1 - 1e-3)).all()
    mean = np.zeros(to.BLOCK)
    us = range(0, 65536, 64)
    for u in us:
        mean += to.decode(*to.encode(x, np.full(to.BLOCK, u), fraction), fraction)
    mean /= len(us)
    top = 2.0 ** (float(to.encode(x, np.zeros(to.BLOCK), fraction)[1][0]) - 127)
    step = np.maximum(np.abs(x) / 2 ** fraction, top * table[1])
    live = np.abs(x) > top * table[1]
    assert (np.abs(mean - x)[live] <= step[live] / 512).all()


# ---------------------------------------------------------------- refusals ----
def _dims(**kw):
    base = dict(T=64, d=128, f=256, E=8, k=2, dtype=1)
    base.update(kw)
    return ctypes.byref(api._Dims(base["T"], base["d"], base["f"], base["E"], base["k"], base["dtype"]))


def _nopts(kind=1, pt=0, eps=1e-5):
    return ctypes.byref(api._NormOpts(kind, pt, eps))


@built
@needs_no_gpu
def test_norm_refusals():
    lib = moe.load_library()
    fwd, bwd, d, o = lib.moe_norm_forward, lib.moe_norm_backward, _dims(), _nopts()
    for bad in (_nopts(kind=2), _nopts(kind=-1), _nopts(pt=3), _nopts(eps=0.0), _nopts(eps=-1.0), _nopts(eps=math.nan),
                _nopts(eps=math.inf), _nopts(eps=1e-38), None):
        assert fwd(d, bad, A, None, A, A, None, A, None, None, None) == 1
        assert bwd(d, bad, A, A, A, A, A, None, A, A, A, A, BIG, None) == 1
        assert lib.moe_norm_backward_workspace_bytes(d, bad) == 0
    for dm, want in ((_dims(d=100), 2), (_dims(d=16392), 2), (_dims(k=9), 1), (_dims(T=-1), 1)):
        assert fwd(dm, o, A, None, A, A, None, A, None, None, None) == want
        assert bwd(dm, o, A, A, A, A, A, None, A, A, A, A, BIG, None) == want
        assert lib.moe_norm_backward_workspace_bytes(dm, o) == 0
    # x, residual, weight, bias, sum, y, mean, rstd
    for args in ((None, None, A, A, None, A, None, None), (A + 8, None, A, A, None, A, None, None),
                 (A, A + 2, A, A, None, A, None, None), (A, None, A + 8, A, None, A, None, None),
                 (A, None, A, A + 4, None, A, None, None), (A, A, A, A, A + 8, A + 16, None, None),
                 (A, A, A, A, A, A, None, None), (A, None, A, A, None, None, None, None),
                 (A, None, A, A, None, A, A + 2, None), (A, None, A, A, None, A, None, A + 1)):
        assert fwd(d, o, *args, None) == 1, args
    assert fwd(d, _nopts(kind=0), A, None, A, A, None, A, None, None, None) == 1   # RMS with a bias
    assert fwd(d, _nopts(kind=0), A, None, A, None, None, A, A, None, None) == 1   # RMS with a mean
    assert fwd(_dims(T=0), o, None, None, None, None, None, None, None, None, None) == 0
    # dy, s, weight, mean, rstd, dx_in, dx, dweight, dbias, ws, bytes
    need = lib.moe_norm_backward_workspace_bytes(d, o)
    assert need >= 2 * 128 * 4
    for args, want in (((None, A, A, A, A, None, A, A, A, A, need), 1), ((A, A + 8, A, A, A, None, A, A, A, A, need), 1),
                       ((A, A, A + 2, A, A, None, A, A, A, A, need), 1), ((A, A, A, None, A, None, A, A, A, A, need), 1),
                       ((A, A, A, A, None, None, A, A, A, A, need), 1), ((A, A, A, A, A, A + 8, A, A, A, A, need), 1),
                       ((A, A, A, A, A, None, None, A, A, A, need), 1), ((A, A, A, A, A, None, A, A + 4, A, A, need), 1),
                       ((A, A, A, A, A, None, A, A, A + 8, A, need), 1), ((A, A, A, A, A, None, A, A, A, A, need - 1), 3),
                       ((A, A, A, A, A, None, A, A, A, None, need), 3), ((A, A, A, A, A, None, A, A, A, A + 64, need), 1)):
        assert bwd(d, o, *args, None) == want, args
    assert bwd(d, _nopts(kind=0), A, A, A, None, A, None, A, A, A, A, BIG, None) == 1   # RMS has no bias


def _grads(*rows):
    return (ctypes.c_int64 * (3 * len(rows)))(*[v for r in rows for v in r])


@built
@needs_no_gpu
def test_grad_norm_refusals():
    lib = moe.load_library()
    good = _grads((A, 5, 0), (0, 0, 1), (A + 2, 9, 1))
    size, fn = lib.moe_grad_norm_workspace_bytes, lib.moe_grad_norm
    assert size(good, 3) >= 16 and size(None, 0) > 0
    for bad in (_grads((A, -1, 0)), _grads((0, 5, 0)), _grads((A + 2, 5, 0)), _grads((A + 1, 5, 1)), _grads((A, 5, 2))):
        assert size(bad, 1) == 0 and fn(bad, 1, 1.0, 1.0, A, A, BIG, None) == 1
    assert fn(_grads((A, (1 << 36) + 1, 0)), 1, 1.0, 1.0, A, A, BIG, None) == 2
    assert fn(good, -1, 1.0, 1.0, A, A, BIG, None) == 1 and fn(None, 1, 1.0, 1.0, A, A, BIG, None) == 1
    assert fn(good, (1 << 20) + 1, 1.0, 1.0, A, A, BIG, None) == 2
    for scale, most in ((math.inf, 1.0), (math.nan, 1.0), (1.0, -1.0), (1.0, math.nan)):
        assert fn(good, 3, scale, most, A, A, BIG, None) == 1
    assert fn(good, 3, 1.0, 1.0, None, A, BIG, None) == 1 and fn(good, 3, 1.0, 1.0, A + 2, A, BIG, None) == 1
    assert fn(good, 3, 1.0, 1.0, A, None, BIG, None) == 3 and fn(good, 3, 1.0, 1.0, A, A + 8, BIG, None) == 1
    assert fn(good, 3, 1.0, 1.0, A, A, 8, None) == 3


def _aopts(**kw):
    base = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1, step=3, state_bits=32, stochastic=0)
    base.update(kw)
    return ctypes.byref(api._AdamOpts(*(base[n] for n in ("lr", "beta1", "beta2", "eps", "weight_decay", "step",
                                                          "state_bits", "stochastic"))))


def _tensors(*rows):
    return (ctypes.c_int64 * (8 * len(rows)))(*[v for r in rows for v in r])


@built
@needs_no_gpu
def test_adam_refusals():
    lib = moe.load_library()
    fn = lib.moe_adam_step
    P = [A + 0x1000 * i for i in range(20)]
    # param, master, m, v, m_scale, v_scale, n, dtype
    good = (P[0], 0, P[1], P[2], P[3], P[4], 5, 1)
    t, g = _tensors(good), _grads((P[9], 5, 0))
    for bad in (dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=math.nan), dict(eps=0.0), dict(eps=math.inf),
                dict(eps=1e-35), dict(weight_decay=math.inf), dict(lr=math.nan), dict(step=0), dict(state_bits=16),
                dict(stochastic=2), dict(stochastic=1), dict(state_bits=8)):  # (the last two without rng)
        assert fn(_aopts(**bad), t, g, 1, None, None, None, None) == 1, bad
    assert fn(None, t, g, 1, None, None, None, None) == 1
    assert fn(_aopts(), t, g, 1, A + 4, None, None, None) == 1
    assert fn(_aopts(), t, g, 1, None, A + 2, None, None) == 1
    assert fn(_aopts(), t, g, 1, None, None, A + 4, None) == 1
    assert fn(_aopts(lr=math.nan, step=0), t, g, 0, A, None, None, None) == 0  # not looked at beside lr_step

    def changed(**kw):
        names = ("param", "master", "m", "v", "m_scale", "v_scale", "n", "dtype")
        row = dict(zip(names, good))
        row.update(kw)
        return _tensors(tuple(row[n] for n in names))
    for bad in (dict(param=0), dict(param=A + 1), dict(dtype=0, param=P[0] + 2), dict(m=0), dict(v=0), dict(m=P[1] + 2),
                dict(v=P[2] + 1), dict(master=P[5] + 2), dict(master=P[5], dtype=0), dict(dtype=2), dict(n=-1), dict(n=6),
                dict(m=P[2]), dict(v=P[0]), dict(master=P[1]), dict(m=P[9])):
        assert fn(_aopts(), changed(**bad), g, 1, None, None, None, None) == 1, bad
    for bad in (dict(m_scale=0), dict(v_scale=0), dict(m_scale=P[4]), dict(v_scale=P[0])):
        assert fn(_aopts(state_bits=8), changed(**bad), g, 1, None, None, A, None) == 1, bad
    assert fn(_aopts(), changed(n=(1 << 36) + 1), _grads((P[9], (1 << 36) + 1, 0)), 1, None, None, None, None) == 2
    # the same tensor twice
    other = (P[10], 0, P[11], P[12], 0, 0, 5, 1)
    assert fn(_aopts(), _tensors(good, good), _grads((P[9], 5, 0), (P[13], 5, 0)), 2, None, None, None, None) == 1
    assert fn(_aopts(), _tensors(good, other[:2] + (P[1],) + other[3:]), _grads((P[9], 5, 0), (P[13], 5, 0)), 2, None,
              None, None, None) == 1
    assert fn(_aopts(), t, None, 1, None, None, None, None) == 1 and fn(_aopts(), None, g, 1, None, None, None, None) == 1
    assert fn(_aopts(), t, g, -1, None, None, None, None) == 1
    assert fn(_aopts(), t, g, (1 << 20) + 1, None, None, None, None) == 2
    assert fn(_aopts(), _tensors((0, 0, 0, 0, 0, 0, 0, 1)), _grads((0, 0, 0)), 1, None, None, None, None) == 0
    val = lib.moe_adam_state_values
    ptr = (ctypes.c_int64 * 1)(A)
    assert val(t, 1, ptr, ptr, 2, None) == 1 and val(t, 1, None, ptr, 1, None) == 1 and val(t, -1, ptr, ptr, 1, None) == 1
    assert val(t, 1, (ctypes.c_int64 * 1)(0), ptr, 1, None) == 1
    assert val(t, 1, (ctypes.c_int64 * 1)(A + 2), ptr, 0, None) == 1
    assert val(changed(m_scale=0), 1, ptr, ptr, 1, None) == 1
    assert val(None, 0, None, None, 1, None) == 0


@built
def test_binding_refusals():
    dims, cpu = moe.Dims(4, 64, 64, 8, 2), torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="kind"):
        moe.NormOptions(kind="batch")
    with pytest.raises(ValueError, match="param_dtype"):
        moe.NormOptions(param_dtype=torch.float16)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.norm_forward(dims, moe.NormOptions(), cpu)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.norm_backward(dims, moe.NormOptions(), cpu, cpu, None, cpu)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.grad_norm([torch.zeros(5)])
    with pytest.raises(ValueError, match="empty"):
        moe.grad_norm([])
    with pytest.raises(ValueError, match="dtype"):
        moe.GradList([torch.zeros(5, dtype=torch.float64)])
    with pytest.raises(ValueError, match="contiguous"):
        moe.GradList([torch.zeros((5, 4)).t()])
    p = [torch.zeros(300), torch.zeros(5)]
    with pytest.raises(ValueError, match="bits"):
        moe.adam_state(p, bits=16)
    st = moe.adam_state(p)
    opts, g = moe.AdamOptions(), [torch.ones(300), torch.ones(5)]
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.adam_step(opts, st, g, lr=1e-3, step=1)
    with pytest.raises(ValueError, match="lr and step"):
        moe.adam_step(opts, st, g, lr=1e-3)
    with pytest.raises(ValueError, match="expected 2"):
        moe.adam_step(opts, st, g[:1], lr=1e-3, step=1)
    with pytest.raises(ValueError, match="rng"):
        moe.adam_step(moe.AdamOptions(stochastic=True), st, g, lr=1e-3, step=1)
    with pytest.raises(ValueError, match="not held in 8 bits"):
        moe.adam_state_values(st)
    f = torch.zeros(600)
    with pytest.raises(ValueError, match="overlap"):
        moe.AdamState([f[:300]], [f[299:599]], [torch.zeros(300)])
    with pytest.raises(ValueError, match="overlap"):
        moe.AdamState([f[:300], f[:300]], [torch.zeros(300), torch.zeros(300)], [torch.zeros(300), torch.zeros(300)])
    with pytest.raises(ValueError, match="elements"):
        moe.AdamState([f[:300]], [torch.zeros(299)], [torch.zeros(300)])
    with pytest.raises(ValueError, match="master"):
        moe.AdamState([f[:300]], [torch.zeros(300)], [torch.zeros(300)], master=[torch.zeros(300)])
    with pytest.raises(ValueError, match="m_scale"):
        moe.AdamState([f[:300]], [torch.zeros(300, dtype=torch.uint8)], [torch.zeros(300, dtype=torch.uint8)])
    with pytest.raises(ValueError, match="m_scale"):
        moe.AdamState([f[:300]], [torch.zeros(300)], [torch.zeros(300)], [torch.zeros(3)], [torch.zeros(3)])
    with pytest.raises(ValueError, match="dtype"):
        moe.AdamState([f[:300]], [torch.zeros(300, dtype=torch.uint8)], [torch.zeros(300)], [torch.zeros(3)], [torch.zeros(3)])


@pytest.mark.parametrize("bits", [8, 32])
def test_states_are_copied_with_their_tensors(bits):
    """A copy works on its own tensors, not on the addresses of the first."""
    st = moe.adam_state([torch.ones(300).bfloat16(), torch.zeros(7)], bits, master=True)
    for other in (copy.deepcopy(st), pickle.loads(pickle.dumps(st))):
        assert other.bits == bits and other.master[1] is None and torch.equal(other.master[0], st.master[0])
        mine, theirs = set(st._rows[k] for k in (0, 1, 2, 3, 8)), set(other._rows[k] for k in (0, 1, 2, 3, 8))
        assert not mine & theirs and other._rows[0] == other.params[0].data_ptr()
    g = moe.GradList([torch.ones(5)])
    h = copy.deepcopy(g)
    assert h._rows[0] == h.tensors[0].data_ptr() != g._rows[0]
    for value in (moe.NormOptions("layer"), moe.AdamOptions(beta2=0.9)):
        assert pickle.loads(pickle.dumps(value)) == value


def test_checked_lists_are_fixed():
    """What the lists hold was read when they were made: it is not exchanged under them."""
    st, g = moe.adam_state([torch.zeros(7)]), moe.GradList([torch.zeros(7)])
    with pytest.raises(AttributeError, match="fixed"):
        st.m = [torch.zeros(7)]
    with pytest.raises(TypeError):
        st.m[0] = torch.zeros(7)
    with pytest.raises(AttributeError, match="fixed"):
        g.tensors = [torch.zeros(7)]
    with pytest.raises(TypeError):
        g.tensors[0] = torch.zeros(7)
    assert moe.grad_norm_workspace_bytes(g) == moe.grad_norm_workspace_bytes(g) > 0 if os.path.exists(
        moe.library_path()) else True


def test_workspace_size_of_a_list_asked_for_by_two_threads(monkeypatch):
    """The second asks while the first one's query runs: both get the size."""
    g, deep, sizes = moe.GradList([torch.ones(5)]), [], []

    class Lib:
        def moe_grad_norm_workspace_bytes(self, ptr, count):
            if not deep:
                deep.append(1)
                sizes.append(moe.grad_norm_workspace_bytes(g))
            return 512

    monkeypatch.setattr(api, "load_library", Lib)
    assert moe.grad_norm_workspace_bytes(g) == 512 and sizes == [512] and moe.grad_norm_workspace_bytes(g) == 512
