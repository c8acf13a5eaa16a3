"""Lists of tensors at the lengths and sizes where the launches are cut: the gradients'
2-norm, the AdamW update and the values of 8-bit states; what autograd is told of a step.
u = 2^-24, 2^-8 bf16's half step; bounds as derived beside the same checks of short lists.
"""
import math

import numpy as np
import pytest
import torch

import mixture_experts_layer_gate_amd as moe
import test_gpu_train_ops as ops
from oracle import train_oracle as to

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8
BF16, F32 = torch.bfloat16, torch.float32


def _say(msg):
    print(msg, flush=True)


# ---------------------------------------------------------- values of states ----
def _values(code, scale, fraction):
    """float64 values of codes by the definition's table."""
    table = torch.from_numpy(to.code_values(fraction)).cuda()
    c = code.long()
    sign = torch.where(c >= 128, -1.0, 1.0).double() if fraction == 3 else 1.0
    v = sign * table[c & 127 if fraction == 3 else c]
    e = scale.long().repeat_interleave(128)[:c.numel()]
    return torch.where(e == 255, torch.full_like(v, math.nan), v * torch.exp2(e.double() - 127.0))


def _random_states(sizes, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    byte = lambda n, lo=0, hi=256: torch.randint(lo, hi, (n,), generator=gen, device="cuda", dtype=torch.uint8)  # noqa: E731
    m, v = ([byte(n) for n in sizes] for _ in range(2))
    ms, vs = ([byte(-(-n // 128), 100, 160) for n in sizes] for _ in range(2))
    for t in ms + vs:
        t[-1] = 255 if t.numel() > 1 else 130
    return moe.AdamState([torch.zeros(n, device="cuda", dtype=BF16) for n in sizes], m, v, ms, vs)


@pytest.mark.parametrize("sizes", [[5] * 56, [130] * 57, [300, 1] * 32, [7] * 126 + [2049], [9000005], [14000077], [23000077]],
                         ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_state_values_of_long_lists_and_large_tensors(dt, sizes):
    _say(f"state values, {len(sizes)} tensors of {sizes[0]}, {dt}")
    st = _random_states(sizes, 4)
    pad = 64
    outs = [[torch.full((n + 2 * pad,), 77.0, device="cuda", dtype=dt) for n in sizes] for _ in range(2)]
    views = [[t[pad:pad + n] for t, n in zip(ts, sizes)] for ts in outs]
    m, r = moe.adam_state_values(st, m=views[0], r=views[1])
    torch.cuda.synchronize()
    for got, codes, scales, fr in ((m, st.m, st.m_scale, 3), (r, st.v, st.v_scale, 4)):
        for a, c, s in zip(got, codes, scales):
            want = _values(c, s, fr).float().to(dt)
            assert torch.equal(torch.isnan(a), torch.isnan(want)) and torch.equal(a.nan_to_num(7.0), want.nan_to_num(7.0))
    for t in outs[0] + outs[1]:
        assert bool((t[:pad] == 77).all()) and bool((t[-pad:] == 77).all())


def test_state_values_into_roots_alone():
    """The type is that of the tensors that are given, the roots' as well as the first moments'."""
    st = _random_states([300, 5], 6)
    m, r = moe.adam_state_values(st, dtype=F32)
    for given in (dict(m=[torch.empty_like(t) for t in m]), dict(r=[torch.empty_like(t) for t in r])):
        a, b = moe.adam_state_values(st, **given)
        assert all(t.dtype is F32 for t in a + b)
        assert all(torch.equal(x.nan_to_num(7.0), y.nan_to_num(7.0)) for x, y in zip(a + b, m + r))
    with pytest.raises(ValueError, match="dtype"):
        moe.adam_state_values(st, m=[t.to(BF16) for t in m], r=r)


# -------------------------------------------------------------------- 2-norm ----
@pytest.mark.parametrize("sizes", [[5] * 167 + [9000], [5] * 168 + [9000], [17] * 169, [17] * 170 + [1], [3] * 337, [3] * 340 + [8193],
                                   [34000003], [68000003, 1]], ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_grad_norm_of_long_lists_and_large_tensors(dt, sizes):
    _say(f"2-norm, {len(sizes)} tensors of {sizes[0]}, {dt}")
    gs = ops._ragged(sizes, (dt,), 8)
    total = math.sqrt(math.fsum(float(g.double().pow(2).sum()) for g in gs))
    out = moe.grad_norm(gs, 0.5, 1.0)
    assert abs(float(out[0]) - 0.5 * total) <= 1.01 * U * 0.5 * total
    f = 0.5 * min(1.0, 1.0 / (0.5 * total + 1e-6))
    assert abs(float(out[1]) - f) <= 1.01 * U * f


# -------------------------------------------------------------------- update ----
@pytest.mark.parametrize("count", [39, 40, 41, 48, 49, 50, 98, 99])
@pytest.mark.parametrize("bits", [32, 8])
def test_adam_lists_around_a_launch(bits, count):
    sizes = [(37 * i) % 140 + 1 for i in range(count)]
    ps, grads = ops._params(sizes, (F32, BF16), 4), ops._ragged(sizes, (BF16, F32, F32), 5)
    st, opts = moe.adam_state(ps, bits), moe.AdamOptions(weight_decay=0.01)
    was = ops._snapshot(st)
    moe.adam_step(opts, st, grads, lr=1e-3, step=1, rng=torch.tensor([11, 12], device="cuda"))
    ops._check_step(st, was, grads, opts, 1e-3, 1, 1.0, 11, 12)


@pytest.mark.parametrize("pd,gd,master,stochastic", [(BF16, F32, True, False), (F32, F32, False, False), (BF16, BF16, False, True),
                                                     (F32, BF16, False, False)])
@pytest.mark.parametrize("bits", [32, 8])
def test_adam_of_large_tensors(bits, pd, gd, master, stochastic):
    """Lists over 128 MB, which stream past the cache: with 32-bit states every element, and windows at the ends and in
    between against the oracle, codes and numbers among them."""
    n = (16 << 20) + 1077
    _say(f"AdamW of {n} elements, {bits} bits, {pd} {gd} master {master} stochastic {stochastic}")
    gen = torch.Generator(device="cuda").manual_seed(2)
    p = (torch.randn(n, generator=gen, device="cuda") * 0.1).to(pd)
    g = torch.randn(n, generator=gen, device="cuda").to(gd)
    st = moe.adam_state([p], bits, master)
    opts, rng = moe.AdamOptions(weight_decay=0.1, stochastic=stochastic), torch.tensor([7, 8], device="cuda")
    moe.adam_step(opts, st, [g], lr=1e-2, step=1, rng=rng)
    g = torch.randn(n, generator=gen, device="cuda").to(gd)
    was = ops._snapshot(st)
    moe.adam_step(opts, st, [g], lr=1e-2, step=2, rng=rng)
    torch.cuda.synchronize()
    b1, b2, gd64 = 0.9, 0.999, g.double()
    if bits == 32:
        m0, v0 = was["m"][0].double(), was["v"][0].double()
        m1, v1 = b1 * m0 + (1 - b1) * gd64, b2 * v0 + (1 - b2) * gd64 ** 2
        tm = (b1 * m0).abs() + ((1 - b1) * gd64).abs()
        assert bool(((st.m[0].double() - m1).abs() <= 4 * U * tm + 2.0 ** -149).all())
        assert bool(((st.v[0].double() - v1).abs() <= 6 * U * v1 + 2.0 ** -148).all())
        w0 = (was["master"] if master else was["params"])[0].double()
        up = 1e-2 / (1 - b1 ** 2) / (torch.sqrt(v1 / (1 - b2 ** 2)) + 1e-8)
        w1 = w0 - up * m1 - 1e-3 * w0
        bound = up * (4 * U * tm + 12 * U * m1.abs()) + 4e-3 * U * w0.abs() + 2 * U * (w0.abs() + w1.abs())
        got = (st.master if master else st.params)[0].double()
        if pd is BF16 and not master:
            bound = bound + (2 if stochastic else 1) * BF * w1.abs().clamp(min=2.0 ** -126)
        assert bool(((got - w1).abs() <= bound).all())
        if master:
            assert torch.equal(st.params[0], st.master[0].to(BF16))
    # windows of whole blocks, against the oracle (codes and numbers among them)
    for a in (0, 4096 * 1000 - 640, n // 256 * 128, (n - 1300) // 128 * 128):
        b = min(n, a + 1408)
        cut = lambda ts, q=1: None if ts is None else [ts[0][a // q:-(-b // q)]]  # noqa: E731
        part = moe.AdamState(cut(st.params), cut(st.m), cut(st.v), cut(st.m_scale, 128), cut(st.v_scale, 128), cut(st.master))
        before = {k: cut(ts, 128 if k.endswith("scale") else 1) for k, ts in was.items()}
        _numbers, first = to.numbers, a
        try:  # the window's elements have the tensor's numbers
            to.numbers = lambda k, base, seed, off: _numbers(k, base + first, seed, off)
            ops._check_step(part, before, [g[a:b]], opts, 1e-2, 2, 1.0, 7, 8)
        finally:
            to.numbers = _numbers


def test_block_training_step_with_8_bit_states():
    """The block's step once more: its update of weights, codes and scales against the formula on its gradients."""
    dims, t, params = ops._block_inputs(70, 256, 256, 8, 2, 3)
    st = moe.adam_state([q.clone() for q in params], 8, True)
    opts = moe.AdamOptions(weight_decay=0.1)
    was = ops._snapshot(st)
    got = ops._block_step(dims, t, st, opts)
    torch.cuda.synchronize()
    flat = moe.AdamState(*[None if ts is None else [None if q is None else q.reshape(-1) for q in ts] for ts in (
        st.params, st.m, st.v, st.m_scale, st.v_scale, st.master)])
    was = {n: None if ts is None else [None if q is None else q.reshape(-1) for q in ts] for n, ts in was.items()}
    ops._check_step(flat, was, [g.reshape(-1) for g in got["grads"]], opts, 1e-3, 1, float(got["norm"][1]),
                    int(t["opt_rng"][0]), int(t["opt_rng"][1]))
    assert all(bool((c != 0).any()) for ts in (st.m, st.v, st.m_scale, st.v_scale) for c in ts)
    assert all(not torch.equal(a, b.reshape(a.shape)) for a, b in zip(st.params, was["params"]))


# ------------------------------------------------------------------ autograd ----
@pytest.mark.parametrize("bits", [32, 8])
def test_autograd_sees_a_step(bits):
    """A graph that saved a weight (or its master) before a step refuses to be differentiated after it."""
    w, u = torch.nn.Parameter(torch.randn(300, device="cuda")), torch.nn.Parameter(torch.randn(5, device="cuda").to(BF16))
    st = moe.adam_state([w, u], bits, True)
    rng = torch.tensor([1, 2], device="cuda")
    grads = [torch.ones(300, device="cuda"), torch.ones(5, device="cuda")]
    for t in (w, u):
        loss = (t * t).sum()
        before = t._version
        moe.adam_step(moe.AdamOptions(), st, grads, lr=1e-3, step=1, rng=rng)
        assert t._version > before
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    master = st.master[1]._version
    moe.adam_step(moe.AdamOptions(), st, moe.GradList(grads), lr=1e-3, step=2, rng=rng)
    assert st.master[1]._version > master
    (w * w).sum().backward()  # a graph made after the step is as before
    assert torch.equal(w.grad, 2 * w)
    # a refused step changes nothing
    before = w._version
    with pytest.raises(moe.MoeError):
        moe.adam_step(moe.AdamOptions(), st, grads, lr=1e-3, step=0, rng=rng)
    assert w._version == before
    # tensors made for inference have no counter
    with torch.inference_mode():
        q = moe.adam_state([torch.ones(9, device="cuda")], bits)
        moe.adam_step(moe.AdamOptions(), q, [torch.ones(9, device="cuda")], lr=1e-3, step=1, rng=rng)
    moe.adam_step(moe.AdamOptions(), q, [torch.ones(9, device="cuda")], lr=1e-3, step=2, rng=rng)


def test_autograd_sees_a_step_of_views():
    """Parameters that are views of one buffer, and of a view's view: the buffer and each of them."""
    flat, other = torch.randn(600, device="cuda"), torch.randn((4, 9), device="cuda")
    ps = [flat[:300], flat[300:600].view(30, 10), other[1], other.view(-1)[18:27], torch.nn.Parameter(flat.new_zeros(7))]
    st, x = moe.adam_state(ps), torch.ones(300, device="cuda", requires_grad=True)
    losses = [(x[: p.numel()] * p.reshape(-1)).sum() for p in ps] + [(x[0] * flat).sum(), (x[0] * other).sum()]
    moe.adam_step(moe.AdamOptions(), st, [torch.ones(p.numel(), device="cuda") for p in ps], lr=1e-3, step=1)
    for loss in losses:
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
