"""The edges of what the norm, the gradient norm and the AdamW update accept:
offsets past 32 bits, moments of every size in 8-bit states, lists of nothing,
stage timing. Against the formulas and the float64 oracle (oracle/train_oracle.py);
u = 2^-24, 2^-8 bf16's half step.
"""
import math

import numpy as np
import pytest
import torch

import mixture_experts_layer_gate_amd as moe
from oracle import train_oracle as to

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8
BF16, F32 = torch.bfloat16, torch.float32


def _say(msg):
    print(msg, flush=True)


def test_tensors_past_32_bit_offsets():
    """A tensor of 2^32 + 5777 elements (bytes past 2^33): its norm, and a step whose first and last elements, and those
    around 2^31 and 2^32, are the formula's."""
    n = 2 ** 32 + 5777  # (the windows below lie apart)
    places = [0, 2 ** 31 - 640, 2 ** 32 - 640, n - 1289]
    g = torch.zeros(n, dtype=BF16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    for a in places:
        g[a:a + 1280] = torch.randn(1280, generator=gen, device="cuda").to(BF16)
    total = math.sqrt(sum(float(g[a:a + 1280].double().pow(2).sum()) for a in places))
    _say("2-norm of 2^32 + 5777 elements")
    out = moe.grad_norm([g, g[:5]], 1.0, 1.0)
    total = math.sqrt(total ** 2 + float(g[:5].double().pow(2).sum()))
    assert abs(float(out[0]) - total) <= 1.01 * U * total
    for bits in (8, 32):
        _say(f"AdamW of 2^32 + 5777 elements, {bits} bits")
        p = torch.full((n,), 0.5, dtype=BF16, device="cuda")
        st = moe.adam_state([p], bits)
        moe.adam_step(moe.AdamOptions(), st, [g], lr=0.25, step=1, rng=torch.tensor([7, 8], device="cuda"))
        torch.cuda.synchronize()
        for a in places:
            # whole blocks of 128 inside the window
            lo = -(-a // 128) * 128 if a else 0
            hi = n if a == places[-1] else lo + 1024
            x = g[lo:hi].float().cpu().numpy()
            m, v = to.adam_moments(x, 1.0, np.zeros(x.size), np.zeros(x.size), 0.9, 0.999, np.float32)
            w = to.adam_update(np.full(x.size, 0.5), m, v, 0.25, 1, 0.9, 0.999, 1e-8, 0.0)
            assert (np.abs(p[lo:hi].double().cpu().numpy() - w) <= (BF + 32 * U) * np.maximum(np.abs(w), 0.25)).all()
            if bits == 8:
                u = to.numbers(hi - lo, lo, 7, 8)
                for y, code, scale, fr in ((m, st.m[0], st.m_scale[0], 3), (np.sqrt(v), st.v[0], st.v_scale[0], 4)):
                    c, e = to.encode(y, u, fr)
                    np.testing.assert_array_equal(code[lo:hi].cpu().numpy(), c)
                    np.testing.assert_array_equal(scale[lo // 128:-(-hi // 128)].cpu().numpy(), e)
            else:
                np.testing.assert_array_equal(st.m[0][lo:hi].cpu().numpy(), m)
        # nothing else moved
        assert float(p[5000:2 ** 31 - 2000].min()) == 0.5 and float(p[2 ** 31 + 2000:2 ** 32 - 2000].max()) == 0.5
        del p, st
        torch.cuda.empty_cache()


def test_norm_past_32_bit_offsets():
    """530000 x 8200 (4.3 G elements): the rows on both sides of each border against their own."""
    T, d = 530000, 8200
    dims, opts = moe.Dims(T, d, 64, 1, 1), moe.NormOptions("layer", 1e-5)
    x = torch.empty((T, d), dtype=BF16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(2)
    block = torch.randn((1000, d), generator=gen, device="cuda")
    for t in range(0, T, 1000):
        x[t:t + 1000] = (block * (1 + t / T)).to(BF16)
    y, _, mean, rstd = moe.norm_forward(dims, opts, x, keep=True)
    dx, dw, db = moe.norm_backward(dims, opts, x, x, None, rstd, mean=mean, want_dbias=True)
    torch.cuda.synchronize()
    few = moe.Dims(64, d, 64, 1, 1)
    for t in (0, 2 ** 31 // d - 32, 2 ** 32 // d - 32, T - 64):
        z = x[t:t + 64].clone()
        a, _, m, r = moe.norm_forward(few, opts, z, keep=True)
        assert torch.equal(a, y[t:t + 64]) and torch.equal(m, mean[t:t + 64]) and torch.equal(r, rstd[t:t + 64])
        e, _, _ = moe.norm_backward(few, opts, z, z, None, r, mean=m)
        assert torch.equal(e, dx[t:t + 64])
    s = torch.zeros(d, dtype=torch.float64, device="cuda")
    mag = torch.zeros(d, dtype=torch.float64, device="cuda")
    for t in range(0, T, 10000):
        s += x[t:t + 10000].double().sum(0)
        mag += x[t:t + 10000].double().abs().sum(0)
    assert bool(((db.double() - s).abs() <= (T / 256 + 64) * U * mag).all())


@pytest.mark.parametrize("exponent", [-149, -140, -127, -125, -100, -75, -60, -20, 0, 20, 60])
def test_codes_of_moments_of_every_size(exponent, rng):
    """Gradients of about 2^exponent: blocks of one size, of wide spreads, of single values; codes and scales equal to
    the definition's on the fp32 moments."""
    n = 128 * 12 + 77
    g = (rng.standard_normal(n) * 2.0 ** exponent).astype(np.float32)
    g[128:512] *= np.exp2(rng.integers(-30, 1, 384)).astype(np.float32)
    g[512:640] = 0
    g[600] = np.float32(2.0 ** exponent)
    g[640:768] = np.float32(1.9375 * 2.0 ** exponent)
    g[768:896] = np.float32(1.9375 * 2.0 ** exponent) * np.float32(1 + 2.0 ** -23)
    _say(f"codes at 2^{exponent}")
    st = moe.adam_state([torch.zeros(n, device="cuda")], 8)
    m, v = np.zeros(n, np.float32), np.zeros(n, np.float32)
    t = torch.from_numpy(g).cuda()
    for k in (1, 2, 3):
        moe.adam_step(moe.AdamOptions(beta1=0.5, beta2=0.75), st, [t], lr=1e-3, step=k, rng=torch.tensor([9, k], device="cuda"))
        m, v = to.adam_moments(g, 1.0, m, v, 0.5, 0.75, np.float32)
        u = to.numbers(n, 0, 9, k)
        new = []
        for x, code, scale, fr in ((m, st.m[0], st.m_scale[0], 3), (np.sqrt(v), st.v[0], st.v_scale[0], 4)):
            c, e = to.encode(x, u, fr)
            np.testing.assert_array_equal(scale.cpu().numpy(), e)
            np.testing.assert_array_equal(code.cpu().numpy(), c)
            new.append(to.decode(c, e, fr).astype(np.float32))
        m, v = new[0], new[1] * new[1]
    assert bool(torch.isfinite(st.params[0]).all())


def test_state_past_the_largest_exponent():
    """Moments at the end of fp32's range: a block whose largest lies above its top code reads as NaN."""
    g = torch.full((256,), 2.0 ** 127 * 1.75, device="cuda")
    g[128:] = 2.0 ** 127 * 1.96875
    st = moe.adam_state([torch.zeros(256, device="cuda")], 8)
    moe.adam_step(moe.AdamOptions(beta1=0.0), st, [g], lr=1e-3, step=1, rng=torch.tensor([1, 1], device="cuda"))
    assert st.m_scale[0].tolist() == [254, 255] and st.v_scale[0].tolist() == [255, 255]
    m, r = moe.adam_state_values(st, dtype=F32)
    assert bool((m[0][:128] == 2.0 ** 127 * 1.75).all()) and bool(torch.isnan(m[0][128:]).all())
    assert bool(torch.isnan(r[0]).all())


def test_empty_tensors_in_lists():
    z = torch.zeros(0, device="cuda")
    for bits in (32, 8):
        st = moe.adam_state([z.clone(), torch.ones(5, device="cuda"), z.clone(), z.clone().bfloat16()], bits, True)
        g = [z, torch.ones(5, device="cuda"), z, z]
        moe.adam_step(moe.AdamOptions(), st, g, lr=1e-2, step=1, rng=torch.tensor([1, 2], device="cuda"))
        assert torch.allclose(st.params[1], torch.full((5,), 0.99, device="cuda"), atol=1e-6)
        if bits == 8:
            m, _ = moe.adam_state_values(st)
            assert [t.numel() for t in m] == [0, 5, 0, 0]
    st = moe.adam_state([z])
    moe.adam_step(moe.AdamOptions(), st, [z], lr=1e-2, step=1)


def test_stage_timing_covers_the_new_calls():
    dims, opts = moe.Dims(4, 64, 64, 8, 2), moe.NormOptions()
    x = torch.randn((4, 64), device="cuda").to(BF16)
    g = [torch.ones(9, device="cuda")]
    st = moe.adam_state([torch.ones(9, device="cuda")])
    moe.timing_enable(4, ["norm", "norm_grad", "grad_norm", "adam"])
    _, s, _, r = moe.norm_forward(dims, opts, x, keep=True)
    moe.norm_backward(dims, opts, x, s, None, r)
    moe.grad_norm(g)
    moe.adam_step(moe.AdamOptions(), st, g, lr=1e-3, step=1)
    torch.cuda.synchronize()
    moe.timing_disable()
    for name in ("norm", "norm_grad", "grad_norm", "adam"):
        ms, n = moe.timing_read(name)
        assert n == 1 and ms > 0


def test_a_stream_of_steps_over_kept_gradients():
    """A GradList and states whose contents change between steps in place, one graph replayed for each: as eager calls on
    lists of the tensors."""
    sizes = [300, 4096, 1, 77777]
    gen = torch.Generator(device="cuda").manual_seed(3)
    ps = [torch.randn(n, generator=gen, device="cuda") for n in sizes]
    grads = [torch.zeros(n, device="cuda") for n in sizes]
    kept, a, b = moe.GradList(grads), moe.adam_state([p.clone() for p in ps], 8), moe.adam_state([p.clone() for p in ps], 8)
    out, ls = torch.zeros(2, device="cuda"), torch.tensor([1e-3, 1.0], dtype=torch.float64, device="cuda")
    rng, opts = torch.tensor([4, 0], device="cuda"), moe.AdamOptions(weight_decay=0.1)

    def step(st, g):
        moe.grad_norm(g, 1.0, 0.5, out=out)
        moe.adam_step(opts, st, g, lr_step=ls, gscale=out[1:], rng=rng)
    step(b, kept)  # zero gradients: weights decay; then back
    for p, q in zip(b.params, ps):
        p.copy_(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a, kept)
    for k in range(1, 5):
        for g in grads:
            g.copy_(torch.randn(g.numel(), generator=gen, device="cuda"))
        ls[1] = k
        rng[1] = k
        graph.replay()
        torch.cuda.synchronize()
        first = out.clone()
        step(b, list(grads))
        torch.cuda.synchronize()
        assert torch.equal(out, first)
        for n in ("params", "m", "v", "m_scale", "v_scale"):
            assert all(torch.equal(x, y) for x, y in zip(getattr(a, n), getattr(b, n))), (k, n)


def test_bench_update_line():
    """bench.py --backward --update: one JSON line that carries the norm's, the gradient norm's and the update's times."""
    import json
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    cmd = [sys.executable, os.path.join(root, "bench.py"), "--backward", "--update", "8", "--wgrad-bf16", "--workload",
           "mixtral_decode_t16", "--steps", "2", "--warmup", "1", "--no-cpu-baseline"]
    _say("bench --backward --update 8")
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stderr[-2000:]
    j = json.loads([l for l in r.stdout.splitlines() if l.startswith("{")][0])
    assert set(j["update"]["stages"]) == {"norm", "norm_grad", "grad_norm", "adam"}
    assert j["update"]["state_bits"] == 8 and all(v["ms"] > 0 for v in j["update"]["stages"].values())


@pytest.mark.parametrize("T,d", [(1030, 520), (1100, 1032), (1030, 4104), (1500, 7168), (2500, 2048), (700, 8192), (300, 12296)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_norm_backward_of_longer_batches(dt, kind, T, d):
    """Batches whose weight gradients are summed from parts of the rows, and wide ones summed by columns: every output, in
    place too, and with the bias' or the weight's gradient alone. Bounds as for the short ones, a part having at most
    T / 256 rows of its own."""
    layer = kind == "layer"
    half = BF if dt is BF16 else U
    _say(f"{kind} {dt} {T} x {d}")
    gen = torch.Generator(device="cuda").manual_seed(T + d)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, dy, di = (rn(T, d) + 0.5 * rn(T, 1)).to(dt), (rn(T, d) * 0.01).to(dt), (rn(T, d) * 0.01).to(dt)
    w = 1 + 0.2 * rn(d)
    dims, opts = moe.Dims(T, d, 64, 8, 2, dt), moe.NormOptions(kind, 1e-5)
    _, s, mean, rstd = moe.norm_forward(dims, opts, x, w, keep=True)
    dx, dw, db = moe.norm_backward(dims, opts, dy, s, w, rstd, mean=mean, dx_in=di, want_dbias=layer)
    nm = mean.double()[:, None] if layer else torch.zeros((T, 1), dtype=torch.float64, device="cuda")
    nr = rstd.double()[:, None]
    h, up = (s.double() - nm) * nr, dy.double()
    g = up * w.double()
    mgh, mg = (g * h).mean(1, keepdim=True), g.mean(1, keepdim=True)
    rx = nr * (g - h * mgh - (mg if layer else 0)) + di.double()
    bound = nr * U * (4 * g.abs() + 50 * h.abs() * (g * h).abs().mean(1, keepdim=True) + 46 * g.abs().mean(1, keepdim=True))
    assert bool(((dx.double() - rx).abs() <= bound + (half + 2 * U) * rx.abs() + 2 * U * di.double().abs()).all())
    rows = -(-T // 256) + 64
    assert bool(((dw.double() - (up * h).sum(0)).abs() <= (rows + 4) * U * (up * h).abs().sum(0)).all())
    if layer:
        assert bool(((db.double() - up.sum(0)).abs() <= rows * U * up.abs().sum(0)).all())
        only = moe.norm_backward(dims, opts, dy, s, w, rstd, mean=mean, dx_in=di, want_dweight=False, want_dbias=True)
        assert torch.equal(only[0], dx) and only[1] is None and torch.equal(only[2], db)
    only = moe.norm_backward(dims, opts, dy, s, w, rstd, mean=mean, dx_in=di)
    assert torch.equal(only[0], dx) and torch.equal(only[1], dw) and only[2] is None
    none = moe.norm_backward(dims, opts, dy, s, w, rstd, mean=mean, dx_in=di, want_dweight=False)
    assert torch.equal(none[0], dx)
    for k in range(3):
        t = [dy.clone(), s.clone(), di.clone()]
        got = moe.norm_backward(dims, opts, t[0], t[1], w, rstd, mean=mean, dx_in=t[2], dx=t[k], want_dbias=layer)
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw) and (not layer or torch.equal(got[2], db))


def test_sum_without_a_residual_is_x():
    """Through the C ABI: the sum's tensor takes x, and y is the norm of it."""
    lib = moe.load_library()
    for T, d, dt in ((5, 64, BF16), (3, 7168, BF16), (4, 1048, F32)):
        dims, opts = moe.Dims(T, d, 64, 8, 2, dt), moe.NormOptions("layer", 1e-5)
        x = torch.randn((T, d), device="cuda").to(dt)
        s, y = torch.zeros_like(x), torch.zeros_like(x)
        st = lib.moe_norm_forward(dims.ref(), opts.ref(), x.data_ptr(), None, None, None, s.data_ptr(), y.data_ptr(), None,
                                  None, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert st == 0 and torch.equal(s, x) and torch.equal(y, moe.norm_forward(dims, opts, x)[0])


def test_state_values_refuse_an_output_twice():
    st = moe.adam_state([torch.zeros(9, device="cuda"), torch.zeros(9, device="cuda")], 8)
    a, b, c = (torch.zeros(9, device="cuda") for _ in range(3))
    with pytest.raises(moe.MoeError):
        moe.adam_state_values(st, m=[a, b], r=[a, c])


@pytest.mark.parametrize("d", [256, 1032, 4104, 7168, 16384])
@pytest.mark.parametrize("offset", [1e2, 1e4, 1e6, -3e7])
def test_layer_norm_of_rows_far_from_zero(offset, d):
    """fp32 rows of unit spread around a large mean. What the mean's own rounding costs is taken back, so that y is off by
    the roundings of the differences (exact where x lies within a factor of two of the mean, else u of it, a size of the
    spread here) and of the row's sums over them: 60 u of a size of sqrt(d), and mean by its rounding as a number."""
    T = 7
    gen = torch.Generator(device="cuda").manual_seed(d)
    x = (torch.randn((T, d), generator=gen, device="cuda").double() * max(1.0, abs(offset) * 2.0 ** -20) + offset).float()
    dims, opts = moe.Dims(T, d, 64, 8, 2, F32), moe.NormOptions("layer", 1e-5)
    y, _, mean, rstd = moe.norm_forward(dims, opts, x, keep=True)
    z = x.double()
    mu = z.mean(1, keepdim=True)
    rs = 1 / torch.sqrt(((z - mu) ** 2).mean(1, keepdim=True) + 1e-5)
    assert bool(((mean.double()[:, None] - mu).abs() <= 1.01 * U * mu.abs() + 60 * U / rs).all())
    assert bool(((rstd.double()[:, None] / rs - 1).abs() <= 60 * U).all())
    h = (z - mu) * rs
    assert bool(((y.double() - h).abs() <= 60 * U * (1 + h.abs())).all())


def test_norm_over_its_own_input_returns_no_row():
    """y over x without a residual: x no longer holds the row that was normalised, so none is handed out for the backward."""
    dims, opts = moe.Dims(5, 64, 64, 8, 2, F32), moe.NormOptions("rms", 1e-6)
    x = torch.randn((5, 64), device="cuda")
    want, row, _, _ = moe.norm_forward(dims, opts, x, keep=True)
    assert row is x
    r = torch.randn_like(x)
    both, s, _, _ = moe.norm_forward(dims, opts, x.clone(), residual=r, keep=True)
    c, q = x.clone(), x.clone()
    got, kept, _, _ = moe.norm_forward(dims, opts, c, y=c, keep=True)
    assert got is c and kept is None and torch.equal(got, want)
    got, kept, _, _ = moe.norm_forward(dims, opts, q, residual=r, y=q, keep=True)  # the sum is apart
    assert got is q and torch.equal(kept, s) and torch.equal(got, both)
    e = torch.zeros((0, 64), device="cuda")
    assert moe.norm_forward(moe.Dims(0, 64, 64, 8, 2, F32), opts, e, y=e)[1] is e
