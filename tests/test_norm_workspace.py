"""The workspace of the norm's gradients: what is asked for is what the form of the call
writes, and a workspace of exactly that size is enough; the dims that the norm takes."""
import ctypes
import os

import pytest
import torch

import mixture_experts_layer_gate_amd as moe
from mixture_experts_layer_gate_amd import api

BF16, F32 = torch.bfloat16, torch.float32
built = pytest.mark.skipif(not os.path.exists(moe.library_path()), reason="HIP library not built")


def _size(T, d, dt, kind):
    return moe.norm_backward_workspace_bytes(moe.Dims(T, d, 64, 1, 1, dt), moe.NormOptions(kind, 1e-5))


@built
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_what_is_asked_for(kind, dt):
    """Columns summed beside the rows (short batches, and rows over 8192 columns at any length): two rows of them at most,
    or a number to each row. Parts: at most 512 rows of columns, twice that with a bias' gradient."""
    for T, d in ((1, 8), (64, 128), (333, 1048), (160, 7168), (1024, 512), (2047, 16384), (100000, 8200)):
        rows = 4 * T if kind == "layer" and d > 8192 else 0
        assert 0 < _size(T, d, dt, kind) <= max(2 * (4 * d + 256), rows + 256), (T, d)
    for T, d in ((1100, 256), (2047, 6144), (8192, 2048), (65536, 7168)):
        assert 4 * d <= _size(T, d, dt, "rms") <= 512 * 4 * d + 256 and _size(T, d, dt, "layer") == 2 * _size(T, d, dt, "rms")


@built
@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="host-only validation test")
def test_less_is_refused():
    A, lib = 0x10000, moe.load_library()
    for T, d in ((64, 128), (2047, 6144), (2047, 16384), (100000, 8200)):
        for kind in ("rms", "layer"):
            dims = ctypes.byref(api._Dims(T, d, 64, 1, 1, 1))
            opts = ctypes.byref(api._NormOpts(int(kind == "layer"), 0, 1e-5))
            need = lib.moe_norm_backward_workspace_bytes(dims, opts)
            mean, db = (A, A) if kind == "layer" else (None, None)
            assert lib.moe_norm_backward(dims, opts, A, A, A, mean, A, None, A, A, db, A, need - 1, None) == 3


@built
@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="host-only validation test")
def test_dims_are_valid_as_a_whole():
    """The layer's dims, experts and width of them included, also for the norm alone."""
    A, lib, opts = 0x10000, moe.load_library(), ctypes.byref(api._NormOpts(0, 0, 1e-6))

    def status(T, f, E, k):
        dims = ctypes.byref(api._Dims(T, 64, f, E, k, 1))
        fwd = lib.moe_norm_forward(dims, opts, A, None, A, None, None, None, None, None, None)
        bwd = lib.moe_norm_backward(dims, opts, A, A, A, None, A, None, None, A, None, A, 1 << 50, None)
        return fwd, bwd, lib.moe_norm_backward_workspace_bytes(dims, opts) > 0
    for bad in ((2 ** 23 + 7, 64, 256, 8), (2 ** 28, 64, 8, 8), (64, 0, 8, 2), (64, 64, 8, 0), (64, 64, 2, 3), (64, 64, 1025, 2)):
        assert status(*bad) == (1, 1, False), bad
    # (these are refused for the output that is missing, behind the dims)
    for good in ((2 ** 23 + 7, 64, 1, 1), (2 ** 23 - 1, 64, 256, 8), (64, 1, 8, 8)):
        assert status(*good) == (1, 1, True), good


@pytest.mark.gpu
@pytest.mark.parametrize("T,d", [(1, 8), (333, 1048), (1024, 512), (700, 7168), (1100, 256), (2047, 6144), (1500, 1032),
                                 (70, 8200), (2600, 16384), (40000, 8200)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_that_much_is_enough(dt, kind, T, d):
    """Exactly the size, whatever it holds, with sentinels behind it; every row far from zero."""
    if dt is F32 and T * d > 1 << 27:
        T //= 4
    print(f"workspace {kind} {dt} {T} x {d}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(T + d)
    x = (torch.randn((T, d), generator=gen, device="cuda") + 300.0).to(dt)
    dy = torch.randn((T, d), generator=gen, device="cuda").to(dt)
    dims, opts = moe.Dims(T, d, 64, 1, 1, dt), moe.NormOptions(kind, 1e-5)
    _, s, mean, rstd = moe.norm_forward(dims, opts, x, keep=True)
    layer = kind == "layer"
    want = moe.norm_backward(dims, opts, dy, s, None, rstd, mean=mean, want_dbias=layer)
    need = moe.norm_backward_workspace_bytes(dims, opts)
    for fill in (0, 255):
        buf = torch.full((need + 4096,), fill, dtype=torch.uint8, device="cuda")
        buf[need:] = 77
        got = moe.norm_backward(dims, opts, dy, s, None, rstd, mean=mean, want_dbias=layer, ws=buf[:need])
        torch.cuda.synchronize()
        assert bool((buf[need:] == 77).all())
        assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(got, want))
