"""The scored router's and the dropout's host code (csrc/router_abi.hip) under
AddressSanitizer and UndefinedBehaviorSanitizer: tests/sanitize/router_host_check.cpp
drives sizing and every refusal, extreme dims included, against that file compiled
with its host code instrumented and the other objects as they are built. Host-only."""
import os
import shlex
import shutil
import subprocess

import pytest
import torch

from mixture_experts_layer_gate_amd import build as b

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DRIVER = os.path.join(ROOT, "tests", "sanitize", "router_host_check.cpp")
FILE = "router_abi.hip"
# host code only: each sanitizer flag applies to the host compilation
SANITIZE = shlex.split("-Xarch_host -fsanitize=address -Xarch_host -fsanitize=undefined "
                       "-Xarch_host -fno-sanitize-recover=undefined -Xarch_host -fno-omit-frame-pointer")


def _others():
    return [os.path.join(b.BUILD, os.path.splitext(s)[0] + ".o") for s in b.SOURCES if s != FILE]


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="host-only checks with placeholder device pointers")
@pytest.mark.skipif(not (os.path.exists("/opt/rocm/bin/hipcc") or shutil.which("hipcc")), reason="hipcc not available")
@pytest.mark.skipif(not all(os.path.exists(o) for o in _others()), reason="library objects not built")
@pytest.mark.timeout(600)
def test_router_host_code_under_sanitizers(tmp_path):
    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, f"{' '.join(cmd)}\n{r.stdout[-1000:]}{r.stderr[-3000:]}"

    hipcc, inc = b.hipcc(), ["-I", b.INCLUDE, "-I", b.CSRC]
    obj, drv, exe = (str(tmp_path / n) for n in ("abi.o", "drv.o", "check"))
    flags = [f for f in b.HIPCC_FLAGS if f != "-O3"] + ["-O1", "-g"]
    run([hipcc, *flags, *SANITIZE, *inc, "-c", os.path.join(b.CSRC, FILE), "-o", obj])
    run([hipcc, *flags, *SANITIZE, *inc, "-x", "hip", "-c", DRIVER, "-o", drv])
    run([hipcc, f"--offload-arch={b.ARCH}", *SANITIZE, drv, obj, *_others(), "-o", exe])
    run([exe])
