"""The 8-bit linear layer's host code (checks, choice, workspace layout) under
AddressSanitizer, with functions that check their arguments in the place of the
launches (tests/asan_linear8.cpp)."""
import os
import subprocess

from matrix_aware_optimizer_muon_amd import build as B

HERE = os.path.dirname(os.path.abspath(__file__))
HOST_ASAN = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fno-omit-frame-pointer"]


def test_host_code_of_the_8_bit_layer(tmp_path):
    exe = str(tmp_path / "asan_linear8")
    r = subprocess.run([B._hipcc(), f"--offload-arch={B.ARCH}", "-std=c++17", "-O1", "-g", *HOST_ASAN, "-I", B.INCLUDE,
                        "-I", B.CSRC, "-x", "hip", os.path.join(B.CSRC, "linear8_api.cpp"), "-x", "hip",
                        os.path.join(HERE, "asan_linear8.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:halt_on_error=1:abort_on_error=0")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    out = r.stdout + r.stderr
    assert "AddressSanitizer" not in out and "LeakSanitizer" not in out, out
    assert r.returncode == 0 and "0 failures" in out, out[-4000:]
