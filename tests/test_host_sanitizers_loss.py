"""The validation layer and workspace arithmetic of the loss calls under
AddressSanitizer and UBSan (CPU only): `vpe_loss_api.cpp` built with g++ against
host stand-ins for the kernel launchers, driven through edge and overflow-prone
sizes.  No GPU code is built with a sanitizer."""
import os
import shutil
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SAN = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer",
       "-g", "-O1"]


def _run(cmd, **kw):
    return subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, **kw)


def test_loss_validation_under_asan_ubsan():
    if shutil.which("g++") is None:
        pytest.skip("no host compiler")
    with tempfile.TemporaryDirectory() as tmp:
        exe = os.path.join(tmp, "host_sanitize_loss")
        r = _run(["g++", "-std=c++17", "-Wall", "-Wextra", "-I", os.path.join(ROOT, "include"), *SAN,
                  os.path.join(ROOT, "tests", "host_sanitize", "driver_loss.cpp"),
                  os.path.join(ROOT, "vocab_sharded_embedding_amd", "csrc", "vpe_loss_api.cpp"),
                  "-o", exe])
        if r.returncode != 0 and "asan" in r.stdout.lower():
            pytest.skip("sanitizer runtime not available: " + r.stdout[-300:])
        assert r.returncode == 0, r.stdout
        r = _run([exe], env={**os.environ, "ASAN_OPTIONS": "detect_leaks=1:abort_on_error=0"})
        assert r.returncode == 0, r.stdout
        assert "all expectations held" in r.stdout
