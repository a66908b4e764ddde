"""Which distillation calls ask for a workspace: the validation layer under
AddressSanitizer and UBSan (CPU only), against host stand-ins for the launchers."""
import os
import re
import shutil
import subprocess
import tempfile

import pytest

import vocab_sharded_embedding_amd as vpe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HERE = os.path.join(ROOT, "tests", "host_sanitize")
CSRC = os.path.join(ROOT, "vocab_sharded_embedding_amd", "csrc")
SAN = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-g", "-O1"]


def test_statistics_of_many_rows_need_no_workspace():
    if shutil.which("g++") is None:
        pytest.skip("no host compiler")
    with tempfile.TemporaryDirectory() as tmp:
        exe = os.path.join(tmp, "driver")
        r = subprocess.run(
            ["g++", "-std=c++17", "-Wall", "-Wextra", "-I", os.path.join(ROOT, "include"), *SAN,
             os.path.join(HERE, "driver_distill_workspace.cpp"),
             os.path.join(HERE, "stub_train_launchers.cpp"),
             os.path.join(CSRC, "vpe_train_api.cpp"), "-o", exe],
            stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
        if r.returncode != 0 and "asan" in r.stdout.lower():
            pytest.skip("sanitizer runtime not available: " + r.stdout[-300:])
        assert r.returncode == 0, r.stdout
        r = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
        assert r.returncode == 0 and "all expectations held" in r.stdout, r.stdout


def test_the_number_of_rows_is_the_headers():
    text = open(os.path.join(ROOT, "include", "vpe_train.h")).read()
    assert int(re.search(r"#define VPE_DISTILL_WHOLE_ROWS (\d+)", text).group(1)) == \
        vpe.VPE_DISTILL_WHOLE_ROWS
