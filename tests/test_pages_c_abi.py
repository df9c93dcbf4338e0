"""The calls for long and shared contexts from C: a C11 program calls each through the header's
prototypes and types (gcc -std=c11 -Wall -Wextra -Werror -pedantic, linked against libmxq.so)
with no GPU visible and checks the host-side answers."""
import os
import shutil
import subprocess

import pytest

import nvfp4_quantization_amd as mxq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_c11_caller(tmp_path):
    if not os.path.exists(mxq.LIB_PATH):
        pytest.fail("libmxq.so is missing: build the library")
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not found")
    exe = str(tmp_path / "mxq_pages_abi_check")
    libdir = os.path.dirname(mxq.LIB_PATH)
    subprocess.run([gcc, "-std=c11", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "c", "mxq_pages_abi_check.c"), "-o", exe, "-L", libdir, "-lmxq",
                    f"-Wl,-rpath,{libdir}"], check=True, capture_output=True, text=True)
    env = dict(os.environ, HIP_VISIBLE_DEVICES="", ROCR_VISIBLE_DEVICES="", CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([exe], env=env, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    assert "all checks passed" in r.stdout
