"""Host AddressSanitizer and UndefinedBehaviorSanitizer on the CPU over the linear layer's host code:
argument checks, workspace layout, plans and launches' arithmetic.  As in test_sanitize_cpu.py the
library is built with the sanitizers on its host side only, and runs in a subprocess with the
sanitizer runtime preloaded."""
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_sanitize_cpu import CLANG, ENV, HERE, HIPCC, ROOT, _runtime


def test_linear_host_code_under_asan_ubsan(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    from mixed_precision_zero_amd.build import SOURCES

    def compile_one(src):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        subprocess.run([HIPCC, "--offload-arch=gfx950", "-O1", "-g1", "-std=c++17", "-fPIC", "-c",
                        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                        "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                        "-Xarch_host", "-fno-omit-frame-pointer",
                        "-I", os.path.join(ROOT, "include"),
                        "-I", os.path.join(ROOT, "mixed_precision_zero_amd", "csrc"), src, "-o", obj],
                       check=True, capture_output=True)
        return obj

    with ThreadPoolExecutor(4) as pool:
        objs = list(pool.map(compile_one, SOURCES))
    so = str(tmp_path / "libneox_zero1_san.so")
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-shared", "-Xarch_host", "-fsanitize=address",
                    "-Xarch_host", "-fsanitize=undefined", *objs, "-o", so], check=True, capture_output=True)
    rt = _runtime([CLANG, "-print-file-name=libclang_rt.asan-x86_64.so"])
    r = subprocess.run([sys.executable, os.path.join(HERE, "host_sanitize_linear_driver.py"), so],
                       env={**os.environ, **ENV, "LD_PRELOAD": rt}, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "host code exercised" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]
