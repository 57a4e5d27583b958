"""Host AddressSanitizer and UndefinedBehaviorSanitizer run of the output layer's losses (no GPU needed).

tests/asan/head_asan.cpp drives their refusals and their workspace plan; like the driver of the other entry points it is
built with sanitizers on host code only (-Xarch_host before each flag) and must finish with exit status 0 and no report.
"""
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from bit_quantized_lora_02_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_head_host_code_under_sanitizers(tmp_path):
    if not os.path.exists(build.HIPCC):
        pytest.skip("hipcc not available")
    flags = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-Xarch_host", "-fsanitize=address", "-Xarch_host",
             "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host",
             "-fno-omit-frame-pointer", "-I", build.INCLUDE, "-I", build.CSRC]
    sources = [os.path.join(ROOT, "tests", "asan", "head_asan.cpp"), *(os.path.join(build.CSRC, s) for s in build.SOURCES)]
    objects = [str(tmp_path / (os.path.basename(s) + ".o")) for s in sources]
    exe = str(tmp_path / "head_asan")

    def run(*args):
        subprocess.check_call([build.HIPCC, *flags, *args], stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)

    with ThreadPoolExecutor(4) as pool:
        list(pool.map(lambda s, o: run("-c", s, "-o", o), sources, objects))
    run(*objects, "-o", exe)
    p = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=dict(os.environ, ASAN_OPTIONS="detect_leaks=1"))
    out = p.stdout + p.stderr
    assert p.returncode == 0 and "Sanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert "head asan driver ok" in out
