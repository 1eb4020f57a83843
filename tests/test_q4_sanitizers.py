"""Host checks of the 4-bit cache's entry points under
UndefinedBehaviorSanitizer (no GPU needed; skipped where one is)."""
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.slow
def test_entry_points_host_checks_are_clean_under_ubsan(tmp_path):
    """The units behind these calls, built with the sanitizer on their host
    code, get sizes at and past their limits (tests/sanitize/q4_extremes.py)."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is visible: this probe runs on machines without one")
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no gcc")
    ubsan = subprocess.run([gcc, "-print-file-name=libubsan.so"], capture_output=True, text=True).stdout.strip()
    if not os.path.isabs(ubsan):
        pytest.skip("no libubsan for this compiler")
    from paged_kv_cache_311_gb300 import build as b

    def compile_one(src):
        obj = str(tmp_path / src.replace(".cu", ".o"))
        subprocess.run([b.nvcc(), *b.ARCH, "-O1", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fsanitize=undefined",
                        "-Xcompiler", "-fno-sanitize-recover=undefined", "-I", os.path.join(ROOT, "include"), "-c",
                        os.path.join(b.CSRC, src), "-o", obj], check=True, capture_output=True)
        return obj

    # pkv_abi.cu holds what the others share; the decode units it refers
    # to are not linked in and not called (symbols are bound lazily)
    with ThreadPoolExecutor(max_workers=5) as ex:
        objs = list(ex.map(compile_one, ["q4_cache.cu", "q4_attention.cu", "q4_attention_f16.cu", "q4_attention_bf16.cu",
                                         "pkv_abi.cu"]))
    lib = str(tmp_path / "libq4_ubsan.so")
    subprocess.run([b.nvcc(), *b.ARCH, "-shared", "-o", lib, *objs], check=True, capture_output=True)
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="", LD_PRELOAD=ubsan, UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "sanitize", "q4_extremes.py"), lib], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=900)
    report = r.stdout[-3000:] + r.stderr[-3000:]
    assert r.returncode == 0, report
    assert "runtime error" not in report and r.stdout.startswith("calls "), report
