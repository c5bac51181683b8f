"""The host code of the operators' entry points under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only, no GPU needed): the host half of the library's
sources, built without its gfx950 half, and tests/sanitize/operators_driver.cpp, which
makes no call that would launch a kernel.  Any report fails the run."""
import concurrent.futures
import glob
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(__file__))
from test_sanitizers import HERE, HIPCC, ROOT, SAN_HOST, _run  # noqa: E402


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
def test_operators_host_code_under_asan_ubsan(tmp_path):
    csrc = os.path.join(ROOT, "segmented_gather_lora_amd", "csrc")
    flags = ["--offload-arch=gfx950", "--offload-host-only", "-O1", "-g", "-std=c++17", "-Xclang", "-target-feature",
             "-Xclang", "-packed-fp32-ops", "-I", os.path.join(ROOT, "include"), "-I", csrc] + SAN_HOST
    srcs = sorted(glob.glob(os.path.join(csrc, "*.hip"))) + [os.path.join(HERE, "operators_driver.cpp")]

    def compile_one(src):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        lang = ["-x", "hip"] if src.endswith(".hip") else []
        _run([HIPCC, *flags, *lang, "-c", src, "-o", obj])
        return obj
    with concurrent.futures.ThreadPoolExecutor(max_workers=4) as ex:
        objs = list(ex.map(compile_one, srcs))
    exe = str(tmp_path / "operators_san")
    # (the kernels themselves are not there)
    _run([HIPCC, "--offload-arch=gfx950", "-Wl,--unresolved-symbols=ignore-in-object-files", *SAN_HOST, *objs, "-o", exe])
    # leak checks stay off: the HIP runtime keeps allocations of its own for the process
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
    r = _run([exe], env=env, timeout=300)
    name, sizes, spans = r.stdout.split()
    assert name == "ok" and int(sizes) > 1000 and int(spans) > 1000
