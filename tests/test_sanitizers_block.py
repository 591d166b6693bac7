"""AddressSanitizer + UndefinedBehaviorSanitizer build (host code only) of the
validation and planning of the calls around the scan, driven by
tests/sanitize/block_fuzz.cpp over edge and random sizes: every call must be
refused before it could launch anything, and no size arithmetic may overflow."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "selective_state_space_21_amd", "csrc")
HERE = os.path.join(ROOT, "tests", "sanitize")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CLANG = "/opt/rocm/llvm/bin/clang++"
ENV = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:halt_on_error=1:abort_on_error=0",
           UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)),
                    reason="needs the ROCm compilers")
def test_block_validation_under_sanitizers(tmp_path):
    flags = ["--offload-host-only", "-O1", "-g", "-std=c++17",
             "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xarch_host", "-fno-sanitize-recover=all",
             "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, "-x", "hip"]
    objs = []
    for src in (os.path.join(CSRC, "block_abi.cpp"), os.path.join(CSRC, "block_plan.cpp"),
                os.path.join(HERE, "block_fuzz.cpp")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        subprocess.run([HIPCC, *flags, "-c", src, "-o", obj], check=True, timeout=600)
        objs.append(obj)
    exe = str(tmp_path / "block_fuzz")
    subprocess.run([CLANG, "-fsanitize=address,undefined", *objs, "-o", exe], check=True, timeout=600)
    for walkers in (None, "5"):
        env = dict(ENV)
        env.pop("SSM_GATED_WALKERS", None)
        if walkers:
            env["SSM_GATED_WALKERS"] = walkers             # the planner's override
        r = subprocess.run([exe, "200000"], env=env, capture_output=True, text=True, timeout=600)
        assert r.returncode == 0 and "no finding" in r.stdout, r.stderr[-3000:]
