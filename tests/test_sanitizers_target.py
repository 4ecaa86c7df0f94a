"""AddressSanitizer and UndefinedBehaviorSanitizer on the host code (argument
checks, launch planning, workspace layout) of the 8-bit rows and the token
log-probabilities, driven by tests/native/target_host_checks.cpp.  Needs a
machine without a GPU: the placeholder addresses must never reach a device."""
import os

import pytest

from tests.test_sanitizers import CLANGXX, CSRC, HIPCC, INCLUDE, NATIVE, ROCM, SAN, _run


@pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="placeholder device addresses: run only without a GPU")
@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANGXX)), reason="ROCm compilers not found")
def test_host_code_under_asan_ubsan(tmp_path):
    host = [f for flag in ["-O1", "-g", *SAN] for f in ("-Xarch_host", flag)]
    # device code is never run here; the tiles' kernels need the optimiser to fit their registers
    common = ["--offload-arch=gfx950", "-std=c++17", "-fPIC", "-Xclang", "-target-feature", "-Xclang",
              "-packed-fp32-ops", "-Xarch_device", "-O1", *host, f"-I{INCLUDE}", f"-I{CSRC}"]
    objs = []
    for s in ("quant.hip", "logprob.hip"):
        objs.append(str(tmp_path / (s[:-4] + ".o")))
        _run([HIPCC, *common, "-c", os.path.join(CSRC, s), "-o", objs[-1]])
    lib = str(tmp_path / "libtarget_san.so")
    _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", lib])
    exe = str(tmp_path / "target_host_checks")
    _run([CLANGXX, "-O1", "-g", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", f"-I{INCLUDE}", f"-I{ROCM}/include",
          os.path.join(NATIVE, "target_host_checks.cpp"), lib, f"-L{ROCM}/lib", "-lamdhip64",
          f"-Wl,-rpath,{tmp_path}", f"-Wl,-rpath,{ROCM}/lib", "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1")
    assert "target host checks passed" in _run([exe], env=env, timeout=300)
