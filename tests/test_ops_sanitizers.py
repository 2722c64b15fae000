"""Host code of the int8 and expert entry points under AddressSanitizer and
UndefinedBehaviorSanitizer, on the CPU: argument checks and kernel choice over
sizes at the ends of their ranges (tests/sanitize/ops_harness.cpp).  Only host
code is instrumented; no kernel is launched."""

import concurrent.futures as cf
import os

from dense_gemm_02_amd import build as B
from test_sanitizers import HERE, ROOT, SAN_ENV, _run


def test_ops_host_code_under_sanitizers(tmp_path):
    hipcc = "/opt/rocm/bin/hipcc"
    san = ["-O1", "-g", "-Xarch_host", "-fsanitize=address,undefined", "-Xarch_host", "-fno-sanitize-recover=all"]
    flags = [f for f in B.HIPCC_FLAGS if f != "-O3"] + san

    def compile_unit(u):
        src, obj, extra = u
        out = str(tmp_path / os.path.basename(obj))
        _run([hipcc] + flags + extra + ["-c", src, "-o", out])
        return out

    with cf.ThreadPoolExecutor(max_workers=min(16, len(os.sched_getaffinity(0)))) as ex:
        objs = list(ex.map(compile_unit, B.units()))
    harness = str(tmp_path / "ops_harness.o")
    _run(["/opt/rocm/llvm/bin/clang++", "-O1", "-g", "-std=c++17", "-fsanitize=address,undefined",
          "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "include"), "-c",
          os.path.join(HERE, "ops_harness.cpp"), "-o", harness])
    exe = str(tmp_path / "ops_san")
    _run([hipcc, "-Xarch_host", "-fsanitize=address,undefined", harness] + objs + ["-o", exe])
    res = _run([exe], env=SAN_ENV)
    assert " 0 failures" in res.stdout, res.stdout
    # every kind of refusal was met
    assert all(f"{s}:0 " not in res.stdout for s in (0, 1, 2, 3, 4, 5, 6, 8)), res.stdout
