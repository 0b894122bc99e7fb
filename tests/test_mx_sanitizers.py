"""The host code of the 4-bit and expert calls (argument checks, size queries, choice of kernel) under AddressSanitizer
and UndefinedBehaviorSanitizer: sizes of every magnitude through tests/sanitize/mx_checks.c, nothing is enqueued."""
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from expand_token_adapter_amd import build as hip_build  # noqa: E402  (build recipe only; nothing is loaded)

SOURCES = [s for s in hip_build.SOURCES if s.split(".")[0] in ("abi", "segments", "mx", "mx_base", "experts")]


@pytest.mark.skipif(not os.path.exists("/opt/rocm/llvm/bin/clang++"), reason="no ROCm clang")
def test_mx_host_checks_under_asan_ubsan(tmp_path):
    san = [f for s in ("-fsanitize=address", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer")
           for f in ("-Xarch_host", s)]
    flags = [f for f in hip_build.HIPCC_FLAGS if f != "-O3"] + ["-O1"]
    objs, cmds = [], []
    for src in SOURCES:
        objs.append(str(tmp_path / (os.path.splitext(src)[0] + ".o")))
        cmds.append([hip_build.hipcc()] + flags + san + ["-I", hip_build.INCLUDE, "-I", hip_build.CSRC, "-c",
                                                         os.path.join(hip_build.CSRC, src), "-o", objs[-1]])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, " ".join(cmd) + "\n" + r.stderr[-3000:]

    with ThreadPoolExecutor(max_workers=4) as ex:
        list(ex.map(run, cmds))
    clang = "/opt/rocm/llvm/bin/clang"
    harness, exe = str(tmp_path / "mx_checks.o"), str(tmp_path / "mx_checks")
    run([clang, "-std=c99", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-I", hip_build.INCLUDE,
         "-c", os.path.join(ROOT, "tests", "sanitize", "mx_checks.c"), "-o", harness])
    run([clang + "++", "-fsanitize=address,undefined", harness] + objs +
        ["-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    res = subprocess.run([exe], env=env, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr[-4000:]
    assert "mx checks: ok" in res.stdout
