"""The host code of the balance and orthogonalisation entry points under
AddressSanitizer and UndefinedBehaviorSanitizer (CPU only), over the shapes and
coefficients that their plans and checks compute with
(tests/sanitize/abi_train_check.cpp); any sanitizer report fails."""
import glob
import os
import subprocess

import pytest

from tests.helpers import ROOT

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
SAN = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
       "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]


def test_train_host_code_is_clean_under_asan_and_ubsan(tmp_path):
    srcs = sorted(glob.glob(os.path.join(ROOT, "grouped_gemm_02_amd", "csrc", "*.hip")))
    srcs.append(os.path.join(ROOT, "tests", "sanitize", "abi_train_check.cpp"))
    flags = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
    objs = [str(tmp_path / (os.path.basename(src) + ".o")) for src in srcs]
    procs = [subprocess.Popen([HIPCC, *flags, *SAN, "-c", src, "-o", obj],
                              stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
             for src, obj in zip(srcs, objs)]
    for p in procs:
        out, _ = p.communicate(timeout=900)
        assert p.returncode == 0, out[-3000:]
    exe = str(tmp_path / "abi_train_check")
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", *SAN, *objs, "-o", exe], capture_output=True, text=True,
                       timeout=900)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and "abi train checks passed" in out, out[-3000:]
    assert "runtime error" not in out and "AddressSanitizer" not in out, out[-3000:]
