"""The binding needs torch and the standard library alone."""
import subprocess
import sys

from tests.helpers import ROOT


def test_binding_without_numpy():
    code = ("import sys; sys.modules['numpy'] = None\n"
            "from grouped_gemm_02_amd import binding as B, inputs\n"
            "b = B.AdamWBuffers([], [], [])\n"
            "assert b.params == () and 'numpy.core' not in sys.modules\n"
            "print('imported')")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "imported" in r.stdout, r.stderr[-2000:]
