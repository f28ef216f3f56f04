"""The expert layer needs torch; the rest of the package does not, star import included."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_star_import_without_torch():
    code = ("import sys; sys.modules['torch'] = None\n"
            "from spgemm_symbolic_row_amd import *\n"
            "print('levels', compute_params(1000, 65536)['levels'])\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and "levels" in r.stdout, r.stderr


def test_star_import_with_torch():
    names = {}
    exec("from spgemm_symbolic_row_amd import *", names)
    assert {"route", "experts", "experts_backward", "clip_grad_norm", "matmul"} <= set(names)
