"""What the package asks of torch before a call: nothing. It is imported at once, and built where there is no torch,
for callers of the C ABI."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
WITHOUT = """
import sys
class Without:
    def find_spec(self, name, path=None, target=None):
        if name == "torch" or name.startswith("torch."):
            raise ModuleNotFoundError("No module named 'torch'", name="torch")
sys.meta_path.insert(0, Without())
"""


def run(code):
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert done.returncode == 0, done.stderr
    return done.stdout


def test_import_does_not_load_torch():
    assert run("import sys, fp32_gemm_nn_amd as mg\nprint('torch' in sys.modules, callable(mg.mi_fp8_gemm), 'rmsnorm' in dir(mg))"
               ).split() == ["False", "True", "True"]


def test_names_once_it_does():
    out = run("import fp32_gemm_nn_amd as mg\n"
              "from fp32_gemm_nn_amd import *\n"
              "assert all(callable(getattr(mg, n)) or n == 'library_path' for n in mg.__all__)\n"
              "assert mg.fp8_gemm is mg.fp8.fp8_gemm and mg.mi_rmsnorm is mg.fp8.mi_rmsnorm and fp8_empty is mg.fp8_empty\n"
              "try:\n    mg.fp8_none\nexcept AttributeError as e:\n    print(e)")
    assert "fp8_none" in out


def test_without_torch():
    out = run(WITHOUT + """
import fp32_gemm_nn_amd as mg
from fp32_gemm_nn_amd import build
try:
    mg.fp8_gemm
except ModuleNotFoundError as e:
    print(e.name)
""")
    assert out.split() == ["torch"]


@pytest.mark.parametrize("torch", [True, False])
def test_build(torch):
    """The library and, where torch is there, the tensor forms' binding (the compilers are stood in for)."""
    out = run((WITHOUT if not torch else "") + """
import os, subprocess
from fp32_gemm_nn_amd import build
made, moved = [], []
class Done:
    returncode = 0
    def __init__(self, cmd, **kw): made.append(cmd[cmd.index("-o") + 1])
    def wait(self): return 0
subprocess.Popen = Done
subprocess.run = Done
gone = []
os.replace, os.remove, os.path.exists = lambda a, b: moved.append(b), gone.append, lambda path: True
build.build()
print(sorted(os.path.basename(m) for m in moved), [os.path.basename(g) for g in gone])
""")
    assert out.strip() == ("['_binding.so', 'libmisgemm.so'] []" if torch else "['libmisgemm.so'] ['_binding.so']")
