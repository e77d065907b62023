"""The package where torch is not installed: the codec's library is built and
loaded as ever; only the calls on torch tensors are missing."""
import os
import subprocess
import sys

from error_bounded_lossy_gb300 import build as ebc_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# a program's first lines: no torch
BLOCK = """
import sys
class Block:
    def find_spec(self, name, path=None, target=None):
        if name.partition(".")[0] == "torch":
            raise ImportError("no torch here")
sys.meta_path.insert(0, Block())
"""


def run(program):
    ebc_build.build()
    r = subprocess.run([sys.executable, "-c", program], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_the_library_is_built_and_loaded():
    run(BLOCK + """
from error_bounded_lossy_gb300 import build
import error_bounded_lossy_gb300 as ebc
assert build.build() == build.LIB
ebc.lib()
assert ebc.ebc_version() == 1
assert ebc.ebc_moe_plan(None, None, 4, 0, 1, 1, None, None, None, None) == ebc.EBC_ERR_INVALID_ARG
""")


def test_everything_else_is_imported_by_star():
    run(BLOCK + """
from error_bounded_lossy_gb300 import *
assert Codec and ebc_compress and EBC_OK == 0
try:
    Experts
except NameError:
    pass
else:
    raise AssertionError
""")


def test_everything_is_imported_by_star_where_torch_is():
    run("""
from error_bounded_lossy_gb300 import *
import error_bounded_lossy_gb300 as ebc
assert Codec and Experts is ebc.Experts and Plan is ebc.Plan and Mx4 is ebc.Mx4
""")


def test_everything_else_is_imported_by_star_where_the_calls_are_not_compiled():
    run("""
from error_bounded_lossy_gb300 import build
build.torch_module = lambda: "/nowhere/calls.so"
from error_bounded_lossy_gb300 import *
assert Codec and "Experts" not in globals()
import error_bounded_lossy_gb300 as ebc
try:
    ebc.Experts
except RuntimeError as e:
    assert "not built" in str(e)
else:
    raise AssertionError
""")
