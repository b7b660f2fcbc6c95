"""The package without torch: its C binding alone needs none."""
import subprocess
import sys

from conftest import ROOT


def _run(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stderr


def test_star_import_without_torch():
    _run("import sys; sys.modules['torch'] = None\n"
         "from table_embedding_bag_amd import *\n"
         "assert tbe_abi_version() == 2 and TBE and 'dropout' not in globals()")


def test_star_import_with_torch_has_the_layers():
    _run("from table_embedding_bag_amd import *\n"
         "assert dropout and scan_step and grouped_linear_backward and TBE")


def test_import_alone_loads_no_torch():
    _run("import sys, table_embedding_bag_amd as t\n"
         "t.tbe_abi_version()\n"
         "assert 'torch' not in sys.modules and 'scan_forward' in t.__all__\n"
         "assert t.dropout and 'torch' in sys.modules")
