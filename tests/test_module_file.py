"""The marshalling module of the paged wrappers, when its file is written anew under a process that has it loaded."""
import os
import shutil
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

from flash_attention_backward_gb300 import build as B  # noqa: E402

LOAD = """
import importlib.util, shutil, sys, torch
old, here = sys.argv[1:]
spec = importlib.util.spec_from_file_location("m._fast", here)
m = importlib.util.module_from_spec(spec)
spec.loader.exec_module(m)
try:
    m.decode()
except TypeError as e:
    assert "9 arguments" in str(e)
try:
    m.bind(*[object()] * 3)
except TypeError as e:
    assert "addresses expected" in str(e)
shutil.copy(old, here)
"""


def test_a_file_that_is_written_anew_leaves_the_process_ending_in_order(tmp_path):
    B.build()
    if B.fast_path() is None or not os.path.exists(B.fast_path()):
        pytest.skip("the module is not built here")
    here = str(tmp_path / "_fast.so")
    shutil.copy(B.fast_path(), here)
    r = subprocess.run([sys.executable, "-c", LOAD, B.fast_path(), here], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
