"""The dense block's host side without a GPU: the limits of its calls, and what building and importing it needs."""
import ctypes
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys

import update_merged_table_gb300 as mt
from update_merged_table_gb300 import build_lib
from test_block_cpu import P, Rows, lib, norm_config  # noqa: F401 (lib: the built library)

MOST_ROWS = (1 << 31) - 4096


def test_row_numbers_leave_room_for_a_tile(lib):  # noqa: F811
    """A kernel adds up to a few hundred rows to a row's number in 32 bits: batches that close to 2^31 are refused."""
    x = Rows(P, 64, None, None)
    packed = Rows(None, 0, P, P)
    row = Rows(P, 64, None, None)
    for n, code, size in ((MOST_ROWS, mt.MT_ENOSPACE, True), (MOST_ROWS + 1, mt.MT_EINVAL, False), ((1 << 31) - 1, mt.MT_EINVAL, False)):
        assert (lib.mt_group_linear_workspace_bytes(n, 2, 64, 32) > 0) == size
        assert (lib.mt_gated_norm_workspace_bytes(n, 64, 1) > 0) == size
        assert lib.mt_group_linear_backward(P, 32, ctypes.byref(x), P, P, 2, n, 64, 32, mt.MT_BF16, None, 0, P, None, None, 0, None) == code
        assert lib.mt_gated_norm_backward(ctypes.byref(norm_config(n=n)), *(ctypes.byref(r) for r in (row, row, packed, row, packed, row, row, row)),
                                          P, None, P, P, None, None, 0, None) == code
        if not size:
            assert lib.mt_group_linear_forward(P, 64, P, P, 2, n, 64, 32, mt.MT_BF16, P, 32, None, None) == code
            assert lib.mt_gated_norm_forward(ctypes.byref(norm_config(n=n)), *(ctypes.byref(row),) * 5, None) == code


def test_library_builds_without_torch(monkeypatch, tmp_path, lib):  # noqa: F811
    """The C library depends on nothing but CUDA: without torch only the Python module is left out."""
    monkeypatch.setattr(build_lib, "BINDING", str(tmp_path / "_mt_block.so"))
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert build_lib.build() == build_lib.LIB
    assert not (tmp_path / "_mt_block.so").exists()


def test_python_module_is_built_anew_for_another_torch(monkeypatch, lib):  # noqa: F811
    started = []
    monkeypatch.setattr(build_lib.subprocess, "Popen", lambda cmd, **kw: started.append(cmd))
    assert build_lib._start_binding(False, False) is None and not started
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.0")
    assert build_lib._start_binding(False, False) is not None and len(started) == 1


def test_all_names_import_without_a_library_or_torch(tmp_path):
    """`from package import *` needs neither the built library nor torch; what does says so when it is used."""
    shutil.copytree(os.path.dirname(build_lib.__file__), tmp_path / "update_merged_table_gb300",
                    ignore=shutil.ignore_patterns("_build", "csrc", "__pycache__"))

    def run(code):
        r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr

    run("""
from update_merged_table_gb300 import *
import torch
assert Packed8 and Table
for f in (lambda: pack8(torch.zeros(2, 32)), lambda: Table(10, 16, device="cpu")):
    try:
        f()
    except RuntimeError as e:
        assert "not built" in str(e), e
    else:
        raise SystemExit("no error")
""")
    run("import sys; sys.modules['torch'] = None\nfrom update_merged_table_gb300 import *\nassert plan_merge and 'Packed8' not in globals()")
