"""More checks of the 8-bit token path on the CPU (see test_i8_host.py): the self-test's arguments, and what is needed
to import the package."""
import importlib.machinery
import os
import shutil
import subprocess
import sys

import pytest

import bit_weight_only_wr_b200 as wr
from test_i8_host import BAD, GEMM, P, UNSUPPORTED, _status


SELFTEST = {k: GEMM[k] for k in ("M", "N", "K", "x", "ldx", "x_scale", "w", "ldw", "w_scale", "y", "ldy")}


@pytest.mark.parametrize("change,status", [
    (dict(M=1), UNSUPPORTED), (dict(M=8), UNSUPPORTED), (dict(K=131072, ldx=131072, ldw=131072), UNSUPPORTED),
    (dict(M=0), BAD), (dict(ldx=104), BAD), (dict(x=None), BAD), (dict(y=P + 4), BAD), (dict(ldy=69), BAD),
])
def test_selftest_refusals(change, status):
    assert _status(wr.wr_selftest_gemm_i8_timeout, **{**SELFTEST, **change}) == status


def test_gemm_i8_needs_no_workspace():
    """The size is 0 whatever the arguments, and the workspace arguments are not among those that are checked: calls with
    none, with one that is not aligned and with a size that is too small are refused (here for ldy) all alike."""
    for shape in ((1, 64, 64), (40, 70, 9728), (333, 2560, 9728), (4096, 19456, 2560), (16, 1, 131071), (0, 1, 1), (1, 1, 131072)):
        assert wr.wr_gemm_i8_workspace_bytes(*shape) == 0
    for workspace, size in ((None, 0), (P + 8, 4), (P, 0), (None, 1 << 40)):
        assert _status(wr.wr_gemm_i8, **{**GEMM, "ldy": 69, "workspace": workspace, "workspace_bytes": size}) == BAD


# ---------------------------------------------------------------- the extension module

def _import_without_module(tmp_path, code, other=None):
    """Runs code with a copy of the package that has no extension module for this Python (`other`: a file there)."""
    pkg = tmp_path / "bit_weight_only_wr_b200"
    pkg.mkdir()
    here = os.path.dirname(wr.LIB_PATH)
    shutil.copy(os.path.join(here, "__init__.py"), pkg)
    os.symlink(wr.LIB_PATH, pkg / "libwr.so")
    if other:
        (pkg / other).write_bytes(b"not a module")
    return subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True, env={**os.environ, "PYTHONPATH": ""})


@pytest.mark.parametrize("other", [None, "_marshal.so", "_marshal.cpython-39-x86_64-linux-gnu.so"])
def test_packed_calls_need_no_extension_module(tmp_path, other):
    """Without the module of this Python (or with another one's) the package imports and its other calls work; those
    that need it say what is missing."""
    r = _import_without_module(tmp_path, """
import numpy as np
import bit_weight_only_wr_b200 as wr
codes = np.arange(16 * 256, dtype=np.uint8).reshape(16, 256) % 4
assert np.array_equal(wr.wr_unpack_codes(2, wr.wr_pack(2, codes), 16, 256), codes)
assert wr.wr_gemm_i8_workspace_bytes(1, 64, 64) == 0
for f in (wr.wr_quantize_rows, wr.wr_gemm_i8, wr.wr_residual_norm):
    try:
        f(1, 2, stream=0)
    except ImportError as e:
        assert f.__name__ in str(e) and "_marshal" in str(e) and "build.py" in str(e)
    else:
        raise AssertionError(f.__name__)
print("done")
""", other)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stderr


def test_a_module_that_does_not_load_is_named_by_the_calls(tmp_path):
    r = _import_without_module(tmp_path, """
import bit_weight_only_wr_b200 as wr
try:
    wr.wr_gemm_i8()
except ImportError as e:
    print("wr_gemm_i8" in str(e) and "_marshal" in str(e))
""", "_marshal" + importlib.machinery.EXTENSION_SUFFIXES[0])
    assert r.stdout.strip() == "True", r.stderr


def test_the_extension_module_carries_the_tag_of_this_python():
    assert wr._marshal.__file__.endswith("_marshal" + importlib.machinery.EXTENSION_SUFFIXES[0])
    assert wr.wr_gemm_i8 is wr._marshal.wr_gemm_i8
