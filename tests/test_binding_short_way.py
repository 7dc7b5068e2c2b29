"""The extension module pa_bind is a short way into the library, not a condition for it: the library loads and builds
without PyTorch, and without that module every call goes through ctypes.  On the CPU, in processes of their own."""
import os
import shutil
import subprocess
import sys

import pytest

import paged_kv_continuous_pa_gb300 as pa
from paged_kv_continuous_pa_gb300 import build as pa_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = "paged_kv_continuous_pa_gb300"
NO_TORCH = "import sys; sys.modules['torch'] = None\n"
PAGES = f"""
import {PACKAGE} as pa
assert pa.load() is not None and pa.pool_bytes(2, 16, 1, 64, pa.PA_BF16) == 2 * 16 * 64 * 2
pages = pa.Pages(8, 16, 2, 4)
"""
CALL = """
import warnings
import torch
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    for _ in range(2):  # arguments that the checks refuse: the long way
        try:
            pa.prompt_attention(*(torch.zeros(4, 2, 64, dtype=torch.bfloat16) for _ in "qkv"),
                                torch.zeros(2, dtype=torch.int32), torch.zeros(4, 2, 64, dtype=torch.bfloat16))
            raise SystemExit("not refused")
        except ValueError as e:
            assert "CUDA" in str(e), e
assert [w.category for w in seen].count(RuntimeWarning) == WARNINGS, [str(w.message) for w in seen]
"""


@pytest.fixture(scope="module", autouse=True)
def built():
    pa_build.build()


def run(code, root=ROOT):
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300,
                       env={**os.environ, "PYTHONPATH": root})
    assert r.returncode == 0, r.stderr[-3000:]


def copy(tmp_path, bind):
    """The package with its library, and with `bind` in pa_bind.so (None: no such file)."""
    to = tmp_path / PACKAGE
    (to / "_lib").mkdir(parents=True)
    shutil.copy(os.path.join(ROOT, PACKAGE, "__init__.py"), to)
    shutil.copy(pa.LIB_PATH, to / "_lib")
    if bind is not None:
        (to / "_lib" / "pa_bind.so").write_bytes(bind)
    return str(tmp_path)


def test_library_loads_without_torch():
    run(NO_TORCH + PAGES)


def test_library_builds_without_torch():
    run(NO_TORCH + f"from {PACKAGE} import build\nassert build.build() == build.LIB_PATH")


def test_calls_without_the_module(tmp_path):
    run(PAGES + CALL.replace("WARNINGS", "1"), copy(tmp_path, None))


def test_calls_with_a_module_that_does_not_load(tmp_path):
    run(PAGES + CALL.replace("WARNINGS", "1"), copy(tmp_path, b"of another torch"))


def test_calls_with_the_module():
    run(PAGES + CALL.replace("WARNINGS", "0") + "assert pa._bind.__name__ == 'pa_bind'")


def test_a_module_that_does_not_compile_leaves_the_library(tmp_path, monkeypatch):
    """The build says so, and leaves no module of older sources behind."""
    stale = tmp_path / "pa_bind.so"
    stale.write_bytes(b"of older sources")
    os.utime(stale, (0, 0))
    monkeypatch.setattr(pa_build, "BIND_PATH", str(stale))
    monkeypatch.setenv("CXX", "false")
    with pytest.warns(RuntimeWarning, match="pa_bind"):
        assert pa_build.build() == pa_build.LIB_PATH
    assert not stale.exists()
    with pytest.raises(RuntimeError, match="pa_bind"):
        pa_build.build_bind()
