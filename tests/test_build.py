"""What has to be there for which calls: the library needs nvcc alone, the target
pass's Python calls a module beside it."""
import os
import shutil
import subprocess
import sys
import time

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = "speculative_decoding_drafter_markov_gb300"


@pytest.fixture
def copy(tmp_path):
    """The package with a library of its own that is up to date, and no module."""
    from speculative_decoding_drafter_markov_gb300 import build
    lib = build.build()
    shutil.copytree(os.path.join(ROOT, PKG), tmp_path / PKG, ignore=shutil.ignore_patterns("_build", "__pycache__"))
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    out = tmp_path / PKG / "_build"
    out.mkdir()
    shutil.copy(lib, out / "libdspark.so")
    os.utime(out / "libdspark.so", (time.time() + 5,) * 2)
    broken = tmp_path / "bin"
    broken.mkdir()
    for name in ("g++", "nvcc"):
        (broken / name).write_text("#!/bin/sh\necho no such compiler >&2\nexit 1\n")
        (broken / name).chmod(0o755)
    return tmp_path, str(broken)


def python(where, code, path=None):
    env = dict(os.environ, PYTHONPATH=str(where))
    if path:
        env["PATH"] = path + os.pathsep + env["PATH"]
    return subprocess.run([sys.executable, "-c", code], cwd=where, env=env, capture_output=True, text=True)


def test_the_library_loads_where_the_module_cannot_be_built(copy):
    where, broken = copy
    r = python(where, f"""
from {PKG} import _lib
assert _lib.load().dspark_version() >= 100
try:
    _lib._target()
except RuntimeError as e:
    assert "bind.cpp" in str(e), e
else:
    raise SystemExit("the module was loaded")
""", broken)
    assert r.returncode == 0, r.stdout + r.stderr


def test_the_module_is_built_when_it_is_first_called(copy):
    where, _ = copy
    before = (where / PKG / "_build" / "libdspark.so").stat().st_mtime
    r = python(where, f"""
from {PKG} import _lib
m = _lib._target()
assert callable(m.page_map) and m.__file__.startswith({str(where)!r}), m.__file__
""")
    assert r.returncode == 0, r.stdout + r.stderr
    assert (where / PKG / "_build" / "libdspark.so").stat().st_mtime == before
    assert not [f for f in os.listdir(where / PKG / "_build") if f.endswith((".o", ".tmp"))]


def test_another_pytorch_does_not_load_this_ones_module(copy):
    """The module of one PyTorch is not current for another, whatever its time."""
    where, broken = copy
    build = f"from {PKG} import build; print(build.build_bind())"
    first = python(where, build)
    assert first.returncode == 0, first.stderr
    os.utime(first.stdout.strip(), (time.time() + 100,) * 2)
    again = python(where, build, broken)  # current: no compiler is called
    assert again.returncode == 0 and again.stdout == first.stdout
    for other in ("torch.__version__ = '1.99.0'", "sysconfig.get_config_var = lambda name: 'cpython-399'"):
        r = python(where, f"import sysconfig, torch; {other}; {build}", broken)
        assert r.returncode != 0 and "bind.cpp" in r.stderr, (other, r.stdout)
