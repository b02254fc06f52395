"""The CPython module goes with one torch and one Python, and the package without it (CPU)."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

import __graft_entry__

PKG = os.path.join(__graft_entry__.ROOT, "paged_kv_cache_476_b200")


@pytest.fixture(scope="module")
def builder():
    b = __graft_entry__._builder()
    b.build()
    return b


class _Compiled(Exception):
    pass


@pytest.fixture
def compiles(builder, monkeypatch):
    """Whether _build_binding goes to the compiler."""
    def run(cmd, **kw):
        raise _Compiled

    monkeypatch.setattr(builder.subprocess, "run", run)

    def check():
        try:
            builder._build_binding(False)
        except _Compiled:
            return True
        return False

    return check


def test_key_names_torch_and_python(builder):
    assert torch.__version__ in builder.binding_key()
    assert f"{sys.version_info[0]}{sys.version_info[1]}" in builder.binding_key()


def test_built_again_only_where_something_changed(builder, compiles, monkeypatch):
    assert not compiles()
    with monkeypatch.context() as m:
        m.setattr(builder, "binding_key", lambda: "torch 0.0, another")
        assert compiles()
    with monkeypatch.context() as m:
        m.setattr(builder, "CXX", "another-compiler")
        assert compiles()
    assert not compiles()


IMPORT = """
import warnings
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    import paged_kv_cache_476_b200 as pkv
assert pkv.__file__.startswith({root!r}), pkv.__file__
assert pkv.pkv_status_string(0)
said = [str(w.message) for w in seen if "_binding.so" in str(w.message)]
print(len(said), pkv._binding.norm_rope(None) is NotImplemented, said)
"""


@pytest.mark.parametrize("how", ["as built", "missing", "another torch", "broken"])
def test_package_without_a_fitting_module(builder, tmp_path, how):
    """The library's own entry points do not depend on torch's C++ layout."""
    to = tmp_path / "paged_kv_cache_476_b200"
    to.mkdir()
    for f in os.listdir(PKG):
        if f.endswith((".py", ".so")):
            shutil.copy2(os.path.join(PKG, f), to / f)
    if how == "missing":
        (to / "_binding.so").unlink()
    elif how == "broken":
        (to / "_binding.so").write_bytes(b"not a library")
    elif how == "another torch":
        with open(to / "build.py", "a") as f:
            f.write("\n\ndef binding_key():\n    return 'torch 0.0, another'\n")
    r = subprocess.run([sys.executable, "-c", IMPORT.format(root=str(tmp_path))], cwd=tmp_path,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    count, handed_on, said = r.stdout.split(" ", 2)
    assert handed_on == "True"
    assert count == ("0" if how == "as built" else "1")
    assert how != "another torch" or "torch 0.0" in said
