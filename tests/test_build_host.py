"""CPU checks of the build: what it compiles, in which order and when."""
import os
import warnings

import pytest

from structured_sparse_gemm_sp24_b200 import build as bld
from structured_sparse_gemm_sp24_b200 import sp24 as B


@pytest.fixture
def fake(monkeypatch, tmp_path):
    """Commands are recorded, their outputs written into a scratch folder."""
    monkeypatch.setattr(bld, "LIB", str(tmp_path / "libsp24.so"))
    monkeypatch.setattr(bld, "BINDING", str(tmp_path / "_binding.so"))
    ran = []

    def run(cmd, verbose):
        name = os.path.basename(cmd[0])
        if name in fail:
            raise RuntimeError(f"{name} failed")
        ran.append(name)
        with open(cmd[cmd.index("-o") + 1], "wb") as f:
            f.write(b"\0".join(c.encode() for c in cmd))

    fail = set()
    monkeypatch.setattr(bld, "_run", run)
    return ran, fail


def test_both_are_built_once(fake):
    ran, _ = fake
    assert bld.build() == bld.LIB
    assert sorted(ran) == ["g++", "nvcc"]
    bld.build()
    assert len(ran) == 2
    bld.build(force=True)
    assert len(ran) == 4


def test_library_is_built_where_the_binding_cannot_be(fake, monkeypatch):
    ran, fail = fake
    fail.add("g++")
    which = bld.shutil.which
    monkeypatch.setattr(bld.shutil, "which", lambda n, *a, **k: None if n == "g++" else which(n, *a, **k))
    with warnings.catch_warnings(record=True) as w:
        warnings.simplefilter("always")
        assert bld.build() == bld.LIB
    assert ran == ["nvcc"] and os.path.exists(bld.LIB)
    assert any("g++" in str(x.message) for x in w)


def test_library_is_built_without_torch(fake, monkeypatch):
    import sys
    ran, _ = fake
    monkeypatch.setitem(sys.modules, "torch", None)      # importing it raises ImportError
    with pytest.warns(RuntimeWarning, match="torch not found"):
        assert bld.build() == bld.LIB
    assert ran == ["nvcc"]


def test_an_error_in_the_binding_leaves_the_library(fake):
    ran, fail = fake
    fail.add("g++")
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        bld.build()
    assert ran == ["nvcc"] and os.path.exists(bld.LIB)


def test_binding_of_another_torch_is_rebuilt(fake, monkeypatch):
    import torch
    ran, _ = fake
    bld.build()
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    bld.build()
    assert ran[2:] == ["g++"]
    bld.build()
    assert len(ran) == 3


def test_binding_of_another_torch_is_not_used(monkeypatch):
    import torch
    bld.build()
    assert B.native().built_for == bld.binding_tag()
    monkeypatch.setattr(B, "_NATIVE", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    with pytest.raises(RuntimeError, match="0.0.1.other.*build"):
        B.native()
