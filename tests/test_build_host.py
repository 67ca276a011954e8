"""The library does not depend on its Python extension: where that cannot be compiled or linked, the build says so and the
C ABI is there all the same."""
import ctypes
import os
import shutil

import pytest


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """build.py with its outputs in a folder of their own, the kernels' objects copied there."""
    from mla_latent_kv_fp8_gb300 import build
    build.build()
    folder = tmp_path / "_build"
    shutil.copytree(build.BUILD, folder)     # (copied with their times: not stale)
    monkeypatch.setattr(build, "BUILD", str(folder))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libmla_decode.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_packed.so"))
    (tmp_path / "_packed.so").write_text("of another torch")
    (folder / "binding.o").unlink()
    return build


@pytest.mark.parametrize("fails", ["compiler", "compile", "headers", "link"])
def test_library_is_built_without_the_extension(elsewhere, monkeypatch, fails):
    build, jobs = elsewhere, elsewhere._binding_jobs

    def broken(force):
        if fails == "headers":
            raise ImportError("no torch")
        commands, obj = jobs(force)
        if fails == "compiler":
            commands = [["/no/such/compiler", "-c", build.BINDING_SRC, "-o", obj]]
        if fails == "compile":
            commands = [[*commands[0][:-4], "-DPY_SSIZE_T_CLEAN=)(", "-include", "/no/such/header", *commands[0][-4:]]]
        if fails == "link":
            with open(obj, "w") as f:
                f.write("no object file")
            commands = []
        return commands, obj

    monkeypatch.setattr(build, "_binding_jobs", broken)
    with pytest.warns(RuntimeWarning, match="extension of the packed operators was not built"):
        path = build.build()
    assert not os.path.exists(build.BINDING)
    assert ctypes.CDLL(path).mla_decode_paged
    assert ctypes.CDLL(path).mla_prefill_ragged


def test_extension_is_built_where_it_can_be(elsewhere):
    elsewhere.build()
    assert os.path.getsize(elsewhere.BINDING) > 1000


def test_packed_operators_say_that_the_extension_is_missing(monkeypatch):
    import builtins

    from mla_latent_kv_fp8_gb300 import _lib, build
    build.build()
    real = builtins.__import__

    def no_extension(name, globals=None, locals=None, fromlist=(), level=0):
        if fromlist and "_packed" in fromlist:
            raise ImportError("no such file")
        return real(name, globals, locals, fromlist, level)

    monkeypatch.setattr(_lib, "_packed", None)
    monkeypatch.setattr(builtins, "__import__", no_extension)
    with pytest.raises(ImportError, match="_packed.so is missing"):
        _lib.mla_gather_latent(None, None, None, None, None, None, None)
    assert _lib.mla_auto_splits(1, 1, 12, 100, 152) >= 1     # what goes through ctypes works
