"""The module of the operators' calls: a module that was built beside another torch,
interpreter or library is not loaded, and does not stay; the library is built whether or
not the module can be."""
import os
import shutil
import subprocess
import sysconfig

import pytest
import torch

import kv_cache_compression_c128_gb300 as kvc

TORCH = os.path.dirname(torch.__file__)
FOREIGN = r"""
#include <Python.h>
static PyObject* bind(PyObject* self, PyObject* args) { Py_RETURN_NONE; }
static PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, 0}, {0, 0, 0, 0}};
static struct PyModuleDef def = {PyModuleDef_HEAD_INIT, "_kvc_call", 0, -1, methods};
PyMODINIT_FUNC PyInit__kvc_call(void) { return PyModule_Create(&def); }
"""


@pytest.fixture
def place(tmp_path, monkeypatch):
    """A folder of its own for what is built, with a library that is up to date."""
    kvc.build()
    monkeypatch.setattr(kvc, "_LIB_DIR", str(tmp_path))
    monkeypatch.setattr(kvc, "LIB_PATH", str(tmp_path / "libkvc.so"))
    monkeypatch.setattr(kvc, "_CALL_PATH", str(tmp_path / "_kvc_call.so"), raising=False)
    monkeypatch.setattr(kvc, "_quick", None)
    (tmp_path / "libkvc.so").write_bytes(b"")
    return tmp_path


@pytest.fixture
def other_torch(tmp_path_factory):
    """The folder of a torch with other libraries than the one here."""
    root = tmp_path_factory.mktemp("torch")
    (root / "lib").mkdir()
    shutil.copy(os.path.join(TORCH, "version.py"), root)
    for name, size in (("libc10.so", 100), ("libtorch_python.so", 200)):
        (root / "lib" / name).write_bytes(bytes(size))
    return root


def _modules(place):
    return sorted(f for f in os.listdir(place) if f.startswith("_kvc_call"))


@pytest.fixture
def compiled(monkeypatch):
    """The commands of a compiler that makes empty files."""
    ran = []

    def run(cmd, **_):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "wb").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(kvc.subprocess, "run", run)
    return ran


def test_what_was_built_beside_others_is_not_loaded(place, other_torch):
    include = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(include, "Python.h")):
        pytest.skip("no Python.h")
    (place / "foreign.c").write_text(FOREIGN)
    subprocess.run(["gcc", "-shared", "-fPIC", f"-I{include}", str(place / "foreign.c"), "-o", str(place / "_kvc_call.so")], check=True)
    kvc._load_torch()
    kvc._load_quick()
    assert kvc._quick is None
    shutil.copy(place / "_kvc_call.so", kvc._call_path(str(other_torch)))
    kvc._load_quick()
    assert kvc._quick is None


def test_the_name_tells_what_it_was_built_for(place, other_torch, monkeypatch, tmp_path_factory):
    names = [kvc._call_path(TORCH), kvc._call_path(str(other_torch))]
    assert names[0] == kvc._call_path(TORCH) and os.path.dirname(names[0]) == str(place)
    version = (other_torch / "version.py").read_text()
    (other_torch / "version.py").write_text(version.replace("git_version", "_git_version"))
    names.append(kvc._call_path(str(other_torch)))
    (other_torch / "lib" / "libc10.so").write_bytes(bytes(101))
    names.append(kvc._call_path(str(other_torch)))
    headers = tmp_path_factory.mktemp("include")
    with monkeypatch.context() as m:
        m.setattr(kvc, "_INCLUDE", str(headers))
        (headers / "kvc.h").write_text(open(os.path.join(os.path.dirname(kvc._HERE), "include", "kvc.h")).read() + "\n")
        names.append(kvc._call_path(TORCH))
    with monkeypatch.context() as m:
        m.setattr(kvc.sysconfig, "get_config_var", lambda name: "cpython-399-another")
        names.append(kvc._call_path(TORCH))
    assert len(set(names)) == len(names)
    (other_torch / "version.py").unlink()
    assert kvc._call_path(str(other_torch)) is None and kvc._call_path("") is None


def test_a_module_that_is_missing_is_built_beside_a_library_that_is_there(place, compiled, other_torch):
    for old in ("_kvc_call.so", os.path.basename(kvc._call_path(str(other_torch)))):
        (place / old).write_bytes(b"")
    assert kvc.build() == kvc.LIB_PATH
    assert [c[0] for c in compiled] == ["g++"]
    assert _modules(place) == [os.path.basename(kvc._call_path(TORCH))]
    kvc.build()
    assert len(compiled) == 1


def test_no_old_module_stays_where_none_can_be_built(place, compiled, other_torch, monkeypatch):
    for why in ("no torch", "no headers"):
        for old in ("_kvc_call.so", os.path.basename(kvc._call_path(str(other_torch)))):
            (place / old).write_bytes(b"")
        with monkeypatch.context() as m:
            if why == "no torch":
                m.setattr(kvc.importlib.util, "find_spec", lambda name: None)
            else:
                m.setenv("CUDA_HOME", str(place / "nowhere"))
            kvc.build()
        assert not compiled and not _modules(place), why


def test_the_module_here_refuses_in_words():
    kvc.build()
    kvc._load_torch()
    kvc._load_quick()
    if kvc._quick is None:
        pytest.skip("built without the interpreter's or torch's headers")
    with pytest.raises(ValueError, match="no CPU path"):
        kvc.dequantize(torch.zeros((2, kvc.KV_PAGE_BYTES), dtype=torch.uint8), torch.zeros(3, dtype=torch.int64),
                       torch.float32, out=torch.zeros((3, 512)))


@pytest.mark.parametrize("how", ["fails", "no compiler", "nothing to run"])
def test_the_library_is_built_without_the_module(place, monkeypatch, how):
    ran = []

    def run(cmd, **_):
        ran.append(cmd[0])
        if cmd[0] == "g++":
            if how == "nothing to run":
                raise FileNotFoundError("g++")
            return subprocess.CompletedProcess(cmd, 1, "", "cannot find -lc10_cuda")
        open(cmd[cmd.index("-o") + 1], "wb").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(kvc.subprocess, "run", run)
    if how == "no compiler":
        monkeypatch.setattr(shutil, "which", lambda name: None)
    (place / "libkvc.so").unlink()
    if how == "no compiler":
        assert kvc.build() == kvc.LIB_PATH
    else:
        with pytest.warns(RuntimeWarning, match="calls go through ctypes"):
            assert kvc.build() == kvc.LIB_PATH
    assert os.path.exists(kvc.LIB_PATH) and not [f for f in _modules(place) if f.endswith(".so")]
    asked = ran.count("g++")
    assert asked == (how != "no compiler")
    if how == "fails":  # not asked again, until something changes
        kvc.build()
        assert ran.count("g++") == asked
        with pytest.warns(RuntimeWarning, match="c10_cuda"):
            kvc.build(force=True)
        assert ran.count("g++") == asked + 1


@pytest.mark.parametrize("gone", ["lib/libc10_cuda.so", "include/c10/cuda/impl/cuda_cmake_macros.h", "lib/libtorch_cpu.so"])
def test_no_compiler_is_asked_beside_a_torch_without_cuda(place, compiled, monkeypatch, gone):
    there = os.path.exists
    monkeypatch.setattr(kvc.os.path, "exists", lambda path: path != os.path.join(TORCH, *gone.split("/")) and there(path))
    kvc.build()
    assert not compiled and not _modules(place)


def test_a_place_that_cannot_be_written_keeps_its_library(place, compiled, monkeypatch):
    def remove(path):
        raise PermissionError(path)

    (place / "_kvc_call.so").write_bytes(b"")
    monkeypatch.setattr(kvc.os, "remove", remove)
    with pytest.warns(RuntimeWarning):
        assert kvc.build() == kvc.LIB_PATH


def test_two_processes_that_remove_the_same_file(place, compiled, monkeypatch):
    def remove(path):
        raise FileNotFoundError(path)

    (place / "_kvc_call.so").write_bytes(b"")
    monkeypatch.setattr(kvc.os, "remove", remove)
    kvc.build()
    assert os.path.exists(kvc._call_path(TORCH)) and len(compiled) == 1
