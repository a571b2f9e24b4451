"""The extension that marshals the paged calls only saves time: where it cannot be
built or loaded, the library is what it was and the calls go through the Python
code behind it."""
import ctypes
import shutil

import pytest
import torch

import sequence_depth_attention_gb300 as moda
from sequence_depth_attention_gb300 import binding
from sequence_depth_attention_gb300 import build as mbuild

from test_abi_paged_args import arguments, ways  # noqa: F401 (a fixture)


@pytest.fixture
def fresh(monkeypatch, tmp_path):
    """binding.py with nothing loaded, and a copy of the extension to spoil."""
    mbuild.build()
    ext = tmp_path / "paged_py.so"
    shutil.copy(binding._EXT, ext)
    shutil.copy(binding._EXT + ".torch", str(ext) + ".torch")
    monkeypatch.setattr(binding, "_EXT", str(ext))
    monkeypatch.setattr(binding, "_lib", None)
    monkeypatch.setattr(binding, "_paged", None)
    return ext


def works(lib):
    assert lib.moda_decode_paged_workspace_bytes(16, 4, 128) > 0
    assert binding.load() is lib and moda.moda_decode_paged_workspace_bytes(16, 4, 128) > 0


def test_a_whole_extension_is_loaded(fresh, recwarn):
    works(binding.load())
    assert (binding._paged is not None) == torch.backends.cuda.is_built()
    assert not [w for w in recwarn if "paged_py" in str(w.message)]


@pytest.mark.skipif(not torch.backends.cuda.is_built(), reason="no extension without CUDA in torch")
@pytest.mark.parametrize("how", ["missing", "not a library", "of another torch", "without a stamp", "without its symbol"])
def test_a_spoiled_extension_costs_time_alone(fresh, how):
    stamp = fresh.with_name("paged_py.so.torch")
    if how == "missing":
        fresh.unlink()
    elif how == "not a library":
        fresh.write_bytes(b"no library")
    elif how == "of another torch":
        stamp.write_text("1.0.0")
    elif how == "without a stamp":
        stamp.unlink()
    else:
        shutil.copy(binding.library_path(), fresh)  # a library that is no module
    with pytest.warns(RuntimeWarning, match="paged_py"):
        lib = binding.load()
    assert binding._paged is None
    works(lib)


@pytest.mark.parametrize("call", ["append", "gather", "decode"])
def test_calls_without_the_extension(ways, call):  # noqa: F811
    rec, _ = ways  # (binding._paged is None there)
    getattr(moda, {"append": "moda_kv_append", "gather": "moda_kv_gather",
                   "decode": "moda_decode_paged"}[call])(**arguments(call, True))
    assert rec.seen is not None


@pytest.mark.parametrize("how", ["no compiler", "no headers"])
def test_the_library_builds_without_the_extension(monkeypatch, tmp_path, how):
    """Objects and library from the tree; the extension's compiler is not there, or fails."""
    mbuild.build()
    shutil.copytree(mbuild.BUILD, tmp_path / "_build", copy_function=shutil.copy2)
    for name in ("LIB", "EXT"):
        monkeypatch.setattr(mbuild, name, str(tmp_path / "_build" / getattr(mbuild, name).rsplit("/", 1)[1]))
    monkeypatch.setattr(mbuild, "BUILD", str(tmp_path / "_build"))
    shutil.os.remove(mbuild.LIB)
    shutil.os.remove(mbuild.EXT)
    which = shutil.which
    compiler = str(tmp_path / "nowhere") if how == "no compiler" else which("false")
    monkeypatch.setattr(mbuild.shutil, "which", lambda x: compiler if x == "g++" else which(x))
    with pytest.warns(RuntimeWarning, match="paged_py"):
        lib = mbuild.build()
    assert ctypes.CDLL(lib).moda_status_string
    # nothing stale is left to be loaded
    assert not shutil.os.path.exists(mbuild.EXT) and not shutil.os.path.exists(mbuild.EXT + ".torch")
