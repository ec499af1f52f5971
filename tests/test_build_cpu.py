"""The build's parts on their own, with nothing compiled: the library without
torch or the compiled checks, the checks' file for one torch and Python only,
and the binding where that file is missing. No GPU."""
import importlib.util

import pytest
import torch

from long_context_prefill_dhsa_b200 import binding, build


@pytest.fixture
def made(monkeypatch):
    """What build() builds, with nothing up to date."""
    made = []
    monkeypatch.setattr(build, "build_library", lambda verbose_ptxas=False: made.append("library"))
    monkeypatch.setattr(build, "build_marshal", lambda: made.append("checks"))
    monkeypatch.setattr(build, "library_up_to_date", lambda: False)
    monkeypatch.setattr(build, "marshal_up_to_date", lambda: False)
    return made


def test_both_are_built(made):
    assert build.build() == build.LIB and sorted(made) == ["checks", "library"]


def test_the_library_needs_no_torch(made, monkeypatch):
    monkeypatch.setattr(importlib.util, "find_spec", lambda name: None)
    assert build.build() == build.LIB and made == ["library"]


def test_the_library_is_built_when_the_checks_are_not(made, monkeypatch):
    def fails():
        raise RuntimeError("no compiler")
    monkeypatch.setattr(build, "build_marshal", fails)
    with pytest.raises(RuntimeError, match="no compiler"):
        build.build()
    assert made == ["library"]


def test_checks_of_another_torch_or_python_are_out_of_date(monkeypatch):
    here = build.marshal_path()
    monkeypatch.setattr(build.importlib.metadata, "version", lambda name: "0.0.1")
    assert build.marshal_path() != here and not build.marshal_up_to_date()
    monkeypatch.undo()
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: "cpython-00")
    assert build.marshal_path() != here and not build.marshal_up_to_date()


def test_a_torch_without_package_metadata(made, monkeypatch):
    here = build.marshal_path()

    def none(name):
        raise build.importlib.metadata.PackageNotFoundError(name)
    monkeypatch.setattr(build.importlib.metadata, "version", none)
    assert build.marshal_path() == here and build.build() == build.LIB and "library" in made


def test_checks_of_another_torch_are_not_loaded(monkeypatch):
    """The binding then checks in Python, says so, and refuses as before."""
    build.build()
    monkeypatch.setattr(binding, "_marshal", None)
    monkeypatch.setattr(build.importlib.metadata, "version", lambda name: "0.0.1")
    bf = torch.zeros(1, 2, 3, 128, dtype=torch.bfloat16)
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.warns(UserWarning, match="checked in Python"):
        with pytest.raises(ValueError):
            binding.tree_attn(bf, bf, bf, n)
    assert binding._marshal is binding._ChecksInPython
    with pytest.raises(ValueError):
        binding.rotary_qkv(bf, bf, torch.zeros(64, dtype=torch.float64))
    with pytest.raises(ValueError):
        binding.cache_evict(bf, bf, torch.zeros(1, 2, 3), torch.zeros(1, 2, 3, dtype=torch.int32), n, 2)


def test_checks_of_this_torch_are_loaded(monkeypatch):
    build.build()
    monkeypatch.setattr(binding, "_marshal", None)
    assert binding._load_marshal().__file__ == build.marshal_path()
