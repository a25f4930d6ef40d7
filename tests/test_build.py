"""What the build leaves where a part of it cannot be made (no compiler runs
here: the commands are stand-ins)."""
import pytest
import torch


@pytest.fixture
def build(monkeypatch, tmp_path):
    from speculative_decoding_verification_75_gb300 import build
    monkeypatch.setattr(build, "LIB", tmp_path / "lib" / "libspecverify.so")
    monkeypatch.setattr(build, "compile_command", lambda unit, out: ["touch", str(out)])
    monkeypatch.setattr(build, "link_command", lambda objects, out: ["touch", str(out)])
    monkeypatch.setattr(build, "binding_command", lambda out: ["touch", str(out)])
    return build


@pytest.mark.parametrize("command", ["false", "/nowhere/g++"])
def test_the_library_is_installed_without_the_binding(build, monkeypatch, command):
    monkeypatch.setattr(build, "binding_command", lambda out: [command])
    with pytest.warns(UserWarning, match="could not be built"):
        assert build.build() == build.LIB
    assert build.LIB.exists() and not build.library_is_stale()
    assert [p.name for p in build.LIB.parent.iterdir()] == [build.LIB.name]


def test_a_library_that_does_not_compile_is_an_error(build, monkeypatch):
    monkeypatch.setattr(build, "compile_command", lambda unit, out: ["false"])
    with pytest.raises(Exception):
        build.build()
    assert not build.LIB.exists()


def test_a_binding_for_another_pytorch_is_built_anew(build, monkeypatch):
    from speculative_decoding_verification_75_gb300 import api, kv
    monkeypatch.setattr(api, "_lib", object())
    build.build()
    assert not build.is_stale()
    before = build.binding_path()
    monkeypatch.setattr(torch, "__version__", "0.1.0")
    assert build.binding_is_stale() and not build.library_is_stale()
    monkeypatch.setattr(kv, "_native", None)
    with pytest.raises(RuntimeError, match="is not built"):
        kv.load_binding()
    build.build()
    assert build.binding_path() != before and not build.is_stale()
