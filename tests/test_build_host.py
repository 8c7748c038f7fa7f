"""The build, where the extension for torch callers cannot be built or the library's compiler
fails (no GPU, and nothing is compiled: the compilers are stand-ins)."""
import sysconfig

import pytest
import torch

from paged_kv_cache_msa_gb300 import binding as B
from paged_kv_cache_msa_gb300 import build as build_mod


@pytest.fixture
def place(tmp_path, monkeypatch):
    """A build into a folder of its own, with stand-ins for both compilers."""
    for name, file in (("OUT_DIR", ""), ("LIB_PATH", "lib.so"), ("STAMP_PATH", "lib.so.sha256"), ("MARSHAL_PATH", "marshal.so")):
        monkeypatch.setattr(build_mod, name, str(tmp_path / file))
    monkeypatch.delenv("MSA_NO_BUILD", raising=False)
    monkeypatch.setattr(build_mod, "_compile", lambda lib, *a, **k: (tmp_path / "lib.so").write_text("library"))
    monkeypatch.setattr(build_mod, "marshal_command", lambda out: ["touch", out])
    monkeypatch.setattr(build_mod, "marshal_digest", lambda: "digest")
    return tmp_path


def test_both_are_built(place):
    assert build_mod.build() == str(place / "lib.so")
    assert sorted(f.name for f in place.iterdir()) == ["lib.so", "marshal.so", "marshal.so.sha256"]


@pytest.mark.parametrize("lacking", ["cuda", "headers"])
def test_the_library_is_built_without_the_extension(place, monkeypatch, lacking):
    """And an extension of an earlier build does not stay beside it; a call that needs it says why."""
    build_mod.build()
    if lacking == "cuda":
        monkeypatch.setattr(torch.version, "cuda", None)
    else:
        monkeypatch.setattr(sysconfig, "get_paths", lambda *a: {"include": str(place / "nowhere")})
    monkeypatch.setattr(build_mod, "marshal_command", lambda out: ["false"])
    assert build_mod.build(force=True) == str(place / "lib.so")
    assert sorted(f.name for f in place.iterdir()) == ["lib.so"]
    monkeypatch.setattr(B, "_marshal", None)
    with pytest.raises(RuntimeError, match="CUDA" if lacking == "cuda" else "headers"):
        B.norm_tensors(B.make_norm_cfg(8), None, None)


def test_a_failed_extension_is_an_error(place, monkeypatch):
    monkeypatch.setattr(build_mod, "marshal_command", lambda out: ["false"])
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        build_mod.build()
    assert sorted(f.name for f in place.iterdir()) == ["lib.so"]


def test_a_failed_library_leaves_no_compiler_running(place, monkeypatch):
    started = []
    start = build_mod.subprocess.Popen

    def keep(*a, **k):
        started.append(start(*a, **k))
        return started[-1]

    def fail(*a, **k):
        raise RuntimeError("nvcc failed")

    monkeypatch.setattr(build_mod.subprocess, "Popen", keep)
    monkeypatch.setattr(build_mod, "_compile", fail)
    monkeypatch.setattr(build_mod, "marshal_command", lambda out: ["sleep", "60"])
    with pytest.raises(RuntimeError, match="nvcc"):
        build_mod.build()
    assert len(started) == 1 and started[0].poll() is not None
    assert list(place.iterdir()) == []
