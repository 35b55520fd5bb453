"""Building where torch or g++ is missing: the C library needs neither."""
import importlib.util
import os
import types

import pytest

from sampling_threshold_filtering_amd import build_native


@pytest.mark.parametrize("spec", [None, types.SimpleNamespace(origin=None),
                                  types.SimpleNamespace(origin="/nowhere/torch/__init__.py")])
def test_without_torch_for_rocm_the_binding_is_left_out(spec, tmp_path, monkeypatch, capsys):
    stale = tmp_path / "_operators.so"
    stale.write_bytes(b"of an earlier build")
    monkeypatch.setattr(build_native, "BINDING", str(stale))
    monkeypatch.setattr(importlib.util, "find_spec", lambda name: spec)
    build_native._build_binding()
    assert not stale.exists()
    assert "left out" in capsys.readouterr().out
    build_native._build_binding()  # nor is there anything to remove


def test_without_gxx_the_binding_is_built_with_hipcc(tmp_path, monkeypatch):
    if build_native._torch_folder() is None:
        pytest.skip("needs torch for ROCm")
    at = tmp_path / "_operators.so"
    monkeypatch.setattr(build_native, "BINDING", str(at))
    monkeypatch.delenv("CXX", raising=False)
    monkeypatch.setattr(build_native.shutil, "which", lambda name: None)
    ran = []
    run = build_native.subprocess.run
    monkeypatch.setattr(build_native.subprocess, "run", lambda cmd, **kw: (ran.append(cmd[0]), run(cmd, **kw))[1])
    build_native._build_binding()
    assert ran == [build_native.HIPCC] and os.path.getsize(at) > 0
