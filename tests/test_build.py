"""The build's order, with the compilers replaced by stand-ins."""
import os
import subprocess

import pytest

from bit_kv_cache_kvarn_gb300 import _build


def _stand_ins(tmp_path, monkeypatch, fails):
    """Compilers that write their -o file, except for commands that `fails` picks."""
    for name in ("BUILD", "LIB", "BINDING"):
        monkeypatch.setattr(_build, name, str(tmp_path / os.path.basename(getattr(_build, name))))

    def run(cmd, **kw):
        if fails(cmd):
            return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("made")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(_build.subprocess, "run", run)


def test_the_library_is_built_without_the_binding(tmp_path, monkeypatch):
    _stand_ins(tmp_path, monkeypatch, lambda cmd: any("serving_binding.cpp" in c for c in cmd))
    with pytest.raises(RuntimeError, match="binding"):
        _build.build()
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.BINDING)


def test_nothing_is_replaced_when_a_kernel_does_not_compile(tmp_path, monkeypatch):
    _stand_ins(tmp_path, monkeypatch, lambda cmd: any("rope_qkv.cu" in c for c in cmd))
    with pytest.raises(RuntimeError, match="rope_qkv"):
        _build.build()
    assert not os.path.exists(_build.LIB) and not os.path.exists(_build.BINDING)
