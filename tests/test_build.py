"""The build: what makes the compiled binding stale.  (The compilers are not
run: a stand-in touches their outputs.)"""
import os
import subprocess

import torch

from paged_kv_decode_attention_gb300 import build as b


def _recorded_build(monkeypatch, tmp_path):
    """build() in an empty folder, as a list of the commands it runs."""
    commands = []

    def touch(cmd, **kw):
        commands.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(b.subprocess, "run", touch)
    monkeypatch.setattr(b, "BUILD", str(tmp_path))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libpkv.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_pkv_binding.so"), raising=False)

    def build():
        commands.clear()
        b.build()
        return [os.path.basename(c[0]) for c in commands]

    return build


def test_another_torch_or_python_makes_the_binding_stale(monkeypatch, tmp_path):
    build = _recorded_build(monkeypatch, tmp_path)
    assert build().count("g++") == 2  # compiled and linked
    assert build() == []
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "2.0.1+cu999")
        assert build() == ["g++", "g++"] and build() == []
    assert build() == []  # the former one is still there
    with monkeypatch.context() as m:
        m.setattr(torch.version, "git_version", "0123456789abcdef")
        assert build() == ["g++", "g++"]
    real = b.sysconfig.get_config_var
    with monkeypatch.context() as m:
        m.setattr(b.sysconfig, "get_config_var", lambda n: "cpython-399-somewhere" if n == "SOABI" else real(n))
        assert build() == ["g++", "g++"]
