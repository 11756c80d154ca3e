"""The build: what makes the compiled binding stale, and which calls need it.
(The compilers are not run: a stand-in touches their outputs.)"""
import os
import subprocess
import sys

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


NO_COMPILER = """
import importlib.util, subprocess, sys
sys.path.insert(0, {root!r})
name = "paged_kv_decode_attention_gb300.build"
spec = importlib.util.spec_from_file_location(name, {root!r} + "/paged_kv_decode_attention_gb300/build.py")
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
b._binding_compile = lambda obj: ["/nonexistent/g++", "-o", obj]
b._binding_tag = lambda: "none"
b.BINDING = "/nonexistent/_pkv_binding.so"
sys.modules[name] = b
import paged_kv_decode_attention_gb300 as pkv
assert pkv.workspace_size(4, 1, 32, 100, 1) > 0
assert pkv.workspace_size_tree(1, 16, 32, 528, 56) > 0
for _ in range(2):
    try:
        pkv.paged_attention_window(*[None] * 6, 1, 1, 0, 1.0)
    except (OSError, RuntimeError):
        continue
    raise SystemExit("the call that needs the binding went on without it")
print("imported")
"""


def test_the_package_imports_where_the_binding_cannot_be_built():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", NO_COMPILER.format(root=root)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "imported" in r.stdout, r.stdout + r.stderr
