"""The compiled part of the binding is this interpreter's and this library's, or none: then every call takes the
interpreted way."""
import os
import subprocess
import sys
import sysconfig
import types

import pytest

from routed_expert_ffn_topk_gb300 import build as build_mod

NAME = "routed_expert_ffn_topk_gb300._binding"


def test_name_and_stale_files(tmp_path):
    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    assert os.path.basename(build_mod.BINDING_PATH) == "_binding" + suffix
    path, untagged = str(tmp_path / ("_binding" + suffix)), tmp_path / "_binding.so"
    untagged.write_bytes(b"another interpreter's")
    build_mod.build_binding(path)
    assert not untagged.exists() and os.path.getsize(path) > 4096
    made = os.stat(path).st_mtime_ns
    build_mod.build_binding(path)
    assert os.stat(path).st_mtime_ns == made
    # older than its source, and no headers to build it anew: nothing is left to load
    os.utime(path, (0, 0))
    build_mod.build_binding(path, python_include=str(tmp_path))
    assert not os.path.exists(path)
    build_mod.build_binding(path, python_include=str(tmp_path))
    assert os.listdir(tmp_path) == []


@pytest.mark.parametrize("module", ["none", "no version", "other version", "cannot be loaded"])
def test_falls_back(monkeypatch, module):
    import routed_expert_ffn_topk_gb300 as package
    from routed_expert_ffn_topk_gb300 import estream as es
    build_mod.build()
    L = es.lib()
    real = es._fast
    assert real is not None and real.version == es.version()

    def setup(*a):
        raise AssertionError("a module of another version was set up")
    fake = types.ModuleType(NAME)
    fake.setup = setup
    if module == "other version":
        fake.version = es.version() + 1
    if module == "cannot be loaded":
        class Finder:
            @staticmethod
            def find_spec(name, path=None, target=None):
                if name == NAME:
                    raise ImportError("built for another interpreter")
        monkeypatch.delitem(sys.modules, NAME)
        monkeypatch.setattr(sys, "meta_path", [Finder] + sys.meta_path)
        monkeypatch.delattr(package, "_binding")
    elif module == "none":
        monkeypatch.setitem(sys.modules, NAME, None)
        monkeypatch.delattr(package, "_binding")
    else:
        monkeypatch.setitem(sys.modules, NAME, fake)
        monkeypatch.setattr(package, "_binding", fake)
    monkeypatch.setattr(es, "_fast", real)
    es._load_fast(L)
    assert es._fast is None


def test_fresh_process():
    """As a program loads it."""
    build_mod.build()
    code = "from routed_expert_ffn_topk_gb300 import estream as es; es.lib(); print(es._fast.__file__)"
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=build_mod.ROOT)
    assert r.returncode == 0 and r.stdout.strip() == build_mod.BINDING_PATH, r.stderr
