"""The build script's commands, with the compiler replaced by a recorder."""
import importlib.util
import os
import subprocess
import types

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_extra_flags_reach_every_compile_and_the_link(tmp_path, monkeypatch):
    spec = importlib.util.spec_from_file_location("_llmoe_build_test", os.path.join(ROOT, "combine_ll_moe_amd", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    monkeypatch.setattr(mod, "LIB", str(tmp_path / "lib.so"))
    calls = []

    def record(cmd, **kw):
        calls.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(subprocess, "run", record)
    assert mod.build(extra_flags=["-gline-tables-only", "-Lsomewhere"]) == str(tmp_path / "lib.so")
    links = [c for c in calls if "-c" not in c]
    assert len(links) == 1 and len(calls) == len(mod.SOURCES) + 1
    for c in calls:
        assert "-gline-tables-only" in c and "-Lsomewhere" in c, c
    assert "-shared" in links[0] and os.path.exists(tmp_path / "lib.so")
