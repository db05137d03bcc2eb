"""The build knows every file that its objects are made of."""
import os
import re

from accelerator_decode_gb300 import build


def test_every_include_is_a_dependency():
    todo, seen = list(build.SOURCES), set()
    while todo:
        path = todo.pop()
        if path in seen:
            continue
        seen.add(path)
        with open(path) as f:
            for name in re.findall(r'^\s*#include "([^"]+)"', f.read(), re.M):
                todo.append(os.path.normpath(os.path.join(os.path.dirname(path), name)))
    known = {os.path.normpath(p) for p in build.DEPS}
    assert {os.path.normpath(p) for p in seen} <= known
    assert all(os.path.exists(p) for p in known)
    assert os.path.normpath(build.__file__) in known            # the flags


def test_an_edited_header_makes_every_object_old(tmp_path, monkeypatch):
    """Each of the files makes what is built from it again, and a source its own object only."""
    jobs = []

    class Done:
        def wait(self):
            return 0

    def popen(cmd):
        jobs.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return Done()

    monkeypatch.setattr(build.subprocess, "Popen", popen)
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, check: open(cmd[cmd.index("-o") + 1], "w").close())
    monkeypatch.setattr(build, "HERE", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    for late in build.DEPS:
        build.build()                                            # everything is there and fresh
        ages = {p: 1000 for p in build.DEPS}
        ages[late] = 4000
        real = os.path.getmtime
        monkeypatch.setattr(build.os.path, "getmtime",
                            lambda p, ages=ages, real=real: ages.get(p, 3000 if str(p).startswith(str(tmp_path)) else real(p)))
        del jobs[:]
        build.build()
        made = {c[-1] for c in jobs}
        assert made == ({late} if late in build.SOURCES else set(build.SOURCES)), late
        monkeypatch.setattr(build.os.path, "getmtime", real)
