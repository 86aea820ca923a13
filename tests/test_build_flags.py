"""What a build compiles again: sources that changed, and objects made with other flags.  The
compiler is a stand-in that records its commands and touches its outputs."""
import os

import pytest

from persistent_tile_pipelined_b200 import build


@pytest.fixture
def project(tmp_path, monkeypatch):
    """Three sources and a header of their own; returns the commands since the last look."""
    csrc, include = tmp_path / "csrc", tmp_path / "include"
    csrc.mkdir()
    include.mkdir()
    (include / "tre.h").write_text("")
    (csrc / "a.h").write_text("")
    for name in ("a.cu", "b.cu", "c.cpp"):
        (csrc / name).write_text('#include "a.h"\n' if name == "a.cu" else '#include "tre.h"\n')
    clock = [1_000_000_000]

    def stamp(path):
        clock[0] += 10
        os.utime(path, (clock[0], clock[0]))

    for folder in (csrc, include):
        for f in folder.iterdir():
            stamp(f)
    commands = []

    def run(cmd):
        commands.append(cmd)
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        stamp(out)

    monkeypatch.setattr(build, "PKG", str(tmp_path))
    monkeypatch.setattr(build, "CSRC", str(csrc))
    monkeypatch.setattr(build, "INCLUDE", str(include))
    monkeypatch.setattr(build, "ENGINE_LIB", str(tmp_path / "libtre.so"))
    monkeypatch.setattr(build, "ENGINE_SOURCES", ["a.cu", "b.cu", "c.cpp"])
    monkeypatch.setattr(build, "_nvcc", lambda: "nvcc")
    monkeypatch.setattr(build.subprocess, "check_call", run)

    def compiled():
        """{source: flags} of what was compiled since the last look, and whether it was linked."""
        got = {os.path.basename(c[c.index("-c") + 1]): c for c in commands if "-c" in c}
        linked = any("-shared" in c for c in commands)
        commands.clear()
        return got, linked

    compiled.touch = lambda name: stamp(csrc / name)
    return compiled


def test_only_what_changed_is_compiled(project):
    build.build_engine()
    got, linked = project()
    assert set(got) == {"a.cu", "b.cu", "c.cpp"} and linked
    build.build_engine()
    assert project() == ({}, False)
    project.touch("a.h")
    build.build_engine()
    got, linked = project()
    assert set(got) == {"a.cu"} and linked


@pytest.mark.parametrize("touched", [None, "b.cu"])
def test_objects_of_other_flags_are_not_taken(project, touched):
    build.build_engine()
    project()
    build.build_engine(extra_flags=["-DTRACE"])
    got, linked = project()
    assert len(got) == 3 and all("-DTRACE" in c for c in got.values()) and linked
    if touched:
        project.touch(touched)
    build.build_engine()
    got, linked = project()
    assert len(got) == 3 and not any("-DTRACE" in c for c in got.values()) and linked
    build.build_engine()
    assert project() == ({}, False)


def test_changed_flags_compile_everything(project, monkeypatch):
    build.build_engine()
    project()
    monkeypatch.setattr(build, "NVCC_FLAGS", [*build.NVCC_FLAGS, "-G"])
    build.build_engine()
    got, linked = project()
    assert len(got) == 3 and all("-G" in c for c in got.values()) and linked


def test_objects_of_a_build_that_stopped_half_way_are_not_taken(project, monkeypatch):
    build.build_engine()
    project()
    run = build.subprocess.check_call

    def stop_at_b(cmd):
        if any(str(c).endswith("b.cu") for c in cmd):
            raise KeyboardInterrupt
        run(cmd)

    monkeypatch.setattr(build.subprocess, "check_call", stop_at_b)
    with pytest.raises(KeyboardInterrupt):
        build.build_engine(extra_flags=["-DTRACE"])
    project()
    monkeypatch.setattr(build.subprocess, "check_call", run)
    build.build_engine()  # the library is still the one of the first build
    project.touch("c.cpp")
    build.build_engine()
    got, linked = project()
    assert {"a.cu", "c.cpp"} <= set(got) and linked
    assert not any("-DTRACE" in c for c in got.values())
