"""What build() leaves behind, with a compiler that only writes its output files."""
import os
import stat

import pytest

from block_quantized_weight_row_gb300 import build as bq_build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A package of two sources whose compilers touch what -o names, and log their lines."""
    src = tmp_path / "csrc"
    src.mkdir()
    include = tmp_path / "include"
    include.mkdir()
    for f in (src / "a.cu", src / "b.cu", src / "p.cu", src / "e.cpp", include / "bq.h"):
        f.write_text("")
    cc = tmp_path / "cc"
    cc.write_text('#!/bin/sh\necho "$@" >> ' + str(tmp_path / "log") + '\nwhile [ "$1" != -o ]; do shift; done\n: > "$2"\n')
    cc.chmod(cc.stat().st_mode | stat.S_IXUSR)
    for name, value in dict(CSRC=src, OBJ_DIR=src / "_build", LIB=tmp_path / "lib.so", PROBE_SRC="p.cu", PROBE_LIB=tmp_path / "probe.so",
                            EXT_SRC="e.cpp", EXT_LIB=tmp_path / "ext.so", INCLUDE=include, HERE=tmp_path).items():
        monkeypatch.setattr(bq_build, name, str(value))
    monkeypatch.setattr(bq_build, "SOURCES", ["a.cu", "b.cu"])
    monkeypatch.setattr(bq_build, "nvcc", lambda: str(cc))
    commands = bq_build.ext_commands

    def ext_commands(tmp):
        obj, compile_, link = commands(tmp)
        return obj, [str(cc), *compile_[1:]], [str(cc), *link[1:]]

    monkeypatch.setattr(bq_build, "ext_commands", ext_commands)

    def built():
        lines = (tmp_path / "log").read_text().splitlines() if (tmp_path / "log").exists() else []
        (tmp_path / "log").write_text("")
        outs = [line.split()[line.split().index("-o") + 1] for line in lines]
        return sorted(os.path.basename(o).split(".tmp")[0] for o in outs)

    return tmp_path, built


def test_everything_is_built_once(tree):
    path, built = tree
    bq_build.build()
    assert built() == ["a.o", "b.o", "e.o", "ext.so", "lib.so", "probe.so"]
    assert all((path / f).exists() for f in ("lib.so", "probe.so", "ext.so"))
    bq_build.build()
    assert built() == []


@pytest.mark.parametrize("step", ["headers", "compile", "link"])
def test_the_library_is_linked_where_the_extension_cannot_be_built(tree, monkeypatch, step):
    path, built = tree
    commands = bq_build.ext_commands

    def failing(tmp):
        if step == "headers":
            raise ImportError("no torch")
        obj, compile_, link = commands(tmp)
        return (obj, ["false"], link) if step == "compile" else (obj, compile_, ["false", *link[1:]])

    monkeypatch.setattr(bq_build, "ext_commands", failing)
    with pytest.raises((ImportError, RuntimeError)):
        bq_build.build()
    assert (path / "lib.so").exists() and (path / "probe.so").exists() and not (path / "ext.so").exists()
    built()
    monkeypatch.setattr(bq_build, "ext_commands", commands)  # mended: the rest follows
    bq_build.build()
    assert (path / "ext.so").exists() and "lib.so" not in built()


def test_the_extension_follows_torch(tree, monkeypatch):
    """Another torch (or Python): only the extension is compiled and linked again, once."""
    path, built = tree
    bq_build.build()
    built()
    monkeypatch.setattr("torch.__version__", "2.999.0")
    bq_build.build()
    assert built() == ["e.o", "ext.so"]
    bq_build.build()
    assert built() == []
