"""Building and loading the optional extension of csrc/marshal.cpp: whatever
keeps it from being built, libpa.so is, and no extension stays behind that was
built for something else."""
import os

import pytest
import torch

from paged_kv_cache_76_gb300 import build


@pytest.fixture
def place(tmp_path, monkeypatch):
    """The extension's files in a folder of their own; libpa.so is up to date."""
    build.build()
    monkeypatch.setattr(build, "MARSHAL", str(tmp_path / os.path.basename(build.MARSHAL)))
    monkeypatch.setattr(build, "MARSHAL_STAMP", str(tmp_path / "marshal.stamp"))
    return tmp_path


def old_one():
    """An extension of an earlier build, and its stamp."""
    for p in (build.MARSHAL, build.MARSHAL_STAMP):
        with open(p, "w") as f:
            f.write("of another torch")


def compiler(path, text):
    path.write_text("#!/bin/sh\n" + text)
    path.chmod(0o755)
    return str(path)


@pytest.mark.parametrize("before", [False, True])
@pytest.mark.parametrize("why", ["compile fails", "half an output", "no compiler", "no torch", "no headers"])
def test_a_build_without_it_still_builds_the_library(place, monkeypatch, capfd, why, before):
    if before:
        old_one()
    if why == "compile fails":
        monkeypatch.setenv("CXX", compiler(place / "cxx", "echo no such library >&2; exit 1\n"))
    elif why == "half an output":
        monkeypatch.setenv("CXX", compiler(place / "cxx", 'for a; do case "$p" in -o) echo x > "$a";; esac; p="$a"; done\n'
                                           "exit 1\n"))
    elif why == "no compiler":
        monkeypatch.setenv("CXX", str(place / "none"))
    elif why == "no torch":
        monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    else:
        monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(place)})
    assert build.build() == build.LIB
    assert not os.path.exists(build.MARSHAL) and not os.path.exists(build.MARSHAL_STAMP)
    assert sorted(p.name for p in place.iterdir()) in ([], ["cxx"])
    assert "_marshal" in capfd.readouterr().err          # left out, and said so
    monkeypatch.undo()


def test_a_build_with_it_replaces_the_old_one_and_then_rests(place, monkeypatch):
    old_one()
    body = 'for a; do case "$p" in -o) echo new > "$a";; esac; p="$a"; done\necho >> "$(dirname "$0")/ran"\n'
    monkeypatch.setenv("CXX", compiler(place / "cxx", body))
    for _ in range(2):
        build.build()
        with open(build.MARSHAL) as f:
            assert f.read() == "new\n"
    assert (place / "ran").read_text() == "\n"           # once
    assert str(torch.__version__) in open(build.MARSHAL_STAMP).read()


class Fake:
    """Stands for the extension: bind must not be reached in one that was built for another torch."""

    def __init__(self, version):
        self.bound = 0
        if version is not None:
            self.torch_version = version

    def bind(self, *addresses):
        self.bound += 1


@pytest.mark.parametrize("version,taken", [(str(torch.__version__), True), ("2.0.0", False), (None, False)])
def test_an_extension_built_for_another_torch_is_not_used(monkeypatch, version, taken):
    from paged_kv_cache_76_gb300 import ops
    build.build()
    fake = Fake(version)
    monkeypatch.setattr(ops.importlib, "import_module", lambda name, package=None: fake)
    monkeypatch.setattr(ops, "_marshal", None)
    assert ops._load_marshal() is (fake if taken else False) and fake.bound == taken
    assert ops._short_way(None) is (fake if taken else False) and fake.bound == taken     # not asked again


def test_the_extension_knows_its_torch():
    from paged_kv_cache_76_gb300 import ops
    build.build()
    if not os.path.exists(build.MARSHAL):
        pytest.skip("the extension is not built here")
    assert ops._load_marshal() and ops._marshal.torch_version == str(torch.__version__)
