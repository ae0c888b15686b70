"""What the build makes again, with compilers that only write down that they were called."""
import os

import pytest

from event_tensor_task_b200 import build as B


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A source tree of two sources, a header and the tensor module; returns a function that builds it and tells what
    was made."""
    here = tmp_path / "package"
    for d in (here / "csrc", tmp_path / "include"):
        d.mkdir(parents=True)
    for name in ("build.py", "csrc/a.cu", "csrc/b.cpp", "csrc/t.cpp", "csrc/h.cuh"):
        (here / name).write_text("")
        os.utime(here / name, (1, 1))
    log = tmp_path / "log"
    cc = tmp_path / "cc"
    cc.write_text(f"""#!/bin/sh
while [ $# -gt 0 ]; do [ "$1" = -o ] && out=$2; shift; done
[ -e {tmp_path}/broken ] && exit 1
echo $(basename $out) >> {log}; echo > $out
""")
    cc.chmod(0o755)
    for name, value in dict(HERE=str(here), ROOT=str(tmp_path), LIB=str(here / "lib.so"), TENSORS=str(here / "t.so"),
                            OBJ=str(here / "_build"), NVCC=str(cc), CXX=str(cc), SOURCES=["csrc/a.cu", "csrc/b.cpp"],
                            TENSORS_SOURCE="csrc/t.cpp").items():
        monkeypatch.setattr(B, name, value)
    monkeypatch.setattr(B, "_tensors_command", lambda: [str(cc), "-o", B.TENSORS])

    def made(**kw):
        if log.exists():
            log.unlink()
        B.build(**kw)
        return sorted(log.read_text().split()) if log.exists() else []

    made.root, made.here = tmp_path, here
    return made


ALL = ["a.cu.o", "b.cpp.o", "lib.so", "t.so"]


def test_only_what_changed_is_made_again(tree):
    assert tree() == ALL and tree() == []
    later = os.path.getmtime(B.LIB) + 5
    os.utime(tree.here / "csrc" / "b.cpp", (later, later))
    os.utime(B._object("csrc/a.cu"), (later - 1, later - 1))
    assert tree() == ["b.cpp.o", "lib.so"]
    for name in ("csrc/b.cpp", "csrc/h.cuh"):
        os.utime(tree.here / name, (1, 1))
    assert tree(force=True) == ALL
    os.utime(tree.here / "csrc" / "h.cuh", (later + 9, later + 9))
    assert tree() == ALL


def test_other_flags_make_the_objects_again(tree):
    assert tree() == ALL
    assert tree(extra=["-G"]) == ["a.cu.o", "b.cpp.o", "lib.so"] and tree(extra=["-G"]) == []
    assert tree() == ["a.cu.o", "b.cpp.o", "lib.so"] and tree() == []


@pytest.mark.parametrize("what", ["torch", "python"])
def test_another_torch_or_python_makes_the_module_again(tree, monkeypatch, what):
    assert tree() == ALL
    if what == "torch":
        monkeypatch.setattr(B.importlib.metadata, "version", lambda name: "99.0")
    else:
        monkeypatch.setattr(B.sysconfig, "get_config_var", lambda name: "cpython-399")
    assert tree() == ["t.so"] and tree() == []


def test_a_failed_build_is_taken_up_again(tree):
    assert tree() == ALL
    (tree.root / "broken").write_text("")
    with pytest.raises(RuntimeError, match="failed"):
        tree(force=True)
    (tree.root / "broken").unlink()
    assert tree() == ALL and tree() == []
