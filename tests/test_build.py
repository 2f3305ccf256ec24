"""What build() compiles, with a stand-in for the compilers."""
import pytest

from ring_attn_gb300 import build as b


@pytest.fixture
def made(monkeypatch, tmp_path):
    """Every command line that build() runs; nothing is compiled."""
    cmds = []
    monkeypatch.setattr(b, "_run", lambda cmd: cmds.append(cmd) or "")
    for name, file in (("BUILD", "_build"), ("LIB", "lib.so"), ("BINDING", "binding.so"), ("BINDING_NOTE", "_build/note.txt")):
        monkeypatch.setattr(b, name, str(tmp_path / file))
    return cmds


def binding_of(cmds):
    return [c for c in cmds if b.BINDING_SRC in c]


def linked(cmds):
    return [c for c in cmds if b.LIB in c]


def test_without_torch_the_library_alone_is_built(made, monkeypatch):
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name: None)
    assert b.build() == b.LIB
    assert len(made) == len(b.SOURCES) + 1 and linked(made) and not binding_of(made)


def test_another_torch_has_the_binding_built_again(made):
    b.build()
    assert len(binding_of(made)) == 1
    open(b.BINDING, "w").close()
    made.clear()
    b.build()
    assert not binding_of(made)
    with open(b.BINDING_NOTE) as f:
        text = f.read()
    with open(b.BINDING_NOTE, "w") as f:
        f.write(text.replace("__version__ = '", "__version__ = '1."))
    b.build()
    assert len(binding_of(made)) == 1


def test_a_binding_that_fails_leaves_the_library(made, monkeypatch):
    record = b._run

    def run(cmd):
        if b.BINDING_SRC in cmd:
            raise RuntimeError("no Python.h")
        return record(cmd)

    monkeypatch.setattr(b, "_run", run)
    with pytest.raises(RuntimeError, match="Python.h"):
        b.build()
    assert linked(made)
    made.clear()
    with pytest.raises(RuntimeError):  # not taken for made
        b.build()
