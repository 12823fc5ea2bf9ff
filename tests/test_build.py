"""Objects of the library are kept only while they are what a fresh build would make (no
compiler runs here: a stand-in writes the files)."""
import os

import pytest

from step_flow_map_b200 import build


class Box:
    """A source tree of two sources and a header, and a compiler that writes down its flags."""

    def __init__(self, tmp, monkeypatch):
        self.root, self.ran = tmp, []
        here, inc = tmp / "pkg", tmp / "include"
        (here / "csrc").mkdir(parents=True)
        inc.mkdir()
        for f, text in (("a.cu", '#include "h.cuh"\n'), ("b.cu", ""), ("h.cuh", "")):
            (here / "csrc" / f).write_text(text)
        (inc / "flashmap.h").write_text("")
        (here / "build.py").write_text("")
        for n, v in dict(HERE=here, ROOT=tmp, LIB=here / "l.so", OBJ_DIR=here / "_build").items():
            monkeypatch.setattr(build, n, str(v))
        monkeypatch.setattr(build, "SRCS", [str(here / "csrc" / f) for f in ("a.cu", "b.cu")])
        monkeypatch.setattr(build, "_run", self.run)
        self.age()

    def age(self):
        """Everything so far was made a minute ago."""
        for d, _, fs in os.walk(self.root):
            for f in fs:
                p = os.path.join(d, f)
                t = os.path.getmtime(p) - 60
                os.utime(p, (t, t))

    def run(self, cmds, verbose):
        for c in cmds:
            out = c[c.index("-o") + 1]
            self.ran.append(os.path.basename(c[-3]) if "-c" in c else "link")
            if "-c" in c:
                text = " ".join(x for x in c if x.startswith("-D")) or "plain"
            else:
                text = "|".join(open(x).read() for x in c if x.endswith(".o"))
            with open(out, "w") as f:
                f.write(text)

    def build(self, **kw):
        self.ran.clear()
        build.build(**kw)
        with open(build.LIB) as f:
            return f.read(), sorted(self.ran)


@pytest.fixture
def box(tmp_path, monkeypatch):
    return Box(tmp_path, monkeypatch)


def touch(p):
    os.utime(p)


def test_only_what_changed_is_compiled(box):
    assert box.build() == ("plain|plain", ["a.cu", "b.cu", "link"])
    assert box.build() == ("plain|plain", [])
    box.age()
    touch(build.SRCS[1])
    assert box.build() == ("plain|plain", ["b.cu", "link"])
    box.age()
    touch(os.path.join(build.HERE, "csrc", "h.cuh"))
    assert box.build() == ("plain|plain", ["a.cu", "link"])


def test_objects_of_other_flags_are_not_linked(box):
    assert box.build(extra=("-DX",))[0] == "-DX|-DX"
    box.age()
    touch(build.SRCS[1])
    assert box.build() == ("plain|plain", ["a.cu", "b.cu", "link"])
    assert box.build(extra=("-DX",))[0] == "-DX|-DX"
    assert box.build(extra=("-DY",))[0] == "-DY|-DY"
    assert box.build() == ("plain|plain", ["link"])


def test_a_change_of_the_build_itself_compiles_anew(box):
    box.build()
    box.age()
    touch(os.path.join(build.HERE, "build.py"))
    assert box.build()[1] == ["a.cu", "b.cu", "link"]


def test_nothing_half_written_is_left_or_linked(box, monkeypatch):
    box.build()
    box.age()
    touch(build.SRCS[0])

    def breaks(cmds, verbose):
        box.run(cmds, verbose)
        raise RuntimeError("the compiler was stopped")
    before = {f: open(os.path.join(build.OBJ_DIR, f)).read() for f in os.listdir(build.OBJ_DIR)}
    monkeypatch.setattr(build, "_run", breaks)
    with pytest.raises(RuntimeError):
        build.build(extra=())
    assert {f: open(os.path.join(build.OBJ_DIR, f)).read() for f in os.listdir(build.OBJ_DIR)} == before
    monkeypatch.setattr(build, "_run", box.run)
    assert box.build()[1] == ["a.cu", "link"]


def test_a_source_that_changes_while_it_is_compiled_is_compiled_again(box, monkeypatch):
    def slow(cmds, verbose):
        box.run(cmds, verbose)
        t = os.path.getmtime(build.SRCS[0]) + 120   # past the start of this build
        os.utime(build.SRCS[0], (t, t))
    monkeypatch.setattr(build, "_run", slow)
    build.build()
    monkeypatch.setattr(build, "_run", box.run)
    assert "a.cu" in box.build()[1]


def test_a_library_of_unknown_objects_counts_by_its_age(box):
    """One that came without the folder of objects is not built again where its sources are older."""
    box.build()
    for f in os.listdir(build.OBJ_DIR):
        os.remove(os.path.join(build.OBJ_DIR, f))
    assert box.build()[1] == []
