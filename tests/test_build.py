"""The library's build with a stand-in compiler: two builds at once, a build that is cut off, a compiler
that fails, sources and flags that change. The stand-in writes its output in two halves; "linking" joins
the objects, and a half-written one shows in the result."""
import os
import subprocess
import sys
import textwrap
import time

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

COMPILER = """\
#!{python}
import os, signal, sys, time
a = sys.argv[1:]
out = a[a.index("-o") + 1]
if "-shared" in a:
    parts = [open(x).read() for x in a[:a.index("-o")] if x.endswith(".o")]
    open(out, "w").write("".join(parts))
    sys.exit(0)
src = a[a.index("-c") + 1]
text = open(src).read()
open(a[a.index("-MF") + 1], "w").write("x: " + src + "\\n")
half = "<" + os.path.basename(src) + " " + text
if os.path.exists(out):
    os.remove(out)
with open(out, "w") as f:
    f.write(half)
    f.flush()
    if "KILL" in text:
        os.kill(os.getppid(), signal.SIGKILL)
        os._exit(1)
    if "FAIL" in text:
        sys.exit(3)
    time.sleep(0.5 if "slow" in text else 0.05)
    f.write(">")
"""

# the build module alone (the package would import torch), on a tree of its own
MODULE = """\
import importlib.util, os, sys, time
spec = importlib.util.spec_from_file_location("build_under_test", {root!r} + "/sparse_dynamic_routing_b200/build.py")
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
b.CSRC, b.OBJ_DIR, b.LIB, b.HEADER = (os.path.join({tmp!r}, x) for x in ("csrc", "build", "lib.so", "csrc/a.cu"))
"""


BUILD = "print(open(b.build()).read())"


class Tree:
    def __init__(self, path):
        self.path = str(path)
        os.makedirs(self.path + "/csrc")
        cc = self.path + "/nvcc"
        with open(cc, "w") as f:
            f.write(COMPILER.format(python=sys.executable))
        os.chmod(cc, 0o755)
        self.env = {**os.environ, "NVCC": cc}

    def write(self, name, text):
        with open(f"{self.path}/csrc/{name}", "w") as f:
            f.write(text)

    def start(self, then):
        """A process that runs these statements with the module as `b`."""
        code = MODULE.format(root=ROOT, tmp=self.path) + textwrap.dedent(then)
        return subprocess.Popen([sys.executable, "-c", code], env=self.env, stdout=subprocess.PIPE, stderr=subprocess.PIPE,
                                text=True)

    def run(self, then):
        p = self.start(then)
        out, err = p.communicate(timeout=120)
        return p.returncode, out.strip(), err

    def build(self):
        return self.run(BUILD)

    def stale(self):
        return self.run("print(b.stale(b.LIB))")[1] == "True"

    def left(self):
        return sorted(x for x in os.listdir(self.path + "/build") if ".tmp" in x)


@pytest.fixture
def tree(tmp_path):
    t = Tree(tmp_path)
    t.write("a.cu", "one slow")
    t.write("b.cu", "two")
    return t


WHOLE = "<a.cu one slow><b.cu two>"


def test_builds_at_once_link_whole_objects(tree):
    runs = []
    for _ in range(4):  # each starts while the one before compiles
        runs.append(tree.start("print(open(b.build(force=True)).read())"))
        time.sleep(0.25)
    for p in runs:
        out, err = p.communicate(timeout=120)
        assert p.returncode == 0 and out.strip() == WHOLE, err[-500:]
    assert tree.left() == []


def test_a_build_that_was_cut_off_leaves_nothing_that_counts(tree):
    tree.write("a.cu", "KILL")
    assert tree.build()[0] != 0
    # the source as it was, older than whatever the cut-off build left
    tree.write("a.cu", "one slow")
    old = time.time() - 100
    for x in ("a.cu", "b.cu"):
        os.utime(f"{tree.path}/csrc/{x}", (old, old))
    rc, out, err = tree.build()
    assert rc == 0 and out == WHOLE, err[-500:]


def test_a_failing_compiler_waits_for_the_others(tree):
    tree.write("a.cu", "FAIL")
    tree.write("b.cu", "two slow")
    rc, _, err = tree.build()
    assert rc != 0 and "CalledProcessError" in err
    time.sleep(0.05)
    names = sorted(os.listdir(tree.path + "/build"))
    assert names == ["b.o", "b.o.d"]  # b's is whole, of a nothing is left
    with open(tree.path + "/build/b.o") as f:
        assert f.read() == "<b.cu two slow>"


def test_what_makes_the_library_stale(tree):
    assert tree.build()[1] == WHOLE
    assert not tree.stale()
    tree.write("b.cu", "three")
    assert tree.stale()
    assert tree.build()[1] == "<a.cu one slow><b.cu three>"


def test_a_source_edited_while_it_compiles_is_compiled_again(tree):
    p = tree.start(BUILD)
    deadline = time.time() + 60
    while not any(x.startswith("a.o") for x in (os.listdir(tree.path + "/build") if os.path.isdir(tree.path + "/build") else [])):
        assert time.time() < deadline
        time.sleep(0.01)
    time.sleep(0.1)
    tree.write("a.cu", "later slow")  # the compiler has read the text before
    assert p.communicate(timeout=120)[0].strip() == WHOLE
    assert tree.build()[1] == "<a.cu later slow><b.cu two>"


def test_changed_flags_make_everything_stale(tree):
    """The flags stand in build.py itself: objects and libraries older than it are made again."""
    assert tree.build()[1] == WHOLE
    rc, out, err = tree.run("""
        obj = b.OBJ_DIR + "/a.o"
        print(b.stale(b.LIB), b._object_is_stale(obj, obj + ".d"))
        later = os.path.join(os.path.dirname(b.LIB), "later.py")
        open(later, "w").close()
        os.utime(later, (time.time() + 5, time.time() + 5))
        b.SELF = later
        print(b.stale(b.LIB), b._object_is_stale(obj, obj + ".d"))
    """)
    assert out.split() == ["False", "False", "True", "True"], err[-500:]
