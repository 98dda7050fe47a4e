"""The build: what the compiler says of the kernels that are to keep their rows in registers, and what is built of
what.  The latter with stand-ins for the compilers, which write their output file and note that they ran."""
from __future__ import annotations

import os
import re
import shutil
import stat
import subprocess
import sys

import pytest

from exact_tiled_attention_fa_gb300 import build as fa_build


def test_norm_and_rotation_kernels_do_not_spill(tmp_path):
    """Bound by bytes with 64 and 128 registers a thread: a spill is memory traffic of its own."""
    src = os.path.join(fa_build.CSRC, "fa_qk_rope.cu")
    r = subprocess.run([fa_build._nvcc(), *fa_build.ARCH, *fa_build.NVCC_FLAGS, "-Xptxas", "-v", "-I", fa_build.INCLUDE, "-c", src,
                        "-o", str(tmp_path / "rope.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    spills = re.findall(r"(\d+) bytes spill stores, (\d+) bytes spill loads", r.stderr)
    assert len(spills) >= 37  # 12 forward and cache forms, 24 gradient forms, the weights' sum
    assert set(spills) == {("0", "0")}, r.stderr


@pytest.fixture
def tree(tmp_path):
    """A copy of the sources with compilers that only note their calls; run(..) builds in a process of its own."""
    pkg = tmp_path / "pkg"
    shutil.copytree(fa_build.CSRC, pkg / "csrc")
    shutil.copytree(fa_build.INCLUDE, tmp_path / "include")
    shutil.copy(fa_build.__file__, pkg / "build.py")
    for name, status in (("nvcc", 0), ("g++", 0), ("bad", 1)):
        f = tmp_path / name
        f.write_text(f"""#!{sys.executable}
import sys
open({str(tmp_path / "calls")!r}, "a").write({name!r} + " " + sys.argv[-1] + "\\n")
open(sys.argv[sys.argv.index("-o") + 1], "w").write("made")
sys.exit({status})
""")
        f.chmod(f.stat().st_mode | stat.S_IXUSR)

    def run(cxx="g++", before="", **kw):
        (tmp_path / "calls").write_text("")
        env = dict(os.environ, NVCC=str(tmp_path / "nvcc"), CXX=str(tmp_path / cxx))
        r = subprocess.run([sys.executable, "-c", f"import sys; sys.path.insert(0, {str(pkg)!r}); {before}\nimport build; build.build(**{kw})"],
                           capture_output=True, text=True, env=env)
        calls = [c.split()[0] for c in (tmp_path / "calls").read_text().splitlines()]
        return r, calls.count("nvcc"), len(calls) - calls.count("nvcc")

    run.pkg = pkg
    return run


@pytest.mark.parametrize("cxx,before", [("bad", ""), ("g++", "sys.modules['torch'] = None")])
def test_library_is_built_without_the_binding(tree, cxx, before):
    """No C++ compiler that can build the binding, or no torch: libfa.so is there all the same, and the error says
    that the binding is not."""
    r, _, _ = tree(cxx, before)
    assert r.returncode != 0 and "libfa.so is built, _fa_binding.so is not" in r.stderr
    assert (tree.pkg / "libfa.so").exists() and not (tree.pkg / "_fa_binding.so").exists()
    r, cuda, host = tree()  # what is there stays; the binding follows
    assert r.returncode == 0 and cuda == 0 and host == 2 and (tree.pkg / "_fa_binding.so").exists()


def test_only_what_changed_is_built(tree):
    n = len(fa_build.sources())
    assert tree()[1:] == (n + 1, 2)
    assert tree()[1:] == (0, 0)
    os.utime(tree.pkg / "csrc" / "fa_binding.cpp")
    assert tree()[1:] == (0, 2)
    os.utime(tree.pkg / "csrc" / "fa_cache.cu")
    assert tree()[1:] == (n + 1, 0)
    os.utime(tree.pkg.parent / "include" / "fa.h")
    assert tree()[1:] == (n + 1, 2)
    assert tree(force=True)[1:] == (n + 1, 2)


def test_binding_is_built_again_for_another_torch_or_python(tree):
    """The binding alone: the library does not depend on them."""
    n = len(fa_build.sources())
    assert tree()[1:] == (n + 1, 2)
    other = "import torch; torch.__version__ += '.other'"
    assert tree(before=other)[1:] == (0, 2)
    assert tree(before=other)[1:] == (0, 0)
    assert tree()[1:] == (0, 2)
    assert tree(before="sys.version = 'another'")[1:] == (0, 2)
