"""The build of the library and of the Python module beside it, with stand-ins for the compilers (they write what
-o names and log their command), on a copy of the package."""
import os
import shutil
import stat
import subprocess
import sys
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = "bit_qk_attention_b200"


@pytest.fixture
def tree(tmp_path):
    """A copy of the sources whose compilers are stand-ins; run(code) runs Python on it and returns the commands."""
    shutil.copytree(os.path.join(ROOT, PKG), tmp_path / PKG,
                    ignore=shutil.ignore_patterns("_build", "*.so", "__pycache__"))
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    tool, log = tmp_path / "tool", tmp_path / "log"
    tool.write_text(textwrap.dedent(f"""\
        #!{sys.executable}
        import sys
        a = sys.argv
        open(a[a.index("-o") + 1], "w").write("built")
        open({str(log)!r}, "a").write(" ".join(a[1:]) + "\\n")
        """))
    tool.chmod(tool.stat().st_mode | stat.S_IXUSR)

    def run(code, fails=False):
        log.write_text("")
        env = dict(os.environ, NVCC=str(tool), CXX=str(tool), PYTHONPATH=str(tmp_path), PYTHONDONTWRITEBYTECODE="1")
        r = subprocess.run([sys.executable, "-c", textwrap.dedent(code)], cwd=tmp_path, env=env, capture_output=True, text=True)
        assert (r.returncode != 0) == fails, r.stdout + r.stderr
        return log.read_text().splitlines()

    run.path = tmp_path / PKG
    return run


NO_TORCH = "import sys; sys.modules['torch'] = None\n"
BUILD = "import runpy; runpy.run_module('bit_qk_attention_b200.build', run_name='__main__')\n"


def test_the_library_is_built_without_torch(tree):
    done = tree(NO_TORCH + BUILD)
    assert (tree.path / "libbinattn.so").exists()
    assert any("-shared" in c and ".cu.o" in c for c in done) and not any(".cpp" in c for c in done)
    assert not [f for f in os.listdir(tree.path) if f.startswith("_paged")]


def test_with_torch_both_are_built_once(tree):
    done = tree(BUILD)
    assert sum(".cpp" in c for c in done) == 1 and any(".cu.o" in c for c in done)
    assert [f for f in os.listdir(tree.path) if f.startswith("_paged")]
    assert tree(BUILD) == []


OTHER_TORCH = """
import importlib.metadata
real = importlib.metadata.version
importlib.metadata.version = lambda name: "9.9.9" if name == "torch" else real(name)
"""


def test_the_module_is_built_again_for_another_torch(tree):
    tree(BUILD)
    done = tree(OTHER_TORCH + BUILD)
    assert len(done) == 1 and ".cpp" in done[0] and 'BA_BUILT_FOR="torch ' in done[0]
    assert tree(OTHER_TORCH + BUILD) == []
    assert len(tree(BUILD)) == 1


def test_the_module_is_named_for_its_python(tree):
    import sysconfig
    tree(BUILD)
    assert [f for f in os.listdir(tree.path) if f.startswith("_paged")] == ["_paged" + sysconfig.get_config_var("EXT_SUFFIX")]


@pytest.mark.parametrize("module", ["built_for = 'torch 1.2.3'", "", None])
def test_a_module_of_another_torch_is_not_called(tree, module):
    """A module for another torch, one from before it said so, and none at all: the message says what to do."""
    if module is not None:
        (tree.path / "_paged.py").write_text(module + "\ndef bind(*a):\n    raise SystemExit('called')\n")
    tree("""
        import bit_qk_attention_b200 as ba
        ba.lib = lambda: None
        try:
            ba._native()
        except RuntimeError as e:
            assert "build it with" in str(e), e
        else:
            raise SystemExit("not refused")
        """)
