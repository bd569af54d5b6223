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
