"""When the build makes its products again (no GPU, no real compiler)."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = """#!/bin/sh
# writes the file after -o; counts in `log`; fails where another compiler writes the same file at that time
while [ $# -gt 0 ]; do if [ "$1" = -o ]; then out=$2; fi; shift; done
mkdir "$out.busy" || { echo "two compilers at $out"; exit 7; }
sleep 0.3
echo "$out" >> "%(log)s"
echo made > "$out"
rmdir "$out.busy"
"""


@pytest.fixture
def tree(tmp_path):
    """A copy of the package whose compilers are scripts; (its root, its log, run)."""
    at = tmp_path / "tree"
    shutil.copytree(os.path.join(ROOT, "q4_weight_matmul_gb300"), at / "q4_weight_matmul_gb300",
                    ignore=shutil.ignore_patterns("_build", "__pycache__", "*.so"))
    shutil.copytree(os.path.join(ROOT, "include"), at / "include")
    log, cc = tmp_path / "log", tmp_path / "bin" / "cc"
    cc.parent.mkdir()
    cc.write_text(FAKE % {"log": log})
    cc.chmod(0o755)
    log.touch()

    def start(code="from q4_weight_matmul_gb300.build import build; build()"):
        return subprocess.Popen([sys.executable, "-c", code], cwd=at, stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                                text=True, env={**os.environ, "NVCC": str(cc), "CXX": str(cc), "PYTHONPATH": str(at)})

    def run(*a):
        p = start(*a)
        out = p.communicate(timeout=300)[0]
        assert p.returncode == 0, out
        made, _ = log.read_text().split(), log.write_text("")
        return [os.path.basename(m).split(".so")[0] for m in made]

    return at, log, start, run


def test_another_torch_or_python_makes_the_binding_again(tree):
    _, _, _, run = tree
    assert "_calls" in run() and run() == []
    other = "import torch; torch.__version__ = '99.0'; from q4_weight_matmul_gb300.build import build; build()"
    assert run(other) == ["_calls"] and run(other) == []
    assert run() == ["_calls"] and run() == []


def test_a_binding_that_cannot_be_imported_says_why(tree):
    at, _, _, run = tree
    run()                                                        # a file that is no library
    code = ("import q4_weight_matmul_gb300 as q\nq.lib = lambda: None\ntry:\n    q._native()\nexcept RuntimeError as e:\n"
            "    assert '_calls.so' in str(e) and str(e.__cause__) in str(e), e\nelse:\n    raise SystemExit(1)")
    assert run(code) == []


def test_builds_at_the_same_time_do_not_write_the_same_files(tree):
    at, log, start, run = tree
    builds = [start() for _ in range(3)]
    for p in builds:
        out = p.communicate(timeout=300)[0]
        assert p.returncode == 0, out
    made = [line for line in log.read_text().split()]
    assert len(made) == len(set(made)) and not list((at / "q4_weight_matmul_gb300").rglob("*.busy"))
    log.write_text("")
    assert run() == []
