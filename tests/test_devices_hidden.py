"""Tests without the gpu mark see no device, whatever is selected beside them: a session over a few tests of its own, with a
stand-in for torch that counts one device unless they are hidden."""

import os
import shutil
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
TORCH = """
import os
class cuda:
    device_count = staticmethod(lambda: 0 if os.environ.get("CUDA_VISIBLE_DEVICES") == "" else 1)
"""
TESTS = """
import os
import pytest
import torch

def test_hidden(): assert torch.cuda.device_count() == 0 and os.environ["CUDA_VISIBLE_DEVICES"] == ""

@pytest.mark.parametrize("n", [1, 2])
def test_fails_by_itself(n): assert torch.cuda.device_count() + n == 1, "a message of its own"

def test_skips(): pytest.skip("for a reason")

@pytest.mark.gpu
def test_marked(): assert torch.cuda.device_count() == 1
"""


@pytest.mark.parametrize("select, outcomes", [
    ([], {"test_hidden": "PASSED", "test_fails_by_itself[1]": "PASSED", "test_fails_by_itself[2]": "FAILED",
          "test_skips": "SKIPPED", "test_marked": "PASSED"}),
    (["-m", "not gpu"], {"test_hidden": "PASSED", "test_fails_by_itself[1]": "PASSED", "test_fails_by_itself[2]": "FAILED",
                         "test_skips": "SKIPPED"}),
    (["-m", "gpu"], {"test_marked": "PASSED"}),
    (["-k", "hidden or marked"], {"test_hidden": "PASSED", "test_marked": "PASSED"}),
])
def test_tests_without_the_mark_see_no_device(tmp_path, select, outcomes):
    (tmp_path / "tests").mkdir()
    (tmp_path / "torch.py").write_text(TORCH)
    (tmp_path / "tests" / "test_some.py").write_text(TESTS)
    shutil.copy(os.path.join(HERE, "conftest.py"), tmp_path / "tests")
    env = {k: v for k, v in os.environ.items() if k not in ("CUDA_VISIBLE_DEVICES", "CLI_TEST_OUTCOMES")}
    env.update(PYTHONPATH=str(tmp_path), PYTEST_DISABLE_PLUGIN_AUTOLOAD="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-v", "-rs", "--rootdir", str(tmp_path), "tests", *select], cwd=tmp_path,
                       env=env, capture_output=True, text=True)
    got = {line.split("::")[1].split()[0]: line.split()[1] for line in r.stdout.splitlines()
           if line.startswith("tests/test_some.py::") and len(line.split()) > 1}
    assert got == outcomes, r.stdout + r.stderr
    assert ("a message of its own" in r.stdout) == ("FAILED" in outcomes.values())
    assert ("for a reason" in r.stdout) == ("SKIPPED" in outcomes.values())
    assert r.returncode == ("FAILED" in outcomes.values())


def test_nor_does_this_one():
    import torch
    assert torch.cuda.device_count() == 0 and not torch.cuda.is_available()
