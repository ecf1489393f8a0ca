import json
import os
import subprocess
import sys
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

REPORT = "CLI_TEST_OUTCOMES"   # where a session without devices writes its tests' outcomes, one a line


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (runs the CUDA path through the C ABI)")
    config.addinivalue_line("markers", "slow: larger CPU cases")


# Tests without the gpu mark see no device.  Several of them give the library invented addresses, and some of those calls
# are valid but for that: where there is a device they would launch kernels on unmapped memory.  So where one is visible,
# those tests run in a session of their own that sees none (a process that has started CUDA keeps its devices), and here
# have the outcome that they had there.

class _Apart:
    def __init__(self, session):
        self.ids = [i.nodeid for i in session.items if i.get_closest_marker("gpu") is None]
        self.root, self.outcomes = str(session.config.rootpath), None

    def outcome(self, node):
        if self.outcomes is None:
            with tempfile.TemporaryDirectory() as folder:
                report = os.path.join(folder, "outcomes")
                r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", *self.ids], cwd=self.root,
                                   env={**os.environ, "CUDA_VISIBLE_DEVICES": "", REPORT: report}, capture_output=True, text=True)
                lines = open(report).read().splitlines() if os.path.exists(report) else []
            self.outcomes = {k: v for k, *v in map(json.loads, lines)}
            self.output = (r.stdout + r.stderr)[-4000:]
        return self.outcomes.get(node, ("failed", "no outcome in the session without devices:\n" + self.output))


def pytest_collection_finish(session):
    session.config.apart = None
    if session.config.option.collectonly or all(i.get_closest_marker("gpu") for i in session.items):
        return
    import torch
    if torch.cuda.device_count():
        session.config.apart = _Apart(session)


@pytest.hookimpl(tryfirst=True)
def pytest_pyfunc_call(pyfuncitem):
    if pyfuncitem.config.apart is None or pyfuncitem.get_closest_marker("gpu") is not None:
        return None
    outcome, text = pyfuncitem.config.apart.outcome(pyfuncitem.nodeid)
    if outcome == "failed":
        pytest.fail(text, pytrace=False)
    if outcome == "skipped":
        pytest.skip(text)
    return True


def pytest_runtest_logreport(report):
    path = os.environ.get(REPORT)
    if path and (report.when == "call" or report.outcome != "passed"):
        text = report.longrepr[2] if isinstance(report.longrepr, tuple) else report.longreprtext
        with open(path, "a") as f:
            f.write(json.dumps([report.nodeid, report.outcome, text]) + "\n")
