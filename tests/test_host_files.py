"""The files whose calls carry made-up addresses run only where no GPU is visible.  In a process
that sees one their tests are skipped with a reason, and run here, in a process of their own that does
not."""
import os
import subprocess
import sys
from types import SimpleNamespace

import pytest

import conftest

HERE = os.path.dirname(os.path.abspath(__file__))


class Item:
    """What the collection hook looks at in a test."""

    def __init__(self, path, gpu=False):
        self.fspath, self.gpu, self.markers = path, gpu, []

    def get_closest_marker(self, name):
        return name == "gpu" and self.gpu

    def add_marker(self, mark):
        self.markers.append(mark)


def test_no_test_is_dropped_beside_a_gpu(monkeypatch):
    config = SimpleNamespace(hook=SimpleNamespace(pytest_deselected=lambda items: None))
    for sees in (True, False):
        monkeypatch.setattr(conftest, "_sees_a_gpu", lambda: sees)
        items = [Item(os.path.join(HERE, name)) for name in (*conftest.NO_GPU_FILES, "test_inputs.py")]
        kept = list(items)
        conftest.pytest_collection_modifyitems(config, kept)
        assert kept == items
        for i in items:
            skipped = [m for m in i.markers if m.name == "skip"]
            assert len(skipped) == (sees and os.path.basename(i.fspath) in conftest.NO_GPU_FILES)
            assert all("test_host_files.py" in m.kwargs["reason"] for m in skipped)


@pytest.mark.skipif(not conftest._sees_a_gpu(), reason="no GPU is visible: the files run in this process")
@pytest.mark.parametrize("name", conftest.NO_GPU_FILES)
def test_file_in_a_process_that_sees_no_gpu(name):
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "not gpu", os.path.join(HERE, name)],
                       cwd=os.path.dirname(HERE), env={**os.environ, "CUDA_VISIBLE_DEVICES": ""}, capture_output=True,
                       text=True, timeout=900)
    assert r.returncode == 0 and " passed" in r.stdout, r.stdout[-3000:]
