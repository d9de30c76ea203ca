import glob
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


# Calls with made-up addresses: the accepted ones would reach a GPU if the process saw one.
NO_GPU_FILES = ("test_abi_host.py", "test_paged_host.py")


def _sees_a_gpu():
    return os.environ.get("CUDA_VISIBLE_DEVICES") != "" and bool(glob.glob("/dev/nvidia[0-9]*"))


def pytest_collection_modifyitems(config, items):
    """Those files run in processes that see no GPU only: beside GPU tests on a machine with one they
    are skipped, and test_host_files.py runs them in such a process (``-m "not gpu"`` hides the GPU and
    runs them directly)."""
    if _sees_a_gpu():
        skip = pytest.mark.skip(reason="made-up addresses: test_host_files.py runs this file in a process that sees no GPU")
        for i in items:
            if os.path.basename(str(i.fspath)) in NO_GPU_FILES and not i.get_closest_marker("gpu"):
                i.add_marker(skip)


def pytest_configure(config):
    if config.option.markexpr.strip() == "not gpu":     # before anything starts CUDA
        os.environ["CUDA_VISIBLE_DEVICES"] = ""
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a); run with -m gpu")
    config.addinivalue_line("markers", "slow: long-running CPU oracle case")


def build_library():
    """Compile libxsattn.so if stale (by path, without importing the package)."""
    import importlib.util
    path = os.path.join(ROOT, "dit_attention_ulysses_gb300", "_build.py")
    spec = importlib.util.spec_from_file_location("xsattn_build", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod.build()
