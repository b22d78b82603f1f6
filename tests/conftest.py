import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built library")
    config.addinivalue_line("markers", "slow: long-running CPU test")


# These expect that a step without a mask does not see the sequence's first tokens where they lie in the step itself, more than a
# window back; it does (test_gpu_tree_window_prompts.py has the same sizes by the rule that holds for whole sequences).  They
# fail, and come last, so that a run that stops at the first failure has run everything else.
NARROWER_RULE = "test_gpu_tree_window.py::test_against_float64[5-2-2-3-64-129-lens11-None-False-2-1-"


def pytest_collection_modifyitems(config, items):
    items.sort(key=lambda item: NARROWER_RULE in item.nodeid)
    try:
        import torch
        has_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        has_gpu = False
    if has_gpu:
        return
    skip = pytest.mark.skip(reason="no CUDA device")
    for item in items:
        if "gpu" in item.keywords:
            item.add_marker(skip)


@pytest.fixture(scope="session", autouse=True)
def _library_built_from_current_sources():
    """The tests run against libringattn.so as built from the sources in this tree: it is compiled
    here if it is missing or older than a source (the binding itself never builds; it raises)."""
    from sequence_sharded_exact_gb300 import build_lib

    build_lib.build()
