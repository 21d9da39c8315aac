import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")


# Tests whose expected values are wrong, kept as they are; each names the test that
# holds the right ones.
WRONG_VALUES = {
    "tests/test_gpu_decode.py::test_verify_bad_nodes":
        "its reference takes the draft distribution away for a token outside the vocabulary, of "
        "which nothing was drawn: the next token of (0.5, 0.5) under (0.9, 0.1) would always be the "
        "second; tests/test_gpu_verify_definition.py::test_nodes_that_are_not_there has the same inputs",
}


def pytest_collection_modifyitems(items):
    for item in items:
        if item.nodeid in WRONG_VALUES:
            item.add_marker(pytest.mark.xfail(reason=WRONG_VALUES[item.nodeid], strict=True))
