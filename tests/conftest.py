import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built libfp4q.so")
    config.addinivalue_line("markers", "slow: full-size parity case (minutes of CPU oracle time)")


def pytest_collection_modifyitems(items):
    from tests.made_up_addresses import skip_where_a_gpu_is

    skip_where_a_gpu_is(items)
