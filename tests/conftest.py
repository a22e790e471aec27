import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")
    config.addinivalue_line("markers", "slow: long-running CPU test")


# Cases that hold a momentum in 8 bits to rounding to nearest at a beta1 where that is wrong: they run, and fail on their
# codes.  test_gpu_momentum_8bit.py holds such sets to the definition.
NEAREST_PAST_ITS_LIMIT = {
    "test_random_sets[18]": "a group has beta1 = 0.98629: 1.125 beta1 = 1.1096 is nearer to 1.125 than to 1",
    "test_random_sets[21]": "a group has beta1 = 0.94451: 1.125 beta1 = 1.06257 is nearer to 1.125 than to 1",
}


def pytest_collection_modifyitems(items):
    for item in items:
        if item.path.name == "test_gpu_tensor_set.py" and item.name in NEAREST_PAST_ITS_LIMIT:
            item.add_marker(pytest.mark.xfail(raises=AssertionError, strict=True,
                                              reason="m never decays there: " + NEAREST_PAST_ITS_LIMIT[item.name]))


@pytest.fixture(scope="session")
def oracle_lib():
    import oracle
    oracle.build(force=False)
    return oracle
