import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
TESTS = os.path.dirname(os.path.abspath(__file__))
if TESTS not in sys.path:
    sys.path.insert(0, TESTS)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built library")
    config.addinivalue_line("markers", "slow: full-size workload, minutes of host work")


# Tests whose expected loss counts each entry of a repeated id for itself (distill_util.distill64), which
# is below the divergence by the entropy of the split and may be negative.  test_distill_repeats_gpu.py
# holds the same calls to the loss of the added-up probabilities.
ENTRIES_APART = ("test_an_id_that_comes_more_than_once[", "test_ids_drawn_with_repetition[",
                 "test_calls_back_to_back[3-131072-64]", "test_calls_back_to_back[700-65536-600]")


def pytest_collection_modifyitems(items):
    for item in items:
        if item.path.name == "test_distill_gpu.py" and item.name.startswith(ENTRIES_APART):
            # the last two draw their ids on the device, with repeats among them
            item.add_marker(pytest.mark.xfail(strict="back_to_back" not in item.name, raises=AssertionError,
                                              reason="its expected loss counts entries of one id apart"))


@pytest.fixture(autouse=True)
def _device_index_checks(request):
    """Under the MHC_CHECK build (MHC_GB300_CHECK=1), every GPU test also
    asserts that no device index check failed while it ran."""
    yield
    if request.node.get_closest_marker("gpu") is None:
        return
    if os.environ.get("MHC_GB300_CHECK", "0") in ("", "0"):
        return
    import gemm_rms_sinkhorn_gb300 as mhc

    site, off, extent = mhc.mhc_testing_check_record()
    assert site == 0, "device index check %d failed: offset %d of %d" % (site, off, extent)
