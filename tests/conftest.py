"""Shared test setup: markers, import path, and the CPU oracle build."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")


# Tests that give an entry point valid arguments with made-up addresses and expect its answer to be
# that there is no device: with one, it would launch kernels on those addresses.
WITHOUT_DEVICE = {
    "test_abi.py": {"test_gemm_size_limits_at_2_31"},
    "test_moe_args.py": {"test_route_entry_rejects_bad_arguments", "test_route_backward_entry_rejects_bad_arguments",
                         "test_plan_entry_rejects_bad_arguments", "test_dispatch_and_combine_entries_reject_bad_arguments",
                         "test_routed_product_entry_rejects_bad_arguments", "test_entries_reject_launches_of_2_32_lanes"},
}


def pytest_collection_modifyitems(items):
    import torch
    if torch.cuda.device_count() == 0:      # counting does not initialise a device
        return
    skip = pytest.mark.skip(reason="made-up addresses: only where no GPU is visible")
    for item in items:
        if item.name in WITHOUT_DEVICE.get(os.path.basename(str(item.path)), ()):
            item.add_marker(skip)


@pytest.fixture(scope="session", autouse=True)
def _oracle_built():
    import oracle
    if not os.path.exists(oracle.LIB_PATH):
        oracle.build(force=False)
    yield
