"""Tests that hand made-up addresses to an entry point past its argument checks are skipped where a GPU is
visible: nothing may launch a kernel on them."""
import ast
import os
import pathlib

import torch

from tests import conftest

HERE = pathlib.Path(__file__).parent


class _Item:
    def __init__(self, path, name):
        self.path, self.name, self.marks = path, name, []

    def add_marker(self, mark):
        self.marks.append(mark.name)


def _past_the_checks():
    """(file, test) of every test that accepts an answer from beyond an entry point's checks."""
    for path in sorted(HERE.glob("test_*.py")):
        if path.name == os.path.basename(__file__):
            continue
        for node in ast.parse(path.read_text()).body:
            if isinstance(node, ast.FunctionDef) and node.name.startswith("test_"):
                called = {n.func.id for n in ast.walk(node) if isinstance(n, ast.Call) and isinstance(n.func, ast.Name)}
                if called & {"passed", "_passed"}:
                    yield path, node.name


def test_skipped_where_a_gpu_is_visible(monkeypatch):
    found = list(_past_the_checks())
    assert {n for _, n in found} >= {"test_gemm_size_limits_at_2_31", "test_entries_reject_launches_of_2_32_lanes"}
    other = _Item(HERE / "test_abi.py", "test_status_strings")
    for devices, want in ((0, []), (1, ["skip"])):
        monkeypatch.setattr(torch.cuda, "device_count", lambda: devices)
        items = [_Item(*f) for f in found] + [other]
        conftest.pytest_collection_modifyitems(items)
        for item in items[:-1]:
            assert item.marks == want, (devices, item.name)
        assert other.marks == []


def test_listed_tests_exist():
    for name, tests in conftest.WITHOUT_DEVICE.items():
        have = {n.name for n in ast.parse((HERE / name).read_text()).body if isinstance(n, ast.FunctionDef)}
        assert tests <= have
