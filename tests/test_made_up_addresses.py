"""Where there is a GPU, no test launches on made-up addresses."""
import ast
import os

import torch

from tests import made_up_addresses, test_abi, test_row_ops

HERE = os.path.dirname(os.path.abspath(__file__))


class Item:
    def __init__(self, function):
        self.function, self.marks = function, []

    def add_marker(self, mark):
        self.marks.append(mark.name)


def names(module):
    return [n for n in dir(module) if n.startswith("test_")]


def test_tests_that_count_on_a_failing_launch_are_skipped(monkeypatch):
    """Every test that takes "accepted, but the launch failed" for an answer
    (ELAUNCH, or RAN which holds it) in the modules' sources."""
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 1)
    count = 0
    for module in (test_abi, test_row_ops):
        items = {n: Item(getattr(module, n)) for n in names(module)}
        made_up_addresses.skip_where_a_gpu_is(items.values())
        with open(module.__file__) as f:
            tree = ast.parse(f.read())
        for node in tree.body:
            if isinstance(node, ast.FunctionDef) and node.name in items:
                used = {getattr(n, "id", getattr(n, "attr", None)) for n in ast.walk(node)}
                if used & {"RAN", "ELAUNCH"}:
                    assert items[node.name].marks == ["skip"], node.name
                    count += 1
    assert count >= 11
    assert Item(test_row_ops.test_rotary_frequencies).marks == []


def test_others_run_where_a_gpu_is():
    assert not made_up_addresses.used_by(test_row_ops.test_rotary_frequencies)
    assert not made_up_addresses.used_by(test_row_ops.test_binding_refusals)
    assert not made_up_addresses.used_by(test_row_ops.test_reference_draws_the_oracles_philox)


def test_nothing_is_skipped_without_a_gpu(monkeypatch):
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 0)
    item = Item(test_row_ops.test_norm_refusals)
    made_up_addresses.skip_where_a_gpu_is([item])
    assert item.marks == []


def test_no_other_module_counts_on_a_failing_launch():
    found = set()
    for name in os.listdir(HERE):
        if name.startswith("test_") and name.endswith(".py") and name != os.path.basename(__file__):
            with open(os.path.join(HERE, name)) as f:
                if "ELAUNCH" in f.read():
                    found.add(name)
    assert found == {"test_abi.py", "test_row_ops.py"}


def test_collection_skips_them(monkeypatch):
    import tests.conftest as conftest

    monkeypatch.setattr(torch.cuda, "device_count", lambda: 1)
    item = Item(test_row_ops.test_norm_refusals)
    conftest.pytest_collection_modifyitems([item])
    assert item.marks == ["skip"]
