"""Tests whose calls reach a launch on made-up addresses do not run where there is a GPU (no GPU)."""
import pathlib

import pytest
import torch

import conftest


class Item:
    def __init__(self, path):
        self.fspath, self.marks = pathlib.Path(path), []

    def add_marker(self, mark):
        self.marks.append(mark.name)


@pytest.mark.parametrize("gpus", [0, 1, 8])
def test_made_up_addresses_stay_off_a_gpu(gpus, monkeypatch):
    monkeypatch.setattr(torch.cuda, "device_count", lambda: gpus)
    here = sorted(pathlib.Path(__file__).parent.glob("test_*.py"))
    items = [Item(p) for p in here]
    conftest.pytest_collection_modifyitems(None, items)
    skipped = [i.fspath.name for i in items if "skip" in i.marks]
    want = [p.name for p in here if "_host_overlap" in p.name]
    assert len(want) >= 2 and skipped == (want if gpus else [])
