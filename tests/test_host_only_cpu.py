"""Tests of made-up addresses never run where a GPU could follow them."""
from __future__ import annotations

from pathlib import Path

import pytest
import torch

import conftest

FILES = sorted(Path(__file__).parent.glob("test_*.py"))


class Item:
    def __init__(self, path):
        self.path, self.markers = path, []

    def add_marker(self, marker):
        self.markers.append(marker.name)


@pytest.mark.parametrize("gpu", [False, True])
def test_made_up_addresses_stay_off_a_gpu(monkeypatch, gpu):
    monkeypatch.setattr(torch.cuda, "is_available", lambda: gpu)
    items = [Item(f) for f in FILES]
    conftest.pytest_collection_modifyitems(items)
    for item in items:
        assert item.markers == (["skip"] if gpu and item.path.name in conftest.MADE_UP_ADDRESSES else [])


def test_every_file_of_made_up_addresses_is_listed():
    """Any host-only test file that calls a C function of the library with whole numbers for addresses."""
    found = {f.name for f in FILES if "\n# Fake" in f.read_text()}
    assert found == set(conftest.MADE_UP_ADDRESSES)
