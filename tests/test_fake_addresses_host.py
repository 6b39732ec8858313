"""Tests that hand the library addresses that are none stay off machines with a GPU, every one of them."""
import pathlib
import re

import pytest

from . import conftest

HERE = pathlib.Path(__file__).parent
ADDRESSES = re.compile(r"fake (device )?address|from (tests)?\.(test_step_host|test_packed_host|test_boundary) import")


class Item:
    def __init__(self, name, *marks):
        self.path, self.marks, self.added = HERE / name, marks, []

    def get_closest_marker(self, name):
        return name if name in self.marks else None

    def add_marker(self, mark):
        self.added.append(mark)


def test_every_module_with_fake_addresses_is_known():
    found = {p.name for p in HERE.glob("test_*.py") if ADDRESSES.search(p.read_text()) and not re.search(r"^pytestmark = pytest.mark.gpu", p.read_text(), re.M)}
    assert found - {"test_fake_addresses_host.py"} == conftest.FAKE_ADDRESSES


@pytest.mark.parametrize("name", sorted(conftest.FAKE_ADDRESSES))
def test_they_are_skipped_where_there_is_a_gpu(name):
    items = [Item(name), Item(name, "gpu"), Item("test_plan_bounds.py")]
    conftest.keep_off_gpus(items, False)
    assert not any(i.added for i in items)
    conftest.keep_off_gpus(items, True)
    assert [len(i.added) for i in items] == [1, 0, 0] and items[0].added[0].name == "skip"
