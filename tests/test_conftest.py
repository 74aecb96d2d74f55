"""Tests that pass made-up addresses to the library never run where a device
would act on them."""
import os
import re
import types

import conftest


class Item:
    def __init__(self, name):
        self.module = types.SimpleNamespace(__name__=name)
        self.marks = []

    def add_marker(self, mark):
        self.marks.append(mark.name)


def test_they_are_skipped_where_there_is_a_device():
    for have in (False, True):
        items = [Item("test_abi"), Item("test_adapter_host"), Item("test_gpu_layer"), Item("test_rings")]
        conftest.skip_made_up_addresses(items, have)
        assert [i.marks for i in items] == ([["skip"], ["skip"], [], []] if have else [[], [], [], []])


def test_no_module_is_missing_from_the_list():
    """(Modules for a GPU pass made-up addresses only where a host check refuses.)"""
    here = os.path.dirname(os.path.abspath(__file__))
    made_up = set()
    for f in os.listdir(here):
        text = open(os.path.join(here, f)).read() if f.startswith("test_") and f.endswith(".py") else ""
        if "pytestmark = pytest.mark.gpu" not in text and f != os.path.basename(__file__) and re.search(
                r"(c_void_p|\bP)\(\(?1 << \d\d\)|base, n = 1 << \d\d", text):
            made_up.add(f[:-3])
    assert made_up == set(conftest.MADE_UP_ADDRESSES)
