"""Which tests run where: those whose addresses are not memory never on a machine
with a GPU, the `gpu` ones never without."""
import pathlib
import types

import pytest
import torch

from tests import conftest


@pytest.mark.parametrize("gpu", [False, True])
def test_collection(monkeypatch, gpu):
    monkeypatch.setattr(torch.cuda, "is_available", lambda: gpu)
    items = []
    for name, keys in (("test_packed_host.py", ()), ("test_rope_in_place_host.py", ()),
                       ("test_binding_host.py", ()), ("test_rope_gpu.py", ("gpu",))):
        marks = []
        items.append(types.SimpleNamespace(path=pathlib.Path("/x") / name, keywords=set(keys),
                                           marks=marks, add_marker=marks.append))
    conftest.pytest_collection_modifyitems(None, items)
    skipped = [bool(i.marks) for i in items]
    assert skipped == ([True, True, False, False] if gpu else [False, False, False, True])
