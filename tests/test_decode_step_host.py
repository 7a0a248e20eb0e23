"""Host side of a decode step (no GPU needed): steps without work, tables and the host's page table, what the example needs."""
import types

import torch

from resident_expert_routed_gb300.decode import DecodeLayer, LanePages, Step


def layer(d=32, heads=4, kv_heads=2, D=64, lanes=3):
    """A layer on the host; nothing in it can be launched."""
    w = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16)  # noqa: E731
    cache = types.SimpleNamespace(n_kv_heads=kv_heads, head_dim=D)
    return DecodeLayer(w((heads + 2 * kv_heads) * D, d), w(d, heads * D), cache, heads, lanes, 8, (None,) * 7, None)


def test_a_step_in_which_every_lane_waits():
    pages = LanePages(3, 8, 16, 4)
    tables = Step(pages, [[], [], []], device="cpu")
    assert tables.n_nodes == 0 and tables.slots.shape == (0,) and tables.mask.shape == (0, 1)
    hidden = torch.zeros((0, 32), dtype=torch.bfloat16)
    out = layer().step(hidden, tables)
    assert out.shape == (0, 32) and out.dtype == torch.bfloat16


def test_a_step_keeps_its_page_table():
    """What the host does with its table afterwards (a lane that ends, pages handed to another) is not the step's."""
    pages = LanePages(2, 8, 16, 4)
    tables = Step(pages, [[-1, 0, 0], [-1]], device="cpu")
    was = tables.table.clone()
    assert was[0, 0] >= 0 and was[1, 0] >= 0
    pages.release(0)
    pages.reserve(1, 60)
    assert torch.equal(tables.table, was)


def test_the_example_does_without_the_test_tree(monkeypatch):
    import importlib
    import sys
    for name in [m for m in sys.modules if m == "tests" or m.startswith("tests.") or m == "examples.tree_decode"]:
        monkeypatch.delitem(sys.modules, name)
    monkeypatch.setitem(sys.modules, "tests", None)                      # any import of it fails
    assert importlib.import_module("examples.tree_decode").HEADS == 8
    monkeypatch.delitem(sys.modules, "examples.tree_decode")
