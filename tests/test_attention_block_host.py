"""The attention block's host side: the bookkeeping of pages and workspaces (no GPU)."""
import copy

import pytest
import torch

from q4_weight_matmul_gb300.attention_block import Pages, Workspaces


def state(p):
    return copy.deepcopy((p.free, p.of, p.length))


def lists(step):
    return {k: v.tolist() for k, v in step.items()}


@pytest.mark.parametrize("new", [{0: 5, 1: 30, 2: 1}, {0: 5, 1: 4, 2: 60}, {2: 1, 1: 4, 0: 17}])
def test_a_refused_step_changes_nothing(new):
    """Six pages of 4 cells, four for a request at most: too many pages in all, or for one request, after earlier requests
    of the batch would have had theirs."""
    pages = Pages(6, 4, 4)
    pages.step({0: 3, 1: 9})
    before = state(pages)
    with pytest.raises(RuntimeError):
        pages.step(new)
    assert state(pages) == before
    step = lists(pages.step({0: 5, 2: 1}))                     # and the next step goes on from there
    assert step["pos"] == [3, 4, 5, 6, 7, 0] and step["kv_len"] == [8, 1]
    assert len({s // 4 for s in step["slot"]} | set(pages.of[1])) == 6


def test_released_pages_are_used_again():
    pages = Pages(5, 4, 4)
    for i in range(40):
        step = lists(pages.step({i: 13, "kept": 0 if i else 3}))
        assert step["kv_len"] == [13, 3] and all(0 <= p < 5 for p in step["table"][0])
        assert set(step["table"][0]) & set(pages.of["kept"]) == set()
        with pytest.raises(RuntimeError):
            pages.step({"other": 1})
        pages.release(i)
    assert pages.length == {"kept": 3} and sorted(pages.free + pages.of["kept"]) == list(range(5))
    with pytest.raises(KeyError):
        pages.release(0)


def test_workspaces_grow_and_stay_for_graphs():
    made = lambda n: lambda: torch.zeros(n, dtype=torch.uint8)  # noqa: E731
    w = Workspaces()
    with pytest.raises(RuntimeError):                                   # a capture makes none
        w.get("attn", 10, made(10), for_graph=True)
    small = w.get("attn", 10, made(10))
    assert w.get("attn", 7, made(7)) is small and w.get("attn", 10, made(10), for_graph=True) is small
    large = w.get("attn", 100, made(100))
    assert large.numel() == 100 and w.get("attn", 10, made(10)) is large
    assert any(t is small for t in w.in_graphs)                         # what the graph writes to is still there
    for n in range(50):
        assert w.get("attn", 50 + n, made(50 + n), for_graph=True) is large
    assert len(w.held) == 1 and len(w.in_graphs) == 2
