"""The example's layer when its cache is full: the step is refused as a whole, and what came before goes on."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def layer_and_step(rows, pages):
    import torch
    from attention_steps import PagedLayer
    layer = PagedLayer(256, 2, 64, rows, pages=pages, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    return layer, lambda new: layer.step(torch.randn(sum(new), 256, generator=g, device="cuda").half(), new)


def same_books(layer):
    assert layer.kv_lens.tolist() == layer.lengths
    refs = [n for n in layer.page_refs.tolist() if n]
    assert sorted(refs) == sorted(layer.holders.values())


def test_a_step_that_does_not_fit_raises():
    layer, step = layer_and_step(3, 6)
    step([40, 16, 17])                                     # 3 + 1 + 2 pages of 16
    same_books(layer)
    before = [t.clone() for t in layer.books()]
    for new in ([0, 1, 0], [9, 0, 0], [1, 1, 1]):
        with pytest.raises(RuntimeError, match="full"):
            step(new)
        assert all((a == b).all() for a, b in zip(before, layer.books()))
        same_books(layer)
    step([8, 0, 15])                                       # what the last pages still take
    same_books(layer)
    layer.truncate([16, 16, 16])
    step([1, 16, 1])
    same_books(layer)


def test_shared_last_pages_need_room():
    layer, step = layer_and_step(3, 4)
    step([20, 0, 0])
    layer.fork([0, 0, 0])
    with pytest.raises(RuntimeError, match="full"):
        step([1, 1, 1])                                    # three copies of the shared page, two free
    same_books(layer)
    step([1, 1, 0])
    same_books(layer)
    assert int((layer.page_refs > 0).sum()) == 4
    step([1, 1, 1])                                        # the last holder keeps it
    same_books(layer)
    layer.compact()
    layer.truncate([0, 3, 30])
    step([4, 0, 2])
    same_books(layer)
