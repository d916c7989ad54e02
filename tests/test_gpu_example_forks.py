"""The example's layer where a fork names parents that are no rows: those rows stay."""
import pytest

from test_gpu_example_full import layer_and_step, same_books

pytestmark = pytest.mark.gpu


def test_parents_that_are_no_rows():
    layer, step = layer_and_step(4, 20)
    step([20, 3, 0, 40])
    layer.fork([-1, 0, 4, 1 << 30])
    assert layer.lengths == [20, 20, 0, 40]
    same_books(layer)
    step([1, 1, 5, 0])
    same_books(layer)
