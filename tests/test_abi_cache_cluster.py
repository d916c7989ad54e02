"""Refusals of the test entry that limits the clusters of the cache's upkeep (no GPU)."""
import pytest

from qkv_projection_gb300 import kaio
from test_abi_attention import passes_validation, refused
from test_abi_cache import book_args


@pytest.mark.parametrize("op", [0, 1, 2])
def test_limit_entry_checks_as_the_entries_do(op):
    fn = lambda args, stream: kaio.lib().kaio_debug_cache_cluster_limit(op, args, 4, stream)   # noqa: E731
    refused(fn, None, "null pointer")
    refused(fn, book_args(size=4), "struct_size")
    refused(fn, book_args(kv_lens=0), "kv_lens is a null")
    passes_validation(fn, book_args())


def test_ops_and_limits():
    for op, most, text in ((-1, 4, "op"), (3, 4, "op"), (0, 0, "most"), (2, -1, "most")):
        refused(lambda args, stream: kaio.lib().kaio_debug_cache_cluster_limit(op, args, most, stream), book_args(), text)
