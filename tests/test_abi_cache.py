"""Refusals of the cache's upkeep and of the scored attention, before anything touches a GPU:
argument blocks with made-up pointers that validation never dereferences."""
import ctypes
import re
import struct

import pytest

from qkv_projection_gb300 import kaio
from test_abi_attention import F32, INVALID, MISALIGNED, paged_args, passes_validation, ptr, refused

COPY = "size caches num_pages page_size kv_heads dim pairs reserved cache strides src dst".split()
BOOKS = ("size batch max_pages num_pages page_size tokens max_moves reserved table_stride page_refs page_table kv_lens "
         "parents q_starts new_lens slots src dst").split()


@pytest.fixture(scope="module")
def L():
    return kaio.lib()


def copy_args(bases=(ptr(0), ptr(1)), steps=((2048, 128, 64),) * 2, **kw):
    a = dict(zip(COPY, [0] * len(COPY)))
    a.update(size=kaio._CACHE_COPY_ARGS.size, caches=2, num_pages=7, page_size=16, kv_heads=2, dim=64, pairs=3,
             src=ptr(2), dst=ptr(3))
    copy_args.keep = ((ctypes.c_void_p * len(bases))(*bases),
                      (ctypes.c_int64 * (3 * len(steps)))(*(x for s in steps for x in s)))
    a["cache"], a["strides"] = (ctypes.addressof(k) for k in copy_args.keep)
    a.update(kw)
    return kaio._CACHE_COPY_ARGS.pack(*a.values())


def book_args(**kw):
    a = dict(zip(BOOKS, [0] * len(BOOKS)))
    a.update(size=kaio._CACHE_ARGS.size, batch=3, max_pages=4, num_pages=7, page_size=16, tokens=5, max_moves=6,
             table_stride=4)
    for i, name in enumerate(BOOKS[9:]):
        a[name] = ptr(i)
    a.update(kw)
    return kaio._CACHE_ARGS.pack(*a.values())


def scored_args(softcap=30.0, reserved2=0, slopes=ptr(10), prefix_lens=ptr(11), doc_starts=ptr(12), **kw):
    kw.setdefault("size", kaio._PAGED_SCORED_ARGS.size)
    return paged_args(**kw) + struct.pack("@fi3P", softcap, reserved2, slopes, prefix_lens, doc_starts)


def test_blocks_have_the_header_s_size_and_order(L):
    text = open(kaio.HEADER).read()
    for name, fields in (("kaio_cache_copy_args", kaio._CACHE_COPY_ARGS), ("kaio_cache_args", kaio._CACHE_ARGS)):
        body = text[:text.index("} " + name + ";")].rsplit("typedef struct {", 1)[1]
        codes = ""
        for line in (x.split("/*")[0].strip().rstrip(";") for x in body.splitlines()):
            if line:
                kind, names = line.split(" ", 1)
                code = "P" if "*" in line else {"uint32_t": "I", "int32_t": "i", "int64_t": "q"}[kind]
                codes += code * (1 if code == "P" else names.count(",") + 1)
        assert "".join(c * int(n or 1) for n, c in re.findall(r"(\d*)([A-Za-z])", fields.format.lstrip("@"))) == codes
    assert kaio._PAGED_SCORED_ARGS.format == kaio._PAGED_ARGS.format + "fi3P"
    for fn, args in ((L.kaio_cache_copy_pages, copy_args(size=4)), (L.kaio_paged_attention_scored, scored_args(size=4)),
                     (L.kaio_paged_attention_scored, scored_args(size=kaio._PAGED_ARGS.size)),
                     *((f, book_args(size=4)) for f in books(L))):
        refused(fn, args, "struct_size")
        refused(fn, None, "null pointer")


def books(L):
    return L.kaio_cache_fork, L.kaio_cache_append, L.kaio_cache_truncate, L.kaio_cache_compact


@pytest.mark.parametrize("kw,text", [
    (dict(caches=-1), "caches"), (dict(dim=60), "dim"), (dict(dim=264), "dim"), (dict(pairs=-1), "pairs"),
    (dict(num_pages=1 << 30), "num_pages"), (dict(page_size=1 << 20, kv_heads=1 << 10), "kv_heads * dim"),
    (dict(page_size=(1 << 30) - 1, kv_heads=(1 << 30) - 1), "kv_heads * dim"),
    (dict(page_size=1 << 15, kv_heads=1 << 8, pairs=1 << 25), "pairs * pieces"),
    (dict(steps=((2048, 128, 64), (2048, 130, 64))), "multiple of 8"), (dict(steps=((2048, 128, 64), (1024, 128, 64))), "share"),
    (dict(bases=(ptr(0), 0)), "null"), (dict(src=0), "src is a null"), (dict(dst=0), "dst is a null"),
    (dict(cache=0), "cache is a null"), (dict(strides=0), "strides is a null"), (dict(dst=ptr(1, 64)), "overlaps input dst"),
])
def test_copy_refusals(L, kw, text):
    refused(L.kaio_cache_copy_pages, copy_args(**kw), text)


def test_copy_alignment_and_what_is_allowed(L):
    refused(L.kaio_cache_copy_pages, copy_args(bases=(ptr(0), ptr(1, 8))), "16-byte", MISALIGNED)
    refused(L.kaio_cache_copy_pages, copy_args(src=ptr(2, 2)), "4-byte", MISALIGNED)
    passes_validation(L.kaio_cache_copy_pages, copy_args())
    passes_validation(L.kaio_cache_copy_pages, copy_args(bases=(ptr(0), ptr(0, 4096)), steps=((4096, 128, 64),) * 2))
    passes_validation(L.kaio_cache_copy_pages, copy_args(caches=0, cache=0, strides=0))


@pytest.mark.parametrize("kw,text", [
    (dict(batch=-1), "batch"), (dict(batch=8193), "at most 8192"), (dict(max_pages=-1), "max_pages"),
    (dict(max_pages=1 << 29), "batch * max_pages"), (dict(num_pages=(1 << 23) + 1), "num_pages"),
    (dict(page_size=0), "page_size"), (dict(num_pages=1 << 20, page_size=1 << 11), "page_size"),
    (dict(table_stride=3), "table_stride"), (dict(table_stride=1 << 41), "table_stride"),
    (dict(page_refs=0), "page_refs is a null"), (dict(page_table=0), "page_table is a null"),
    (dict(kv_lens=0), "kv_lens is a null"), (dict(page_table=ptr(0, 8)), "overlap"), (dict(kv_lens=ptr(1, 40)), "overlap"),
])
def test_book_refusals(L, kw, text):
    for fn in books(L):
        refused(fn, book_args(**kw), text)


def test_refusals_of_each_book_entry(L):
    fork, append, truncate, compact = books(L)
    refused(fork, book_args(parents=0), "parents is a null")
    refused(fork, book_args(parents=ptr(2)), "overlaps input parents")
    refused(truncate, book_args(new_lens=0), "new_lens is a null")
    refused(append, book_args(q_starts=0), "without q_starts")
    for name in ("slots", "src", "dst"):
        refused(append, book_args(**{name: 0}), f"{name} is a null")
        refused(append, book_args(**{name: ptr(4)}), "overlaps input q_starts")
    refused(append, book_args(tokens=-1), "tokens")
    refused(compact, book_args(max_moves=-1), "max_moves")
    refused(compact, book_args(src=0), "src is a null")
    refused(compact, book_args(dst=ptr(0)), "overlap")
    refused(append, book_args(batch=0), "without sequences")
    refused(compact, book_args(batch=0), "without sequences")
    for fn in books(L):
        refused(fn, book_args(kv_lens=ptr(2, 2)), "4-byte", MISALIGNED)
        passes_validation(fn, book_args())
        passes_validation(fn, book_args(batch=0, tokens=0, max_moves=0))
        passes_validation(fn, book_args(num_pages=0, page_refs=0))
    passes_validation(append, book_args(q_starts=0, tokens=3))
    passes_validation(fork, book_args(q_starts=0, slots=0, src=0, dst=0, tokens=-7, max_moves=-7))
    passes_validation(compact, book_args(max_moves=0, src=0, dst=0))


@pytest.mark.parametrize("kw,text", [
    (dict(softcap=-1.0), "softcap"), (dict(softcap=257.0), "softcap"), (dict(softcap=float("nan")), "softcap"),
    (dict(softcap=float("inf")), "softcap"), (dict(softcap=1e-38), "softcap"), (dict(scale=1e-38), "softcap"),
    (dict(out=ptr(10)), "overlaps input slopes"), (dict(lse=ptr(11)), "overlaps input prefix_lens"),
    (dict(workspace=ptr(12)), "overlaps input doc_starts"), (dict(dtype=F32), "F16 or BF16"), (dict(window=-1), "window"),
    (dict(q_starts=0), "without q_starts"), (dict(q=0), "q is a null"),
])
def test_scored_attention_refusals(L, kw, text):
    refused(L.kaio_paged_attention_scored, scored_args(**kw), text)


def test_scored_attention_alignment_and_what_is_allowed(L):
    for name in ("slopes", "prefix_lens", "doc_starts"):
        refused(L.kaio_paged_attention_scored, scored_args(**{name: ptr(20, 2)}), f"{name}", MISALIGNED)
        passes_validation(L.kaio_paged_attention_scored, scored_args(**{name: 0}))
    passes_validation(L.kaio_paged_attention_scored, scored_args(softcap=0.0))
    passes_validation(L.kaio_paged_attention_scored, scored_args(softcap=256.0, scale=0.0))
    passes_validation(L.kaio_paged_attention_scored, scored_args(0.0, 0, 0, 0, 0))


def test_bindings_refuse_what_does_not_fit():
    import torch
    i32 = torch.int32
    refs, table, lens = torch.zeros(4, dtype=i32), torch.zeros(2, 3, dtype=i32), torch.zeros(2, dtype=i32)
    for call in (lambda: kaio.cache_fork(refs, table, lens, lens, 16), lambda: kaio.cache_truncate(refs, table, lens, lens, 16),
                 lambda: kaio.cache_copy_pages([], refs, refs),
                 lambda: kaio.paged_attention(torch.zeros(2, 4, 64).half(), torch.zeros(1, 16, 4, 64).half(),
                                              torch.zeros(1, 16, 4, 64).half(), table, lens, softcap=30.0)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    with pytest.raises(TypeError, match="torch.Tensor"):
        kaio.cache_fork([1], table, lens, lens, 16)
    for v in (1.5, "3", None):
        with pytest.raises(TypeError, match="tokens"):
            kaio.cache_append(refs, table, lens, None, v, 16)
        with pytest.raises(TypeError, match="max_moves"):
            kaio.cache_compact(refs, table, lens, 16, v)
