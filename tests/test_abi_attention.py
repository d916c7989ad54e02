"""Host-side checks of the rotary and paged-attention entries (no GPU): argument
blocks and the order of the refusals, with made-up pointers that validation never
dereferences."""
import pytest

from qkv_projection_gb300 import kaio

INVALID, MISALIGNED, CUDA_ERR, UNSUPPORTED = (kaio.KAIO_ERR_INVALID_VALUE, kaio.KAIO_ERR_MISALIGNED,
                                              kaio.KAIO_ERR_CUDA, kaio.KAIO_ERR_UNSUPPORTED_DEVICE)
F32, F16, BF16 = kaio.KAIO_DTYPE_F32, kaio.KAIO_DTYPE_F16, kaio.KAIO_DTYPE_BF16

ROPE = ("size dtype tokens heads kv_heads dim pairs axes s0 s1 s2 s3 interleaved inverse num_pages page_size "
        "q k v q_out k_cache v_cache positions inv_freq slots q_ts q_hs o_ts o_hs k_ts k_hs v_ts v_hs "
        "kc_ps kc_ss kc_hs vc_ps vc_ss vc_hs pos_stride").split()
PAGED = ("size dtype batch tokens heads kv_heads dim page_size num_pages max_pages max_new causal window sinks "
         "scale reserved q k_cache v_cache table kv_lens q_starts out lse workspace workspace_bytes "
         "q_ts q_hs o_ts o_hs k_ps k_ss k_hs v_ps v_ss v_hs table_stride").split()


@pytest.fixture(scope="module")
def L():
    return kaio.lib()


def ptr(i, off=0):
    return (1 << 40) + i * (1 << 36) + off


def rope_args(**kw):
    a = dict(zip(ROPE, [0] * len(ROPE)))
    a.update(size=kaio._ROPE_ARGS.size, dtype=F16, tokens=5, heads=4, kv_heads=2, dim=64, pairs=32, axes=2, s0=20,
             s1=12, num_pages=3, page_size=16, pos_stride=5, q_ts=256, q_hs=64, o_ts=256, o_hs=64, k_ts=128, k_hs=64,
             v_ts=128, v_hs=64, kc_ps=2048, kc_ss=128, kc_hs=64, vc_ps=2048, vc_ss=128, vc_hs=64)
    for i, name in enumerate("q k v q_out k_cache v_cache positions inv_freq slots".split()):
        a[name] = ptr(i)
    a.update(kw)
    return kaio._ROPE_ARGS.pack(*a.values())


def paged_args(**kw):
    a = dict(zip(PAGED, [0] * len(PAGED)))
    a.update(size=kaio._PAGED_ARGS.size, dtype=BF16, batch=3, tokens=5, heads=4, kv_heads=2, dim=64, page_size=16,
             num_pages=7, max_pages=4, max_new=5, causal=1, scale=0.125, workspace_bytes=1 << 30, q_ts=256, q_hs=64,
             o_ts=256, o_hs=64, k_ps=2048, k_ss=128, k_hs=64, v_ps=2048, v_ss=128, v_hs=64, table_stride=4)
    for i, name in enumerate("q k_cache v_cache table kv_lens q_starts out lse workspace".split()):
        a[name] = ptr(i)
    a.update(kw)
    return kaio._PAGED_ARGS.pack(*a.values())


def refused(fn, args, text, status=INVALID):
    assert fn(args, None) == status, kaio.last_error()
    assert text in kaio.last_error(), kaio.last_error()


def passes_validation(fn, args):
    """Past its argument checks; without a GPU the first CUDA call then fails."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: made-up pointers go no further than the argument checks")
    assert fn(args, None) in (CUDA_ERR, UNSUPPORTED), kaio.last_error()


def test_blocks_have_the_header_s_size_and_order(L):
    for fn, pack in ((L.kaio_rope, rope_args), (L.kaio_rope_append, rope_args), (L.kaio_paged_attention, paged_args)):
        refused(fn, pack(size=8), "struct_size 8")
        refused(fn, None, "null pointer")
    text = open(kaio.HEADER).read()
    for name, fields in (("kaio_rope_args", kaio._ROPE_ARGS), ("kaio_paged_attention_args", kaio._PAGED_ARGS)):
        body = text[:text.index("} " + name + ";")].rsplit("typedef struct {", 1)[1]
        codes = ""
        for line in body.splitlines():
            line = line.split("/*")[0].strip().rstrip(";")
            if not line:
                continue
            if "*" in line:
                codes += "P"
                continue
            kind, names = line.split(" ", 1)
            code = {"uint32_t": "I", "int32_t": "i", "float": "f", "uint64_t": "Q", "int64_t": "q"}[kind]
            for n in names.split(","):
                codes += code * (int(n.split("[")[1].rstrip("]")) if "[" in n else 1)
        import struct
        assert struct.Struct("@" + codes).size == fields.size
        expand = lambda f: "".join(c * int(n or 1) for n, c in __import__("re").findall(r"(\d*)([A-Za-z])", f))  # noqa: E731
        assert expand(fields.format.lstrip("@")) == codes


@pytest.mark.parametrize("kw,text", [
    (dict(dtype=F32), "F16 or BF16"), (dict(dtype=9), "F16 or BF16"), (dict(dim=60), "dim"), (dict(dim=264), "dim"),
    (dict(dim=0), "dim"), (dict(pairs=0), "pairs"), (dict(pairs=33), "pairs"), (dict(axes=0), "axes"),
    (dict(axes=5), "axes"), (dict(s0=-1, s1=33), "negative"), (dict(s0=19), "sum to 31"), (dict(axes=1), "sum to 20"),
    (dict(tokens=-1), "tokens"), (dict(heads=0), "heads"), (dict(tokens=1 << 29, heads=8), "tokens * heads"),
    (dict(q_ts=252), "multiple of 8"), (dict(q_ts=-256), "non-negative"), (dict(o_ts=0), "below dim"),
    (dict(q=None), "null"), (dict(q_out=None), "null"), (dict(positions=None), "null"), (dict(inv_freq=None), "null"),
    (dict(q_out=ptr(0, 64)), "overlaps input q"), (dict(q_out=ptr(6)), "overlaps input positions"),
    (dict(q_out=ptr(0), o_ts=512), "overlaps input q"), (dict(pos_stride=-1), "positions_axis_stride"),
])
def test_rope_refusals(L, kw, text):
    kw = {k: 0 if v is None else v for k, v in kw.items()}
    refused(L.kaio_rope, rope_args(**kw), text)
    refused(L.kaio_rope_append, rope_args(**kw), text)


@pytest.mark.parametrize("kw,text", [
    (dict(inverse=1), "inverse"), (dict(kv_heads=0), "kv_heads"), (dict(page_size=0), "page_size"),
    (dict(num_pages=-1), "num_pages"), (dict(k=0), "k is a null"), (dict(slots=0), "slots is a null"),
    (dict(k_cache=0), "k_cache is a null"), (dict(kc_ss=0), "below dim"), (dict(v_ts=100), "v: stride"),
    (dict(k_cache=ptr(5)), "k_cache and v_cache"), (dict(v_cache=ptr(3, 128)), "q_out and v_cache"),
    (dict(k_cache=ptr(2, -1024)), "overlaps input v"), (dict(k_cache=ptr(0, 1024)), "overlaps input q"),
])
def test_rope_append_refusals(L, kw, text):
    refused(L.kaio_rope_append, rope_args(**kw), text)


def test_rope_alignment_and_what_is_allowed(L):
    for name in ("q", "q_out", "k", "v", "k_cache", "v_cache"):
        refused(L.kaio_rope_append, rope_args(**{name: ptr(20, 8)}), name, MISALIGNED)
    for name in ("positions", "inv_freq", "slots"):
        refused(L.kaio_rope_append, rope_args(**{name: ptr(20, 2)}), name, MISALIGNED)
    passes_validation(L.kaio_rope, rope_args(q_out=ptr(0)))                       # in place
    passes_validation(L.kaio_rope, rope_args(k=0, v=0, k_cache=0, v_cache=0, slots=0, kv_heads=0))
    passes_validation(L.kaio_rope, rope_args(q_hs=0))                             # a broadcast input
    passes_validation(L.kaio_rope_append, rope_args(v_cache=ptr(4, 4096), kc_ps=4096, vc_ps=4096))   # one buffer


@pytest.mark.parametrize("kw,text", [
    (dict(dtype=F32), "F16 or BF16"), (dict(dim=4), "dim"), (dict(dim=136), "dim"), (dict(dim=60), "dim"),
    (dict(heads=5), "multiple of kv_heads"), (dict(kv_heads=0), "kv_heads"), (dict(heads=0), "multiple of kv_heads"),
    (dict(page_size=8), "page_size"), (dict(page_size=48), "page_size"), (dict(page_size=2048), "page_size"),
    (dict(window=-1), "window"), (dict(sinks=-1), "sinks"), (dict(scale=float("inf")), "scale"),
    (dict(scale=float("nan")), "scale"), (dict(batch=-1), "batch"), (dict(tokens=1 << 30), "tokens"),
    (dict(max_new=-1), "max_new"), (dict(q_starts=0), "without q_starts"), (dict(q_ts=4), "multiple of 8"),
    (dict(k_ss=12), "multiple of 8"), (dict(o_hs=32), "below dim"), (dict(table_stride=-1), "table_stride"),
    (dict(q=0), "q is a null"), (dict(kv_lens=0), "kv_lens is a null"), (dict(table=0), "page_table is a null"),
    (dict(out=0), "out is a null"), (dict(workspace=0), "workspace is a null"), (dict(out=ptr(0)), "overlaps input q"),
    (dict(out=ptr(1, 512)), "overlaps input k_cache"), (dict(lse=ptr(6, 64)), "overlap"),
    (dict(workspace=ptr(2, 256)), "overlaps input v_cache"),
])
def test_paged_attention_refusals(L, kw, text):
    refused(L.kaio_paged_attention, paged_args(**kw), text)


def test_paged_attention_alignment_and_what_is_allowed(L):
    for name in ("q", "k_cache", "v_cache", "out", "workspace"):
        refused(L.kaio_paged_attention, paged_args(**{name: ptr(20, 8)}), name, MISALIGNED)
    for name in ("table", "kv_lens", "q_starts", "lse"):
        refused(L.kaio_paged_attention, paged_args(**{name: ptr(20, 2)}), "4-byte", MISALIGNED)
    passes_validation(L.kaio_paged_attention, paged_args())
    passes_validation(L.kaio_paged_attention, paged_args(lse=0, q_starts=0, tokens=3))
    passes_validation(L.kaio_paged_attention, paged_args(num_pages=0, k_cache=0, v_cache=0))
    passes_validation(L.kaio_paged_attention, paged_args(v_cache=ptr(1, 4096), k_ps=4096, v_ps=4096))


def test_workspace_query_refuses_null(L):
    assert L.kaio_paged_attention_workspace(None) == INVALID and "null" in kaio.last_error()


def test_bindings_refuse_cpu_tensors():
    import torch
    x = torch.zeros(2, 4, 64, dtype=torch.float16)
    pos, inv = torch.zeros(2, dtype=torch.int32), torch.ones(32)
    cache = torch.zeros(1, 16, 4, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA device"):
        kaio.rope(x, pos, inv)
    with pytest.raises(ValueError, match="CUDA device"):
        kaio.rope_append(x, x, x, pos, inv, cache, cache, pos)
    with pytest.raises(ValueError, match="CUDA device"):
        kaio.paged_attention(x, cache, cache, pos[:, None], pos)
    with pytest.raises(TypeError, match="float16 or"):
        kaio.rope(x.float(), pos, inv)
