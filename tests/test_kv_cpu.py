"""Refusals of the rotary, cache-append and attention entry points (every call here fails on the host before anything
would be enqueued, with made-up addresses), and the frequencies of the rotary positions."""
import ctypes
import math
import os

import pytest
import torch

import q4_dequant_gemv_block_amd as q4

BASE = 1 << 40  # an address no check dereferences
GIB = 1 << 30


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(q4.LIB_PATH):
        from q4_dequant_gemv_block_amd import build
        build.build()
    return q4.load_library()


def heads(at, heads=8, dim=128, kind=q4.Q4_TYPE_F16, **over):
    f = dict(data=BASE + at, token_stride=heads * dim, head_stride=dim, type=kind)
    f.update(over)
    return q4.Heads(**f)


def cache(**over):
    hk, page, dim = over.get("kv_heads", 2), over.get("page_size", 16), over.get("head_dim", 128)
    f = dict(k=BASE + 16 * GIB, v=BASE + 32 * GIB, k_page_stride=hk * page * dim, k_head_stride=page * dim, k_slot_stride=dim,
             v_page_stride=hk * page * dim, v_head_stride=page * dim, v_slot_stride=dim, pages=10, page_size=page,
             kv_heads=hk, head_dim=dim, type=q4.Q4_TYPE_F16)
    f.update(over)
    return q4.CacheDesc(**f)


def batch(**over):
    f = dict(block_table=BASE + 64 * GIB, table_stride=4, table_pages=4, seqs=3, query_start=BASE + 65 * GIB,
             context_len=BASE + 66 * GIB, max_query=0, max_context=0)
    f.update(over)
    return q4.BatchDesc(**f)


def refused(lib, status, want, text):
    assert status == want, (status, q4.last_error())
    assert text in q4.last_error(), q4.last_error()


def ref(x):
    return None if x is None else ctypes.byref(x)


POS, FREQ = BASE + 70 * GIB, BASE + 71 * GIB


@pytest.mark.parametrize("over,want,text", [
    (dict(tokens=0), -1, "tokens"), (dict(tokens=1 << 28), -1, "tokens"), (dict(heads=0), -1, "heads"),
    (dict(dim=0, rot=0), -1, "head_dim"), (dict(dim=1026), -1, "head_dim"),
    (dict(rot=3), -1, "rot_dim"), (dict(rot=130), -1, "rot_dim"), (dict(rot=0), -1, "rot_dim"), (dict(rot=-2), -1, "rot_dim"),
    (dict(layout=2), -1, "layout"), (dict(mscale=math.nan), -1, "mscale"), (dict(mscale=math.inf), -1, "mscale"),
    (dict(pos=None), -1, "positions"), (dict(pos=POS + 2), -2, "positions"), (dict(freq=None), -1, "inv_freq"),
    (dict(freq=FREQ + 4), -2, "inv_freq"),
    (dict(x=None), -1, "null x"), (dict(out=None), -1, "null out"), (dict(x=heads(0, data=None)), -1, "null x"),
    (dict(x=heads(0, kind=7)), -1, "type"), (dict(x=heads(1)), -2, "aligned"),
    (dict(x=heads(0, token_stride=-1)), -1, "stride"),
    (dict(out=heads(GIB, head_stride=64)), -1, "overlap each other"),
    (dict(out=heads(GIB, token_stride=0)), -1, "overlap each other"),
    (dict(out=heads(2)), -1, "overlaps x"), (dict(out=heads(0, kind=q4.Q4_TYPE_F32)), -1, "overlaps x"),
    (dict(out=heads(70 * GIB)), -1, "overlaps positions"), (dict(out=heads(71 * GIB)), -1, "overlaps positions"),
])
def test_rope_refusals(lib, over, want, text):
    a = dict(x=heads(0), out=heads(GIB), pos=POS, freq=FREQ, tokens=5, heads=8, dim=128, rot=128, layout=0, mscale=1.0)
    a.update(over)
    st = lib.q4_rope(ref(a["x"]), ref(a["out"]), a["pos"], a["freq"], a["tokens"], a["heads"], a["dim"], a["rot"],
                     a["layout"], a["mscale"], None)
    refused(lib, st, want, text)


CACHE_REFUSALS = [
    (dict(cache=None), -1, "null cache"), (dict(cache=cache(k=None)), -1, "null cache"),
    (dict(cache=cache(type=q4.Q4_TYPE_F32)), -1, "binary16 or bfloat16"), (dict(cache=cache(pages=0)), -1, "pages"),
    (dict(cache=cache(page_size=12)), -1, "page_size"), (dict(cache=cache(page_size=0)), -1, "page_size"),
    (dict(cache=cache(page_size=1 << 17)), -1, "page_size"), (dict(cache=cache(kv_heads=0)), -1, "kv_heads"),
    (dict(cache=cache(k_slot_stride=64)), -1, "overlap each other"), (dict(cache=cache(v_page_stride=-8)), -1, "stride"),
    (dict(batch=None), -1, "null batch"), (dict(batch=batch(block_table=None)), -1, "null batch"),
    (dict(batch=batch(query_start=BASE + 2)), -2, "aligned"), (dict(batch=batch(seqs=0)), -1, "seqs"),
    (dict(batch=batch(table_pages=0)), -1, "block table"), (dict(batch=batch(table_pages=1 << 27)), -1, "block table"),
    (dict(batch=batch(table_stride=3)), -1, "stride"), (dict(batch=batch(max_query=-1)), -1, "max_query"),
]


@pytest.mark.parametrize("over,want,text", CACHE_REFUSALS + [
    (dict(tokens=0), -1, "tokens"), (dict(k=None), -1, "null k"), (dict(v=None), -1, "null v"),
    (dict(v=heads(2 * GIB, 2, kind=q4.Q4_TYPE_F32)), -1, "one type"), (dict(q=None), -1, "go together"),
    (dict(q_out=None), -1, "go together"), (dict(q_out=heads(4 * GIB, kind=q4.Q4_TYPE_BF16)), -1, "cache's type"),
    (dict(q_out=heads(3 * GIB + 2)), -1, "q_out overlaps"), (dict(q_out=heads(GIB)), -1, "q_out overlaps"),
    (dict(q_out=heads(16 * GIB)), -1, "q_out overlaps"), (dict(q_out=heads(64 * GIB)), -1, "q_out overlaps"),
    (dict(k=heads(16 * GIB, 2)), -1, "overlaps an input"), (dict(v=heads(32 * GIB, 2)), -1, "overlaps an input"),
    (dict(q=heads(32 * GIB)), -1, "q overlaps the cache"), (dict(cache=cache(v=BASE + 16 * GIB)), -1, "same memory"), (dict(pos=16 * GIB + BASE), -1, "overlaps an input"),
    (dict(rot=130), -1, "rot_dim"), (dict(freq=None), -1, "inv_freq"), (dict(layout=9), -1, "layout"),
    (dict(pos=POS + 1), -2, "positions"),
])
def test_append_refusals(lib, over, want, text):
    a = dict(cache=cache(), batch=batch(), k=heads(GIB, 2), v=heads(2 * GIB, 2), q=heads(3 * GIB), q_out=heads(4 * GIB),
             tokens=5, pos=None, freq=FREQ, rot=128, layout=0)
    a.update(over)
    st = lib.q4_kv_append(ref(a["cache"]), ref(a["batch"]), ref(a["k"]), ref(a["v"]), ref(a["q"]), ref(a["q_out"]), 8,
                          a["tokens"], a["pos"], a["freq"], a["rot"], a["layout"], 1.0, None)
    refused(lib, st, want, text)


@pytest.mark.parametrize("over,want,text", CACHE_REFUSALS + [
    (dict(cache=cache(head_dim=80)), -1, "head_dim"), (dict(q_heads=7), -1, "multiple of kv_heads"),
    (dict(cache=cache(k=BASE + 16 * GIB + 8)), -2, "16-byte"), (dict(cache=cache(v_slot_stride=132)), -2, "multiples of 8"),
    (dict(tokens=0), -1, "tokens"), (dict(q=None), -1, "null q"), (dict(out=None), -1, "null out"),
    (dict(q=heads(GIB, kind=q4.Q4_TYPE_F32)), -1, "cache's type"), (dict(out=heads(2 * GIB, kind=q4.Q4_TYPE_BF16)), -1, "cache's type"),
    (dict(q=heads(GIB + 8)), -2, "16-byte"), (dict(q=heads(GIB, token_stride=1028)), -2, "multiples of 8"),
    (dict(lse=BASE + 3 * GIB + 2), -2, "lse"), (dict(scale=0.0), -1, "scale"), (dict(scale=-1.0), -1, "scale"),
    (dict(scale=math.nan), -1, "scale"), (dict(scale=math.inf), -1, "scale"), (dict(scale=3e38), -1, "scale"),
    (dict(window=-1), -1, "window"),
    (dict(out=heads(GIB)), -1, "overlaps an input"), (dict(out=heads(16 * GIB)), -1, "overlaps an input"),
    (dict(out=heads(65 * GIB)), -1, "overlaps the batch"), (dict(lse=BASE + 32 * GIB), -1, "overlaps an input"),
    (dict(lse=BASE + 2 * GIB), -1, "must not overlap"), (dict(out=heads(2 * GIB, head_stride=0)), -1, "overlap each other"),
])
def test_attention_refusals(lib, over, want, text):
    a = dict(cache=cache(), batch=batch(), q=heads(GIB), out=heads(2 * GIB), lse=None, q_heads=8, tokens=5, scale=0.1, window=0)
    a.update(over)
    st = lib.q4_attention_paged(ref(a["cache"]), ref(a["batch"]), ref(a["q"]), ref(a["out"]), a["lse"], a["q_heads"],
                                a["tokens"], a["scale"], a["window"], BASE + 80 * GIB, GIB, None)
    refused(lib, st, want, text)


def test_strides_of_single_tokens_do_not_count(lib):
    """torch gives a dimension of one entry any stride: it is no misalignment (the call fails on the workspace only)."""
    c, b = cache(), batch(table_pages=2000, table_stride=2000, max_context=32000)
    odd = heads(GIB, token_stride=1025)
    st = lib.q4_attention_paged(ref(c), ref(b), ref(odd), ref(heads(2 * GIB)), None, 8, 1, 0.1, 0, None, 0, None)
    refused(lib, st, -3, "workspace")
    st = lib.q4_attention_paged(ref(c), ref(b), ref(odd), ref(heads(2 * GIB)), None, 8, 2, 0.1, 0, None, 0, None)
    refused(lib, st, -2, "multiples of 8")


def test_attention_workspace(lib):
    c, b = cache(), batch(table_pages=2000, table_stride=2000, max_context=32000)
    need = lib.q4_attention_paged_workspace_bytes(ref(c), ref(b), 8, 5, 0)
    assert q4.last_error() == ""
    args = (ref(c), ref(b), ref(heads(GIB)), ref(heads(2 * GIB)), None, 8, 5, 0.1, 0)
    assert need > 0  # a long context of few heads is cut
    refused(lib, lib.q4_attention_paged(*args, None, 0, None), -3, "workspace")
    refused(lib, lib.q4_attention_paged(*args, BASE + 80 * GIB, need - 1, None), -3, "workspace")
    refused(lib, lib.q4_attention_paged(*args, BASE + 80 * GIB + 8, need, None), -2, "workspace")
    refused(lib, lib.q4_attention_paged(*args, BASE + 16 * GIB, need, None), -1, "overlaps an input")
    refused(lib, lib.q4_attention_paged(*args, BASE + 2 * GIB, need, None), -1, "must not overlap")
    assert lib.q4_attention_paged_workspace_bytes(ref(cache(head_dim=80)), ref(b), 8, 5, 0) == 0
    assert "head_dim" in q4.last_error()


def test_parts_of_packed_rows_are_not_taken_for_overlapping(lib):
    """q turned in place in the packed q/k/v rows of tokens: refused only for what comes after the overlap checks."""
    row = (8 + 2 + 2) * 128
    q, k, v = (heads(GIB + 2 * off, n, token_stride=row) for off, n in ((0, 8), (1024, 2), (1280, 2)))
    st = lib.q4_kv_append(ref(cache(k=BASE + GIB + 2 * 1024)), ref(batch()), ref(k), ref(v), ref(q), ref(q), 8, 5, None, FREQ, 128, 0, 1.0, None)
    refused(lib, st, -1, "overlaps")  # the cache lies in them
    wide = heads(GIB, 9, token_stride=row)
    st = lib.q4_kv_append(ref(cache()), ref(batch()), ref(k), ref(v), ref(wide), ref(wide), 9, 5, None, FREQ, 128, 0, 1.0, None)
    refused(lib, st, -1, "q_out overlaps")  # head 8 is the first of k


def test_python_refusals():
    x = torch.zeros(2, 3, 4, dtype=torch.float16)
    pos, freq = torch.zeros(2, dtype=torch.int32), torch.ones(2, dtype=torch.float64)
    with pytest.raises(ValueError):
        q4.q4_rope(x, pos, freq)  # not on a GPU
    with pytest.raises(ValueError):
        q4.KVCache(torch.zeros(2, 1, 8, 64, dtype=torch.float16), torch.zeros(2, 1, 8, 64, dtype=torch.float16))
    with pytest.raises(TypeError):
        q4.KVCache(torch.zeros(2, 1, 8, 64), torch.zeros(2, 1, 8, 64))
    with pytest.raises(TypeError):
        q4.KVBatch(torch.zeros(2, 2, dtype=torch.int64), torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        q4.KVBatch(torch.zeros(2, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))


def test_frequencies():
    f, m = q4.rope_frequencies(8, 10000.0, device="cpu")
    assert f.dtype == torch.float64 and m == 1.0
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-14, atol=0)
    lin, m = q4.rope_frequencies(8, 10000.0, "linear", 4.0, device="cpu")
    assert torch.allclose(lin, f / 4, rtol=1e-14, atol=0) and m == 1.0
    ntk, _ = q4.rope_frequencies(8, 10000.0, "ntk", 4.0, device="cpu")
    assert float(ntk[0]) == 1.0 and abs(float(ntk[3]) / float(f[3]) - 0.25) < 1e-12  # fastest as before, slowest as linear
    # over 4096 positions pair 0 of 64 makes 652 turns (kept), the last 0.0869 (divided by the factor)
    f, _ = q4.rope_frequencies(128, 10000.0, device="cpu")
    y, m = q4.rope_frequencies(128, 10000.0, "yarn", 8.0, 4096, device="cpu")
    turns = 4096 * f / (2 * math.pi)
    assert abs(m - (0.1 * math.log(8.0) + 1)) < 1e-15
    assert torch.equal(y[turns >= 32 * 1.2], f[turns >= 32 * 1.2])
    assert torch.allclose(y[turns <= 0.8], f[turns <= 0.8] / 8, rtol=1e-14, atol=0)
    between = (y / f)[(turns < 28) & (turns > 1.2)]
    assert bool((between[1:] < between[:-1]).all()) and bool((between < 1).all()) and bool((between > 1 / 8).all())


@pytest.mark.parametrize("args", [(7,), (0,), (8, 1.0), (8, 1e4, "linear", 0.5), (8, 1e4, "yarn", 2.0), (2, 1e4, "ntk", 2.0),
                                  (8, 1e4, "other", 2.0), (8, 1e4, "yarn", 2.0, 4096, 1.0, 1.0), (8, math.inf)])
def test_frequencies_refusals(args):
    with pytest.raises(ValueError):
        q4.rope_frequencies(*args, device="cpu")
