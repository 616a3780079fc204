"""Refusals that follow from where the tensors of the cache operators lie: strides whose products pass 64 bits, caches
that overlap themselves or each other.  Every call here fails on the host, with made-up addresses."""
import pytest

import q4_dequant_gemv_block_amd as q4
from test_kv_cpu import BASE, FREQ, GIB, POS, batch, cache, heads, lib, ref, refused  # noqa: F401 (lib: a fixture)

FAR = 1 << 40  # the largest stride


@pytest.mark.parametrize("which", ["x", "out"])
def test_rope_strides_that_pass_64_bits(lib, which):
    """2^24 tokens 2^40 elements apart: the span's end is in front of its beginning, and would overlap nothing."""
    a = dict(x=heads(0), out=heads(GIB))
    a[which] = heads(0, token_stride=FAR)
    st = lib.q4_rope(ref(a["x"]), ref(a["out"]), POS, FREQ, 1 << 24, 8, 128, 128, 0, 1.0, None)
    refused(lib, st, -1, "strides of %s reach too far" % which)


def test_append_strides_that_pass_64_bits(lib):
    def call(**over):
        a = dict(cache=cache(), batch=batch(), k=heads(GIB, 2), v=heads(2 * GIB, 2), q=heads(3 * GIB), q_out=heads(4 * GIB))
        a.update(over)
        return lib.q4_kv_append(ref(a["cache"]), ref(a["batch"]), ref(a["k"]), ref(a["v"]), ref(a["q"]), ref(a["q_out"]), 8,
                                1 << 24, None, FREQ, 128, 0, 1.0, None)
    for name in ("k", "v", "q", "q_out"):
        refused(lib, call(**{name: heads(3 * GIB, token_stride=FAR)}), -1, "strides of %s reach too far" % name)
    for over in (dict(k_page_stride=FAR), dict(v_page_stride=FAR)):
        refused(lib, call(cache=cache(pages=1 << 30, **over)), -1, "strides of the cache reach too far")
    refused(lib, call(batch=batch(seqs=1 << 24, table_stride=FAR)), -1, "stride reaches too far")


def test_attention_strides_that_pass_64_bits(lib):
    def call(**over):
        a = dict(cache=cache(), batch=batch(), q=heads(GIB), out=heads(2 * GIB))
        a.update(over)
        return lib.q4_attention_paged(ref(a["cache"]), ref(a["batch"]), ref(a["q"]), ref(a["out"]), None, 8, 1 << 24, 0.1, 0,
                                      BASE + 80 * GIB, 8 * GIB, None)
    for name in ("q", "out"):
        refused(lib, call(**{name: heads(3 * GIB, token_stride=FAR)}), -1, "strides of %s reach too far" % name)
    refused(lib, call(cache=cache(pages=1 << 30, v_page_stride=FAR)), -1, "strides of the cache reach too far")
    refused(lib, call(batch=batch(seqs=1 << 24, table_stride=FAR)), -1, "stride reaches too far")
    assert lib.q4_attention_paged_workspace_bytes(ref(cache(pages=1 << 30, k_page_stride=FAR)), ref(batch()), 8, 5, 0) == 0
    assert "too far" in q4.last_error()


def append(lib, c, **over):
    """An append to that cache that is refused behind the checks of the cache (q without q_out) if those pass."""
    dim = c.head_dim
    k, v = heads(GIB, c.kv_heads, dim), heads(2 * GIB, c.kv_heads, dim)
    return lib.q4_kv_append(ref(c), ref(batch()), ref(k), ref(v), ref(heads(3 * GIB, 8, dim)), None, 8, 5, None, FREQ, 64,
                            0, 1.0, None)


@pytest.mark.parametrize("over", [
    dict(k_head_stride=128),                                         # heads in each other's slots
    dict(v_head_stride=128),
    dict(k_page_stride=16 * 128),                                    # a page where the next head is
    dict(v_page_stride=2 * 16 * 128 - 1),                            # one element too near
    dict(k_page_stride=128, k_head_stride=10 * 128, k_slot_stride=19 * 128),  # pages innermost: 2 heads reach 20
])
def test_append_to_a_cache_that_overlaps_itself(lib, over):
    refused(lib, append(lib, cache(**over)), -1, "heads of the cache overlap each other")


@pytest.mark.parametrize("over", [
    dict(k_page_stride=16 * 2 * 128, k_slot_stride=2 * 128, k_head_stride=128),  # slots outside heads
    dict(v_page_stride=128, v_head_stride=10 * 128, v_slot_stride=20 * 128),     # pages innermost
    dict(k_page_stride=1 << 20, k_head_stride=1 << 13, k_slot_stride=136),       # gaps
    dict(kv_heads=1, k_head_stride=0, v_head_stride=5),                          # a stride that is never used
    dict(pages=1, k_page_stride=0),
])
def test_append_to_any_layout(lib, over):
    refused(lib, append(lib, cache(**over)), -1, "go together")


K = BASE + 16 * GIB
PAGE = 2 * 16 * 128  # elements of a page of the keys: 2 heads of 16 slots


@pytest.mark.parametrize("over", [
    dict(v=K), dict(v=K + 2 * 128), dict(v=K + 2), dict(v=K + 2 * (10 * PAGE - 1)),  # behind the keys' beginning
    dict(v=K - 2 * 128), dict(v=K - 2 * (10 * PAGE - 1)),                             # in front of it
    # page by page, but one element, or one slot, too few between
    dict(v=K + 2 * (PAGE - 1), k_page_stride=2 * PAGE, v_page_stride=2 * PAGE),
    dict(v=K + 2 * PAGE, k_page_stride=2 * PAGE - 128, v_page_stride=2 * PAGE - 128),
    # head by head (each head's values behind its keys), the values one slot early
    dict(v=K + 2 * 15 * 128, k_head_stride=2 * 16 * 128, v_head_stride=2 * 16 * 128, k_page_stride=2 * PAGE, v_page_stride=2 * PAGE),
    # slot by slot, half a head apart
    dict(v=K + 2 * 64, k_slot_stride=256, v_slot_stride=256, k_head_stride=4096, v_head_stride=4096, k_page_stride=8192, v_page_stride=8192),
])
def test_append_to_keys_and_values_that_overlap(lib, over):
    refused(lib, append(lib, cache(**dict(dict(k=K), **over))), -1, "same memory")


@pytest.mark.parametrize("over", [
    dict(v=K + 2 * 10 * PAGE), dict(v=K - 2 * 10 * PAGE),                                 # one behind the other
    dict(v=K + 2 * PAGE, k_page_stride=2 * PAGE, v_page_stride=2 * PAGE),                  # page by page
    dict(v=K - 2 * PAGE, k_page_stride=2 * PAGE, v_page_stride=2 * PAGE),
    dict(v=K + 2 * 16 * 128, k_head_stride=2 * 16 * 128, v_head_stride=2 * 16 * 128, k_page_stride=2 * PAGE, v_page_stride=2 * PAGE),
    dict(v=K + 2 * 128, k_slot_stride=256, v_slot_stride=256, k_head_stride=4096, v_head_stride=4096, k_page_stride=8192, v_page_stride=8192),
    # a page's values in another order than its keys
    dict(v=K + 2 * PAGE, k_page_stride=2 * PAGE, v_page_stride=2 * PAGE, v_slot_stride=256, v_head_stride=128),
    # the layers of a model page by page, this one's keys and values 3 and 8 places in
    dict(k=K + 2 * 3 * PAGE, v=K + 2 * 8 * PAGE, k_page_stride=20 * PAGE, v_page_stride=20 * PAGE),
    dict(k=K + 2 * 8 * PAGE, v=K + 2 * 3 * PAGE, k_page_stride=20 * PAGE, v_page_stride=20 * PAGE),
])
def test_append_to_keys_and_values_beside_each_other(lib, over):
    refused(lib, append(lib, cache(**dict(dict(k=K), **over))), -1, "go together")
