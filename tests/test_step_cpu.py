"""Refusals of the entry points of a step with drafted trees: every call here fails on the host before anything would be
enqueued, with made-up addresses."""
import ctypes
import math
import random

import pytest
import torch

import q4_dequant_gemv_block_amd as q4
from test_kv_cpu import BASE, CACHE_REFUSALS, FREQ, GIB, POS, batch, cache, heads, lib, ref, refused  # noqa: F401

STEP = dict(table_in=1, table_in_stride=4, held_in=2, past_len=3, new_len=4, free_pages=5, free_capacity=9, free_count=6,
            parents=7, table=8, table_stride=4, held=9, query_start=10, context_len=11, missing=12, free_left=13,
            positions=14, slots=15, mask=16, mask_words=1, seqs=3, table_pages=4, page_size=16, tokens=5)
POINTERS = [n for n, t in q4.StepDesc._fields_ if t is ctypes.c_void_p]


def step(**over):
    f = {n: BASE + v * GIB if n in POINTERS else v for n, v in STEP.items()}
    f.update(over)
    return q4.StepDesc(**f)


@pytest.mark.parametrize("over,want,text", [
    (dict(seqs=0), -1, "seqs"), (dict(seqs=65537), -1, "seqs"), (dict(tokens=0), -1, "tokens"), (dict(tokens=1 << 28), -1, "tokens"),
    (dict(page_size=12), -1, "page_size"), (dict(page_size=0), -1, "page_size"), (dict(table_pages=0), -1, "block table"),
    (dict(table_pages=1 << 27), -1, "block table"), (dict(table_stride=3), -1, "stride"), (dict(table_in_stride=3), -1, "stride"),
    (dict(table_stride=-4), -1, "stride"), (dict(free_capacity=-1), -1, "free_capacity"), (dict(free_capacity=1 << 31), -1, "free_capacity"),
    (dict(mask_words=0), -1, "mask_words"), (dict(mask_words=17), -1, "mask_words"), (dict(mask=None), -1, "mask_words"),
    (dict(mask=BASE + 16 * GIB + 4), -2, "mask"), (dict(slots=BASE + 15 * GIB + 4), -2, "slots"),
    (dict(table=BASE + GIB + 16), -1, "table overlaps table_in"), (dict(table=BASE + GIB, table_stride=5), -1, "table overlaps table_in"),
    (dict(held=BASE + 2 * GIB), -1, "held overlaps held_in"), (dict(context_len=BASE + 3 * GIB), -1, "context_len overlaps past_len"),
    (dict(free_left=BASE + 6 * GIB), -1, "free_left overlaps free_count"), (dict(positions=BASE + 7 * GIB), -1, "positions overlaps parents"),
    (dict(query_start=BASE + 11 * GIB - 12), -1, "query_start overlaps context_len"), (dict(slots=BASE + 16 * GIB - 32), -1, "slots overlaps mask"),
    (dict(held=BASE + GIB), -1, "held overlaps table_in"), (dict(table=BASE + 5 * GIB), -1, "table overlaps free_pages"),
] + [(dict([(n, None)]), -1, n) for n in POINTERS if n not in ("parents", "mask")]
  + [(dict([(n, BASE + STEP[n] * GIB + 2)]), -2, n) for n in POINTERS])
def test_assign_refusals(lib, over, want, text):
    refused(lib, lib.q4_kv_assign(ref(step(**over)), None), want, text)


def test_assign_without_free_pages_needs_no_list(lib):
    """No free pages at all: no list (the call fails on another argument only)."""
    refused(lib, lib.q4_kv_assign(ref(step(free_pages=None, free_capacity=0, held=None)), None), -1, "null held")
    refused(lib, lib.q4_kv_assign(None, None), -1, "null step")


GAIN = BASE + 72 * GIB


@pytest.mark.parametrize("over,want,text", [
    (dict(tokens=0), -1, "tokens"), (dict(heads=0), -1, "heads"), (dict(dim=1026), -1, "head_dim"), (dict(rot=3), -1, "rot_dim"),
    (dict(rot=130), -1, "rot_dim"), (dict(layout=2), -1, "layout"), (dict(mscale=math.nan), -1, "mscale"), (dict(pos=None), -1, "positions"),
    (dict(pos=POS + 2), -2, "positions"), (dict(freq=None), -1, "inv_freq"), (dict(eps=-1e-6), -1, "eps"), (dict(eps=math.nan), -1, "eps"),
    (dict(eps=math.inf), -1, "eps"), (dict(gain_type=5), -1, "gains"), (dict(gain=GAIN + 1), -2, "gains"),
    (dict(gain=GAIN + 2, gain_type=2), -2, "gains"), (dict(x=None), -1, "null x"), (dict(out=heads(2)), -1, "overlaps x"),
    (dict(out=heads(72 * GIB - 256)), -1, "overlaps the gain"), (dict(out=heads(70 * GIB)), -1, "overlaps positions"),
])
def test_norm_rope_refusals(lib, over, want, text):
    a = dict(x=heads(0), out=heads(GIB), gain=GAIN, gain_type=0, eps=1e-6, pos=POS, freq=FREQ, tokens=5, heads=8, dim=128, rot=128,
             layout=0, mscale=1.0)
    a.update(over)
    st = lib.q4_norm_rope(ref(a["x"]), ref(a["out"]), a["gain"], a["gain_type"], a["eps"], a["pos"], a["freq"], a["tokens"], a["heads"],
                          a["dim"], a["rot"], a["layout"], a["mscale"], None)
    refused(lib, st, want, text)


@pytest.mark.parametrize("over,want,text", CACHE_REFUSALS + [
    (dict(tokens=0), -1, "tokens"), (dict(k=None), -1, "null k"), (dict(q=None), -1, "go together"), (dict(eps=math.inf), -1, "eps"),
    (dict(gain_type=9), -1, "gains"), (dict(k_gain=GAIN + 1), -2, "gains"), (dict(q_out=heads(72 * GIB - 1024)), -1, "q_out overlaps"),
    (dict(q_out=heads(73 * GIB - 1024)), -1, "q_out overlaps"), (dict(cache=cache(v=BASE + 16 * GIB)), -1, "same memory"),
    (dict(q_gain=BASE + 16 * GIB), -1, "overlaps an input"), (dict(k_gain=BASE + 32 * GIB), -1, "overlaps an input"),
])
def test_append_norm_refusals(lib, over, want, text):
    a = dict(cache=cache(), batch=batch(), k=heads(GIB, 2), v=heads(2 * GIB, 2), q=heads(3 * GIB), q_out=heads(4 * GIB),
             tokens=5, q_gain=GAIN, k_gain=GAIN + GIB, gain_type=0, eps=1e-6)
    a.update(over)
    st = lib.q4_kv_append_norm(ref(a["cache"]), ref(a["batch"]), ref(a["k"]), ref(a["v"]), ref(a["q"]), ref(a["q_out"]), 8,
                               a["tokens"], a["q_gain"], a["k_gain"], a["gain_type"], a["eps"], None, FREQ, 128, 0, 1.0, None)
    refused(lib, st, want, text)


MASK = BASE + 74 * GIB


@pytest.mark.parametrize("over,want,text", CACHE_REFUSALS + [
    (dict(mask=None), -1, "null mask"), (dict(mask=MASK + 4), -2, "mask"), (dict(words=0), -1, "mask_words"), (dict(words=17), -1, "mask_words"),
    (dict(cache=cache(head_dim=80)), -1, "head_dim"), (dict(q_heads=7), -1, "multiple of kv_heads"), (dict(tokens=0), -1, "tokens"),
    (dict(q=None), -1, "null q"), (dict(q=heads(GIB + 8)), -2, "16-byte"), (dict(scale=0.0), -1, "scale"), (dict(window=-1), -1, "window"),
    (dict(out=heads(GIB)), -1, "overlaps an input"), (dict(out=heads(74 * GIB - 1024)), -1, "overlaps the mask"),
    (dict(lse=MASK), -1, "overlaps the mask"), (dict(workspace=MASK - 256), -1, "overlaps the mask"),
    (dict(workspace=None), -3, "workspace"), (dict(out=heads(65 * GIB)), -1, "overlaps the batch"),
])
def test_attention_tree_refusals(lib, over, want, text):
    a = dict(cache=cache(), batch=batch(table_pages=2000, table_stride=2000, max_context=32000, max_query=5), q=heads(GIB), out=heads(2 * GIB),
             mask=MASK, words=1, lse=None, q_heads=8, tokens=5, scale=0.1, window=0, workspace=BASE + 80 * GIB)
    a.update(over)
    st = lib.q4_attention_tree(ref(a["cache"]), ref(a["batch"]), ref(a["q"]), ref(a["out"]), a["mask"], a["words"], a["lse"], a["q_heads"],
                               a["tokens"], a["scale"], a["window"], a["workspace"], GIB, None)
    refused(lib, st, want, text)


RULES = dict(seqs=3, query_start=20, history=21, history_stride=100, history_tokens=100, history_len=22, prompt_len=23, draft=24, mask=25,
             mask_words=1, repetition=26, presence=27, frequency=28, bias_start=29, bias_tokens=30, bias_values=31, biases=4, allowed=32,
             allowed_stride=300, allowed_rows=5, allowed_row=33)
RULE_POINTERS = [n for n, t in q4.RulesDesc._fields_ if t is ctypes.c_void_p]


def rules(**over):
    f = {n: BASE + v * GIB if n in RULE_POINTERS else v for n, v in RULES.items()}
    f.update(over)
    return q4.RulesDesc(**f)


@pytest.mark.parametrize("over,want,text", [
    (dict(rows=0), -1, "rows"), (dict(rows=1 << 25), -1, "rows"), (dict(vocab=0), -1, "vocab"), (dict(vocab=1 << 25), -1, "vocab"),
    (dict(type=3), -1, "type"), (dict(stride=-1), -1, "stride"), (dict(out_stride=8000), -1, "overlap each other"),
    (dict(logits=None), -1, "logits"), (dict(tokens=None), -1, "tokens"), (dict(logits=BASE + 2), -2, "logits"), (dict(out=BASE + GIB + 1), -2, "out"),
    (dict(tokens=BASE + 2 * GIB + 2), -2, "tokens"), (dict(workspace=None), -3, "workspace"), (dict(bytes=7), -3, "workspace"),
    (dict(workspace=BASE + 3 * GIB + 4), -2, "workspace"), (dict(out=BASE + 4), -1, "out overlaps logits"), (dict(out=BASE, out_stride=9100), -1, "out overlaps logits"),
    (dict(tokens=BASE + 16), -1, "tokens overlaps logits"), (dict(workspace=BASE + GIB), -1, "out overlaps workspace"),
    (dict(rules=rules(seqs=0)), -1, "seqs"), (dict(rules=rules(query_start=None)), -1, "without query_start"),
    (dict(rules=rules(history_len=None)), -1, "go together"), (dict(rules=rules(history=None)), -1, "go together"),
    (dict(rules=rules(history_tokens=0)), -1, "history_tokens"), (dict(rules=rules(history_stride=99)), -1, "history_stride"),
    (dict(rules=rules(history=None, history_len=None)), -1, "prompt_len without history"), (dict(rules=rules(draft=None)), -1, "a mask without draft"),
    (dict(rules=rules(mask_words=0)), -1, "mask_words"), (dict(rules=rules(mask=None)), -1, "mask_words"), (dict(rules=rules(mask_words=17)), -1, "mask_words"),
    (dict(rules=rules(biases=-1)), -1, "biases"), (dict(rules=rules(bias_values=None)), -1, "go together"), (dict(rules=rules(bias_start=None)), -1, "go together"),
    (dict(rules=rules(allowed_rows=0)), -1, "allowed_rows"), (dict(rules=rules(allowed=None)), -1, "allowed_row without allowed"),
    (dict(rules=rules(allowed_stride=-1)), -1, "allowed_stride"),
    (dict(rules=rules(history_stride=1 << 40, seqs=1 << 24)), -1, "reaches too far"),
] + [(dict(rules=rules(**{n: BASE + RULES[n] * GIB + 2})), -2, n) for n in RULE_POINTERS]
  + [(dict(rules=rules(**{n: BASE + GIB})), -1, "out overlaps " + n) for n in RULE_POINTERS]
  + [(dict(rules=rules(**{n: BASE + 2 * GIB})), -1, "tokens overlaps " + n) for n in RULE_POINTERS])
def test_logits_refusals(lib, over, want, text):
    a = dict(logits=BASE, type=2, stride=9000, rows=5, vocab=9000, rules=rules(), out=BASE + GIB, out_stride=9000, tokens=BASE + 2 * GIB,
             workspace=BASE + 3 * GIB, bytes=GIB)
    a.update(over)
    st = lib.q4_logits_argmax(a["logits"], a["type"], a["stride"], a["rows"], a["vocab"], ref(a["rules"]), a["out"], a["out_stride"], a["tokens"],
                              a["workspace"], a["bytes"], None)
    refused(lib, st, want, text)


def test_logits_workspace(lib):
    """None for rows of one slice, a key of 8 bytes for each slice of a row otherwise."""
    assert q4.logits_argmax_workspace_bytes(1, 1000) == 0
    assert q4.logits_argmax_workspace_bytes(1, 151936) >= 8 * (151936 // 8192)
    assert q4.logits_argmax_workspace_bytes(0, 1000) == 0 and q4.logits_argmax_workspace_bytes(1, 1 << 25) == 0


ACCEPT = dict(query_start=1, context_len=2, choice=3, draft=4, parents=5, accepted=6, next=7, path=8, lens=9, history=10)


@pytest.mark.parametrize("over,want,text", [
    (dict(seqs=0), -1, "seqs"), (dict(seqs=1 << 25), -1, "seqs"), (dict(tokens=0), -1, "tokens"), (dict(history_tokens=0), -1, "history_tokens"),
    (dict(history_stride=3), -1, "history_stride"), (dict(history_stride=-1), -1, "history_stride"),
    (dict(path=BASE + 4 * GIB), -1, "path overlaps draft"), (dict(lens=BASE + 2 * GIB), -1, "lens overlaps context_len"),
    (dict(accepted=BASE + 7 * GIB), -1, "accepted overlaps next"), (dict(history=BASE + 4 * GIB), -1, "history overlaps draft"),
] + [(dict([(n, None)]), -1, n) for n in ACCEPT if n not in ("parents", "history")] + [(dict([(n, BASE + v * GIB + 2)]), -2, n) for n, v in ACCEPT.items()])
def test_accept_refusals(lib, over, want, text):
    a = {n: BASE + v * GIB for n, v in ACCEPT.items()}
    a.update(dict(seqs=3, tokens=9, history_stride=40, history_tokens=40))
    a.update(over)
    st = lib.q4_tree_accept(a["query_start"], a["context_len"], a["seqs"], a["choice"], a["draft"], a["parents"], a["tokens"], a["accepted"],
                            a["next"], a["path"], a["lens"], a["history"], a["history_stride"], a["history_tokens"], None)
    refused(lib, st, want, text)


def layers(*descs):
    return (q4.CacheDesc * len(descs))(*descs)


FAR = dict(k=BASE + 17 * GIB, v=BASE + 33 * GIB)  # a second layer beside cache()


@pytest.mark.parametrize("over,want,text", [(dict(caches=layers(o["cache"])) if o.get("cache") else o, w, t)
                                            for o, w, t in CACHE_REFUSALS if o.get("cache", 1) is not None] + [
    (dict(caches=None), -1, "null cache"), (dict(layers=0), -1, "layers"), (dict(layers=513), -1, "layers"), (dict(tokens=0), -1, "tokens"),
    (dict(path=None), -1, "path"), (dict(path=BASE + 2), -2, "path"), (dict(accepted=None), -1, "accepted"),
    (dict(caches=layers(cache(), cache(pages=11, **FAR))), -1, "same sizes"), (dict(caches=layers(cache(), cache(k_page_stride=1 << 13, **FAR))), -1, "same sizes"),
    (dict(caches=layers(cache(), cache(type=1, **FAR))), -1, "same sizes"), (dict(caches=layers(cache(), cache())), -1, "same memory"),
    (dict(caches=layers(cache(), cache(k=BASE + 32 * GIB, v=BASE + 48 * GIB))), -1, "same memory"),
    (dict(caches=layers(cache(), cache(k=None, v=BASE))), -1, "null cache"), (dict(path=BASE + 16 * GIB), -1, "overlaps an input"),
    (dict(caches=layers(cache(), cache(k=BASE + 17 * GIB, v=BASE + 16 * GIB + 256))), -1, "same memory"),
    (dict(caches=layers(cache(k_head_stride=0))), -1, "overlap each other"),
])
def test_move_refusals(lib, over, want, text):
    a = dict(caches=layers(cache(), cache(**FAR)), batch=batch(), path=BASE, accepted=BASE + GIB, tokens=5)
    a.update(over)
    n = a.get("layers", len(a["caches"]) if a["caches"] is not None else 1)
    refused(lib, lib.q4_kv_move(a["caches"], n, ref(a["batch"]), a["path"], a["accepted"], a["tokens"], None), want, text)


def test_layers_of_one_tensor_are_apart(lib):
    """Layers, or keys and values, side by side in each page of one tensor: their spans overlap, they do not (the call
    fails on the path only)."""
    hk, page, dim = 2, 16, 128
    one = hk * page * dim
    wide = dict(k_page_stride=4 * one, v_page_stride=4 * one)
    at = BASE + 16 * GIB
    both = layers(*(cache(k=at + 4 * i * one, v=at + 4 * i * one + 2 * one, **wide) for i in range(2)))
    refused(lib, lib.q4_kv_move(both, 2, ref(batch()), None, BASE, 5, None), -1, "null path")
    q4.last_error()
    close = layers(*(cache(k=at + 4 * i * one - 16 * i, v=at + 4 * i * one + 2 * one, **wide) for i in range(2)))
    refused(lib, lib.q4_kv_move(close, 2, ref(batch()), BASE, BASE + GIB, 5, None), -1, "same memory")


def test_many_layers_of_one_tensor(lib):
    """Keys and values of 40 layers side by side in each page, in any order and over two tensors: none meet, and any
    block moved into a neighbour (the last one's is the first one's next page) does."""
    hk, page, dim = 2, 16, 128
    one = 2 * hk * page * dim  # bytes
    wide = dict(k_page_stride=40 * one // 2, v_page_stride=40 * one // 2)
    tensors = (BASE + 16 * GIB + 2, BASE + 17 * GIB)  # 20 layers each
    for seed in range(8):
        rng = random.Random(seed)
        places = [t + i * one for t in tensors for i in range(40)]
        rng.shuffle(places)
        at = rng.randrange(80)
        for shift in (0, 2, -2, one - 2, 2 - one):
            moved = list(places)
            moved[at] += shift
            caches = layers(*(cache(k=moved[2 * i], v=moved[2 * i + 1], **wide) for i in range(40)))
            if shift:
                refused(lib, lib.q4_kv_move(caches, 40, ref(batch()), BASE, BASE + GIB, 5, None), -1, "same memory")
            else:
                refused(lib, lib.q4_kv_move(caches, 40, ref(batch()), None, BASE, 5, None), -1, "null path")


def test_python_checks():
    """Shapes, types and places that the Python layer refuses before any call."""
    cpu = torch.zeros(3, 4)
    with pytest.raises(ValueError):
        q4.q4_logits_argmax(cpu)
    with pytest.raises(ValueError):
        q4.q4_norm_rope(torch.zeros(1, 1, 8), None)
    with pytest.raises(ValueError):
        q4.KVLayers([])
    with pytest.raises(ValueError):
        q4.KVStep(0, 4, 16, 5, device="cpu")
    with pytest.raises(ValueError):
        q4.LogitRules(presence=torch.zeros(3))
    with pytest.raises(TypeError):
        q4.LogitRules(presence=[0.0])
