"""Refusals of q4_tree_accept_stored, and workspaces made for the largest call: every call here fails on the host before
anything would be enqueued, with made-up addresses."""
import pytest
import torch

import q4_dequant_gemv_block_amd as q4
from test_kv_cpu import BASE, GIB, batch, cache, lib, ref, refused  # noqa: F401

NAMES = dict(query_start=1, context_len=2, choice=3, draft=4, parents=5, accepted=6, next=7, path=8, lens=9, history=10, slots=11)
OUTPUTS = ("accepted", "next", "path", "lens", "history")


@pytest.mark.parametrize("over,want,text", [
    (dict(seqs=0), -1, "seqs"), (dict(tokens=0), -1, "tokens"), (dict(history_stride=3), -1, "history_stride"),
    (dict(slots=BASE + 11 * GIB + 4), -2, "slots"), (dict(slots=BASE + 4 * GIB, draft=None), -1, "null draft"),
] + [(dict([(n, None)]), -1, n) for n in NAMES if n not in ("parents", "history", "slots")]
  + [(dict([(n, BASE + v * GIB + 2)]), -2, n) for n, v in NAMES.items()]
  + [(dict([(n, BASE + 11 * GIB + 68)]), -1, n + " overlaps slots") for n in OUTPUTS])
def test_refusals(lib, over, want, text):
    a = {n: BASE + v * GIB for n, v in NAMES.items()}
    a.update(dict(seqs=3, tokens=9, history_stride=40, history_tokens=40))
    a.update(over)
    st = lib.q4_tree_accept_stored(a["query_start"], a["context_len"], a["seqs"], a["choice"], a["draft"], a["parents"], a["slots"],
                                   a["tokens"], a["accepted"], a["next"], a["path"], a["lens"], a["history"], a["history_stride"],
                                   a["history_tokens"], None)
    refused(lib, st, want, text)


def enough_for_logits(lib, rows, vocab, given):
    """Whether a workspace of `given` bytes serves a call (which then fails on its rules)."""
    st = lib.q4_logits_argmax(BASE, q4.Q4_TYPE_F32, vocab, rows, vocab, ref(q4.RulesDesc(seqs=0)), None, 0, BASE - GIB, BASE - 64 * GIB, given,
                              None)
    assert st == -3 or (st == -1 and "seqs" in q4.last_error()), q4.last_error()
    return st == -1


@pytest.mark.parametrize("vocab", [1, 2048, 2049, 8192, 8193, 32000, 50021, 151936, 1 << 24])
def test_a_logits_workspace_serves_fewer_rows(lib, vocab):
    """A workspace for so many rows and entries serves every call of fewer rows, or fewer entries."""
    sizes = [*range(1, 70), 127, 128, 129, 255, 256, 257, 511, 512, 513, 1000, 4097, 70001]
    for rows in sizes:
        given = q4.logits_argmax_workspace_bytes(rows, vocab)
        assert given >= q4.logits_argmax_workspace_bytes(max(rows - 1, 1), vocab)
        for fewer in sizes:
            if fewer <= rows:
                for v in (vocab, vocab // 2, vocab // 3, 9000, 2049):
                    assert not 1 <= v <= vocab or enough_for_logits(lib, fewer, v, given), (rows, fewer, v)


SIZES = [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 24, 31, 32, 33, 40, 63, 64, 65, 100, 127, 128, 129, 200, 513, 2048, 9000]


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("q_heads", [2, 8, 14, 40])
def test_an_attention_workspace_serves_fewer_tokens(lib, dim, q_heads):
    """attention_workspace_most covers every batch of up to so many new tokens, whatever its sequences, lengths, hints and
    window, of both kinds of attention, and is no more than the most that one of them takes."""
    c = cache(head_dim=dim, pages=9000)
    most = {n: lib.q4_attention_workspace_most(ref(c), q_heads, n) for n in SIZES}
    needed = 0
    for n in SIZES:
        for pages in (1, 4, 40, 400, 4000):
            for seqs in (1, 2, 3, 16, 64, 65, 300):
                for query in (0, 1, n // 2, n):
                    for context in (0, pages * 9):
                        for window in (0, 100, 4000):
                            b = batch(table_pages=pages, table_stride=pages, seqs=seqs, max_query=query, max_context=context)
                            for fn in (lib.q4_attention_paged_workspace_bytes, lib.q4_attention_tree_workspace_bytes):
                                needed = max(needed, fn(ref(c), ref(b), q_heads, n, window))
        assert needed <= most[n], n  # of this many or fewer
    assert needed == most[SIZES[-1]]
    assert lib.q4_attention_workspace_most(ref(c), q_heads, 0) == 0 and "tokens" in q4.last_error()
    assert lib.q4_attention_workspace_most(ref(c), 7, 4) == 0 and "multiple of kv_heads" in q4.last_error()
    assert lib.q4_attention_workspace_most(ref(cache(head_dim=80)), q_heads, 4) == 0 and "head_dim" in q4.last_error()
    assert lib.q4_attention_workspace_most(None, q_heads, 4) == 0 and "null cache" in q4.last_error()


def test_masks_have_words():
    """A mask of no words is refused; it would be as none at all, by which rows see every drafted token up to their own."""
    for words in (1, 16):
        q4._mask(torch.zeros(3, words, dtype=torch.int64), 3, -1)
    with pytest.raises(ValueError, match="words"):
        q4._mask(torch.zeros(3, 0, dtype=torch.int64), 3, -1)
