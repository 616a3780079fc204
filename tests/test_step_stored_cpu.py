"""Refusals of q4_tree_accept_stored: every call here fails on the host before anything would be enqueued, with made-up
addresses."""
import pytest

from test_kv_cpu import BASE, GIB, lib, refused  # noqa: F401

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
