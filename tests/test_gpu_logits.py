"""q4_logits_argmax against the same rules row by row on the host: bit for bit where each step is rounded to binary32, and
within those roundings of the formula in 64 bits."""
import math

import numpy as np
import pytest
import torch

import step_ref
from gpu_util import lib, say

pytestmark = pytest.mark.gpu


def make(seqs, rows_of, vocab, seed, tree=None, history=True, biases=5, grammar=True, allowed_rows=False, penalties=True, length=40, start=None):
    rng = np.random.default_rng(seed)
    rows = sum(rows_of)
    over = {}
    if start is not None or rows_of != [1] * seqs:
        over["query_start"] = np.concatenate([[0], np.cumsum(rows_of)]).astype(np.int32) if start is None else np.asarray(start, np.int32)
    if history:
        over["history"] = rng.integers(-2, vocab + 2, (seqs, length)).astype(np.int32)
        over["history"][:, : length // 2] = rng.integers(0, min(vocab, 7), (seqs, length // 2))
        over["history_lens"] = rng.integers(0, length + 5, seqs).astype(np.int32)
        over["history_lens"][0] = length
        over["prompt_lens"] = rng.integers(0, length, seqs).astype(np.int32)
    if tree is not None:
        over["draft"] = rng.integers(0, min(vocab, 9), rows).astype(np.int32)
        if tree:
            over["mask"] = step_ref.mask_rows([step_ref.tree(n, rng) for n in rows_of], tree).numpy()
    if penalties:
        over["repetition"] = rng.uniform(1.0, 2.0, seqs).astype(np.float32)
        over["presence"], over["frequency"] = (rng.uniform(-1.0, 2.0, seqs).astype(np.float32) for _ in range(2))
    if biases:
        over["bias_start"] = np.concatenate([[0], np.cumsum(rng.integers(0, biases + 1, seqs))]).astype(np.int32)
        n = int(over["bias_start"][-1])
        over["bias_tokens"] = rng.integers(-1, min(vocab, 12) + 1, n).astype(np.int32)  # equal ones among them
        over["bias_values"] = rng.normal(0, 5, n).astype(np.float32)
    words = -(-vocab // 32)
    if grammar:
        held = 3 if allowed_rows else rows
        over["allowed"] = rng.integers(-2 ** 31, 2 ** 31, (held, words)).astype(np.int32)
        if allowed_rows:
            over["allowed_rows"] = rng.integers(-1, 4, rows).astype(np.int32)
    return step_ref.Rules(seqs, **over)


def check(q4, logits, rules, with_out=True):
    rows, vocab = logits.shape
    dev = logits.cuda()
    out = torch.full((rows, vocab), 55.0, device="cuda") if with_out else None
    tokens = torch.full((rows,), -77, dtype=torch.int32, device="cuda")
    q4.q4_logits_argmax(dev, rules.device(q4), out=out, tokens=tokens)
    torch.cuda.synchronize()
    host, got = logits.float().numpy(), tokens.tolist()
    for t in range(rows):
        want = rules.apply(host, t)
        if want is None:
            assert got[t] == -77 and (out is None or bool((out[t] == 55.0).all()))
            continue
        assert got[t] == rules.pick(want), t
        if out is not None:
            o = out[t].cpu().numpy()
            assert np.array_equal(np.isnan(o), np.isnan(want))
            assert np.array_equal(o[~np.isnan(o)], want[~np.isnan(want)]), t
    return out, tokens


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("vocab", [1, 3, 31, 33, 1000, 1023, 1025, 4099, 32003, 151936])
def test_vocabularies(vocab, dtype):
    """One row and a few, every rule at once, vocabularies that end inside words, vectors and slices."""
    q4 = lib()
    for seqs in (1, 3):
        rules = make(seqs, [1] * seqs, vocab, vocab)
        logits = (3 * torch.randn(seqs, vocab, generator=torch.Generator().manual_seed(vocab))).to(dtype)
        say("logits", seqs, vocab, dtype)
        check(q4, logits, rules)


@pytest.mark.parametrize("over", [dict(history=False, biases=0, grammar=False, penalties=False), dict(biases=0), dict(history=False), dict(penalties=False),
                                  dict(grammar=False), dict(allowed_rows=True), dict(history=False, biases=0), dict(history=False, biases=400, length=40),
                                  dict(length=3000), dict(length=1)])
@pytest.mark.parametrize("tree", [None, 0, 1, 2])
def test_rules(over, tree):
    """Rules left out, in every combination of lists; rows of single tokens, chains and trees of sequences of which some
    have none."""
    q4 = lib()
    rows_of = [1] * 6 if tree is None else [5, 0, 1, 70, 9, 64]
    rules = make(6, rows_of, 5003, 3, tree=tree, **over)
    logits = 3 * torch.randn(sum(rows_of), 5003, generator=torch.Generator().manual_seed(1))
    check(q4, logits, rules)
    check(q4, logits, rules, with_out=False)


@pytest.mark.parametrize("rows,vocab", [(1, 9000), (40, 60000), (100, 60000), (400, 20000), (1100, 900), (300, 8192)])
def test_slices(rows, vocab):
    """Rows and vocabularies for every length of a slice."""
    q4 = lib()
    rules = make(rows, [1] * rows, vocab, rows)
    logits = torch.randn(rows, vocab, generator=torch.Generator().manual_seed(2))
    check(q4, logits, rules)


def test_against_the_formula():
    """Within the roundings of the formula in 64 bits: each of the up to five steps rounds once, by 2^-24 of what it has."""
    q4 = lib()
    rules = make(4, [1] * 4, 3001, 8, biases=300, length=400)
    logits = 3 * torch.randn(4, 3001)
    out, _ = check(q4, logits, rules)
    for t in range(4):
        exact = rules.apply(logits.numpy(), t, np.float64)
        on = np.isfinite(exact)
        # no step has more than |x| repetition + frequency count + presence + bias
        size = 2 * np.abs(logits[t].numpy()) + 2 * 400 + 2 + 25
        assert np.array_equal(np.isfinite(out[t].cpu().numpy()), on)
        assert bool((np.abs(out[t].cpu().numpy()[on] - exact[on]) <= 5 * 2.0 ** -24 * size[on]).all())


def test_ties_and_nothing_left():
    """Ties go to the lowest index, over slices too; -0 and +0 are equal; NaN and -infinity are never picked; rows where
    nothing is left give -1; +infinity wins."""
    q4 = lib()
    v = 20000
    x = torch.full((9, v), -1.0)
    x[0, [19999, 8192, 77]] = 4.0
    x[1, 5], x[1, 3000] = -0.0, 0.0
    x[2] = float("nan")
    x[3] = -float("inf")
    x[4] = float("nan")
    x[4, 15000] = -3e38
    x[5, 9], x[5, 18000] = float("inf"), float("inf")
    x[6] = torch.finfo(torch.float32).min
    x[7, 12000] = 1.0
    x[7, 12001] = float("nan")
    assert q4.q4_logits_argmax(x.cuda()).tolist() == [77, 5, -1, -1, 15000, 9, 0, 12000, 0]
    assert q4.q4_logits_argmax(x[8].expand(3, v).cuda()).tolist() == [0, 0, 0]  # one row for all
    words = -(-v // 32)
    allowed = torch.zeros(9, words, dtype=torch.int32)
    allowed[8, 300] = -2 ** 31
    allowed[7, 375] = 3  # 12000, 12001
    got = q4.q4_logits_argmax(x.cuda(), q4.LogitRules(allowed=allowed.cuda()))
    assert got.tolist() == [-1] * 7 + [12000, 9631]
    bias = q4.LogitRules(bias_start=torch.tensor([0, 2], dtype=torch.int32, device="cuda"), bias_tokens=torch.tensor([4, 9], dtype=torch.int32, device="cuda"),
                         bias_values=torch.tensor([-math.inf, math.inf], device="cuda"))
    assert q4.q4_logits_argmax(torch.zeros(1, v, device="cuda"), bias).tolist() == [9]
    assert q4.q4_logits_argmax(torch.zeros(0, v, device="cuda")).shape == (0,)


def test_in_place_and_strides():
    """out is the logits themselves; rows that lie apart, at odd places; a workspace of the caller's."""
    q4 = lib()
    rules = make(5, [1] * 5, 4001, 4)
    logits = 2 * torch.randn(5, 4001)
    want, tokens = check(q4, logits, rules)
    for width, at in ((4001, 0), (4005, 3), (5000, 1)):
        wide = torch.zeros(5, width, device="cuda")
        part = wide[:, at : at + 4001]
        part.copy_(logits)
        rest = wide.clone()
        out = torch.zeros(5, 4013, device="cuda")[:, 5:4006]
        ws = torch.full((q4.logits_argmax_workspace_bytes(5, 4001),), 0xAB, dtype=torch.uint8, device="cuda")
        assert torch.equal(q4.q4_logits_argmax(part, rules.device(q4), out=out, workspace=ws), tokens)
        assert torch.equal(out, want) and torch.equal(wide, rest)
        q4.q4_logits_argmax(part, rules.device(q4), out=part)
        assert torch.equal(part, want)
        wide[:, at : at + 4001] = rest[:, at : at + 4001]
        assert torch.equal(wide, rest)


def test_rows_outside():
    """Rows in front of the first sequence and behind the last are left as they are."""
    q4 = lib()
    rng = np.random.default_rng(1)
    rules = step_ref.Rules(3, query_start=np.array([2, 4, 4, 7], np.int32), history=rng.integers(0, 900, (3, 20)).astype(np.int32),
                           history_lens=np.array([20, 3, 11], np.int32), presence=np.array([1, 2, 3], np.float32), draft=rng.integers(0, 900, 9).astype(np.int32))
    check(q4, torch.randn(9, 900), rules)
    rules.draft = np.concatenate([rules.draft, rules.draft])
    check(q4, torch.randn(18, 9000), rules)


def test_captured_with_new_lists():
    """A graph replayed with other logits, texts, lengths and grammars in the same tensors, eager calls in between."""
    q4 = lib()
    vocab, seqs = 30011, 4
    sets = [make(seqs, [1] * seqs, vocab, s, length=60, biases=9) for s in range(4)]
    logits = [3 * torch.randn(seqs, vocab, generator=torch.Generator().manual_seed(s)) for s in range(4)]
    names = ("history", "history_lens", "prompt_lens", "repetition", "presence", "frequency", "allowed")
    fixed = {n: torch.as_tensor(getattr(sets[0], n)).cuda() for n in names}
    x, out = torch.zeros(seqs, vocab, device="cuda"), torch.zeros(seqs, vocab, device="cuda")
    tokens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    rules = q4.LogitRules(**fixed)
    q4.q4_logits_argmax(x, rules, out=out, tokens=tokens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q4.q4_logits_argmax(x, rules, out=out, tokens=tokens)
    for r, l in zip(sets, logits):
        r.bias_start = r.bias_tokens = r.bias_values = None
        for n in names:
            fixed[n].copy_(torch.as_tensor(getattr(r, n)))
        x.copy_(l)
        graph.replay()
        torch.cuda.synchronize()
        for t in range(seqs):
            want = r.apply(l.numpy(), t)
            assert np.array_equal(out[t].cpu().numpy(), want) and int(tokens[t]) == r.pick(want)
        check(q4, l, r)


def test_many_rows():
    """More rows than a launch has along an axis, some of them without anything allowed."""
    q4 = lib()
    rows, vocab = 70001, 40
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(rows, vocab, device="cuda", generator=g)
    allowed = torch.randint(-2 ** 31, 2 ** 31, (rows, 2), device="cuda", generator=g).to(torch.int32)
    allowed[::1000] = 0
    open_ = (allowed.repeat_interleave(32, 1)[:, :vocab] >> (torch.arange(vocab, device="cuda") % 32)) & 1
    want = torch.where(open_.bool(), x, -math.inf)
    out = torch.zeros_like(x)
    tokens = q4.q4_logits_argmax(x, q4.LogitRules(allowed=allowed), out=out)
    assert torch.equal(out, want)
    assert torch.equal(tokens, torch.where(want.amax(1) > -math.inf, want.argmax(1), -1).int())
    y = torch.randn(66000, 2100, device="cuda", generator=g)  # and of two slices
    assert torch.equal(q4.q4_logits_argmax(y), y.argmax(1).int())


def test_far_rows():
    """Rows whose offsets pass 2^32 bytes, read and written."""
    q4 = lib()
    stride, vocab = (1 << 30) + 32, 9001
    flat = torch.zeros(2 * stride + vocab, dtype=torch.float16, device="cuda")
    x = flat.as_strided((3, vocab), (stride, 1))
    y = torch.randn(3, vocab, generator=torch.Generator().manual_seed(1)).half().cuda()
    x.copy_(y)
    far = torch.zeros(2 * stride + vocab, device="cuda")
    out = far.as_strided((3, vocab), (stride, 1))
    presence = torch.ones(3, device="cuda")
    history = y.argmax(1, keepdim=True).int()
    tokens = q4.q4_logits_argmax(x, q4.LogitRules(history=history, history_lens=torch.ones(3, dtype=torch.int32, device="cuda"), presence=presence), out=out)
    want = y.float().scatter_add(1, history.long(), -presence[:, None])
    assert torch.equal(out, want) and torch.equal(tokens, want.argmax(1).int())


def test_two_streams():
    """Two calls at once, each with its own workspace and rules."""
    q4 = lib()
    jobs = []
    for seed in range(2):
        r = make(6, [1] * 6, 50021, seed, length=300, biases=20)
        x = torch.randn(6, 50021, generator=torch.Generator().manual_seed(seed))
        out, tokens = check(q4, x, r)
        jobs.append((x.cuda(), r.device(q4), out, tokens, torch.cuda.Stream(),
                     torch.empty(q4.logits_argmax_workspace_bytes(6, 50021), dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    got = [[torch.empty_like(j[2]) for _ in range(10)] for j in jobs]
    picks = [[], []]
    torch.cuda.synchronize()
    for n in range(10):
        for i, (x, r, _, _, stream, ws) in enumerate(jobs):
            picks[i].append(q4.q4_logits_argmax(x, r, out=got[i][n], workspace=ws, stream=stream))
    torch.cuda.synchronize()
    for i, j in enumerate(jobs):
        assert all(torch.equal(o.view(torch.int32), j[2].view(torch.int32)) for o in got[i]) and all(torch.equal(p, j[3]) for p in picks[i])


def test_no_sequences_are_refused():
    q4 = lib()
    zero, none = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(0, device="cuda")
    for over in (dict(query_start=zero), dict(repetition=none), dict(bias_start=zero, bias_tokens=zero, bias_values=torch.zeros(1, device="cuda")),
                 dict(allowed=torch.zeros(2, 2, dtype=torch.int32, device="cuda"), seqs=0)):
        with pytest.raises(ValueError):
            q4.LogitRules(**over)


def test_quotients():
    """Logits and repetitions of every size, results that overflow or have few bits among them: each quotient and product
    is rounded once."""
    q4 = lib()
    rng = np.random.default_rng(5)
    seqs, vocab = 40, 5003
    x = torch.from_numpy(rng.integers(0, 2 ** 32, (seqs, vocab), dtype=np.uint64).astype(np.uint32).view(np.float32))
    repetition = np.abs(rng.integers(1, 0x7F800000, seqs).astype(np.uint32).view(np.float32))
    repetition[:8] = np.array([1.0, 1.1, 3.0, 2.0 ** -140, 1.17549435e-38, 3.4e38, 1 - 2.0 ** -24, 0.75], np.float32)
    x[8:16] = torch.from_numpy((np.float32(2.0 ** -126) * rng.uniform(0.25, 4.0, (8, vocab))).astype(np.float32))  # around the normal ones' end
    repetition[8:16] = np.array([2.0, 4.0, 1.5, 0.5, 1.0, 1.0 + 2.0 ** -23, 3.0, 8.0], np.float32)
    with np.errstate(all="ignore"):
        check(q4, x, step_ref.Rules(seqs, history=np.tile(np.arange(vocab, dtype=np.int32), (seqs, 1)), history_lens=np.full(seqs, vocab, np.int32),
                                    repetition=repetition))


def test_many_biases():
    """More biases in a row than a workgroup has threads, most tokens several times; some rows with just as many, and
    biases of zero."""
    q4 = lib()
    rng = np.random.default_rng(6)
    for vocab in (700, 20011):
        counts = [2000, 512, 513, 0, 511, 5000]
        start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        values = rng.normal(0, 5, start[-1]).astype(np.float32)
        values[::3] = 0.0
        values[1::7] = rng.integers(0, 9, len(values[1::7])).astype(np.uint32).view(np.float32)  # bits like small places
        check(q4, torch.randn(6, vocab), step_ref.Rules(6, bias_start=start, bias_tokens=rng.integers(-2, vocab + 2, start[-1]).astype(np.int32),
                                                        bias_values=values, history=rng.integers(0, vocab, (6, 30)).astype(np.int32),
                                                        history_lens=np.full(6, 30, np.int32), presence=np.ones(6, np.float32)))
