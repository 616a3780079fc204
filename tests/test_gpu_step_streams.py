"""The operators of a step with drafted trees on a stream that is not the current one, behind work there that has yet to
make their inputs: nothing but the launch itself comes after that work is queued, and nothing but that stream is waited
for."""
import pytest
import torch

from gpu_util import lib, say

pytestmark = pytest.mark.gpu
NAMES = ("assign", "norm", "append", "tree", "pick", "accept", "move")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(q4, name):
    """The input that the stream makes, and a function that makes what else a call needs and gives the call itself, which
    returns what it writes."""
    g = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    freq, _ = q4.rope_frequencies(128)
    table, start, ctx = i32([[3, 1, 0], [2, 5, 4]]), i32([0, 5, 9]), i32([40, 44])
    batch = q4.KVBatch(table, start, ctx)
    base = [n(6, 2, 16, 128).half() for _ in range(2)]
    history = torch.randint(0, 30000, (2, 50), device="cuda", generator=g, dtype=torch.int32)
    mask = torch.tensor([1, 3, 7, 11, 19, 1, 3, 7, 15], device="cuda").view(9, 1)

    def assign():
        step, left, count = q4.KVStep(2, 3, 16, 9, 1), i32([9, 8, 7, 6]), i32([4])
        written = [step.block_table, step.held, step.query_start, step.context_lens, step.missing, step.free_count, step.positions, step.slots, step.mask]
        return lambda x, **on: [q4.q4_kv_assign(step, table, x[0], x[1], x[2], left, count, **on)] and written

    def norm():
        pos = i32(range(9))
        return lambda x, **on: [q4.q4_norm_rope(x, None, 1e-6, pos, freq, **on)]

    def append():
        kv = [t.clone() for t in base]
        cache = q4.KVCache(*kv)
        return lambda x, **on: [q4.q4_kv_append_norm(cache, batch, x[:, 8:10], x[:, 10:], q=x[:, :8], inv_freq=freq, **on)] + kv

    def tree():
        cache = q4.KVCache(*base)
        return lambda x, **on: [q4.q4_attention_tree(cache, batch, x, mask, **on)]

    def pick():
        rules = q4.LogitRules(query_start=start, history=history, history_lens=i32([50, 20]), presence=torch.ones(2, device="cuda"))
        out = torch.zeros(9, 30000, device="cuda")
        return lambda x, **on: [q4.q4_logits_argmax(x, rules, out=out, **on), out]

    def accept():
        text, slots = torch.zeros(2, 60, dtype=torch.int32, device="cuda"), torch.arange(9, device="cuda")
        return lambda x, **on: [*q4.q4_tree_accept(batch, x[0], x[1], parents=x[2], history=text, slots=slots, **on), text]

    def move():
        kv = [t.clone() for t in base]
        layers = q4.KVLayers([q4.KVCache(*kv)])
        return lambda x, **on: [q4.q4_kv_move(layers, batch, x[:9], x[9:], **on)] and kv

    real = dict(assign=lambda: i32([[1, 2], [16, 30], [5, 4]]), norm=lambda: n(9, 12, 128).half(), append=lambda: n(9, 12, 128).half(),
                tree=lambda: n(9, 8, 128).half(), pick=lambda: n(9, 30000),
                accept=lambda: i32([[4, 9, 1, 1, 3, 5, 5, 5, 5], [0, 4, 7, 9, 8, 0, 5, 5, 5], [-1, 0, 0, 1, 1, -1, 0, 1, 2]]),
                move=lambda: i32([0, 2, 4, -1, -1, 0, 3, -1, -1, 3, 2]))[name]()
    return real, dict(assign=assign, norm=norm, append=append, tree=tree, pick=pick, accept=accept, move=move)[name]


@pytest.mark.parametrize("name", NAMES)
def test_behind_work_on_another_stream(name):
    q4 = lib()
    real, make = prepare(q4, name)
    say("stream", name)
    want = [x.clone() for x in make()(real)]
    given = torch.zeros_like(real)
    stale = [x.clone() for x in make()(given)]
    assert not all(torch.equal(a, b) for a, b in zip(stale, want))  # what a launch on the current stream would give
    call = make()
    side, made, slow = torch.cuda.Stream(), torch.cuda.Event(), torch.randn(8192, 8192, device="cuda").half()
    with torch.cuda.stream(side):
        slow @ slow  # (its first use sets the library up)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            slow @ slow
        given.copy_(real)
        made.record()
    got = call(given, stream=side)
    waits = not made.query()
    side.synchronize()
    assert waits, "the inputs were there before the call: nothing was tested"
    for a, b in zip(got, want):
        assert torch.equal(a, b)
