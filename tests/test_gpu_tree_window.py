"""Windows over chains of new tokens: the masks of chains, without the tokens outside of a window that is shorter than they
are, give what causal attention gives with that window; as they are, the mask alone decides about new tokens."""
import pytest
import torch

import step_ref
from gpu_util import lib, say
from test_gpu_attention_tree import check, setup

pytestmark = pytest.mark.gpu


def chain(new, tokens, window):
    """Row i of a sequence sees its last `window` new tokens up to its own (0: all), in masks of two words."""
    mask = torch.zeros(tokens, 2, dtype=torch.int64)
    at = 0
    for n in new:
        for i in range(n):
            for j in range(max(0, i - window + 1) if window else 0, i + 1):
                bit = 1 << (j & 63)
                mask[at, j >> 6] |= bit if bit < 1 << 63 else -(1 << 63)
            at += 1
    return mask


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("lens,window,hq", [([(40, 90), (5, 300)], 16, 4), ([(40, 90), (5, 300)], 40, 4), ([(100, 130), (1, 9)], 33, 8),
                                            ([(100, 700), (128, 128)], 64, 2), ([(9, 9)], 1, 4)])
def test_chains(lens, window, hq, dtype):
    q4 = lib()
    say("window", lens, window, dtype)
    batch, q, k, v, _ = setup(lens, 16, hq, 2, 64, dtype, 2, 5)
    within = chain(batch.new, batch.tokens, window)
    exact = step_ref.TreeExact(q, k, v, batch, within, 64 ** -0.5, window)
    check(q4, batch, q, k, v, within, window, exact=exact)
    n = int(batch.start[-1])
    causal = q4.q4_attention_paged(q4.KVCache(k.cuda(), v.cuda()), batch.device(q4), q.cuda(), window=window)
    assert bool(((causal[:n].double().cpu() - exact.out[:n]).abs() <= exact.bound[:n]).all())
    whole = chain(batch.new, batch.tokens, 0)
    check(q4, batch, q, k, v, whole, window)
    if window >= max(batch.new):
        assert torch.equal(whole, within)
