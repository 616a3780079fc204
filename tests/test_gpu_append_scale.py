"""The factor of the rotation (mscale, as scaling for long contexts wants it) on the way into the cache."""
import pytest
import torch

import kv_ref
from gpu_util import lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rot", [64, 32])
def test_queries_and_keys_are_scaled_and_values_are_not(layout, rot):
    """yarn's frequencies and factor, as a program passes both on: the rotated elements of q and k times the factor
    (so scores of heads rotated whole times its square), the others and the values as they are."""
    q4 = lib()
    freq, mscale = q4.rope_frequencies(rot, 1e4, "yarn", 8.0, 4096)
    assert mscale > 1.2
    g = torch.Generator().manual_seed(rot)
    q, k, v = (torch.randn(5, h, 64, generator=g) for h in (4, 2, 2))
    kc, vc = (torch.zeros(4, 2, 8, 64, dtype=torch.float16, device="cuda") for _ in range(2))
    batch = kv_ref.Batch([(5, 20)], 8, spare=1)
    turned = q4.q4_kv_append(q4.KVCache(kc, vc), batch.device(q4), k.cuda(), v.cuda(), q=q.cuda(), inv_freq=freq,
                             layout=layout, mscale=mscale)
    pos = torch.arange(15, 20)
    at = [(int(batch.table[0, p // 8]), p % 8) for p in range(15, 20)]
    got_k, got_v = (torch.stack([c[a, :, s] for a, s in at]).cpu() for c in (kc, vc))
    assert torch.equal(got_v, v.half())
    for got, x in ((turned.cpu(), q), (got_k, k)):
        want = kv_ref.rotate(x.double(), pos, freq.cpu(), layout, mscale)
        bound = kv_ref.rotate_bound(x.double(), pos, freq.cpu(), layout, torch.float16, mscale)
        assert bool(((got.double() - want).abs() <= bound).all())
