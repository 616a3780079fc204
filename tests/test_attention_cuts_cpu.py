"""The calls of tests/attention_cuts.py are cut as they say, and are complete: a change of the rule that takes a kernel
out of the tests' reach fails here."""
import pytest
import torch

import kv_ref
from attention_cuts import Exact, cases, shim


@pytest.fixture(scope="module")
def shape(tmp_path_factory):
    return shim(str(tmp_path_factory.mktemp("shape")))


def test_every_kernel_is_reached():
    have = {(c.rows, c.dim, c.whole, c.window > 0) for c in cases()}
    want = {(r, d, w, x) for r in (16, 32, 64, 128) for d in (64, 96, 128, 256) for w in (True, False) for x in (True, False)}
    assert have == want


@pytest.mark.parametrize("case", cases(), ids=repr)
def test_cut(shape, case):
    assert shape(case) == (case.rows, case.whole)


@pytest.mark.parametrize("window", [0, 5])
def test_the_64_bit_forms_agree(window):
    """The form with each sequence's keys side by side against the one that goes row by row, and that a mask or a
    window that is off by one key would be seen."""
    batch = kv_ref.Batch([(3, 20), (1, 9), (0, 4), (4, 2), (1, 0)], 8, seed=1, pad_rows=2)
    g = torch.Generator().manual_seed(1)
    q = torch.randn(batch.tokens, 4, 64, generator=g).half()
    k, v = (torch.randn(batch.pages, 2, 8, 64, generator=g).half() for _ in range(2))
    want, lse, bound, lse_bound = kv_ref.attention(q, k, v, batch, 0.125, window)
    got = Exact(q, k, v, batch, 0.125, window)
    assert bool(((got.out - want).abs() <= 1e-13).all()) and bool(((got.bound - bound).abs() <= 1e-13).all())
    some = torch.isfinite(lse)
    assert bool((torch.isfinite(got.lse) == some).all())
    assert bool(((got.lse - lse)[some].abs() <= 1e-13).all()) and bool(((got.lse_bound - lse_bound).abs() <= 1e-13)[some].all())
    if window:
        other = Exact(q, k, v, batch, 0.125, window - 1)
    else:
        batch.ctx = [max(c - 1, 0) for c in batch.ctx]
        other = Exact(q, k, v, batch, 0.125, 0)
    assert bool(((other.out - want).abs() > bound).any(2).any(1)[:4].all())
