"""The calls of tree_cuts are cut as they say, and together reach every kernel of attention over trees."""
import pytest

import tree_cuts


@pytest.fixture(scope="module")
def shape(tmp_path_factory):
    return tree_cuts.shim(str(tmp_path_factory.mktemp("shape")))


@pytest.mark.parametrize("case", tree_cuts.cases(), ids=repr)
def test_cut(shape, case):
    assert shape(case) == (case.rows, case.whole)


def test_every_kernel_is_reached():
    got = {(c.dim, c.rows, c.whole) for c in tree_cuts.cases()}
    want = {(d, r, w) for d in (64, 96, 128, 256) for r in (16, 32, 64, 128) for w in (True, False)}
    assert got == want | {(d, 256, False) for d in (96, 128)}
