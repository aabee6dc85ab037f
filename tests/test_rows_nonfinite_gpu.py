"""NaN and infinities in the queries and keys of qa_tree_attn and
qa_cross_attn: what they reach must not depend on how a call's keys are cut
into workers' ranges, so that every case is taken with requests that one
worker finishes, with requests of a few parts, and of many."""
import numpy as np
import pytest

from _util import f64
from test_rows_attn_gpu import NAN, Case

pytestmark = pytest.mark.gpu

# (kind, rows of a request, requests, keys): on a grid of 152 workers (8 KV heads: 19 for many rows) a request of one page
# or tile is whole, forty of 17 pages are cut into about 4 parts, six of 3 tiles into about 3, and a single one into as
# many parts as it has pages or tiles
FEW = [("whole", 200, 8), ("few parts", 40, 257), ("many parts", 1, 400)]
MANY = [("whole", 60, 60), ("few parts", 6, 300), ("many parts", 1, 2300)]
CASES = [(kind, rows, *x) for kind, rows in (("tree", 6), ("cross", 4)) for x in FEW] + \
        [(kind, rows, *x) for kind, rows in (("tree", 33), ("cross", 90)) for x in MANY]


def case(kind, rows, n, keys):
    c = Case(70, [rows] * n, [keys] * n, 16, 8, kind)
    clean, bound = c.reference()
    return c, clean, bound


def check(got, clean, bound, hit):
    """NaN exactly where `hit` says so, and the rest as without them."""
    got = f64(got)
    assert np.array_equal(np.isnan(got), hit), f"{np.isnan(got).sum()} values are NaN, {hit.sum()} should be"
    assert (np.abs(got - clean) <= bound)[~hit].all()


@pytest.mark.parametrize("kind, rows, parts, n, keys", CASES)
def test_nan_in_a_query(kind, rows, parts, n, keys):
    c, clean, bound = case(kind, rows, n, keys)
    hit = np.zeros(clean.shape, bool)
    for row, head in ((1, 5), (rows * n - 1, 12)):
        c.q[row, head, 77] = NAN
        hit[row, head] = True
    check(c.call(), clean, bound, hit)


@pytest.mark.parametrize("kind, rows, parts, n, keys", CASES)
@pytest.mark.parametrize("where", ["first", "middle", "last"])
def test_nan_in_every_key_of_a_range(kind, rows, parts, n, keys, where):
    """All cached keys of a page (or of the tile's 128 around it) are NaN in one KV head."""
    c, clean, bound = case(kind, rows, n, keys)
    step = 16 if rows < 10 else 128
    pieces = -(-keys // step)
    begin = {"first": 0, "middle": pieces // 2, "last": pieces - 1}[where] * step
    b, head = n // 2, 3
    for pos in range(begin, min(begin + step, keys)):
        c.k[c.table[b, pos // 16], pos % 16, head] = NAN
    hit = np.zeros(clean.shape, bool)
    hit[rows * b:rows * (b + 1), 2 * head:2 * head + 2] = True
    check(c.call(), clean, bound, hit)


@pytest.mark.parametrize("kind, rows, parts, n, keys", CASES)
def test_nan_in_every_key(kind, rows, parts, n, keys):
    c, clean, bound = case(kind, rows, n, keys)
    hit = np.zeros(clean.shape, bool)
    for pos in range(c.keys[0]):
        c.k[c.table[0, pos // 16], pos % 16, 6] = NAN
    hit[:rows, 12:14] = True
    check(c.call(), clean, bound, hit)
