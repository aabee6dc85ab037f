"""NaN and infinities in the queries and keys of qa_tree_attn and
qa_cross_attn: what they reach must not depend on how a call's keys are cut
into workers' ranges, so that every case is taken with requests that one
worker finishes, with requests of a few parts, and of many."""
import numpy as np
import pytest

import _rows
import workloads as wl
from _util import f64
from test_rows_attn_gpu import INF, NAN, Case

pytestmark = pytest.mark.gpu

MINUS = INF | 0x8000

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


def positive(c, dim=9):
    """Queries above 0 in one dim, so that an infinity in that dim of a key makes its score as infinite."""
    q = wl.bf16_to_f64(c.q)
    q[..., dim] = 0.5 + np.abs(q[..., dim])
    c.q = wl.bf16_bits(q.astype(np.float32))


def hidden(c, b, positions):
    """The reference with positions of request b hidden from its rows."""
    vis = [np.ones((n, m), bool) for n, m in zip(c.rows, c.keys)] if c.kind == "cross" else _rows.tree_visible(c.parents, c.rows, c.past)
    vis[b][:, positions] = False
    return _rows.attention(wl.bf16_to_f64(c.q), wl.bf16_to_f64(c.k), wl.bf16_to_f64(c.v), c.table, c.rows, c.keys, vis)


@pytest.mark.parametrize("kind, rows, parts, n, keys", CASES)
def test_a_score_of_minus_infinity_has_no_weight(kind, rows, parts, n, keys):
    c = Case(71, [rows] * n, [keys] * n, 16, 8, kind)
    positive(c)
    b, last = n // 2, c.keys[n // 2] - 1
    gone = sorted({0, 3, keys // 2} | set(range(16, min(32, keys))) | ({last} if kind == "cross" else set()))
    ref, bound = hidden(c, b, gone)
    for pos in gone:
        c.k[c.table[b, pos // 16], pos % 16, :, 9] = MINUS
    got = f64(c.call())
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= bound).all()


@pytest.mark.parametrize("kind, rows, parts, n, keys", CASES)
def test_rows_with_such_scores_only_are_zero(kind, rows, parts, n, keys):
    c = Case(72, [rows] * n, [keys] * n, 16, 8, kind)
    positive(c)
    clean, bound = c.reference()
    b = n // 2
    for pos in range(c.keys[b]):
        c.k[c.table[b, pos // 16], pos % 16, 2, 9] = MINUS
    got = f64(c.call())
    zero = np.zeros(clean.shape, bool)
    zero[rows * b:rows * (b + 1), 4:6] = True
    assert (got[zero] == 0).all()
    assert (np.abs(got - clean) <= bound)[~zero].all()


@pytest.mark.parametrize("rows", [1, 5, 40])
def test_a_row_whose_own_key_is_all_it_sees(rows):
    """Row 0 of an empty cache sees its own key alone, the others their ancestors and themselves."""
    for what in ("-inf", "inf", "nan"):
        c = Case(73, [rows, 2], [0, 20], 16, 8, "tree")
        c.parents[:rows] = [-1] + [0] * (rows - 1)
        positive(c)
        if what == "-inf":
            ref, bound = hidden(c, 0, [0])
        else:
            ref, bound = c.reference()
        c.k[c.table[0, 0], 0, :, 9] = {"-inf": MINUS, "inf": INF, "nan": NAN}[what]
        got = f64(c.call())
        if what == "-inf":
            assert (got[0] == 0).all()
            assert (np.abs(got - ref) <= bound).all()
        else:
            assert np.isnan(got[:rows]).all()
            assert (np.abs(got - ref) <= bound)[rows:].all()


@pytest.mark.parametrize("kind, rows, parts, n, keys", CASES)
def test_a_score_of_infinity_is_nan(kind, rows, parts, n, keys):
    c = Case(74, [rows] * n, [keys] * n, 16, 8, kind)
    positive(c)
    clean, bound = c.reference()
    c.k[c.table[0, 0], 5, 7, 9] = INF
    hit = np.zeros(clean.shape, bool)
    hit[:rows, 14:16] = True
    check(c.call(), clean, bound, hit)


@pytest.mark.parametrize("kind, rows, parts, n, keys", CASES)
def test_a_cached_infinite_value_is_no_number_behind_it(kind, rows, parts, n, keys):
    c, clean, bound = case(kind, rows, n, keys)
    c.v[c.table[0, keys // 32], 1, 4, 50] = INF
    got = f64(c.call())
    hit = np.zeros(clean.shape, bool)
    hit[:rows, 8:10, 50] = True
    assert not np.isfinite(got[hit]).any()
    assert (np.abs(got - clean) <= bound)[~hit].all()
