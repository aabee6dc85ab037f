"""GPU parity of qa_append_rows (rows normed, rotated and written to the paged
bf16 cache) against the definition in 64 bits: rotated results are roundings
of values within the fp32 error (_util), everything else bit for bit."""
import numpy as np
import pytest

import _kvq
import _rows
import workloads as wl
from _util import assert_rounded_match, bits, to_dev

pytestmark = pytest.mark.gpu
import torch  # noqa: E402

import paged_kv_gqa_attention_gb300 as qa  # noqa: E402


class Case:
    def __init__(self, seed, rows, past, hq, hkv, norm=True, axes=0, tree=False, extra=0):
        rng = np.random.default_rng(seed)
        self.rows, self.past, self.hq, self.hkv = list(rows), list(past), hq, hkv
        total = sum(rows) + extra
        self.table, pages = _rows.page_table(rng, [a + b for a, b in zip(rows, past)])
        self.k_pool, self.v_pool = _rows.pool(rng, pages, hkv), _rows.pool(rng, pages, hkv)
        self.q, self.k, self.v = (wl.normal_bf16(rng, (total, h, 128)) for h in (hq, hkv, hkv))
        self.cu = _rows.cumulative(rows)
        self.gains = [wl.bf16_to_f64(wl.bf16_bits(rng.uniform(0.5, 1.5, size=128).astype(np.float32))).astype(np.float32)
                      for _ in range(2)] if norm else [None, None]
        self.parents = np.concatenate([_rows.tree(rng, n) for n in rows] + [np.zeros(extra, np.int32)]).astype(np.int32) if tree else None
        self.positions = rng.integers(0, 1 << 18, size=(axes, total)).astype(np.int32) if axes else None
        self.axis = rng.integers(0, axes, size=64).astype(np.uint8) if axes else None

    def turned(self):
        """The rotary positions [axes, rows], those of the depths where none are given."""
        if self.positions is not None:
            return self.positions[:, :sum(self.rows)]
        first, out = 0, []
        for n, past in zip(self.rows, self.past):
            t = np.arange(n) - 1 if self.parents is None else self.parents[first:first + n]
            out.append(past + _rows.depths(t))
            first += n
        return np.concatenate(out)[None]

    def args(self):
        d = lambda x: None if x is None else to_dev(x)  # noqa: E731
        return dict(n_past=to_dev(np.array(self.past, np.int32)), parents=d(self.parents), positions=d(self.positions),
                    q_gain=d(self.gains[0]), k_gain=d(self.gains[1]), pair_axis=self.axis, debug_checks=True)

    def call(self, q="own", k=None, v=None, pools=None, **kw):
        self.pools = pools or [to_dev(self.k_pool), to_dev(self.v_pool)]
        a = self.args() | kw
        q = to_dev(self.q) if isinstance(q, str) else q
        return qa.qa_append_rows(q, to_dev(self.k) if k is None else k, to_dev(self.v) if v is None else v, to_dev(self.cu),
                                 to_dev(self.table), *self.pools, **a)

    def check(self, q_out, keep=None):
        """keep: the rows that have been written (default all)."""
        n = sum(self.rows)
        keep = np.arange(n) if keep is None else np.asarray(keep)
        pos = self.turned()
        if q_out is not None:
            ref, size = _kvq.rope(wl.bf16_to_f64(self.q[:n]), pos, self.gains[0], self.axis)
            assert_rounded_match(bits(q_out)[keep], ref[keep], size[keep], "q")
        page, slot = _rows.places(self.table, self.past, self.rows)
        page, slot = page[keep], slot[keep]
        got = [bits(p) for p in self.pools]
        ref, size = _kvq.rope(wl.bf16_to_f64(self.k[:n]), pos, self.gains[1], self.axis)
        assert_rounded_match(got[0][page, slot], ref[keep], size[keep], "k")
        np.testing.assert_array_equal(got[1][page, slot], self.v[:n][keep])
        for g, before in zip(got, (self.k_pool, self.v_pool)):  # every other slot as it was
            rest = np.ones(g.shape[:2], bool)
            rest[page, slot] = False
            np.testing.assert_array_equal(g[rest], before[rest])


@pytest.mark.parametrize("rows, past", [
    ([1], [0]), ([1], [15]), ([3], [16]), ([8], [257]), ([16], [0]), ([17, 1], [15, 16]), ([0, 5, 0, 2, 0], [3, 9, 0, 31, 7]),
    ([8] * 33, list(range(33))), ([1] * 100, list(range(0, 1000, 10))), ([2000, 31], [5, 0]), ([300] * 16, list(range(0, 160, 10))),
])
@pytest.mark.parametrize("tree", [False, True])
def test_rows(rows, past, tree):
    c = Case(len(rows) + rows[0], rows, past, 16, 8, tree=tree)
    c.check(c.call())


@pytest.mark.parametrize("hq, hkv", [(1, 1), (2, 1), (3, 3), (6, 3), (5, 5), (14, 7), (8, 8), (8, 4)])
@pytest.mark.parametrize("norm, axes", [(True, 0), (False, 3), (True, 4), (False, 1)])
def test_heads_and_axes(hq, hkv, norm, axes):
    c = Case(hq + hkv, [9, 30, 1], [7, 100, 0], hq, hkv, norm=norm, axes=axes, tree=axes == 0)
    c.check(c.call())


def test_without_queries():
    c = Case(3, [9, 30], [7, 100], 16, 8, tree=True)
    assert c.call(q=None) is None
    c.check(None)


@pytest.mark.parametrize("rows", [[4], [200, 777, 31]])
def test_without_rotation_bits_are_kept(rows):
    c = Case(4, rows, [21] * len(rows), 16, 8)
    rng = np.random.default_rng(5)
    c.q, c.k, c.v = (rng.integers(0, 1 << 16, size=x.shape).astype(np.uint16) for x in (c.q, c.k, c.v))  # NaN, infinities and all
    got = c.call(rotate=False, positions=None, q_gain=None, k_gain=None, pair_axis=None)
    np.testing.assert_array_equal(bits(got), c.q)
    page, slot = _rows.places(c.table, c.past, c.rows)
    np.testing.assert_array_equal(bits(c.pools[0])[page, slot], c.k)
    np.testing.assert_array_equal(bits(c.pools[1])[page, slot], c.v)


@pytest.mark.parametrize("rows, stable", [([7, 3], 0), ([400, 300], 1)])
def test_rows_of_a_fused_projection_in_place(rows, stable):
    c = Case(6, rows, [5, 40], 16, 8, axes=3)
    n = sum(rows)
    x = torch.full((n, 33, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    x[:, :16], x[:, 16:24], x[:, 24:32] = to_dev(c.q), to_dev(c.k), to_dev(c.v)
    out = c.call(q=x[:, :16], k=x[:, 16:24], v=x[:, 24:32], stable_metadata=stable)
    c.check(out)
    again = c.call(q=x[:, :16], k=x[:, 16:24], v=x[:, 24:32], q_out=x[:, :16], stable_metadata=stable)
    c.check(again)
    assert torch.equal(x[:, :16], out) and bool((x[:, 32] == 7).all())
    np.testing.assert_array_equal(bits(x[:, 16:24].contiguous()), c.k)


def test_no_n_past_is_zero():
    c = Case(7, [33, 2], [0, 0], 16, 8, tree=True)
    c.check(c.call(n_past=None))


def test_deep_trees_and_long_requests():
    # a line of 300 rows by parents: deeper than a warp's window of 64; and every row a child of row 0
    for parents in (np.arange(300) - 1, np.array([-1] + [0] * 299), np.array([-1] * 300), np.array([-1] + [(i - 1) // 2 for i in range(1, 300)])):
        c = Case(8, [300], [20], 2, 1)
        c.parents = parents.astype(np.int32)
        c.check(c.call())


def test_rows_behind_the_last_request_stay():
    c = Case(9, [9, 2], [7, 3], 16, 8, tree=True, extra=6)
    out = torch.full((17, 16, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    c.call(q_out=out)
    c.check(out[:11])
    assert bool((out[11:] == 5).all())


def test_bad_positions_pages_lengths_and_parents():
    c = Case(10, [20, 5], [7, 3], 16, 8, axes=2)
    c.positions[0, 3], c.positions[1, 22] = -1, 1 << 18
    out = torch.full((25, 16, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    c.call(q_out=out, debug_checks=False)
    assert qa.qa_device_status() == 0x10
    good = np.array([i for i in range(25) if i not in (3, 22)])
    c.check(out, good)
    assert bool((out[[3, 22]] == 5).all())
    with pytest.raises(qa.QAError, match="bad position"):
        c.call()

    # a bad page: its rows have no place, but their queries are there
    c = Case(11, [40, 5], [7, 3], 16, 8)
    lost = [i for i in range(40) if 16 <= 7 + i < 32]
    c.table, kept = c.table.copy(), c.table
    c.table[0, 1] = c.k_pool.shape[0]
    out = c.call(debug_checks=False)
    assert qa.qa_device_status() == 0x1
    c.table = kept
    rest = np.array([i for i in range(45) if i not in lost])
    c.check(None, rest)
    ref, size = _kvq.rope(wl.bf16_to_f64(c.q), c.turned(), c.gains[0], None)
    assert_rounded_match(bits(out), ref, size, "q")

    # past the page-table row; and n_past that is no length
    c = Case(12, [20, 5], [7, 3], 16, 8)
    cap = c.table.shape[1] * 16
    real = c.past[0]
    c.past[0] = cap - 6
    c.table[0] = np.where(c.table[0] < 0, 0, c.table[0])
    c.call(debug_checks=False)
    assert qa.qa_device_status() == 0x2
    page, slot = _rows.places(c.table, [cap - 6], [6])
    np.testing.assert_array_equal(bits(c.pools[1])[page, slot], c.v[:6])
    for bad in (-1, cap + 1, 2 ** 31 - 1):
        c = Case(12, [20, 5], [7, 3], 16, 8)
        c.past[0] = bad
        out = torch.full((25, 16, 128), 5.0, dtype=torch.bfloat16, device="cuda")
        c.call(q_out=out, debug_checks=False)
        assert qa.qa_device_status() == 0x2
        c.past[0] = real
        c.check(None, np.arange(20, 25))
        assert bool((out[:20] == 5).all())

    # parents that are none count as -1
    c = Case(13, [30], [7], 16, 8, tree=True)
    bad = c.parents.copy()
    bad[[5, 9, 20]] = 5, -3, 2 ** 31 - 1
    c.parents = bad
    out = c.call(debug_checks=False)
    assert qa.qa_device_status() == 0x20
    bad[[5, 9, 20]] = -1
    c.check(out)


def test_bad_segments():
    c = Case(14, [10, 20, 5], [7, 3, 0], 16, 8)
    c.cu[3] = 36  # past the rows: that request is no request
    c.call(debug_checks=False)
    assert qa.qa_device_status() == 0x4
    c.check(None, np.arange(30))
    c = Case(15, [10, 20, 5], [0, 0, 0], 16, 8)
    c.cu[1] = 33
    c.call(debug_checks=False)
    assert qa.qa_device_status() & 0x4


def test_positions_past_the_rotation():
    """n_past plus depth is checked as positions are."""
    c = Case(16, [4], [0], 2, 1)
    wide = (1 << 18) // 16 + 1
    c.past, c.table = [(1 << 18) - 2], np.zeros((1, wide), np.int32)
    c.table[0, -2:] = [0, 1] if c.k_pool.shape[0] > 1 else [0, 0]
    out = torch.full((4, 2, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    c.call(q_out=out, debug_checks=False)
    assert qa.qa_device_status() == 0x10
    assert bool((out[2:] == 5).all()) and not bool((out[:2] == 5).all())


def test_no_rows():
    c = Case(17, [3], [5], 16, 8)
    z = torch.zeros(0, 8, 128, dtype=torch.bfloat16, device="cuda")
    qa.qa_append_rows(None, z, z, to_dev(np.zeros(2, np.int32)), to_dev(c.table), to_dev(c.k_pool), to_dev(c.v_pool), debug_checks=True)
    # rows that no request owns
    pools = [to_dev(c.k_pool), to_dev(c.v_pool)]
    qa.qa_append_rows(None, to_dev(c.k), to_dev(c.v), to_dev(np.zeros(2, np.int32)), to_dev(c.table), *pools, debug_checks=True)
    assert np.array_equal(bits(pools[0]), c.k_pool) and np.array_equal(bits(pools[1]), c.v_pool)


@pytest.mark.parametrize("batch", [33, 1024, 1025, 4096])
def test_many_requests(batch):
    rng = np.random.default_rng(batch)
    rows = rng.integers(0, 4, batch).tolist()
    c = Case(18, rows, rng.integers(0, 20, batch).tolist(), 2, 1, tree=True)
    c.check(c.call())


def test_one_row_equals_the_decode_append():
    c = Case(19, [1] * 9, list(range(0, 180, 20)), 16, 8)
    out = c.call()
    c.check(out)
    pools = [to_dev(c.k_pool), to_dev(c.v_pool)]
    ref = qa.qa_decode_append(to_dev(c.q), to_dev(c.k), to_dev(c.v), to_dev(c.gains[0]), to_dev(c.gains[1]), to_dev(c.table),
                              to_dev(np.array(c.past, np.int32) + 1), *pools, debug_checks=True)
    page, slot = _rows.places(c.table, c.past, c.rows)
    ref_k, size = _kvq.rope(wl.bf16_to_f64(c.k), c.turned(), c.gains[1], None)
    assert_rounded_match(bits(pools[0])[page, slot], ref_k, size, "k of the decode append")
    assert torch.equal(pools[1], c.pools[1])
    assert ref.shape == out.shape


def test_graph_stream_and_levels():
    c = Case(20, [8, 20], [30, 41], 16, 8, tree=True)
    want = c.call()
    c.check(want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for level in (0, 1, 2):
        got = c.call(stream=side, stable_metadata=level)
        side.synchronize()
        assert torch.equal(got, want)
    q, k, v, cu, table = (to_dev(x) for x in (c.q, c.k, c.v, c.cu, c.table))
    pools = [to_dev(c.k_pool), to_dev(c.v_pool)]
    out = torch.zeros_like(want)
    a = c.args() | dict(debug_checks=False)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qa.qa_append_rows(q, k, v, cu, table, *pools, out, **a)
    d = Case(21, [8, 20], [30, 41], 16, 8, tree=True)
    for dst, src in ((q, d.q), (k, d.k), (v, d.v), (a["parents"], d.parents), (a["n_past"], np.array([29, 0], np.int32))):
        dst.copy_(to_dev(src))
    graph.replay()
    torch.cuda.synchronize()
    c.q, c.k, c.v, c.parents, c.past, c.pools = d.q, d.k, d.v, d.parents, [29, 0], pools
    c.check(out)


def test_pages_past_four_gigabytes():
    pages = (5 << 30) // (16 * 8 * 128 * 2)
    c = Case(22, [40, 3], [100, 20], 16, 8)
    n = c.k_pool.shape[0]
    big = [torch.zeros(pages, 16, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kept = c.table
    c.table = np.where(kept >= 0, kept + pages - n, -1).astype(np.int32)
    for p, src in zip(big, (c.k_pool, c.v_pool)):
        p[pages - n:] = to_dev(src)
    out = c.call(pools=big)
    c.table, c.pools = kept, [p[pages - n:] for p in big]
    c.check(out)
    assert all(not bool(p[:pages - n].any()) for p in big)
