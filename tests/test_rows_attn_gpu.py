"""GPU parity of qa_tree_attn and qa_cross_attn against the definition in 64
bits (_rows.attention, which derives the bound), and their refusals on the
device."""
import threading

import numpy as np
import pytest

import _rows
import test_kvq_decode_gpu
import workloads as wl
from _util import bits, f64, to_dev

pytestmark = pytest.mark.gpu
import torch  # noqa: E402

import paged_kv_gqa_attention_gb300 as qa  # noqa: E402

NAN = wl.bf16_bits(np.array([np.nan], np.float32))[0]
INF = wl.bf16_bits(np.array([np.inf], np.float32))[0]


class Case:
    """Host inputs of one call: a tree, a chain or cross attention (keys: the states)."""

    def __init__(self, seed, rows, keys, hq, hkv, kind, size=1.5, extra=0, width=None):
        rng = np.random.default_rng(seed)
        self.rows, self.hq, self.hkv, self.kind = list(rows), hq, hkv, kind
        self.past = list(keys)
        self.keys = [p + n if kind != "cross" else p for p, n in zip(self.past, self.rows)]
        self.table, pages = _rows.page_table(rng, self.keys, width=width)
        self.k, self.v = _rows.pool(rng, pages, hkv), _rows.pool(rng, pages, hkv)
        for p in (self.k, self.v):
            _rows.poison(p, self.table, self.keys)
        total = sum(self.rows) + extra
        self.q = wl.bf16_bits((size * rng.standard_normal((total, hq, 128))).astype(np.float32))
        self.cu = _rows.cumulative(self.rows)
        self.parents = None
        if kind == "tree":
            flat = [_rows.tree(rng, n) for n in self.rows] + [np.zeros(extra, np.int32)]
            self.parents = np.concatenate(flat).astype(np.int32)
        self.most = max(1, max(self.rows))

    def reference(self, scale=None):
        visible = None if self.kind == "cross" else _rows.tree_visible(self.parents, self.rows, self.past)
        return _rows.attention(wl.bf16_to_f64(self.q), wl.bf16_to_f64(self.k), wl.bf16_to_f64(self.v), self.table, self.rows,
                               self.keys, visible, scale)

    def call(self, q=None, most=None, **kw):
        q = to_dev(self.q) if q is None else q
        kw.setdefault("debug_checks", True)
        args = (q, to_dev(self.cu), to_dev(np.array(self.past, np.int32)), to_dev(self.table), to_dev(self.k), to_dev(self.v),
                most or self.most)
        if self.kind == "cross":
            return qa.qa_cross_attn(*args, **kw)
        return qa.qa_tree_attn(*args, parents=None if self.parents is None else to_dev(self.parents), **kw)

    def check(self, got, what="", scale=None):
        ref, bound = self.reference(scale)
        n = sum(self.rows)
        got = f64(got)[:n]
        d = np.abs(got - ref[:n])
        finite, bad = bool(np.isfinite(got).all()), d > bound[:n]
        assert finite, f"{what}: values that are not finite"
        n_bad = int(bad.sum())
        assert n_bad == 0, f"{what}: {n_bad} of {bad.size} outside the bound, worst {np.max(d / bound[:n]):.2f} of it, first at {np.argwhere(bad)[0]}"


@pytest.mark.parametrize("rows, past", [
    ([1], [0]), ([1], [1]), ([2], [15]), ([8], [0]), ([8], [8]), ([8], [9]), ([5], [16]), ([8], [257]), ([8, 1, 3], [31, 700, 47]),
    ([0, 4, 0, 8], [5, 0, 0, 100]), ([7] * 40, list(range(0, 400, 10))),
])
@pytest.mark.parametrize("kind", ["tree", "chain"])
def test_few_rows(rows, past, kind):
    c = Case(len(rows) + rows[0], rows, past, 16, 8, kind)
    c.check(c.call())


@pytest.mark.parametrize("rows, past", [([16], [100]), ([9, 16], [0, 1000]), ([12] * 20, list(range(3, 1003, 50))), ([1, 16], [40, 41])])
def test_up_to_sixteen_rows(rows, past):
    c = Case(7, rows, past, 16, 8, "tree")
    c.check(c.call())


@pytest.mark.parametrize("rows, past", [
    ([17], [0]), ([64], [0]), ([64], [1]), ([64], [63]), ([33], [64]), ([64], [65]), ([40], [1000]), ([64, 20, 1], [127, 0, 500]),
    ([0, 30, 0], [0, 130, 4]), ([50] * 12, list(range(0, 1200, 100))),
])
@pytest.mark.parametrize("kind", ["tree", "chain"])
def test_many_rows(rows, past, kind):
    c = Case(len(rows) + rows[0], rows, past, 16, 8, kind)
    c.check(c.call())


@pytest.mark.parametrize("hq, hkv", [(1, 1), (2, 1), (2, 2), (4, 2), (3, 3), (6, 3), (8, 4), (5, 5), (10, 5), (6, 6), (7, 7), (14, 7), (8, 8)])
@pytest.mark.parametrize("rows", [[3, 8, 1], [31, 2, 16], [64, 20, 3]])
def test_heads(hq, hkv, rows):
    c = Case(hq * 10 + hkv, rows, [90, 0, 333], hq, hkv, "tree")
    c.check(c.call())


@pytest.mark.parametrize("rows, states", [
    ([1], [1]), ([1], [0]), ([3, 0, 2], [16, 5, 17]), ([4, 1], [390, 13]), ([16], [500]), ([32], [64]), ([33], [63]), ([128], [65]),
    ([129], [200]), ([300, 1, 257], [129, 1000, 31]), ([200, 40], [0, 700]), ([65] * 10, list(range(1, 1001, 100))),
])
@pytest.mark.parametrize("hq, hkv", [(16, 8), (8, 8), (3, 3)])
def test_cross(rows, states, hq, hkv):
    c = Case(sum(rows), rows, states, hq, hkv, "cross")
    c.check(c.call())


def test_rows_without_states_are_zero():
    for rows in ([5, 3], [70, 40]):
        c = Case(3, rows, [0, 33], 16, 8, "cross")
        got = c.call(out=torch.full((sum(rows), 16, 128), 9.0, dtype=torch.bfloat16, device="cuda"))
        assert bool((got[:rows[0]] == 0).all())
        c.check(got)


@pytest.mark.parametrize("most", [8, 16, 32, 64])
def test_a_larger_max_rows_serves_smaller_requests(most):
    c = Case(5, [3, 8, 1], [200, 3, 77], 16, 8, "tree")
    c.check(c.call(most=most))


@pytest.mark.parametrize("rows", [[4] * 3, [20] * 3, [50] * 3])
def test_long_context(rows):
    c = Case(11, rows, [20000, 3000, 9], 16, 8, "tree")
    c.check(c.call())


@pytest.mark.parametrize("rows", [1, 12, 33])
def test_largest_batch(rows):
    rng = np.random.default_rng(1)
    c = Case(12, [rows] * 1024, rng.integers(0, 60, 1024).tolist(), 2, 1, "tree")
    c.check(c.call())


@pytest.mark.parametrize("kind, most, group", [("tree", 8, 2), ("tree", 16, 1), ("tree", 64, 2), ("cross", 300, 2), ("cross", 300, 1)])
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_mixed_lengths(kind, most, group, seed):
    """Lengths at the borders of pages and tiles between long ones and none at all, so that ranges of workers begin and
    end on, before and behind a job's first and last tile."""
    rng = np.random.default_rng(seed)
    border = [0, 1, 15, 16, 17, 127, 128, 129, 255, 256, 257, 400]
    n = int(rng.integers(20, 60))
    keys = [int(rng.choice(border)) if rng.random() < 0.8 else int(rng.integers(300, 3000)) for _ in range(n)]
    rows = [int(rng.choice([0, 1, most, int(rng.integers(1, most + 1))])) for _ in range(n)]
    rows[0] = most
    c = Case(100 + seed, rows, keys, 4 * group, 4, kind)
    c.check(c.call())


@pytest.mark.parametrize("rows", [8, 32, 64])
def test_deep_and_flat_trees(rows):
    for parents in ([-1] * rows, [-1] + [0] * (rows - 1), [i - 1 for i in range(rows)], [i // 2 - 1 if i < 2 else (i - 1) // 2 for i in range(rows)]):
        c = Case(13, [rows], [75], 16, 8, "tree")
        c.parents = np.array(parents, np.int32)
        c.check(c.call())


@pytest.mark.parametrize("rows, kind", [([6, 2], "tree"), ([60, 9], "tree"), ([6, 2], "cross"), ([200, 9], "cross")])
@pytest.mark.parametrize("size", [0.0, 12.0, 60.0])
def test_flat_and_sharp_scores(rows, kind, size):
    c = Case(14, rows, [300, 40], 16, 8, kind, size=size)
    c.check(c.call())


@pytest.mark.parametrize("rows", [[5], [40]])
def test_rising_scores(rows):
    """Every tile's largest score is above all before it, and then below."""
    c = Case(15, rows, [400], 16, 8, "tree")
    q = wl.bf16_to_f64(c.q)
    for name in ("rise", "fall"):
        k = np.where(np.isnan(wl.bf16_to_f64(c.k)), np.nan, 0.01)
        for j in range(c.keys[0]):
            x = j if name == "rise" else c.keys[0] - j
            k[c.table[0, j // 16], j % 16] = x / 16.0
        c.k = wl.bf16_bits(k.astype(np.float32))
        c.q = wl.bf16_bits((np.abs(q) * 0.5).astype(np.float32))
        c.check(c.call(), name)


def test_scale():
    for rows in ([4], [50]):
        c = Case(16, rows, [90], 16, 8, "tree")
        c.check(c.call(scale=0.25), scale=0.25)


@pytest.mark.parametrize("hq, rows", [(16, [8, 3]), (8, [16, 3]), (16, [16, 9]), (16, [64, 30]), (8, [64, 30])])
@pytest.mark.parametrize("past", [50, 0, 125, 300])
def test_hidden_rows_may_hold_anything(hq, rows, past):
    """NaN and infinities in a drafted row's key or value reach that row and those behind it in the tree, no other."""
    c = Case(17, rows, [past, 0], hq, 8, "tree")
    c.parents[:rows[0]] = [-1, 0, 0, 1] + [2] * (rows[0] - 4)
    clean, bound = c.reference()
    at = c.past[0] + 1  # row 1: its row and row 3's see it
    page, slot = c.table[0, at // 16], at % 16
    behind = [1, 3]
    others = [i for i in range(sum(rows)) if i not in behind]
    for what in ("value inf", "value nan", "key nan", "key inf", "value -inf in one dim"):
        d = Case(17, rows, [past, 0], hq, 8, "tree")
        d.parents = c.parents
        if what == "value inf":
            d.v[page, slot] = INF
        elif what == "value nan":
            d.v[page, slot] = NAN
        elif what == "key nan":
            d.k[page, slot] = NAN
        elif what == "key inf":
            d.k[page, slot] = INF
        else:
            d.v[page, slot, :, 77] = INF | 0x8000
        got = f64(d.call())
        assert (np.abs(got - clean)[others] <= bound[others]).all(), what
        hit = got[behind]
        if what == "value inf":
            assert (hit == np.inf).all()
        elif what == "value nan":
            assert np.isnan(hit).all()
        elif what == "value -inf in one dim":
            assert (hit[..., 77] == -np.inf).all()
            rest = [x for x in range(128) if x != 77]
            assert (np.abs(hit - clean[behind])[..., rest] <= bound[behind][..., rest]).all()
        elif what == "key nan":
            assert np.isnan(hit).all()


@pytest.mark.parametrize("kind, rows", [("tree", [3, 5]), ("tree", [30, 41]), ("cross", [3, 5]), ("cross", [130, 41])])
def test_rows_behind_the_last_request_stay(kind, rows):
    c = Case(18, rows, [70, 5], 16, 8, kind, extra=9)
    out = torch.full((sum(rows) + 9, 16, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    got = c.call(out=out)
    c.check(got)
    assert bool((got[sum(rows):] == 3).all())


@pytest.mark.parametrize("rows", [[4, 7], [20, 41]])
def test_strided_queries_and_unaligned_output(rows):
    c = Case(19, rows, [70, 5], 16, 8, "tree")
    n = sum(rows)
    x = torch.full((n, 33, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    x[:, 3:19] = to_dev(c.q)
    # an output 16 bytes behind a 32-byte boundary
    flat = torch.full((n * 2048 + 16,), 5.0, dtype=torch.bfloat16, device="cuda")
    out = flat[8:8 + n * 2048].view(n, 16, 128)
    assert out.data_ptr() % 32 == 16
    c.check(c.call(q=x[:, 3:19], out=out))
    assert bool((flat[:8] == 5).all()) and bool((flat[-8:] == 5).all())


@pytest.mark.parametrize("kind, rows", [("tree", [3, 5, 8]), ("tree", [30, 41, 8]), ("cross", [150, 41, 8])])
def test_bad_pages_lengths_and_segments(kind, rows):
    def fresh():
        return Case(20, rows, [100, 200, 40], 16, 8, kind)

    # a bad page is left out: as if its positions were not there
    c = fresh()
    cut = c.table.copy()
    cut[1, 3], cut[1, 4] = c.k.shape[0], -7
    good, c.table = c.table, cut
    with pytest.raises(qa.QAError, match="bad page"):
        c.call()
    out = torch.zeros(sum(rows), 16, 128, dtype=torch.bfloat16, device="cuda")
    c.call(out=out, debug_checks=False)
    assert qa.qa_device_status() == 0x1
    c.table = good
    vis = [np.ones((n, m), bool) for n, m in zip(c.rows, c.keys)] if kind == "cross" else _rows.tree_visible(c.parents, c.rows, c.past)
    vis[1][:, 48:80] = False
    ref, bound = _rows.attention(wl.bf16_to_f64(c.q), wl.bf16_to_f64(c.k), wl.bf16_to_f64(c.v), good, c.rows, c.keys, vis)
    assert (np.abs(f64(out) - ref) <= bound).all()

    # bad lengths: that request's rows are zero
    for bad in (-1, c.table.shape[1] * 16 + 1):
        c = fresh()
        full = c.past[1]
        c.past[1] = bad
        out = torch.full((sum(rows), 16, 128), 9.0, dtype=torch.bfloat16, device="cuda")
        c.call(out=out, debug_checks=False)
        assert qa.qa_device_status() == 0x2
        c.past[1] = full
        ref, bound = c.reference()
        a, b = int(c.cu[1]), int(c.cu[2])
        assert bool((out[a:b] == 0).all())
        rest = list(range(a)) + list(range(b, sum(rows)))
        assert (np.abs(f64(out) - ref) <= bound)[rest].all()

    # more rows than max_rows
    c = fresh()
    out = torch.full((sum(rows), 16, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    most = sorted(rows)[-2]
    c.call(out=out, most=most, debug_checks=False)
    assert qa.qa_device_status() == 0x2
    ref, bound = c.reference()
    for r in range(3):
        a, b = int(c.cu[r]), int(c.cu[r + 1])
        if rows[r] > most:
            assert bool((out[a:b] == 0).all())
        else:
            assert (np.abs(f64(out) - ref) <= bound)[a:b].all()

    # malformed segments: those requests' rows are not written
    c = fresh()
    c.cu[1] = c.cu[2] + 2
    out = torch.full((sum(rows), 16, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    c.call(out=out, most=64 if kind == "tree" else 200, debug_checks=False)
    assert qa.qa_device_status() & 0x4
    c = fresh()
    c.cu[3] += 1
    out = torch.full((sum(rows), 16, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    c.call(out=out, debug_checks=False)
    assert qa.qa_device_status() == 0x4
    assert bool((out[int(c.cu[2]):] == 9).all())


@pytest.mark.parametrize("kind, most", [("tree", 8), ("tree", 50), ("cross", 8), ("cross", 160)])
@pytest.mark.parametrize("what", ["begins behind its end", "begins below 0", "ends behind the rows", "all three"])
def test_malformed_segments_leave_the_others_as_they_are(kind, most, what):
    """Requests whose segments are well formed, and do not overlap, have their results; every other row stays."""
    cu = {"begins behind its end": [2 + most, 3, 3 + most, 8 + most], "begins below 0": [-1, 4, 4 + most, 9 + most],
          "ends behind the rows": [0, most, most + 5, 10 ** 6], "all three": [-7, -3, 5, 2 ** 31 - 1]}[what]
    total, keys = 2 * most + 12, [300, 77, 129]
    good = {"begins behind its end": [1, 2], "begins below 0": [1, 2], "ends behind the rows": [0, 1], "all three": []}[what]
    rng = np.random.default_rng(24)
    # a case of the good requests alone gives the reference; the call has all three
    rows = [cu[r + 1] - cu[r] if r in good else 0 for r in range(3)]
    c = Case(25, rows, keys, 16, 8, kind)
    ref, bound = c.reference()
    q = wl.normal_bf16(rng, (total, 16, 128))
    parents, first = np.full(total, -1, np.int32), 0
    for r, n in enumerate(rows):
        if n:
            q[cu[r]:cu[r] + n] = c.q[first:first + n]
            if kind == "tree":
                parents[cu[r]:cu[r] + n] = c.parents[first:first + n]
        first += n
    out = torch.full((total, 16, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    args = (to_dev(q), to_dev(np.array(cu, np.int32)), to_dev(np.array(keys, np.int32)), to_dev(c.table), to_dev(c.k), to_dev(c.v), most, out)
    if kind == "cross":
        qa.qa_cross_attn(*args)
    else:
        qa.qa_tree_attn(*args, parents=to_dev(parents))
    assert qa.qa_device_status() == 0x4
    got, owned, first = f64(out), np.zeros(total, bool), 0
    for r, n in enumerate(rows):
        if n:
            at = slice(cu[r], cu[r] + n)
            owned[at] = True
            assert (np.abs(got[at] - ref[first:first + n]) <= bound[first:first + n]).all(), r
        first += n
    assert (got[~owned] == 9).all()
    assert owned.sum() == sum(rows)


@pytest.mark.parametrize("rows", [[8], [50]])
def test_bad_parents_count_as_roots(rows):
    c = Case(21, rows, [33], 16, 8, "tree")
    bad = c.parents.copy()
    bad[5], bad[7], bad[3] = 5, -2, 2 ** 31 - 1
    c.parents = bad
    out = torch.zeros(sum(rows), 16, 128, dtype=torch.bfloat16, device="cuda")
    c.call(out=out, debug_checks=False)
    assert qa.qa_device_status() == 0x20
    c.parents = np.where(np.isin(np.arange(rows[0]), [3, 5, 7]), -1, bad).astype(np.int32)
    c.check(out)


def test_no_rows_at_all():
    z = torch.zeros(0, 16, 128, dtype=torch.bfloat16, device="cuda")
    c = Case(22, [3], [40], 16, 8, "tree")
    args = (to_dev(np.zeros(2, np.int32)), to_dev(np.array([40], np.int32)), to_dev(c.table), to_dev(c.k), to_dev(c.v))
    assert qa.qa_tree_attn(z, *args, 8, debug_checks=True).shape == (0, 16, 128)
    assert qa.qa_cross_attn(z, *args, 800, debug_checks=True).shape == (0, 16, 128)
    # rows, but of no request
    q = torch.ones(4, 16, 128, dtype=torch.bfloat16, device="cuda")
    for fn, most in ((qa.qa_tree_attn, 8), (qa.qa_tree_attn, 60), (qa.qa_cross_attn, 500)):
        out = torch.full_like(q, 4.0)
        fn(q, *args, most, out, debug_checks=True)
        assert bool((out == 4).all())


@pytest.mark.parametrize("kind, rows", [("tree", [8] * 6), ("tree", [40] * 6), ("cross", [170] * 3)])
def test_calls_repeat_bit_for_bit_whatever_the_workspace_holds(kind, rows):
    c = Case(23, rows, [700, 900, 20, 1500, 3, 64][:len(rows)], 16, 8, kind)
    size = qa.qa_rows_attn_workspace_size(c.most)
    ws = torch.full((size,), 0xff, dtype=torch.uint8, device="cuda")  # NaN in every float
    first = c.call(workspace=ws)
    c.check(first)
    for level in (0, 1, 2):
        ws.fill_(0x7f)
        torch.cuda.synchronize()
        assert torch.equal(c.call(workspace=ws, stable_metadata=level), first)


def test_a_larger_workspace_serves_fewer_rows():
    for hq, hkv in ((16, 8), (8, 8), (2, 1), (6, 3)):
        sizes = [qa.qa_rows_attn_workspace_size(n, n_q_heads=hq, n_kv_heads=hkv) for n in range(1, 200)]
        assert sizes == sorted(sizes)


def test_chained_layers_share_a_workspace():
    """Calls one behind another on a stream, trees and cross attention in turn, at each level of stable_metadata."""
    cases = [Case(30 + i, rows, keys, 16, 8, kind) for i, (rows, keys, kind) in enumerate([
        ([8, 3, 8], [900, 50, 300], "tree"), ([40, 3], [900, 50], "tree"), ([150, 3], [800, 90], "cross"), ([2, 2], [33, 1], "cross")])]
    ws = torch.empty(max(qa.qa_rows_attn_workspace_size(c.most) for c in cases), dtype=torch.uint8, device="cuda")
    alone = [c.call(workspace=ws) for c in cases]
    for c, x in zip(cases, alone):
        c.check(x)
    args = []
    for c in cases:
        a = [to_dev(c.q), to_dev(c.cu), to_dev(np.array(c.past, np.int32)), to_dev(c.table), to_dev(c.k), to_dev(c.v), c.most]
        kw = {} if c.kind == "cross" else dict(parents=to_dev(c.parents))
        args.append((qa.qa_cross_attn if c.kind == "cross" else qa.qa_tree_attn, a, kw))
    torch.cuda.synchronize()
    for level in (0, 1, 2):
        outs = [[torch.empty_like(x) for x in alone] for _ in range(20)]
        for row in outs:
            for (fn, a, kw), out in zip(args, row):
                fn(*a, out, workspace=ws, stable_metadata=level, **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for row in outs for x, y in zip(row, alone))
    assert qa.qa_device_status() == 0


@pytest.mark.parametrize("rows, kind", [([8, 3, 8], "tree"), ([40, 3, 12], "tree"), ([4, 1, 2], "cross"), ([150, 3, 64], "cross")])
def test_workspace_shared_with_the_decodes(rows, kind):
    """A step of one token over either cache, which counts its splits in the workspace, and drafted rows, in turn."""
    lens = (6000, 3, 9000, 700)
    x = wl.decode_workload(45, lens, num_pages=1100, max_pages=600)
    d = [to_dev(x[n]) for n in ("q", "k_pages", "v_pages", "page_table", "seq_lens")]
    w = test_kvq_decode_gpu.setup(44, lens)
    y = [to_dev(w[n]) for n in ("q", "k_pages", "v_pages", "table", "lens")]
    c = Case(26, rows, [900, 50, 2000], 16, 8, kind)
    size = max(qa.qa_rows_attn_workspace_size(c.most), qa.qa_kvq_decode_workspace_size(4, 0),
               qa.qa_decode_workspace_size(4, 9000, num_pages=1100, max_pages_per_seq=600))
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    one, four, many = qa.qa_decode_attn(*d), qa.qa_kvq_decode_attn(*y), c.call()
    c.check(many)
    for _ in range(3):
        got = c.call(workspace=ws, out=torch.full_like(many, 7.0), debug_checks=False)
        assert torch.equal(got, many)
        got = qa.qa_decode_attn(*d, torch.full_like(one, 7.0), workspace=ws)
        assert torch.equal(got, one)
        got = qa.qa_kvq_decode_attn(*y, torch.full_like(four, 7.0), workspace=ws)
        assert torch.equal(got, four)
        assert not ws[:4096 * 8 * 4].any()
    assert qa.qa_device_status() == 0


def test_streams_graphs_and_threads():
    c = [Case(40, [8, 5], [600, 30], 16, 8, "tree"), Case(41, [44, 5], [600, 30], 16, 8, "tree"), Case(42, [140], [555], 16, 8, "cross")]
    want = [x.call() for x in c]
    # a side stream, and a graph captured on it and replayed with other contents in the same buffers
    side = torch.cuda.Stream()
    for x, w in zip(c, want):
        x.check(w)
        q, cu, past, table, k, v = (to_dev(y) for y in (x.q, x.cu, np.array(x.past, np.int32), x.table, x.k, x.v))
        parents = None if x.parents is None else to_dev(x.parents)
        kw = {} if x.kind == "cross" else dict(parents=parents)
        fn = qa.qa_cross_attn if x.kind == "cross" else qa.qa_tree_attn
        ws = torch.empty(qa.qa_rows_attn_workspace_size(x.most), dtype=torch.uint8, device="cuda")
        out = torch.zeros_like(w)
        torch.cuda.synchronize()
        got = fn(q, cu, past, table, k, v, x.most, stream=side, **kw)
        side.synchronize()
        assert torch.equal(got, w)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            for _ in range(3):
                fn(q, cu, past, table, k, v, x.most, out, workspace=ws, **kw)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
        y = Case(140, x.rows, [p - 7 for p in x.past], 16, 8, x.kind)
        for dst, src in ((q, y.q), (past, np.array(y.past, np.int32))):
            dst.copy_(to_dev(src))
        if parents is not None:
            parents.copy_(to_dev(y.parents))
        x.q, x.past, x.parents = y.q, y.past, y.parents
        x.keys = [p + n if x.kind != "cross" else p for p, n in zip(x.past, x.rows)]
        graph.replay()
        torch.cuda.synchronize()
        x.check(out, "replay")

    # host threads with streams and workspaces of their own
    errors = []

    def work(i):
        try:
            x = c[i]
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                first = x.call(debug_checks=False)
                for _ in range(20):
                    got = x.call(debug_checks=False)
                s.synchronize()
                assert torch.equal(first, got)
                x.check(got)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


@pytest.mark.parametrize("rows", [[3, 2], [40, 2]])
def test_pages_past_four_gigabytes(rows):
    pages = (5 << 30) // (16 * 8 * 128 * 2)
    c = Case(50, rows, [100, 20], 16, 8, "tree")
    n = c.k.shape[0]
    pools = []
    for p in (c.k, c.v):
        big = torch.empty(pages, 16, 8, 128, dtype=torch.bfloat16, device="cuda")
        big[pages - n:] = to_dev(p)
        pools.append(big)
    table = np.where(c.table >= 0, c.table + pages - n, -1).astype(np.int32)
    got = qa.qa_tree_attn(to_dev(c.q), to_dev(c.cu), to_dev(np.array(c.past, np.int32)), to_dev(table), *pools, c.most,
                          parents=to_dev(c.parents), debug_checks=True)
    c.check(got)


def test_one_row_equals_the_decode():
    """A chain of one row a request is the single-token decode; cross attention of it too."""
    rng = np.random.default_rng(60)
    past = rng.integers(0, 900, 20).tolist()
    c = Case(61, [1] * 20, past, 16, 8, "chain")
    got = c.call()
    c.check(got)
    lens = to_dev(np.array(c.keys, np.int32))
    ref = qa.qa_decode_attn(to_dev(c.q), to_dev(c.k), to_dev(c.v), to_dev(c.table), lens)
    _, bound = c.reference()
    assert (np.abs(f64(got) - f64(ref)) <= 2 * bound).all()
    cross = qa.qa_cross_attn(to_dev(c.q), to_dev(c.cu), lens, to_dev(c.table), to_dev(c.k), to_dev(c.v), 1, debug_checks=True)
    assert np.array_equal(bits(cross), bits(got))


def test_a_job_may_take_longer_than_a_wait():
    """The last worker of 19 has 1.9 million tiles of the first request, 2.4 s of them, before three jobs of one tile: more
    than the 2 s that a wait inside the kernel lasts.  512 pages with keys of 0 make up that request again and again, but
    for its last page, whose keys score 181 more: the others' share is below 2^-230, and the result the mean of 16 values."""
    long_pages, rows, pages = 18 << 20, [1024, 192], 514
    rng = np.random.default_rng(80)
    v = wl.normal_bf16(rng, (pages, 16, 8, 128))
    k = np.zeros(v.shape, np.float32)
    k[-2:] = 16.0
    table = (torch.arange(2 * long_pages, dtype=torch.int32, device="cuda") % (pages - 2)).view(2, long_pages)
    table[0, -1], table[1, 0] = pages - 2, pages - 1
    keys = torch.tensor([16 * long_pages, 16], dtype=torch.int32, device="cuda")
    q = torch.ones(sum(rows), 16, 128, dtype=torch.bfloat16, device="cuda")
    got = qa.qa_cross_attn(q, to_dev(_rows.cumulative(rows)), keys, table, to_dev(wl.bf16_bits(k)), to_dev(v), max(rows), debug_checks=True)
    mean = np.repeat(wl.bf16_to_f64(v[-2:]).mean(1), 2, axis=1)  # [request, query head, 128]
    # probabilities of 1, sums of 16 bf16 values in fp32 and one rounding of the result to bf16
    bound = 2.0 ** -8 * np.abs(mean) + 2.0 ** -18
    for part, ref, most in zip(torch.split(got, rows), mean, bound):
        assert (np.abs(f64(part) - ref) <= most).all()
