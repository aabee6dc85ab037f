"""qa_tree_accept on the GPU against the definition (whole numbers and moved
bits, all exact), and the calls of a drafting decoder in a row."""
import numpy as np
import pytest

import _kvq
import _rows
import workloads as wl
from _util import bits, f64, to_dev

pytestmark = pytest.mark.gpu
import torch  # noqa: E402

import paged_kv_gqa_attention_gb300 as qa  # noqa: E402


class Case:
    def __init__(self, seed, rows, past, layers=2, hkv=8, tokens=6, chain=False, agree=0.8):
        rng = np.random.default_rng(seed)
        self.rows, self.past, self.layers = list(rows), list(past), layers
        self.table, pages = _rows.page_table(rng, [a + b for a, b in zip(rows, past)])
        self.pools = [[rng.integers(0, 1 << 16, size=(pages, 16, hkv, 128)).astype(np.uint16) for _ in range(layers)] for _ in range(2)]
        trees = [_rows.tree(rng, n) for n in rows]
        self.parents = None if chain else np.concatenate(trees).astype(np.int32)
        total = sum(rows)
        self.draft = rng.integers(0, tokens, total).astype(np.int32)
        self.target = rng.integers(0, tokens, total).astype(np.int32)
        first = 0
        for n, t in zip(rows, trees):  # often the token of a child
            t = np.arange(n) - 1 if chain else t
            for i in range(n):
                children = np.nonzero(t == i)[0]
                if len(children) and rng.random() < agree:
                    self.target[first + i] = self.draft[first + rng.choice(children)]
            first += n
        self.cu = _rows.cumulative(rows)
        self.most = max(1, max(rows))

    def call(self, most=None, **kw):
        self.dev = [[to_dev(p) for p in side] for side in self.pools]
        return qa.qa_tree_accept(to_dev(self.draft), to_dev(self.target), None if self.parents is None else to_dev(self.parents),
                                 to_dev(self.cu), to_dev(np.array(self.past, np.int32)), to_dev(self.table), *self.dev,
                                 most or self.most, **({"debug_checks": True} | kw))

    def check(self, got, most=None, skipped=(), still=()):
        """skipped: requests that are not settled; still: pairs (request, place on its path) that are not moved."""
        count, path, token = (x.cpu().numpy() for x in got)
        paths, tokens = _rows.accept(self.draft, self.target, self.parents, self.rows)
        most = most or self.most
        want = np.full((len(self.rows), most), -1, np.int32)
        for b, p in enumerate(paths):
            if b in skipped:
                paths[b], tokens[b] = [], None
            else:
                want[b, :len(p)] = p
        np.testing.assert_array_equal(count, [len(p) for p in paths])
        np.testing.assert_array_equal(path, want)
        np.testing.assert_array_equal(token, [-1 if t is None else t for t in tokens])
        for side, dev in zip(self.pools, self.dev):
            for pool, d in zip(side, dev):
                ref = pool.copy()
                for b, p in enumerate(paths):
                    at = lambda i: (self.table[b, (self.past[b] + i) // 16], (self.past[b] + i) % 16)  # noqa: E731, B023
                    for j, i in enumerate(p):
                        if (b, j) not in still:
                            ref[at(j)] = pool[at(i)]
                np.testing.assert_array_equal(bits(d), ref)
        return paths


@pytest.mark.parametrize("rows, past", [
    ([1], [0]), ([1], [31]), ([2], [15]), ([8], [13]), ([64], [0]), ([64], [9]), ([33, 32, 31, 1], [1, 2, 3, 4]),
    ([0, 7, 0], [4, 40, 0]), ([20] * 50, list(range(50))),
])
@pytest.mark.parametrize("layers, hkv, chain", [(1, 8, False), (3, 2, False), (2, 8, True), (0, 1, False)])
def test_settles(rows, past, layers, hkv, chain):
    for agree in (0.0, 0.8, 1.0):
        c = Case(len(rows) + rows[0] + layers, rows, past, layers, hkv, chain=chain, agree=agree)
        paths = c.check(c.call())
        if agree == 1.0 and chain and max(rows) > 1 and layers:
            assert max(len(p) for p in paths) > 1


def test_sixty_four_layers_and_every_head_count():
    for hkv in range(1, 9):
        c = Case(hkv, [12, 3], [20, 0], 64 if hkv == 3 else 2, hkv, agree=1.0)
        c.check(c.call())


@pytest.mark.parametrize("batch, layers", [(2, 2), (80, 64)])
def test_a_pool_listed_several_times_is_settled_once(batch, layers):
    """Layers that share a cache, and keys and values in one pool.  With 80 requests of 64 layers the CTAs of a pool's
    later mentions start when those of its first are done."""
    rows = [24] * batch
    c = Case(10, rows, [5] * batch, 3, 2)
    keep = np.arange(24) % 3 != 1  # every path leaves rows out, so that it moves them
    keep[0] = True
    last = np.maximum.accumulate(np.where(keep, np.arange(24), 0))
    one = np.where(np.arange(24) > 0, np.concatenate(([0], last[:-1])), -1)
    c.parents = np.tile(one, batch).astype(np.int32)
    tokens = np.where(keep, 1, 2)
    c.draft = np.tile(tokens, batch).astype(np.int32)
    c.target = np.ones(24 * batch, np.int32)
    c.dev = [[to_dev(p) for p in side] for side in c.pools]
    (a, b, _), (d, e, _) = c.dev
    ks, vs = ([a, b, a, a] * layers)[:layers], ([d, a, b, e] * layers)[:layers]
    got = qa.qa_tree_accept(to_dev(c.draft), to_dev(c.target), to_dev(c.parents), to_dev(c.cu), to_dev(np.array(c.past, np.int32)),
                            to_dev(c.table), ks, vs, 24, debug_checks=True)
    c.dev = [[a, b], [d, e if layers > 3 else d]]
    c.pools = [c.pools[0][:2], [c.pools[1][0], c.pools[1][1] if layers > 3 else c.pools[1][0]]]
    paths = c.check(got)
    assert paths == [list(np.nonzero(keep)[0])] * batch


def test_ties_go_to_the_first_row():
    c = Case(1, [6], [5], 1)
    c.parents = np.array([-1, 0, 0, 0, 2, 2], np.int32)
    c.draft = np.array([9, 4, 7, 7, 1, 1], np.int32)
    c.target = np.array([7, 0, 1, 1, 3, 8], np.int32)
    paths = c.check(c.call())
    assert paths == [[0, 2, 4]]


def test_roots_other_than_row_zero_are_never_accepted():
    c = Case(2, [5], [5], 1)
    c.parents = np.array([-1, -1, 0, 1, -1], np.int32)
    c.draft = np.array([1, 1, 1, 1, 1], np.int32)
    c.target = np.array([1, 1, 1, 1, 1], np.int32)
    assert c.check(c.call()) == [[0, 2]]


def test_any_token_is_a_token():
    c = Case(3, [4], [5], 1)
    c.parents = np.array([-1, 0, 1, 2], np.int32)
    c.draft = np.array([0, -1, -2 ** 31, 2 ** 31 - 1], np.int32)
    c.target = np.array([-1, -2 ** 31, 2 ** 31 - 1, -1], np.int32)
    assert c.check(c.call()) == [[0, 1, 2, 3]]


def test_refusals_on_the_device():
    rows, past = [20, 7, 12], [10, 3, 30]
    c = Case(4, rows, past, agree=1.0)
    c.past[1] = -1
    got = c.call(debug_checks=False)
    assert qa.qa_device_status() == 0x2
    c.past[1] = 3
    c.check(got, skipped=[1])
    with pytest.raises(qa.QAError, match="bad length"):
        c.call(most=12)
    got = c.call(most=12, debug_checks=False)
    assert qa.qa_device_status() == 0x2
    c.check(got, most=12, skipped=[0])

    c = Case(4, rows, past, agree=1.0)
    c.cu[3] += 1
    got = c.call(debug_checks=False)
    assert qa.qa_device_status() == 0x4
    c.check(got, skipped=[2])

    # a bad page: rows from or to it stay
    c = Case(5, [20], [10], agree=1.0, chain=False)
    c.parents = np.array([-1] + [0] * 9 + [5, 10, 11] + [0] * 7, np.int32)
    c.draft = np.arange(20).astype(np.int32)
    c.target[:] = 99
    c.target[0], c.target[5], c.target[10], c.target[11] = 5, 10, 11, 12
    table = c.table
    c.table = table.copy()
    c.table[0, 1] = -1  # positions 16 .. 31: rows 6 .. 19
    got = c.call(debug_checks=False)
    assert qa.qa_device_status() == 0x1
    c.table = table
    assert c.check(got, still=[(0, 2), (0, 3), (0, 4)]) == [[0, 5, 10, 11, 12]]

    c = Case(6, [9], [10], agree=1.0)
    bad = c.parents.copy()
    bad[4], bad[7] = 4, -9
    c.parents = bad
    got = c.call(debug_checks=False)
    assert qa.qa_device_status() == 0x20
    c.parents = np.where(np.isin(np.arange(9), [4, 7]), -1, bad).astype(np.int32)
    c.check(got)


def test_given_outputs_streams_levels_and_a_graph():
    c = Case(7, [20, 7, 12], [10, 3, 30], agree=1.0)
    outs = [torch.full(s, 77, dtype=torch.int32, device="cuda") for s in ((3,), (3, 64), (3,))]
    got = c.call(most=64, n_accepted=outs[0], path=outs[1], next_token=outs[2])
    assert all(a is b for a, b in zip(got, outs))
    c.check(got, most=64)
    side = torch.cuda.Stream()
    for level in (0, 1, 2):
        torch.cuda.synchronize()
        got = c.call(stream=side, stable_metadata=level)
        c.check(got)
    d = Case(8, [20, 7, 12], [10, 3, 30], agree=1.0)
    dev = [to_dev(x) for x in (c.draft, c.target, c.parents, c.cu, np.array(c.past, np.int32), d.table)]
    pools = [[to_dev(p) for p in s] for s in d.pools]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qa.qa_tree_accept(*dev, *pools, 64, *outs)
    for dst, src in zip(dev, (d.draft, d.target, d.parents)):
        dst.copy_(to_dev(src))
    graph.replay()
    torch.cuda.synchronize()
    d.dev = pools
    d.check(outs, most=64)


def test_drafting_run():
    """Two layers of a decoder with cross attention for several drafted steps: states laid into pages, drafted rows appended,
    attended, cross-attended and settled, each call on the cache that the calls before it left; against the definitions
    on a cache of its own that holds accepted rows only."""
    rng = np.random.default_rng(9)
    layers, hq, hkv, batch, states = 2, 16, 8, 3, [40, 130, 17]
    gains = [wl.bf16_to_f64(wl.bf16_bits(rng.uniform(0.5, 1.5, 128).astype(np.float32))).astype(np.float32) for _ in range(2)]
    dg = [to_dev(g) for g in gains]
    # the encoder's states, once
    st_table, st_pages = _rows.page_table(rng, states)
    st = [[wl.normal_bf16(rng, (sum(states), hkv, 128)) for _ in range(2)] for _ in range(layers)]
    st_pool = [[torch.full((st_pages, 16, hkv, 128), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(layers)]
    st_cu, d_states, d_st_table = to_dev(_rows.cumulative(states)), to_dev(np.array(states, np.int32)), to_dev(st_table)
    for x, p in zip(st, st_pool):
        qa.qa_append_rows(None, to_dev(x[0]), to_dev(x[1]), st_cu, d_st_table, *p, rotate=False, debug_checks=True)
    table, pages = _rows.page_table(rng, [200] * batch)
    pool = [[torch.full((pages, 16, hkv, 128), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(layers)]
    d_table = to_dev(table)
    past = [0, 0, 0]
    held = [[[np.zeros((0, hkv, 128)) for _ in range(2)] for _ in range(batch)] for _ in range(layers)]  # accepted rows
    ws = torch.empty(qa.qa_rows_attn_workspace_size(64), dtype=torch.uint8, device="cuda")
    for step in range(5):
        rows = [[20, 31, 7], [1, 8, 16], [40, 64, 3], [5, 5, 5], [16, 1, 64]][step]
        total, most = sum(rows), max(rows)
        trees = [_rows.tree(rng, n, back=4) for n in rows]
        parents = np.concatenate(trees).astype(np.int32)
        draft = rng.integers(0, 4, total).astype(np.int32)
        target = rng.integers(0, 4, total).astype(np.int32)
        cu, d_past, d_parents = to_dev(_rows.cumulative(rows)), to_dev(np.array(past, np.int32)), to_dev(parents)
        turn = np.concatenate([p + _rows.depths(t) for p, t in zip(past, trees)])
        new = []
        for layer in range(layers):
            q, k, v = (wl.normal_bf16(rng, (total, h, 128)) for h in (hq, hkv, hkv))
            qr = qa.qa_append_rows(to_dev(q), to_dev(k), to_dev(v), cu, d_table, *pool[layer], n_past=d_past, parents=d_parents,
                                   q_gain=dg[0], k_gain=dg[1])
            out = qa.qa_tree_attn(qr, cu, d_past, d_table, *pool[layer], most, parents=d_parents, workspace=ws, stable_metadata=1)
            cross = qa.qa_cross_attn(out, cu, d_states, d_st_table, *st_pool[layer], most, workspace=ws, stable_metadata=1)
            assert qa.qa_device_status() == 0
            # the definitions: rows of this step as the calls rounded them, the cache's as held
            kr = [f64(pool[layer][0])[p, s] for p, s in [_rows.places(table, past, rows)]][0]
            ref_k, size = _kvq.rope(wl.bf16_to_f64(k), turn, gains[1], None)
            assert (np.abs(kr - ref_k) <= 2.0 ** -8 * np.abs(ref_k) + 2.0 ** -18 * size).all()
            vr = wl.bf16_to_f64(v)
            new.append((kr, vr))
            cu_n = _rows.cumulative(rows)
            keys = [p + n for p, n in zip(past, rows)]
            flat = [np.full((-(-sum(keys) // 16) + batch + 1, 16, hkv, 128), np.nan) for _ in range(2)]
            t2, at = np.full((batch, 40), -1, np.int32), 0
            for b in range(batch):
                for side in range(2):
                    x = np.concatenate((held[layer][b][side], new[layer][side][cu_n[b]:cu_n[b + 1]]))
                    pad = np.concatenate((x, np.full((-len(x) % 16, hkv, 128), np.nan))).reshape(-1, 16, hkv, 128)
                    flat[side][at:at + len(pad)] = pad
                t2[b, :len(pad)] = np.arange(at, at + len(pad))
                at += len(pad)
            ref, bound = _rows.attention(f64(qr), flat[0], flat[1], t2, rows, keys, _rows.tree_visible(parents, rows, past))
            assert (np.abs(f64(out) - ref) <= bound).all()
            ref, bound = _rows.attention(f64(out), f64(st_pool[layer][0]), f64(st_pool[layer][1]), st_table, rows, states, None)
            assert (np.abs(f64(cross) - ref) <= bound).all()
        count, path, token = qa.qa_tree_accept(to_dev(draft), to_dev(target), d_parents, cu, d_past, d_table,
                                               [p[0] for p in pool], [p[1] for p in pool], most, debug_checks=True)
        paths, tokens = _rows.accept(draft, target, parents, rows)
        assert count.tolist() == [len(p) for p in paths] and token.tolist() == [int(t) for t in tokens]
        assert [[x for x in row if x >= 0] for row in path.tolist()] == paths
        for layer in range(layers):
            for b in range(batch):
                for side in range(2):
                    rows_b = new[layer][side][cu_n[b]:cu_n[b + 1]][paths[b]]
                    held[layer][b][side] = np.concatenate((held[layer][b][side], rows_b))
        past = [p + len(x) for p, x in zip(past, paths)]
        for layer in range(layers):  # the cache now holds the accepted rows, in order
            for side in range(2):
                got = f64(pool[layer][side])
                for b in range(batch):
                    p, s = _rows.places(table[b:b + 1], [0], [past[b]])
                    np.testing.assert_array_equal(got[p, s], held[layer][b][side])
    assert sum(past) > 5 * batch  # a step accepts row 0 of each request, so more of them means drafted tokens were accepted
