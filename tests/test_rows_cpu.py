"""Host side of drafted rows over the paged cache and of cross attention,
without a GPU: the refusals of every entry point, the Python checks, and the
test definitions against ones written another way."""
import ctypes

import numpy as np
import pytest

import _kvq
import _rows
import workloads as wl
import paged_kv_gqa_attention_gb300 as qa
from test_kvq_cpu import FAKE, ODD, params, refused, rope

TWO = ctypes.c_void_p(0x1002)


def append(q=FAKE, ldq=0, k=FAKE, ldk=0, v=FAKE, ldv=0, cu=FAKE, past=FAKE, parents=FAKE, batch=2, total=5, table=FAKE,
           kp=FAKE, vp=FAKE, qo=FAKE, ldqo=0, r="rope", p=None):
    return qa._lib.qa_append_rows(q, ldq, k, ldk, v, ldv, cu, past, parents, batch, total, table, kp, vp, qo, ldqo,
                                  rope() if r == "rope" else r, p or params())


def tree_attn(q=FAKE, ldq=0, cu=FAKE, past=FAKE, parents=FAKE, batch=2, total=5, max_rows=4, table=FAKE, kp=FAKE, vp=FAKE,
              out=FAKE, p=None):
    return qa._lib.qa_tree_attn(q, ldq, cu, past, parents, batch, total, max_rows, table, kp, vp, out, p or params())


def cross_attn(q=FAKE, ldq=0, cu=FAKE, past=FAKE, batch=2, total=5, max_rows=4, table=FAKE, kp=FAKE, vp=FAKE, out=FAKE, p=None):
    return qa._lib.qa_cross_attn(q, ldq, cu, past, batch, total, max_rows, table, kp, vp, out, p or params())


def accept(draft=FAKE, target=FAKE, parents=FAKE, cu=FAKE, past=FAKE, batch=2, total=5, max_rows=4, table=FAKE, layers=1,
           kp=(0x1000,), vp=(0x1000,), n=FAKE, path=FAKE, nxt=FAKE, p=None):
    def pools(x):
        return None if x is None else (ctypes.c_void_p * max(1, len(x)))(*x)

    return qa._lib.qa_tree_accept(draft, target, parents, cu, past, batch, total, max_rows, table, layers, pools(kp), pools(vp),
                                  n, path, nxt, p or params())


@pytest.mark.parametrize("fn", [append, tree_attn, cross_attn, accept])
def test_rows_and_params_refuse(fn):
    most = 1024 if fn in (tree_attn, cross_attn) else 4096
    refused(fn(batch=0), "batch")
    refused(fn(batch=-3), "batch")
    refused(fn(batch=most + 1), "batch")
    refused(fn(total=-1), "total_rows")
    refused(fn(total=2**30 + 1), "total_rows")
    refused(fn(cu=None), "NULL")
    refused(fn(table=None), "NULL")
    refused(fn(kp=None), "NULL")
    refused(fn(vp=None), "NULL")
    refused(fn(cu=TWO), "aligned")
    refused(fn(past=TWO), "aligned")
    refused(fn(table=TWO), "aligned")
    if fn is not cross_attn:
        refused(fn(parents=TWO), "aligned")
    for field, bad in (("head_dim", 64), ("n_kv_heads", 9), ("n_kv_heads", 0), ("n_q_heads", 24), ("page_size", 32),
                       ("num_pages", 0), ("max_pages_per_seq", 0), ("abi_version", 99), ("stable_metadata", 3), ("scale", -1.0)):
        refused(fn(p=params(**{field: bad})), "")


def test_append_refuses():
    refused(append(k=None), "NULL")
    refused(append(v=None), "NULL")
    refused(append(qo=None), "NULL")
    for name in ("q", "k", "v", "kp", "vp", "qo"):
        refused(append(**{name: ODD}), "aligned")
    refused(append(ldq=2040), "ldq")
    refused(append(ldq=2052), "ldq")
    refused(append(ldk=1016), "ldk")
    refused(append(ldv=2**31 + 8), "ldv")
    refused(append(ldqo=-8), "ldq_out")
    refused(append(ldq=4096), "row stride")  # in place
    refused(append(ldqo=4096), "row stride")
    refused(append(r=rope(theta=0.5)), "theta")
    refused(append(r=rope(k_gain=None)), "gain")
    refused(append(r=rope(rms_eps=0.0)), "rms_eps")
    refused(append(r=rope(n_axes=5)), "n_axes")
    refused(append(r=rope(n_axes=2, positions=None)), "positions")
    refused(append(r=rope(q_gain=0x1004)), "aligned")
    axes = np.zeros(64, np.uint8)
    axes[7] = 1
    refused(append(r=rope(pair_axis=axes.ctypes.data)), "pair_axis[7]")
    # nothing to do, nothing launched: empty tensors have no address
    assert append(total=0, q=None, qo=None, k=None, v=None) == 0
    assert append(total=0) == 0
    assert append(total=0, past=None, parents=None, r=None) == 0


@pytest.mark.parametrize("fn", [tree_attn, cross_attn])
def test_attention_refuses(fn):
    for name in ("q", "past", "out"):
        refused(fn(**{name: None}), "NULL")
    for name in ("q", "kp", "vp", "out"):
        refused(fn(**{name: ODD}), "aligned")
    refused(fn(max_rows=0), "max_rows")
    refused(fn(max_rows=-1), "max_rows")
    refused(fn(ldq=2040), "ldq")
    refused(fn(ldq=2052), "ldq")
    refused(fn(p=params(num_pages=2**27)), "num_pages")
    refused(fn(batch=1024, p=params(max_pages_per_seq=2**20 + 1)), "max_pages_per_seq")
    assert fn() in (-1, -3)  # no workspace; without a GPU, no device
    assert "workspace" in qa.qa_last_error() or "device" in qa.qa_last_error()
    assert fn(total=0, q=None, out=None) == 0
    # blocks of 64 rows times pages: the largest call that is taken, and the next
    fits = params(max_pages_per_seq=2**20)
    assert fn(batch=1024, max_rows=64, p=fits) in (-1, -3)
    assert "max_pages_per_seq" not in qa.qa_last_error()


@pytest.mark.parametrize("fn", [tree_attn, cross_attn])
def test_positions_whose_tiles_end_past_31_bits_are_refused(fn):
    """2^31 - 128 positions end a tile of 128 keys below 2^31; one page more does not."""
    for pages in (2**27 - 7, 2**27 - 1):
        refused(fn(batch=1, p=params(max_pages_per_seq=pages)), "above 134217720")
    assert fn(batch=1, p=params(max_pages_per_seq=2**27 - 8)) in (-1, -3)  # no workspace; without a GPU, no device
    assert "max_pages_per_seq" not in qa.qa_last_error()


def test_row_limits():
    refused(tree_attn(max_rows=65), "[1, 64]")
    refused(accept(max_rows=65), "[1, 64]")
    refused(accept(max_rows=0), "[1, 64]")
    refused(cross_attn(batch=1024, max_rows=65, p=params(max_pages_per_seq=2**20)), "max_rows / 64")
    refused(cross_attn(max_rows=2**31 - 1, p=params(max_pages_per_seq=2**30)), "max_pages_per_seq")
    refused(cross_attn(max_rows=2**31 - 1, p=params(max_pages_per_seq=2**26)), "max_rows / 64")
    assert qa._lib.qa_rows_attn_workspace_size(0, params()) == 0 and "max_rows" in qa.qa_last_error()
    assert qa._lib.qa_rows_attn_workspace_size(4, params(n_kv_heads=3)) == 0
    with pytest.raises(qa.QAError):
        qa.qa_rows_attn_workspace_size(0)
    with pytest.raises(qa.QAError):
        qa.qa_rows_attn_workspace_size(8, n_q_heads=16, n_kv_heads=4)


def test_accept_refuses():
    refused(accept(layers=-1), "n_layers")
    refused(accept(layers=65), "n_layers")
    for name in ("draft", "target", "past", "n", "path", "nxt"):
        refused(accept(**{name: None}), "NULL")
    for name in ("draft", "target", "n", "path", "nxt"):
        refused(accept(**{name: TWO}), "aligned")
    refused(accept(layers=2, kp=(0x1000, 0), vp=(0x1000, 0x1000)), "NULL")
    refused(accept(layers=2, kp=(0x1000, 0x1000), vp=(0x1000, 0x1008)), "aligned")


def test_accept_refuses_pools_that_overlap():
    """A pool may be listed several times (layers that share a cache); another one that begins inside it may not."""
    pages = 3
    size = pages * 16 * 8 * 128 * 2
    p = params(num_pages=pages)
    a = 1 << 30
    for kp, vp in (((a,), (a + 16,)), ((a,), (a + size - 16,)), ((a, a + 2 * size), (a, a + size + 256)), ((a, a + size), (a - 16, a - size))):
        refused(accept(layers=len(kp), kp=kp, vp=vp, p=p), "overlap")


def test_python_checks():
    torch = pytest.importorskip("torch")
    rows = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    pool = torch.zeros(3, 16, 8, 128, dtype=torch.bfloat16)
    cu, table = torch.zeros(2, dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32)
    past, ids = torch.zeros(1, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError, match="k must be a torch.Tensor"):
        qa.qa_append_rows(None, None, rows, cu, table, pool, pool)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        qa.qa_append_rows(None, rows, rows, cu, table, pool, pool)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        qa.qa_tree_attn(rows, cu, past, table, pool, pool, 4)
    with pytest.raises(TypeError, match="q must be a torch.Tensor"):
        qa.qa_cross_attn(None, cu, past, table, pool, pool, 4)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        qa.qa_cross_attn(rows, cu, past, table, pool, pool, 4)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        qa.qa_tree_accept(ids, ids, None, cu, past, table, [pool], [pool], 4)
    with pytest.raises(TypeError, match="draft must be a torch.Tensor"):
        qa.qa_tree_accept(None, ids, None, cu, past, table, [pool], [pool], 4)


# ------------------------------------------------- the definitions themselves

def test_trees_and_what_a_row_sees():
    rng = np.random.default_rng(1)
    for n in (1, 2, 7, 64):
        parents = _rows.tree(rng, n)
        assert ((parents >= -1) & (parents < np.arange(n))).all()
        seen, depth = _rows.seen(parents), _rows.depths(parents)
        # reachability by powers of the edges' matrix
        edges = np.eye(n, dtype=bool)
        for i, p in enumerate(parents):
            if p >= 0:
                edges[i, p] = True
        reach = np.linalg.matrix_power(edges.astype(object), n) > 0
        np.testing.assert_array_equal(seen, reach)
        np.testing.assert_array_equal(depth, seen.sum(1) - 1)


def test_attention_definition():
    """Two requests over pages in any order, against a loop over rows and heads."""
    rng = np.random.default_rng(2)
    rows, past, H, Hq = [3, 2], [19, 0], 2, 4
    keys = [p + n for p, n in zip(past, rows)]
    table, pages = _kvq.page_table(rng, keys)
    k_pool, v_pool = (wl.bf16_to_f64(wl.normal_bf16(rng, (pages, 16, H, 128))) for _ in range(2))
    q = wl.bf16_to_f64(wl.normal_bf16(rng, (5, Hq, 128)))
    parents = [np.array([-1, 0, 0], np.int32), np.array([-1, -1], np.int32)]
    visible = [np.concatenate((np.ones((n, p), bool), _rows.seen(t)), 1) for n, p, t in zip(rows, past, parents)]
    got, bound = _rows.attention(q, k_pool, v_pool, table, rows, keys, visible)
    t = 0
    for b in range(2):
        for i in range(rows[b]):
            see = [j for j in range(keys[b]) if j < past[b] or _rows.seen(parents[b])[i, j - past[b]]]
            for h in range(Hq):
                k = np.array([k_pool[table[b, j // 16], j % 16, h // 2] for j in see])
                v = np.array([v_pool[table[b, j // 16], j % 16, h // 2] for j in see])
                s = k @ q[t, h] / np.sqrt(128)
                w = np.exp(s - s.max())
                np.testing.assert_allclose(got[t, h], w @ v / w.sum(), rtol=1e-12, atol=1e-13)
            t += 1
    assert (bound >= 0).all() and bound.max() < 0.1
