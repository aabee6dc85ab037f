"""GPU parity of qa_rope_rows (per-head QK-norm and rotary positions with
several axes on packed rows) against the definition in 64 bits: every bf16
result is a rounding of a value within the fp32 error (_util)."""
import numpy as np
import pytest

import _kvq
import workloads as wl
from _util import assert_rounded_match, bits, to_dev

pytestmark = pytest.mark.gpu
import torch  # noqa: E402

import paged_kv_gqa_attention_gb300 as qa  # noqa: E402


def inputs(seed, rows, hq, hkv, dim, axes, norm):
    rng = np.random.default_rng(seed)
    q, k = wl.normal_bf16(rng, (rows, hq, dim)), wl.normal_bf16(rng, (rows, hkv, dim))
    pos = rng.integers(0, 1 << 18, size=(axes, rows)).astype(np.int32)
    pos[:, 0] = 0
    pos[-1, -1] = (1 << 18) - 1
    gains = [wl.bf16_to_f64(wl.bf16_bits(rng.uniform(0.5, 1.5, size=dim).astype(np.float32))).astype(np.float32)
             for _ in range(2)] if norm else [None, None]
    axis = rng.integers(0, axes, size=dim // 2).astype(np.uint8)
    return q, k, pos, gains, axis


def check(got, x, pos, gain, axis, what):
    ref, size = _kvq.rope(wl.bf16_to_f64(x), pos, gain, axis)
    assert_rounded_match(bits(got), ref, size, what)


def run(q, k, pos, gains, axis, **kw):
    dq, dk = to_dev(q), None if k is None else to_dev(k)
    g = [None if x is None else to_dev(x) for x in gains]
    return qa.qa_rope_rows(dq, dk, to_dev(pos), q_gain=g[0], k_gain=g[1], pair_axis=axis, debug_checks=True, **kw)


@pytest.mark.parametrize("rows, hq, hkv, dim, axes, norm", [
    (1, 16, 8, 128, 3, True), (1, 1, 1, 64, 1, False), (2, 16, 8, 128, 1, True), (3, 14, 14, 64, 2, False),
    (5, 5, 3, 128, 4, True), (33, 3, 1, 64, 3, True), (200, 16, 8, 128, 3, False), (257, 40, 5, 128, 2, True),
    (1031, 16, 8, 128, 3, True), (2900, 14, 14, 64, 2, False), (4099, 2, 1, 128, 1, True),
])
def test_matches_the_definition(rows, hq, hkv, dim, axes, norm):
    q, k, pos, gains, axis = inputs(rows, rows, hq, hkv, dim, axes, norm)
    qo, ko = run(q, k, pos, gains, axis)
    check(qo, q, pos, gains[0], axis, "q")
    check(ko, k, pos, gains[1], axis, "k")


def test_default_axis_and_queries_alone():
    q, _, pos, gains, _ = inputs(2, 19, 16, 8, 128, 1, True)
    qo, ko = run(q, None, pos[0], gains, None)
    assert ko is None
    check(qo, q, pos, gains[0], None, "q")


@pytest.mark.parametrize("rows, stable", [(7, False), (700, True)])
def test_rows_of_a_fused_projection(rows, stable):
    q, k, pos, gains, axis = inputs(3, rows, 16, 8, 128, 3, True)
    x = torch.full((rows, 33, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    x[:, :16], x[:, 16:24], x[:, 24:] = to_dev(q), to_dev(k), 7.0
    g = [to_dev(v) for v in gains]
    dpos = to_dev(pos)
    torch.cuda.synchronize()
    # into fresh rows, then in place: the same bits, and the rest of the rows untouched
    qo, ko = qa.qa_rope_rows(x[:, :16], x[:, 16:24], dpos, q_gain=g[0], k_gain=g[1], pair_axis=axis, stable_metadata=stable)
    check(qo, q, pos, gains[0], axis, "q")
    check(ko, k, pos, gains[1], axis, "k")
    qa.qa_rope_rows(x[:, :16], x[:, 16:24], dpos, x[:, :16], x[:, 16:24], q_gain=g[0], k_gain=g[1], pair_axis=axis,
                    stable_metadata=stable, debug_checks=True)
    assert torch.equal(x[:, :16], qo) and torch.equal(x[:, 16:24], ko) and bool((x[:, 24:] == 7).all())


def test_bad_positions_leave_their_rows():
    q, k, pos, gains, axis = inputs(4, 40, 16, 8, 128, 3, True)
    pos[1, 3], pos[2, 17], pos[0, 39] = -1, 1 << 18, 2 ** 31 - 1
    bad = [3, 17, 39]
    dq, dk = to_dev(q), to_dev(k)
    qo, ko = torch.full_like(dq, 5.0), torch.full_like(dk, 5.0)
    with pytest.raises(qa.QAError, match="bad position"):
        run(q, k, pos, gains, axis, q_out=qo, k_out=ko)
    assert bool((qo[bad] == 5).all()) and bool((ko[bad] == 5).all())
    ok = np.setdiff1d(np.arange(40), bad)
    check(qo[torch.from_numpy(ok).cuda()], q[ok], pos[:, ok], gains[0], axis, "q")
    assert qa.qa_device_status() == 0  # read and cleared


def test_no_rows():
    q, k = torch.zeros(0, 16, 128, dtype=torch.bfloat16, device="cuda"), None
    qo, _ = qa.qa_rope_rows(q, k, torch.zeros(1, 0, dtype=torch.int32, device="cuda"))
    assert qo.shape == (0, 16, 128)


def test_refused_tensors():
    q, k, pos, gains, axis = inputs(6, 8, 16, 8, 128, 2, True)
    dq, dk, dpos, g = to_dev(q), to_dev(k), to_dev(pos), [to_dev(v) for v in gains]
    for bad, error, word in (
            (dict(q=dq.float()), TypeError, "bfloat16"), (dict(q=dq[0]), ValueError, "dims"),
            (dict(q=dq.transpose(1, 2)), ValueError, "contiguous"), (dict(q=dq[:1].expand(8, 16, 128)), ValueError, "overlap"),
            (dict(q=dq.cpu()), ValueError, "CUDA"), (dict(k=dk[:7]), ValueError, "shapes"), (dict(k=dk[:, :, :64].contiguous()), ValueError, "shapes"),
            (dict(positions=dpos[:, :5]), ValueError, "positions"), (dict(positions=dpos.long()), TypeError, "int32"),
            (dict(positions=dpos.T), ValueError, "positions"), (dict(positions=None), ValueError, "required"),
            (dict(q_out=torch.empty_like(dq[:7])), ValueError, "shapes"), (dict(q_gain=g[0][:64]), ValueError, "head_dim"),
            (dict(q_gain=None), qa.QAError, "both"), (dict(pair_axis=[0] * 63), ValueError, "pair_axis"),
            (dict(pair_axis=[-1] * 64), ValueError, "pair_axis"), (dict(pair_axis=3), TypeError, "pair_axis"),
            (dict(pair_axis=[2] * 64), qa.QAError, "pair_axis"), (dict(stream=5), TypeError, "stream"),
            (dict(rope_theta="x"), TypeError, "rope_theta"), (dict(rms_eps=0.0), qa.QAError, "rms_eps"),
            (dict(stable_metadata=3), qa.QAError, "stable_metadata")):
        args = dict(dict(q=dq, k=dk, positions=dpos, q_gain=g[0], k_gain=g[1], pair_axis=axis), **bad)
        with pytest.raises(error, match=word):
            qa.qa_rope_rows(**args)


def test_smallest_frequency_base():
    """theta 1: every pair turns by a radian a position, 41721 turns at the last one."""
    q, k, pos, gains, axis = inputs(8, 9, 16, 8, 128, 1, False)
    pos = np.array([[0, 1, 2, 3, 1000, 65537, 131072, 262142, 262143]], np.int32)
    got, _ = qa.qa_rope_rows(to_dev(q), None, to_dev(pos), rope_theta=1.0)
    want, size = _kvq.rope(wl.bf16_to_f64(q), pos, None, axis, theta=1.0)
    torch.cuda.synchronize()
    assert_rounded_match(bits(got), want, size, "theta 1")


def test_refused_when_checked():
    """A refusal of a checked call, too, is an exception."""
    rows = 2**31  # of no heads: only the positions take memory
    empty, pos = torch.empty(rows, 0, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(rows, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="rows"):
        qa.qa_rope_rows(empty, None, pos, debug_checks=True)
    pos = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 16, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError, match="debug_checks"):
        qa.qa_rope_rows(q, None, pos, debug_checks=np.zeros(2))
    with pytest.raises(ValueError, match="stable_metadata"):
        qa.qa_rope_rows(q, None, pos, stable_metadata=2**32)


def test_kinds_of_pair_axis():
    q, k, pos, gains, axis = inputs(7, 8, 16, 8, 128, 3, True)
    dq, dpos = to_dev(q), to_dev(pos)
    outs = [qa.qa_rope_rows(dq, None, dpos, pair_axis=x)[0] for x in (axis, axis.tolist(), bytes(axis), axis.astype(np.int64), tuple(axis))]
    for o in outs:
        check(o, q, pos, None, axis, "q")


def test_graph_and_other_stream():
    q, k, pos, gains, axis = inputs(5, 65, 16, 8, 128, 3, True)
    dq, dk, dpos, g = to_dev(q), to_dev(k), to_dev(pos), [to_dev(v) for v in gains]
    qo, ko = torch.empty_like(dq), torch.empty_like(dk)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()

    def call():
        qa.qa_rope_rows(dq, dk, dpos, qo, ko, q_gain=g[0], k_gain=g[1], pair_axis=axis, stream=s)

    call()
    torch.cuda.synchronize()
    first = qo.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    qo.zero_()
    dq.copy_(to_dev(q))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(qo, first)
    check(qo, q, pos, gains[0], axis, "q")


def test_agrees_with_the_decode_append():
    w = wl.decode_append_workload(41, (33, 250, 1000, 1), num_pages=96, max_pages=64)
    d = {n: to_dev(w[n]) for n in ("q_new", "k_new", "v_new", "q_gain", "k_gain", "page_table", "seq_lens", "k_pages", "v_pages")}
    q1 = qa.qa_decode_append(d["q_new"], d["k_new"], d["v_new"], d["q_gain"], d["k_gain"], d["page_table"], d["seq_lens"],
                             d["k_pages"], d["v_pages"])
    q2, _ = qa.qa_rope_rows(d["q_new"], d["k_new"], d["seq_lens"] - 1, q_gain=d["q_gain"], k_gain=d["k_gain"])
    torch.cuda.synchronize()
    # the same formula in fp32, summed in another order: a rare last-bit difference
    assert int((q1 != q2).sum()) <= max(4, q1.numel() // 200)
