"""GPU tests of qa_kvq_write and qa_kvq_read: every byte of the pools against
the format's definition (bit for bit), and the values read back."""
import numpy as np
import pytest

import _kvq
import workloads as wl
from _util import bits, to_dev

pytestmark = pytest.mark.gpu
import torch  # noqa: E402

import paged_kv_gqa_attention_gb300 as qa  # noqa: E402


def setup(seed, lens, past, hkv, width=None):
    rng = np.random.default_rng(seed)
    lens, past = np.asarray(lens), np.asarray(past)
    T = int(lens.sum())
    w = dict(k=wl.normal_bf16(rng, (T, hkv, 128)), v=wl.normal_bf16(rng, (T, hkv, 128)), cu=wl.cu_from_lengths(lens),
             past=past.astype(np.int32))
    w["table"], pages = _kvq.page_table(rng, lens + past, width=width)
    for n in ("k_pages", "v_pages"):
        w[n] = rng.integers(0, 256, size=(pages, hkv * _kvq.HEAD_BYTES), dtype=np.uint8)
    return w


def expected(w, skip=()):
    out = {}
    for n, x in (("k_pages", w["k"]), ("v_pages", w["v"])):
        pool = w[n].copy()
        for r in range(len(w["past"])):
            if r not in skip:
                _kvq.put_rows(pool, w["table"][r], int(w["past"][r]), x[w["cu"][r]:w["cu"][r + 1]], n == "k_pages")
        out[n] = pool
    return out


def write(w, **kw):
    d = {n: to_dev(w[n]) for n in ("table", "cu", "past")}
    pools = {n: torch.from_numpy(w[n].copy()).cuda() for n in ("k_pages", "v_pages")}
    k, v = kw.pop("k", None), kw.pop("v", None)
    k, v = to_dev(w["k"]) if k is None else k, to_dev(w["v"]) if v is None else v
    past = None if kw.pop("no_past", False) else d["past"]
    qa.qa_kvq_write(k, v, d["cu"], d["table"], pools["k_pages"], pools["v_pages"], n_past=past, **kw)
    torch.cuda.synchronize()
    return pools, d


def check_pools(pools, want):
    for n in ("k_pages", "v_pages"):
        np.testing.assert_array_equal(pools[n].cpu().numpy(), want[n], err_msg=n)


CASES = [
    ([1], [0], 8), ([1, 1, 1], [15, 16, 17], 8), ([16], [0], 1), ([15, 16, 17, 0, 1], [0, 0, 0, 3, 31], 8),
    ([33, 5, 64], [7, 30, 1], 3), ([0, 0, 40], [0, 9, 0], 2), ([300, 299], [0, 1000], 8), ([2] * 70, list(range(70)), 5),
    ([0, 0], [0, 5], 8), ([1031], [3], 8), ([37] * 33, [15] * 33, 1),
]


@pytest.mark.parametrize("lens, past, hkv", CASES)
def test_write_is_bit_exact(lens, past, hkv):
    w = setup(len(lens) + hkv, lens, past, hkv)
    pools, _ = write(w, debug_checks=True)
    check_pools(pools, expected(w))


@pytest.mark.parametrize("lens, past, hkv", CASES)
def test_read_is_the_stored_value(lens, past, hkv):
    w = setup(100 + len(lens), lens, past, hkv)
    rng = np.random.default_rng(7)
    for n in ("k_pages", "v_pages"):
        w[n] = _kvq.random_pool(rng, w[n].shape[0], hkv)
    d = {n: to_dev(w[n]) for n in ("table", "cu", "past", "k_pages", "v_pages")}
    T = len(w["k"])
    k, v = qa.qa_kvq_read(d["k_pages"], d["v_pages"], d["table"], d["cu"], T, n_past=d["past"], debug_checks=True)
    for got, n in ((k, "k_pages"), (v, "v_pages")):
        for r in range(len(lens)):
            s, m, c = _kvq.rows(w[n], w["table"][r], past[r], lens[r], n == "k_pages")
            # s n is exact in fp32, the sum is rounded to fp32 and then to bf16
            want = wl.bf16_bits((m + s * c).astype(np.float32)).reshape(m.shape).transpose(1, 0, 2)
            np.testing.assert_array_equal(bits(got)[w["cu"][r]:w["cu"][r + 1]], want)


def test_unusual_values():
    w = setup(11, [48], [0], 2)
    x = wl.bf16_to_f64(w["k"]).astype(np.float32)
    x[0, 0, :32] = 3.25  # constant
    x[1, 0, 5] = np.inf
    x[2, 1, 40] = -np.inf
    x[4, 0, 70:80] = 3.3e38  # a range past fp32
    x[4, 0, 80:90] = -3.3e38
    x[5, 0, :32] = 0.0
    x[6, 0] = np.float32(2.0 ** -130)  # subnormal spread
    x[6, 0, ::3] = 0.0
    x[7, 0] *= 1e30
    x[8, 0] *= 1e-30
    x[9, 0, 31] = 5000.0  # one large value
    x[10, 1] = -0.0
    x[11, 0, ::2], x[11, 0, 1::2] = 0.0, -0.0
    b = wl.bf16_bits(x).reshape(x.shape)
    b[3, 0, 100] = 0x7FC0  # NaN (bf16_bits takes finite inputs and infinities)
    b[3, 1, 64] = 0xFFC1
    w["k"] = w["v"] = b
    pools, d = write(w, debug_checks=True)
    want = expected(w)
    # of a group of zeros the sign of m is open: -0 + s n and +0 + s n are the same value
    for n in ("k_pages", "v_pages"):
        got = pools[n].cpu().numpy()
        s0, m0, c0 = _kvq.rows(got, w["table"][0], 0, 48, n == "k_pages")
        s1, m1, c1 = _kvq.rows(want[n], w["table"][0], 0, 48, n == "k_pages")
        np.testing.assert_array_equal(s0, s1)
        np.testing.assert_array_equal(m0, m1)
        np.testing.assert_array_equal(c0, c1)
    k, v = qa.qa_kvq_read(pools["k_pages"], pools["v_pages"], d["table"], d["cu"], 48)
    nan = torch.isnan(k)
    assert torch.equal(nan, torch.isnan(v))
    groups = nan.reshape(48, 2, 4, 32)
    assert bool((groups.any(-1) == groups.all(-1)).all())
    assert {tuple(i) for i in groups.all(-1).nonzero().tolist()} == {(1, 0, 0), (2, 1, 1), (3, 0, 3), (3, 1, 2), (4, 0, 2)}
    assert bool((k[0, 0, :32] == 3.25).all()) and bool((k[5, 0, :32] == 0).all())


def test_rounding_at_ties():
    # groups 0, s, 2 s ... with halves: codes at exact ties go to the even one
    x = np.zeros((16, 1, 128), np.float32)
    for t in range(16):
        s = np.float32(2.0 ** (t - 8))
        x[t, 0] = np.tile(np.arange(32) * s / 2, 4)
        x[t, 0, ::32] = 0
        x[t, 0, 31::32] = 15 * s
    w = setup(12, [16], [0], 1)
    w["k"] = w["v"] = wl.bf16_bits(x).reshape(x.shape)
    pools, _ = write(w)
    check_pools(pools, expected(w))


def test_strided_rows_and_no_past():
    w = setup(13, [20, 45], [0, 0], 8)
    x = torch.full((65, 40, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    x[:, 16:24], x[:, 24:32] = to_dev(w["k"]), to_dev(w["v"])
    pools, _ = write(w, k=x[:, 16:24], v=x[:, 24:32], no_past=True, debug_checks=True, stable_metadata=True)
    check_pools(pools, expected(w))


def test_bad_pages_lengths_and_segments():
    w = setup(14, [40, 20, 33, 16], [0, 5, 0, 0], 8, width=4)
    good = w["table"].copy()
    w["table"][0, 1] = w["k_pages"].shape[0]
    w["table"][2, 0] = -7
    with pytest.raises(qa.QAError, match="bad page"):
        write(w, debug_checks=True)
    pools, _ = write(w)
    qa.qa_device_status()
    want = {n: x.copy() for n, x in expected(w, skip=(0, 2)).items()}
    for n, x in (("k_pages", w["k"]), ("v_pages", w["v"])):  # the pages of requests 0 and 2 that are good
        _kvq.put_rows(want[n], good[0], 0, x[0:16], n == "k_pages")
        _kvq.put_rows(want[n], good[0], 32, x[32:40], n == "k_pages")
        _kvq.put_rows(want[n], good[2], 16, x[60 + 16:60 + 33], n == "k_pages")
    check_pools(pools, want)

    w = setup(15, [40, 20], [0, 0], 8, width=3)
    w["past"] = np.array([20, -1], np.int32)  # 60 positions of a 48-position row; a negative past
    w["table"][0] = [0, 1, 2]
    with pytest.raises(qa.QAError, match="bad length"):
        write(w, debug_checks=True)
    pools, _ = write(w)
    qa.qa_device_status()
    want = {n: w[n].copy() for n in ("k_pages", "v_pages")}
    for n, x in (("k_pages", w["k"]), ("v_pages", w["v"])):
        _kvq.put_rows(want[n], w["table"][0], 20, x[:28], n == "k_pages")
    check_pools(pools, want)

    for cu in ([0, 10, 59], [0, 70, 60], [1, 10, 60], [0, -5, 60], [0, 40, 20]):
        w = setup(16, [40, 20], [0, 0], 8)
        w["cu"] = np.array(cu, np.int32)
        with pytest.raises(qa.QAError, match="bad segments"):
            write(w, debug_checks=True)
        assert qa.qa_device_status() == 0


def test_no_rows_at_all():
    w = setup(17, [0, 0, 0], [0, 4, 16], 8)
    pools, _ = write(w, debug_checks=True)
    check_pools(pools, w)


def test_skipped_rows_of_a_read_stay():
    w = setup(18, [40, 20], [0, 0], 8)
    w["table"][0, 1] = -1
    rng = np.random.default_rng(3)
    for n in ("k_pages", "v_pages"):
        w[n] = _kvq.random_pool(rng, w[n].shape[0], 8)
    d = {n: to_dev(w[n]) for n in ("table", "cu", "k_pages", "v_pages")}
    k, v = (torch.full((60, 8, 128), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qa.qa_kvq_read(d["k_pages"], d["v_pages"], d["table"], d["cu"], 60, k, v)
    assert qa.qa_device_status() == 1
    for x in (k, v):
        same = (x == 9).all(-1).all(-1).cpu().numpy()
        np.testing.assert_array_equal(same, (np.arange(60) >= 16) & (np.arange(60) < 32))


def test_pages_past_four_gigabytes():
    # pools of 4.6 GB each: byte offsets past 32 bits
    w = setup(19, [35], [10], 8)
    pages = 450000
    w["table"] = np.array([[449990, 5, 449999]], np.int32)
    pools = {n: torch.zeros(pages, 10240, dtype=torch.uint8, device="cuda") for n in ("k_pages", "v_pages")}
    d = {n: to_dev(w[n]) for n in ("table", "cu", "past", "k", "v")}
    qa.qa_kvq_write(d["k"], d["v"], d["cu"], d["table"], pools["k_pages"], pools["v_pages"], n_past=d["past"], debug_checks=True)
    small = {n: np.zeros((3, 10240), np.uint8) for n in pools}
    for n, x in (("k_pages", w["k"]), ("v_pages", w["v"])):
        _kvq.put_rows(small[n], [0, 1, 2], 10, x, n == "k_pages")
        np.testing.assert_array_equal(pools[n][torch.tensor([449990, 5, 449999], device="cuda")].cpu().numpy(), small[n])
    k, _ = qa.qa_kvq_read(pools["k_pages"], pools["v_pages"], d["table"], d["cu"], 35, n_past=d["past"])
    assert float((k.float() - d["k"].float()).abs().max()) < 0.5


def test_graph_replay_reads_new_contents():
    w = setup(20, [17, 60], [3, 40], 8)
    pools, d = write(w)
    k, v = to_dev(w["k"]), to_dev(w["v"])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    with torch.cuda.graph(graph, stream=s):
        qa.qa_kvq_write(k, v, d["cu"], d["table"], pools["k_pages"], pools["v_pages"], n_past=d["past"], stream=s)
        qa.qa_kvq_read(pools["k_pages"], pools["v_pages"], d["table"], d["cu"], 77, ko, vo, n_past=d["past"], stream=s)
    w2 = setup(21, [17, 60], [3, 40], 8)
    k.copy_(to_dev(w2["k"]))
    v.copy_(to_dev(w2["v"]))
    graph.replay()
    torch.cuda.synchronize()
    w["k"], w["v"] = w2["k"], w2["v"]
    check_pools(pools, expected(w))
    s_, m, c = _kvq.quantise(w2["k"])[1][..., 0], _kvq.quantise(w2["k"])[1][..., 1], _kvq.quantise(w2["k"])[0]
    want = _kvq.f32(m)[..., None] + _kvq.f32(s_)[..., None] * c.reshape(77, 8, 4, 32).astype(np.float32)
    np.testing.assert_array_equal(bits(ko), wl.bf16_bits(want).reshape(77, 8, 128))
