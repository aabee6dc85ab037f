"""GPU parity of qa_kvq_decode_attn and qa_kvq_decode_step against attention
over the 4-bit cache in 64 bits (_kvq.decode, with its error bound), and a
serving run through all the operators of the 4-bit cache."""
import threading

import numpy as np
import pytest

import _kvq
import oracle
import workloads as wl
from _util import assert_close, assert_rounded_match, bits, f64, to_dev

pytestmark = pytest.mark.gpu
import torch  # noqa: E402

import paged_kv_gqa_attention_gb300 as qa  # noqa: E402

EPS, THETA = wl.RMS_EPS, wl.ROPE_THETA


def setup(seed, lens, hq=16, hkv=8, width=None, q_scale=1.5, poison=True):
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int32)
    table, pages = _kvq.page_table(rng, lens, width=width)
    w = dict(table=table, lens=lens, q=wl.bf16_bits((q_scale * rng.standard_normal((len(lens), hq, 128))).astype(np.float32)))
    w["q"] = w["q"].reshape(len(lens), hq, 128)
    for n in ("k_pages", "v_pages"):
        w[n] = _kvq.random_pool(rng, pages, hkv)
        if poison:
            _kvq.poison_after(w[n], table, lens)
    return w


def attn(w, **kw):
    d = {n: to_dev(w[n]) for n in ("q", "k_pages", "v_pages", "table", "lens")}
    return qa.qa_kvq_decode_attn(d["q"], d["k_pages"], d["v_pages"], d["table"], d["lens"], **kw)


def check(got, w, what, scale=None, q=None):
    ref, bound = _kvq.decode(wl.bf16_to_f64(w["q"]) if q is None else q, w["k_pages"], w["v_pages"], w["table"], w["lens"], scale)
    g = f64(got)
    assert np.isfinite(g).all(), f"{what}: non-finite"
    over = np.abs(g - ref) > bound
    assert not over.any(), f"{what}: {int(over.sum())} of {over.size} past the bound, worst {np.max(np.abs(g - ref) / np.maximum(bound, 1e-30)):.3g} times it, error {np.max(np.abs(g - ref)[over]):.3g}"
    assert np.linalg.norm(g - ref) <= 5e-3 * np.linalg.norm(ref), what


@pytest.mark.parametrize("lens", [
    (1,), (2, 15, 16, 17, 31, 32, 33), (127, 128, 129, 1), (2000,), (16,) * 40, (3000, 1, 2500, 33), (0, 5, 0, 700, 0),
    (9000, 40, 1, 4000),
])
@pytest.mark.parametrize("hq, hkv", [(16, 8), (8, 8), (2, 1), (6, 3)])
def test_lengths_and_heads(lens, hq, hkv):
    w = setup(len(lens) * 10 + hq, lens, hq, hkv)
    check(attn(w, debug_checks=True), w, f"{lens} {hq}/{hkv}")


@pytest.mark.parametrize("hq, hkv", [(1, 1), (4, 2), (4, 4), (10, 5), (12, 6), (7, 7)])
def test_other_heads(hq, hkv):
    w = setup(hq, (1, 300, 77, 1025), hq, hkv)
    check(attn(w, debug_checks=True), w, f"{hq}/{hkv}")


def test_many_requests():
    rng = np.random.default_rng(5)
    w = setup(5, rng.integers(0, 120, size=700))
    out = attn(w, debug_checks=True)
    check(out, w, "700 requests")
    assert not bits(out)[w["lens"] == 0].any()


def test_long_context():
    w = setup(6, (33333, 20001))
    check(attn(w), w, "long")


def test_sharp_and_flat_scores():
    w = setup(7, (500, 1000, 64), q_scale=12.0)  # one position takes nearly all
    check(attn(w), w, "sharp")
    w = setup(8, (500, 1000, 64), q_scale=0.0)
    check(attn(w), w, "flat")
    w = setup(9, (700, 18))
    check(attn(w, scale=0.01), w, "small scale", scale=0.01)


def test_rising_scores():
    # the running maximum moves on every page: later keys lie ever further along q
    w = setup(10, (400,), 2, 1, poison=False)
    heads = w["k_pages"].reshape(w["k_pages"].shape[0], 1, 1280)
    q0 = wl.bf16_to_f64(w["q"])[0, 0]
    for pos in range(400):
        x = (q0 * (0.01 * pos)).astype(np.float32)
        _kvq.put_rows(w["k_pages"], w["table"][0], pos, wl.bf16_bits(x).reshape(1, 1, 128), True)
    assert heads.shape[2] == 1280
    check(attn(w), w, "rising")
    w["table"][0] = w["table"][0][::-1].copy()
    check(attn(w), w, "falling")


def test_nan_in_a_cached_group_stays_in_its_head():
    w = setup(11, (50, 60))
    nan = np.array([0x7FC0, 0x7FC0], np.uint16).view(np.uint8)
    heads = w["v_pages"].reshape(-1, 8, 1280)
    heads[w["table"][0][1], 3, 1024 + 16 * 4 + 4 * 2:][:4] = nan  # token 20, group 2, KV head 3
    got = f64(attn(w))
    bad = np.isnan(got)
    assert bad[0, 6:8, 64:96].all() and bad.sum() == 64
    heads[w["table"][0][1], 3, 1024 + 16 * 4 + 4 * 2:][:4] = np.array([0x3E00, 0xBF80], np.uint16).view(np.uint8)
    check(attn(w), w, "mended")


def test_heads_and_groups_of_very_different_size():
    # query heads 2^40 apart in size over one KV head, and an infinite one: each by itself
    w = setup(36, (300, 41))
    q = wl.bf16_to_f64(w["q"]).astype(np.float32)
    q[:, 1::4] *= np.float32(2.0 ** -40)
    q[:, 2::4] *= np.float32(2.0 ** 30)
    w["q"] = wl.bf16_bits(q).reshape(q.shape)
    g = f64(attn(w))
    small = dict(w, q=w["q"][:, 0::2]), dict(w, q=w["q"][:, 1::2])
    for i, part in enumerate(small):
        ref, bound = _kvq.decode(wl.bf16_to_f64(part["q"]), w["k_pages"], w["v_pages"], w["table"], w["lens"])
        keep = [h for h in range(8) if (2 * h + i) % 4 != 2]  # scores of 2^30: one token takes all, in any arithmetic
        assert (np.abs(g[:, i::2] - ref)[:, keep] <= bound[:, keep]).all()
    assert np.isfinite(g).all()
    w = setup(37, (300, 41))
    ref, bound = _kvq.decode(wl.bf16_to_f64(w["q"]), w["k_pages"], w["v_pages"], w["table"], w["lens"])
    w["q"][0, 5, 77] = 0x7F80
    g = f64(attn(w))
    assert not np.isfinite(g[0, 5]).any()
    g[0, 5], ref[0, 5] = 0, 0
    assert (np.abs(g - ref) <= bound).all()
    # value groups 2^90 apart in one head: each to its own accuracy
    w = setup(38, (700, 30))
    heads = w["v_pages"].reshape(-1, 8, 1280)
    params = heads[:, :, 1024:].copy().view(np.uint16).reshape(-1, 8, 16, 4, 2)
    scale = np.array([2.0 ** -60, 1.0, 2.0 ** 30, 2.0 ** -20], np.float32)[None, None, None, :, None]
    heads[:, :, 1024:] = wl.bf16_bits((_kvq.f32(params) * scale).astype(np.float32)).reshape(params.shape).view(np.uint8).reshape(-1, 8, 256)
    _kvq.poison_after(w["v_pages"], w["table"], w["lens"])
    g = f64(attn(w))
    ref, bound = _kvq.decode(wl.bf16_to_f64(w["q"]), w["k_pages"], w["v_pages"], w["table"], w["lens"])
    assert (np.abs(g - ref) <= bound).all()
    for grp in range(4):
        sl = np.s_[:, :, 32 * grp:32 * grp + 32]
        assert np.linalg.norm((g - ref)[sl]) <= 5e-3 * np.linalg.norm(ref[sl])


def params_view(pool, hkv=8):
    """The parameters of a pool as a writable bit view [pages, heads, 16 tokens, 4 groups, 2]."""
    return pool.reshape(pool.shape[0], hkv, 1280)[:, :, 1024:].view(np.uint16).reshape(pool.shape[0], hkv, 16, 4, 2)


def place_score(w, b, pos, nats):
    """Gives request b's token `pos` constant key groups whose score is the largest of its head's others plus `nats`,
    for the query heads of every KV head (q . K = sum_g m_g sum_{d in g} q_d: an equation each for four minima)."""
    n = int(w["lens"][b])
    ks, km, kn = _kvq.rows(w["k_pages"], w["table"][b], 0, n, True)
    q = wl.bf16_to_f64(w["q"])[b].reshape(8, -1, 128)
    sc = np.einsum("hgd,htd->hgt", q, km + ks * kn)
    sc[..., pos] = -np.inf
    want = sc.max(-1) + nats * 128 ** 0.5
    sums = q.reshape(8, -1, 4, 32).sum(-1)
    sm = np.zeros((8, 4, 2), np.float32)
    for h in range(8):
        sm[h, :, 1] = np.linalg.lstsq(sums[h], want[h], rcond=None)[0]
    params_view(w["k_pages"])[w["table"][b][pos // 16], :, pos % 16] = wl.bf16_bits(sm).reshape(sm.shape)


@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("log2_ratio", [17, 24, 60])
@pytest.mark.parametrize("hq", [16, 8])
def test_a_huge_value_of_no_weight(where, log2_ratio, hq):
    """A token whose values are 2^17 and more times the others' and whose probability is e^-60 of the largest: the
    others' part of the output stays exact to the bound, in its own group and the rest."""
    w = setup(42, (700, 41, 5000), hq)
    for b, n in enumerate(w["lens"]):
        pos = {"first": 0, "middle": int(n) // 2, "last": int(n) - 1}[where]
        place_score(w, b, pos, -60.0)
        group = params_view(w["v_pages"])[w["table"][b][pos // 16], :, pos % 16, 1]
        group[...] = wl.bf16_bits(_kvq.f32(group) * np.float32(2.0 ** log2_ratio)).reshape(group.shape)
    check(attn(w), w, f"{where}, 2^{log2_ratio}")


@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("hq", [16, 8])
def test_a_sink_without_a_value(where, hq):
    """A token that takes nearly all of the softmax and whose value groups are 0 + 2^-30 n: the output is what the
    others' probabilities of e^-19 give, all alike, so that their roundings would not average out."""
    w = setup(43, (700, 41, 3000), hq)
    for n in ("k_pages", "v_pages"):
        params_view(w[n])[...] = wl.bf16_bits(np.array([0.0, 0.0] if n == "k_pages" else [0.171875, -1.25], np.float32))
    for b, n in enumerate(w["lens"]):
        pos = {"first": 0, "middle": int(n) // 2, "last": int(n) - 1}[where]
        place_score(w, b, pos, 19.0)
        params_view(w["v_pages"])[w["table"][b][pos // 16], :, pos % 16] = wl.bf16_bits(np.array([2.0 ** -30, 0.0], np.float32))
    for n in ("k_pages", "v_pages"):
        _kvq.poison_after(w[n], w["table"], w["lens"])
    check(attn(w), w, where)


def test_constant_groups():
    # s = 0 in every value group: the output is the minimum's average; in every key group: all scores of a token equal m sum q
    w = setup(39, (200, 3))
    for n in ("k_pages", "v_pages"):
        heads = w[n].reshape(-1, 8, 1280)
        params = heads[:, :, 1024:].copy().view(np.uint16).reshape(-1, 8, 16, 4, 2)
        params[..., 0] = 0
        heads[:, :, 1024:] = params.view(np.uint8).reshape(-1, 8, 256)
        _kvq.poison_after(w[n], w["table"], w["lens"])
    check(attn(w), w, "constant groups")


@pytest.mark.parametrize("batch", [2049, 4096])
def test_largest_batches(batch):
    rng = np.random.default_rng(batch)
    w = setup(batch, rng.integers(0, 70, size=batch), 4, 2)
    check(attn(w, debug_checks=True), w, f"batch {batch}")
    s = step_setup(batch, rng.integers(1, 40, size=batch), 2, 1)
    out, d = run_step(s, debug_checks=True)
    got = {n: d[n].cpu().numpy() for n in ("k_pages", "v_pages")}
    q, _ = _kvq.rope(wl.bf16_to_f64(s["q"]), (s["lens"] - 1)[None], s["q_gain"], None)
    check(out, dict(s, **got), f"step of batch {batch}", q=wl.bf16_to_f64(wl.bf16_bits(q.astype(np.float32)).reshape(q.shape)))


def test_more_pages_than_32_bit_products_serve():
    # 4096 requests of 129 pages, 528384 in all, over three requests' worth of real pages
    w = setup(40, (2064, 2050, 2049), 2, 1)
    ref, bound = _kvq.decode(wl.bf16_to_f64(w["q"]), w["k_pages"], w["v_pages"], w["table"], w["lens"])
    pick = np.arange(4096) % 3
    big = dict(w, q=w["q"][pick], table=w["table"][pick], lens=w["lens"][pick])
    g = f64(attn(big, debug_checks=True))
    assert (np.abs(g - ref[pick]) <= bound[pick]).all()


def test_no_tokens_at_all():
    w = setup(41, (0, 0, 0))
    assert not bits(attn(w, out=torch.full((3, 16, 128), 7.0, dtype=torch.bfloat16, device="cuda"), debug_checks=True)).any()


def test_bad_pages_and_lengths():
    w = setup(12, (100, 40, 50, 20), width=8)
    w["table"][0, 2] = -5
    w["table"][2, 0] = 10 ** 6
    with pytest.raises(qa.QAError, match="bad page"):
        attn(w, debug_checks=True)
    out = attn(w)
    assert qa.qa_device_status() == 1
    # the page is left out: as if its positions were not there
    keep = setup(12, (100, 40, 50, 20), width=8)
    keep["table"][0, :6] = np.delete(keep["table"][0, :7], 2)
    keep["table"][2, :3] = np.delete(keep["table"][2, :4], 0)
    keep["lens"] = np.array([84, 40, 34, 20], np.int32)
    check(out, keep, "bad page left out")
    w = setup(13, (100, 40, 50), width=8)
    w["lens"] = np.array([129, 40, -1], np.int32)
    out = attn(w)
    assert qa.qa_device_status() == 2
    assert not bits(out)[[0, 2]].any()
    w["lens"] = np.array([0, 40, 0], np.int32)
    check(out, w, "others")


def test_bad_page_at_the_end_of_a_split_request():
    w = setup(14, (4000, 8), width=260)
    w["table"][0, 249] = -1  # the last page
    out = attn(w)
    assert qa.qa_device_status() == 1
    w["lens"] = np.array([249 * 16, 8], np.int32)
    w["table"][0, 249] = 0
    check(out, w, "last page bad")
    w = setup(15, (33,), width=260)
    w["table"][:] = -1  # nothing left
    out = attn(w)
    assert qa.qa_device_status() == 1 and not bits(out).any()


def test_workspace_is_reusable_and_calls_repeat():
    size = qa.qa_kvq_decode_workspace_size(300, 0)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for seed, lens in ((21, (5000, 3)), (22, (100,) * 300), (23, (70, 8000, 9)), (21, (5000, 3))):
        w = setup(seed, lens)
        a = attn(w, workspace=ws)
        check(a, w, str(lens[:3]))
        assert torch.equal(a, attn(w, workspace=ws))
    if size > 256:  # the arrival counters are zero between calls
        torch.cuda.synchronize()
    with pytest.raises(qa.QAError, match="workspace"):
        attn(w, workspace=ws[:128])


def test_workspace_shared_with_the_bf16_decode():
    """Layers of both caches take turns on one workspace; requests are split over more than 16 workers, whose groups
    have counters of their own."""
    lens = (6000, 3, 9000, 700)
    w, x = setup(44, lens), wl.decode_workload(45, lens, num_pages=1100, max_pages=600)
    ref = oracle.decode(x["q"], x["k_pages"], x["v_pages"], x["page_table"], x["seq_lens"])
    size = max(qa.qa_kvq_decode_workspace_size(4, 0), qa.qa_decode_workspace_size(4, 9000, num_pages=1100, max_pages_per_seq=600))
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    dx = {n: to_dev(x[n]) for n in ("q", "k_pages", "v_pages", "page_table", "seq_lens")}
    for i in range(4):
        out = torch.full((4, 16, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        qa.qa_decode_attn(dx["q"], dx["k_pages"], dx["v_pages"], dx["page_table"], dx["seq_lens"], out, workspace=ws)
        assert_close(f64(out), ref, f"bf16 layer {i}")
        out = torch.full((4, 16, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        check(attn(w, workspace=ws, out=out, debug_checks=True), w, f"4-bit layer {i}")
        assert not ws[:4096 * 8 * 4].any()


@pytest.mark.parametrize("batch, hq, hkv", [(4018, 8, 8), (4019, 8, 8), (4096, 16, 8), (4096, 7, 7), (4096, 2, 1)])
def test_long_requests_in_the_largest_batches(batch, hq, hkv):
    """Requests over more than 16 workers among so many that the groups' counters have little room, or none."""
    w = setup(46, (20000, 20, 13000), hq, hkv)
    ref, bound = _kvq.decode(wl.bf16_to_f64(w["q"]), w["k_pages"], w["v_pages"], w["table"], w["lens"])
    pick = np.ones(batch, int)
    pick[[100, batch - 1]] = 0, 2
    pick[101] = 2
    ws = torch.zeros(qa.qa_kvq_decode_workspace_size(batch, 0, n_q_heads=hq, n_kv_heads=hkv), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        g = f64(attn(dict(w, q=w["q"][pick], table=w["table"][pick], lens=w["lens"][pick]), workspace=ws, debug_checks=True))
        assert (np.abs(g - ref[pick]) <= bound[pick]).all()
        assert not ws[:4096 * 8 * 4].any()


@pytest.mark.parametrize("level", [0, 1, 2])
def test_stable_metadata_levels(level):
    w = setup(24, (700, 1, 90, 3000))
    d = {n: to_dev(w[n]) for n in ("q", "k_pages", "v_pages", "table", "lens")}
    ws = torch.zeros(qa.qa_kvq_decode_workspace_size(4, 0), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(d["q"]) for _ in range(6)]
    torch.cuda.synchronize()
    x = d["q"]
    for o in outs:  # each call's query is the last one's output, as between layers
        qa.qa_kvq_decode_attn(x, d["k_pages"], d["v_pages"], d["table"], d["lens"], o, workspace=ws, stable_metadata=level)
        x = o
    torch.cuda.synchronize()
    prev = w["q"]
    for i, o in enumerate(outs):
        check(o, dict(w, q=prev), f"layer {i}")
        prev = bits(o)


def test_two_streams_and_graphs():
    ws, outs, ref, graphs = [], [], [], []
    data = [setup(30, (900, 20, 333)), setup(31, (64, 2222))]
    for w in data:
        d = {n: to_dev(w[n]) for n in ("q", "k_pages", "v_pages", "table", "lens")}
        s = torch.cuda.Stream()
        wsp = torch.zeros(qa.qa_kvq_decode_workspace_size(len(w["lens"]), 0), dtype=torch.uint8, device="cuda")
        out = torch.empty_like(d["q"])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            qa.qa_kvq_decode_attn(d["q"], d["k_pages"], d["v_pages"], d["table"], d["lens"], out, workspace=wsp, stream=s)
            qa.qa_kvq_decode_attn(d["q"], d["k_pages"], d["v_pages"], d["table"], d["lens"], out, workspace=wsp, stream=s)
        graphs.append((g, s, d))
        ws.append(wsp)
        outs.append(out)
    for _ in range(20):
        for g, s, _d in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for w, o in zip(data, outs):
        check(o, w, "replayed on its own stream")
    del ref


def test_host_threads_with_batches_of_their_own():
    """Calls of two host threads interleave; their kernels need different amounts of shared memory."""
    data = [setup(35, (40,)), setup(36, (3,) * 2000)]
    want = [attn(w) for w in data]
    torch.cuda.synchronize()
    failed = []

    def serve(w, ref):
        try:
            s = torch.cuda.Stream()
            d = {n: to_dev(w[n]) for n in ("q", "k_pages", "v_pages", "table", "lens")}
            ws = torch.zeros(qa.qa_kvq_decode_workspace_size(len(w["lens"]), 0), dtype=torch.uint8, device="cuda")
            out = torch.empty_like(d["q"])
            torch.cuda.synchronize()
            for _ in range(400):
                qa.qa_kvq_decode_attn(d["q"], d["k_pages"], d["v_pages"], d["table"], d["lens"], out, workspace=ws, stream=s)
            s.synchronize()
            assert torch.equal(out, ref)
        except Exception as e:  # noqa: BLE001 - whatever it is, the test shows it
            failed.append(e)

    threads = [threading.Thread(target=serve, args=x) for x in zip(data, want)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not failed, failed


def test_workspace_made_inside_a_call_on_another_stream():
    w = setup(33, (3000, 10))
    d = {n: to_dev(w[n]) for n in ("q", "k_pages", "v_pages", "table", "lens")}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = [qa.qa_kvq_decode_attn(d["q"], d["k_pages"], d["v_pages"], d["table"], d["lens"], stream=s) for _ in range(5)]
    s.synchronize()
    for o in outs:
        check(o, w, "other stream")


def test_page_locked_host_query_and_output():
    w = setup(34, (100, 300))
    d = {n: to_dev(w[n]) for n in ("k_pages", "v_pages")}
    q = torch.from_numpy(w["q"].view(np.int16)).view(torch.bfloat16).pin_memory()
    table, lens = torch.from_numpy(w["table"]).pin_memory(), torch.from_numpy(w["lens"]).pin_memory()
    out = torch.empty_like(q).pin_memory()
    qa.qa_kvq_decode_attn(q, d["k_pages"], d["v_pages"], table, lens, out,
                          workspace=torch.zeros(qa.qa_kvq_decode_workspace_size(2, 0), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    check(out, w, "host buffers")


def test_pages_past_four_gigabytes():
    w = setup(35, (40,))
    d = {n: to_dev(w[n]) for n in ("q", "lens")}
    ids = [449990, 5, 449999]
    big = {n: torch.zeros(450000, 10240, dtype=torch.uint8, device="cuda") for n in ("k_pages", "v_pages")}
    for n in big:
        big[n][torch.tensor(ids, device="cuda")] = torch.from_numpy(w[n][w["table"][0]]).cuda()
    out = qa.qa_kvq_decode_attn(d["q"], big["k_pages"], big["v_pages"], torch.tensor([ids], dtype=torch.int32, device="cuda"), d["lens"])
    check(out, w, "far pages")


# ------------------------------------------------------------------ the step

def step_setup(seed, lens, hq=16, hkv=8, axes=0, width=None):
    w = setup(seed, lens, hq, hkv, width)
    rng = np.random.default_rng([seed, 1])
    B = len(lens)
    for n, h in (("q", hq), ("k", hkv), ("v", hkv)):
        w[n] = wl.normal_bf16(rng, (B, h, 128))
    for n in ("q_gain", "k_gain"):
        w[n] = wl.bf16_to_f64(wl.bf16_bits(rng.uniform(0.5, 1.5, size=128).astype(np.float32))).astype(np.float32)
    w["positions"] = rng.integers(0, 1 << 18, size=(axes, B)).astype(np.int32) if axes else None
    w["pair_axis"] = rng.integers(0, axes, size=64).astype(np.uint8) if axes else None
    return w


def run_step(w, d=None, **kw):
    names = ("q", "k", "v", "q_gain", "k_gain", "table", "lens", "k_pages", "v_pages")
    d = d or {n: to_dev(w[n]) for n in names}
    pos = None if w["positions"] is None else to_dev(w["positions"])
    out = qa.qa_kvq_decode_step(d["q"], d["k"], d["v"], d["q_gain"], d["k_gain"], d["table"], d["lens"], d["k_pages"],
                                d["v_pages"], positions=pos, pair_axis=w["pair_axis"], **kw)
    return out, d


def new_rows(pools, w, d):
    """The appended rows as stored (bf16 of m + s n), K and V."""
    B = len(w["lens"])
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    return qa.qa_kvq_read(d["k_pages"], d["v_pages"], d["table"], cu, B, n_past=d["lens"] - 1)


def check_step(w, what, **kw):
    out, d = run_step(w, debug_checks=True, **kw)
    pos = (w["lens"] - 1)[None] if w["positions"] is None else w["positions"]
    q_ref, q_size = _kvq.rope(wl.bf16_to_f64(w["q"]), pos, w["q_gain"], w["pair_axis"])
    k_ref, k_size = _kvq.rope(wl.bf16_to_f64(w["k"]), pos, w["k_gain"], w["pair_axis"])
    # the pools: everything but the new rows as before, V's new row bit for bit
    got = {n: d[n].cpu().numpy() for n in ("k_pages", "v_pages")}
    want = {n: w[n].copy() for n in got}
    for b in range(len(w["lens"])):
        at = int(w["lens"][b]) - 1
        _kvq.put_rows(want["v_pages"], w["table"][b], at, w["v"][b:b + 1], False)
        _kvq.put_rows(want["k_pages"], w["table"][b], at, wl.bf16_bits(k_ref[b:b + 1].astype(np.float32)).reshape(1, -1, 128), True)
    np.testing.assert_array_equal(got["v_pages"], want["v_pages"])
    # K's new row is quantised from bf16 roundings of fp32 results, a few of which round the other way (_util):
    # one moves a code by one, or its group's s or m, and with it 32 codes by at most one
    differ = got["k_pages"] != want["k_pages"]
    assert differ.sum() <= max(24, 0.004 * len(w["lens"]) * w["k"].shape[1] * 80), f"{what}: {differ.sum()} bytes"
    for b in range(len(w["lens"])):
        at = int(w["lens"][b]) - 1
        s, m, n = _kvq.rows(got["k_pages"], w["table"][b], at, 1, True)
        val = (m + s * n)[:, 0]
        err = np.abs(val - k_ref[b])
        # half a step (s within 2^-8 of range / 15: up to 15 * 2^-8 steps more), and K's bf16 rounding
        assert (err <= s[:, 0] * (0.5 + 15 * 2.0 ** -8) + 2.0 ** -8 * np.abs(k_ref[b]) + 2.0 ** -18 * k_size[b]).all()
        if differ[w["table"][b][at // 16]].any():
            want["k_pages"][w["table"][b][at // 16]] = got["k_pages"][w["table"][b][at // 16]]
    np.testing.assert_array_equal(got["k_pages"], want["k_pages"])
    # the output: attention of the rounded query over the cache as it now is; a query that rounds the other way is within
    # 2^-8 of a few of its values, which the bound's allowance for scores covers
    q = wl.bf16_to_f64(wl.bf16_bits(q_ref.astype(np.float32)).reshape(q_ref.shape))
    check(out, dict(w, **got), what, q=q)
    return out, d


@pytest.mark.parametrize("lens", [(1,), (1, 15, 16, 17, 127, 128, 129), (2000,), (16,) * 40, (3000, 1, 2500, 33), (18000, 2)])
@pytest.mark.parametrize("axes", [0, 3])
def test_step(lens, axes):
    check_step(step_setup(50 + len(lens), lens, axes=axes), f"step {lens}")


@pytest.mark.parametrize("hq, hkv", [(8, 8), (2, 1), (1, 1), (6, 3), (10, 5)])
def test_step_heads(hq, hkv):
    check_step(step_setup(60 + hq, (1, 300, 77, 1025), hq, hkv, axes=2), f"step {hq}/{hkv}")


def test_step_many():
    rng = np.random.default_rng(61)
    check_step(step_setup(61, rng.integers(1, 70, size=600), axes=3), "600 short requests")


def test_step_rows_of_a_fused_projection():
    w = step_setup(62, (33, 250, 1000))
    names = ("q_gain", "k_gain", "table", "lens")
    x = torch.full((3, 40, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    x[:, :16], x[:, 16:24], x[:, 24:32] = to_dev(w["q"]), to_dev(w["k"]), to_dev(w["v"])
    pools = lambda: {n: to_dev(w[n]) for n in ("k_pages", "v_pages")}  # noqa: E731
    base = {n: to_dev(w[n]) for n in names}
    a, _ = run_step(w, dict(base, **pools(), q=x[:, :16], k=x[:, 16:24], v=x[:, 24:32]))
    b, _ = run_step(w)
    assert torch.equal(a, b)


def test_step_equals_the_three_calls():
    w = step_setup(63, np.random.default_rng(63).integers(1, 900, size=40), axes=3)
    out, d = run_step(w)
    e = {n: to_dev(w[n]) for n in d}
    pos = to_dev(w["positions"])
    q, k = qa.qa_rope_rows(e["q"], e["k"], pos, q_gain=e["q_gain"], k_gain=e["k_gain"], pair_axis=w["pair_axis"])
    cu = torch.arange(41, dtype=torch.int32, device="cuda")
    qa.qa_kvq_write(k, e["v"], cu, e["table"], e["k_pages"], e["v_pages"], n_past=e["lens"] - 1)
    three = qa.qa_kvq_decode_attn(q, e["k_pages"], e["v_pages"], e["table"], e["lens"])
    torch.cuda.synchronize()
    assert_close(f64(out), f64(three), "step against the three calls")
    assert int((d["k_pages"] != e["k_pages"]).sum()) <= 64 and torch.equal(d["v_pages"], e["v_pages"])


def test_step_of_non_finite_rows():
    w = step_setup(67, (40, 33, 20))
    w["v"][0, 2, 70] = 0x7FC0  # NaN in a value group: that group of the head's outputs
    w["v"][1, 5, 3] = 0xFF80  # -inf
    # inf in a key: its mean square is inf, so the norm leaves x / inf = 0 of the finite dims and inf / inf = NaN of dim
    # 9, which the rotation spreads to its partner 9 + 64; the groups of the two, 0 and 2, are NaN, and so every score
    w["k"][2, 4, 9] = 0x7F80
    out, d = run_step(w)
    nan = np.isnan(f64(out))
    want = np.zeros_like(nan)
    want[0, 4:6, 64:96] = want[1, 10:12, 0:32] = want[2, 8:10] = True
    np.testing.assert_array_equal(nan, want)
    k, v = new_rows(None, w, d)
    assert bool(torch.isnan(v[0, 2, 64:96]).all()) and int(torch.isnan(v).sum()) == 64
    assert bool(torch.isnan(k[2, 4].view(4, 32)[[0, 2]]).all()) and int(torch.isnan(k).sum()) == 64
    assert bool((k[2, 4].view(4, 32)[[1, 3]] == 0).all())


def test_step_refusals_on_the_device():
    w = step_setup(64, (20, 30, 40, 50), axes=3, width=5)
    before = {n: w[n].copy() for n in ("k_pages", "v_pages")}
    w["positions"][1, 1] = -1
    w["positions"][2, 2] = 1 << 18
    good = w["lens"].copy()
    w["lens"] = np.array([0, 30, 40, 50], np.int32)
    out, d = run_step(w)
    assert qa.qa_device_status() == 0x12
    assert not bits(out)[:3].any() and bits(out)[3].any()
    got = d["k_pages"].cpu().numpy()
    changed = np.nonzero((got != before["k_pages"]).any(1))[0].tolist()
    assert changed == [int(w["table"][3][49 // 16])]
    # a bad last page: the new token has no place, the rest is attended
    w = step_setup(65, (40, 33), width=5)
    w["table"][0, 2] = -1
    out, d = run_step(w)
    assert qa.qa_device_status() == 1
    ref = dict(w, lens=np.array([32, 33], np.int32), k_pages=d["k_pages"].cpu().numpy(), v_pages=d["v_pages"].cpu().numpy())
    q, _ = _kvq.rope(wl.bf16_to_f64(w["q"]), (w["lens"] - 1)[None], w["q_gain"], None)
    check(out, ref, "last page bad", q=wl.bf16_to_f64(wl.bf16_bits(q.astype(np.float32)).reshape(q.shape)))
    del good


def test_step_graph_replay_grows_the_cache():
    # one captured step, replayed with lengths that the graph itself advances
    w = step_setup(66, (5, 31, 300), width=24)
    rng = np.random.default_rng(66)
    table, pages = _kvq.page_table(rng, (24 * 16,) * 3, width=24)
    w["table"] = table
    for n in ("k_pages", "v_pages"):
        w[n] = _kvq.random_pool(rng, pages, 8)
    d = {n: to_dev(w[n]) for n in ("q", "k", "v", "q_gain", "k_gain", "table", "lens", "k_pages", "v_pages")}
    ws = torch.zeros(qa.qa_kvq_decode_workspace_size(3, 0), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(d["q"])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        with torch.cuda.stream(s):
            qa.qa_kvq_decode_step(d["q"], d["k"], d["v"], d["q_gain"], d["k_gain"], d["table"], d["lens"], d["k_pages"],
                                  d["v_pages"], out, workspace=ws, stream=s)
            d["lens"].add_(1)
    d["lens"].copy_(to_dev(w["lens"]))
    for i in range(20):
        fresh = {n: wl.normal_bf16(rng, w[n].shape) for n in ("q", "k", "v")}
        for n in fresh:
            d[n].copy_(to_dev(fresh[n]))
        g.replay()
        torch.cuda.synchronize()
    got = {n: d[n].cpu().numpy() for n in ("k_pages", "v_pages")}
    lens = w["lens"] + 19
    q, _ = _kvq.rope(wl.bf16_to_f64(fresh["q"]), (lens - 1)[None], w["q_gain"], None)
    check(out, dict(w, lens=lens, **got), "twentieth step", q=wl.bf16_to_f64(wl.bf16_bits(q.astype(np.float32)).reshape(q.shape)))
    assert (d["lens"].cpu().numpy() == w["lens"] + 20).all() and qa.qa_device_status() == 0


def grown(seed, lens, tokens, axes):
    """A layer's cache of `lens` tokens with room for `tokens` more, and the new rows of each of them."""
    rng = np.random.default_rng(seed)
    B = len(lens)
    table, pages = _kvq.page_table(rng, np.asarray(lens) + tokens)
    w = dict(table=table, k_pages=_kvq.random_pool(rng, pages, 8), v_pages=_kvq.random_pool(rng, pages, 8))
    w["rows"] = [{n: wl.normal_bf16(rng, (B, h, 128)) for n, h in (("q", 16), ("k", 8), ("v", 8))} for _ in range(tokens)]
    for n in ("q_gain", "k_gain"):
        w[n] = wl.bf16_to_f64(wl.bf16_bits(rng.uniform(0.5, 1.5, size=128).astype(np.float32))).astype(np.float32)
    w["positions"] = rng.integers(0, 1 << 18, size=(tokens, axes, B)).astype(np.int32) if axes else None
    w["pair_axis"] = rng.integers(0, axes, size=64).astype(np.uint8) if axes else None
    return w


@pytest.mark.parametrize("read_back", [False, True])
@pytest.mark.parametrize("axes", [0, 3])
@pytest.mark.parametrize("level", [1, 2])
def test_chained_steps_at_stable_metadata_levels(level, axes, read_back):
    """Six tokens through two layers' caches, queued without a host synchronise, rings filled and angles computed before
    the call before is done: every output, every row read back and the pools are those of calls made one at a time at
    level 0, and those are right."""
    lens, tokens = np.array([5000, 0, 13, 15, 16, 700]), 6
    layers = [grown(seed, lens, tokens, axes) for seed in (80, 81)]
    dev = [[{n: to_dev(x) for n, x in row.items()} for row in w["rows"]] for w in layers]
    fixed = [{n: to_dev(w[n]) for n in ("q_gain", "k_gain", "table")} for w in layers]
    pos = [None if w["positions"] is None else [to_dev(x) for x in w["positions"]] for w in layers]
    n_of = [(lens + 1 + i).astype(np.int32) for i in range(tokens)]
    dn, last = [to_dev(n) for n in n_of], [to_dev(n - 1) for n in n_of]
    cu = torch.arange(len(lens) + 1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(qa.qa_kvq_decode_workspace_size(len(lens), 0), dtype=torch.uint8, device="cuda")

    def run(level, after):
        pools = [{n: to_dev(w[n]) for n in ("k_pages", "v_pages")} for w in layers]
        torch.cuda.synchronize()
        got = []
        for i in range(tokens):
            for j, w in enumerate(layers):
                r, f, p = dev[j][i], fixed[j], pools[j]
                out = qa.qa_kvq_decode_step(r["q"], r["k"], r["v"], f["q_gain"], f["k_gain"], f["table"], dn[i], p["k_pages"],
                                            p["v_pages"], positions=pos[j] and pos[j][i], pair_axis=w["pair_axis"],
                                            workspace=ws, stable_metadata=level)
                got.append(out)
                if read_back:
                    got += qa.qa_kvq_read(p["k_pages"], p["v_pages"], f["table"], cu, len(lens), n_past=last[i],
                                          stable_metadata=level)
                after(i, j, p, out)
        torch.cuda.synchronize()
        return got + [p[n] for p in pools for n in p]

    def right(i, j, p, out):
        w = layers[j]
        at = (n_of[i] - 1)[None] if w["positions"] is None else w["positions"][i]
        q, _ = _kvq.rope(wl.bf16_to_f64(w["rows"][i]["q"]), at, w["q_gain"], w["pair_axis"])
        k, size = _kvq.rope(wl.bf16_to_f64(w["rows"][i]["k"]), at, w["k_gain"], w["pair_axis"])
        now = dict(table=w["table"], lens=n_of[i], **{n: x.cpu().numpy() for n, x in p.items()})
        check(out, now, f"token {i} layer {j}", q=wl.bf16_to_f64(wl.bf16_bits(q.astype(np.float32)).reshape(q.shape)))
        v_codes, v_sm = _kvq.quantise(w["rows"][i]["v"])
        for b, n in enumerate(n_of[i]):
            s, m, c = (x[:, 0] for x in _kvq.rows(now["v_pages"], w["table"][b], n - 1, 1, False))
            np.testing.assert_array_equal(c, v_codes[b])
            np.testing.assert_array_equal(s[:, ::32], wl.bf16_to_f64(v_sm[b][..., 0]))
            np.testing.assert_array_equal(m[:, ::32], wl.bf16_to_f64(v_sm[b][..., 1]))
            s, m, c = (x[:, 0] for x in _kvq.rows(now["k_pages"], w["table"][b], n - 1, 1, True))
            # as in check_step: half a step of s, s itself within 2^-8, and K's rounding to bf16
            assert (np.abs(m + s * c - k[b]) <= s * (0.5 + 15 * 2.0 ** -8) + 2.0 ** -8 * np.abs(k[b]) + 2.0 ** -18 * size[b]).all()

    want = run(0, right)
    for _ in range(3):
        got = run(level, lambda *a: None)
        assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))
    assert qa.qa_device_status() == 0


@pytest.mark.parametrize("lens, hq, hkv", [((5000, 3), 16, 8), ((9000, 40, 1, 4000), 16, 8), ((70,) * 300, 16, 8),
                                           ((16000, 12000), 2, 1), ((3000, 257), 6, 3), ((0, 0), 16, 8)])
def test_counters_are_zero_after_every_call(lens, hq, hkv):
    """Those of requests and those of the groups that merge requests over more than 16 workers, on a workspace whose
    partials are of other sizes every time."""
    ws = torch.zeros(qa.qa_kvq_decode_workspace_size(300, 0), dtype=torch.uint8, device="cuda")
    w = setup(47, lens, hq, hkv)
    for _ in range(2):
        check(attn(w, workspace=ws), w, "attention")
        assert not ws[:4096 * 8 * 4].any()
    if min(lens) > 0:
        w = step_setup(48, lens, hq, hkv)
        check_step(w, "step", workspace=ws)
        assert not ws[:4096 * 8 * 4].any()


# ------------------------------------------------------------------ served together

def test_serving_run():
    """Prompts with image positions rotated, attended and quantised into the
    cache; tokens decoded by the fused step; a second chunk attended over the
    cache read back.  Every stage against the definitions on what the stage
    before it left."""
    rng = np.random.default_rng(70)
    lens = np.array([37, 5, 130])
    hq, hkv, T = 16, 8, 172
    axis = qa.qa_rope_axes([24, 20, 20], interleaved=True)
    gains = [wl.bf16_to_f64(wl.bf16_bits(rng.uniform(0.5, 1.5, size=128).astype(np.float32))).astype(np.float32) for _ in range(2)]
    dg = [to_dev(g) for g in gains]
    qkv = wl.normal_bf16(rng, (T, 32, 128))
    x = to_dev(qkv)
    pos = np.concatenate([np.stack((n // 7 + np.arange(n) // 12, np.arange(n) // 4 % 3, np.arange(n) % 4)) for n in lens], 1).astype(np.int32)
    cu = to_dev(wl.cu_from_lengths(lens))
    table, pages = _kvq.page_table(rng, lens + 40)
    dtable = to_dev(table)
    kp, vp = (torch.full((pages, 10240), 0xAB, dtype=torch.uint8, device="cuda") for _ in range(2))

    # the prompt: in place in the projection's rows, then attention through a bf16 scratch pool
    q, k = qa.qa_rope_rows(x[:, :16], x[:, 16:24], to_dev(pos), q_gain=dg[0], k_gain=dg[1], pair_axis=axis)
    v = x[:, 24:].contiguous()
    ref, size = _kvq.rope(wl.bf16_to_f64(qkv[:, :16]), pos, gains[0], axis)
    assert_rounded_match(bits(q), ref, size, "prompt q")
    sk, sv = (torch.zeros(pages, 16, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out = qa.qa_prefill_attn(q, k, v, cu, dtable, sk, sv)
    assert_close(f64(out), oracle.prefill(bits(q), bits(k), bits(v), wl.cu_from_lengths(lens)), "prompt attention")
    qa.qa_kvq_write(k, x[:, 24:], cu, dtable, kp, vp)

    # tokens
    n = lens.copy()
    for i in range(4):
        n += 1
        row = wl.normal_bf16(rng, (3, 32, 128))
        r = to_dev(row)
        p3 = np.stack((n + 3, n + 3, n + 3)).astype(np.int32)
        out = qa.qa_kvq_decode_step(r[:, :16], r[:, 16:24], r[:, 24:], dg[0], dg[1], dtable, to_dev(n.astype(np.int32)), kp, vp,
                                    positions=to_dev(p3), pair_axis=axis, debug_checks=True)
        qr, _ = _kvq.rope(wl.bf16_to_f64(row[:, :16]), p3, gains[0], axis)
        w = dict(k_pages=kp.cpu().numpy(), v_pages=vp.cpu().numpy(), table=table, lens=n)
        check(out, w, f"token {i}", q=wl.bf16_to_f64(wl.bf16_bits(qr.astype(np.float32)).reshape(qr.shape)))

    # a second chunk over the cache, read back as whole bf16 pages (their last slots are not read)
    padded = -(-(n + 20) // 16) * 16
    starts = wl.cu_from_lengths(padded)
    ck, cv = qa.qa_kvq_read(kp, vp, dtable, to_dev(starts), int(padded.sum()), debug_checks=True)
    pool_k, pool_v = ck.view(-1, 16, 8, 128), cv.view(-1, 16, 8, 128)
    ident = np.full((3, int(padded.max()) // 16), -1, np.int32)
    for b in range(3):
        ident[b, :padded[b] // 16] = starts[b] // 16 + np.arange(padded[b] // 16)
    new = wl.normal_bf16(rng, (60, 32, 128))
    xn = to_dev(new)
    cn = wl.cu_from_lengths([20, 20, 20])
    args = [xn[:, a:b].contiguous() for a, b in ((0, 16), (16, 24), (24, 32))]
    before = bits(pool_k), bits(pool_v)
    out = qa.qa_prefill_chunk_attn(*args, to_dev(cn), to_dev(n.astype(np.int32)), to_dev(ident), pool_k, pool_v, debug_checks=True)
    ref = oracle.prefill_chunk(bits(args[0]), bits(args[1]), bits(args[2]), cn, n.astype(np.int32), ident, *before)
    assert_close(f64(out), ref["out"] if isinstance(ref, dict) else ref, "chunk over the read-back cache")
    qa.qa_kvq_write(args[1], args[2], to_dev(cn), dtable, kp, vp, n_past=to_dev(n.astype(np.int32)), debug_checks=True)
    k2, _ = qa.qa_kvq_read(kp, vp, dtable, to_dev(cn), 60, n_past=to_dev(n.astype(np.int32)))
    codes, sm = _kvq.quantise(bits(args[1]))
    val = wl.bf16_to_f64(sm[..., 1])[..., None] + wl.bf16_to_f64(sm[..., 0])[..., None] * codes.reshape(60, 8, 4, 32)
    np.testing.assert_array_equal(bits(k2), wl.bf16_bits(val.astype(np.float32)).reshape(60, 8, 128))
