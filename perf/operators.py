"""Cases, plain forms and exact results of the rotary-position and 4-bit-cache operators.

Five operators make up serving with a cache held in 4 bits:

    rope    per-head QK-norm and rotary positions with several axes, on packed query and key rows
    write   K and V rows quantised to 4 bits as they are written to their pages, and their values read back
    read    the values of cached rows as packed bf16 rows
    attn    paged grouped-query decode attention over the 4-bit cache
    step    norm, rotation, quantised append and attention of one new token a request

``run`` computes them with elementary torch operations, or, where ``own`` is true, with the calls a serving program
makes of the package.  ``exact`` has each result in 64 bits, written from the operators' definitions.

The cache: pages of 16 tokens, 1280 bytes for each KV head.  A group is 32 consecutive dims of one token's head; it has
a bf16 scale s, a bf16 minimum m and 32 codes n of 4 bits, and stands for the values m + s n.  The first 1024 bytes hold
the codes: of K, token t's dim 32 g + 8 c + j is nibble j of the 4-byte word at 64 t + 16 c + 4 g; of V, token
8 u + 2 p + e's dim 32 g + 4 r + i is nibble i of the 2-byte word at 512 u + 64 r + 16 p + 4 g + 2 e.  The last 256
bytes hold (s, m) of token t's group g at 16 t + 4 g.
"""
import math
import random

import torch

own = False

PAGE = 16
HEAD_BYTES = 1280
CODE_BYTES = 1024
GROUP = 32
ROPE_THETA = 1.0e6
RMS_EPS = 1.0e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step's rows of 32 requests: text positions, three axes interleaved over the pairs
        dict(name="rope step", op="rope", rows=32, hq=16, hkv=8, dim=128, axes=3, interleaved=True, norm=True, fused=False),
        # a packed prompt bucket with video frames in it, q and k inside the fused projection's rows
        dict(name="rope prompt", op="rope", rows=16111, hq=16, hkv=8, dim=128, axes=3, interleaved=True, norm=True, fused=True),
        # an image encoder's rows: two axes (height, width), 64-wide heads, no norm
        dict(name="rope image", op="rope", rows=4095, hq=14, hkv=14, dim=64, axes=2, interleaved=False, norm=False, fused=False),
        # one token each of 64 requests, appended to its page
        dict(name="write tokens", op="write", batch=64, lo=1, hi=1, past=1999, hkv=8, len_seed=1),
        # prompts of up to 4096 tokens, written whole
        dict(name="write prompts", op="write", batch=16, lo=500, hi=4096, past=0, hkv=8, len_seed=2),
        # short cached prompts read back for the next chunk's attention
        dict(name="read short", op="read", batch=16, lo=53, hi=430, past=0, hkv=8, len_seed=3),
        # long contexts read back
        dict(name="read long", op="read", batch=8, lo=2000, hi=16000, past=0, hkv=8, len_seed=4),
        # a single caller: latency
        dict(name="attn single", op="attn", batch=1, lo=257, hi=257, hq=16, hkv=8, len_seed=5),
        # the ordinary decode batch
        dict(name="attn batch", op="attn", batch=32, lo=200, hi=2000, hq=16, hkv=8, len_seed=6),
        # the long-context decode batch
        dict(name="attn long", op="attn", batch=64, lo=2000, hi=16000, hq=16, hkv=8, len_seed=7),
        # the whole step for a few callers
        dict(name="step few", op="step", batch=5, lo=1, hi=700, hq=16, hkv=8, axes=3, len_seed=8),
        # the whole step for a full batch, positions from the lengths
        dict(name="step full", op="step", batch=128, lo=100, hi=4000, hq=16, hkv=8, axes=0, len_seed=9),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attn", "attn", "step"])
    if op == "rope":
        dim = rng.choice([64, 128, 128])
        axes = rng.choice([1, 2, 3, 3])
        hkv = _spread(rng, 1, 16)
        return dict(op=op, rows=_spread(rng, 1, 16000), hq=hkv * rng.choice([1, 2]), hkv=hkv, dim=dim, axes=axes,
                    interleaved=axes > 1 and rng.random() < 0.5, norm=rng.random() < 0.7, fused=rng.random() < 0.5)
    hkv = rng.choice([1, 2, 4, 6, 8, 8, 8, 8])
    if op in ("write", "read"):
        batch = _spread(rng, 1, 128)
        hi = _spread(rng, 1, 30000 // batch)
        return dict(op=op, batch=batch, lo=_spread(rng, 1, hi), hi=hi, past=rng.choice([0, _spread(rng, 1, 2000)]),
                    hkv=hkv, len_seed=rng.randrange(1 << 20))
    batch = _spread(rng, 1, 256)
    hi = _spread(rng, 1, min(16000, 400000 // batch))
    case = dict(op=op, batch=batch, lo=_spread(rng, 1, hi), hi=hi, hq=hkv * rng.choice([1, 2, 2]), hkv=hkv,
                len_seed=rng.randrange(1 << 20))
    if op == "step":
        case["axes"] = rng.choice([0, 3])
    return case


def _lengths(case):
    rng = random.Random(case["len_seed"])
    return [rng.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]


def _pasts(case):
    rng = random.Random(case["len_seed"] + 1)
    return [rng.randint(0, case["past"]) if case["past"] else 0 for _ in range(case["batch"])]


def _sections(axes, dim):
    """Rotation pairs of each axis: three axes 24 : 20 : 20 of every 64 pairs, two halves, or all."""
    if axes == 3:
        return [12 * dim // 64, 10 * dim // 64, 10 * dim // 64]
    return [dim // 4, dim // 4] if axes == 2 else [dim // 2]


def work(case):
    if case["op"] == "rope":
        heads = case["hq"] + case["hkv"]
        n = case["rows"] * heads * case["dim"]
        return {"bytes": 4 * n + 4 * max(1, case["axes"]) * case["rows"], "flops": 6 * n}
    lens = _lengths(case)
    if case["op"] == "write":
        n = sum(lens) * case["hkv"]  # rows read, cache written, values returned
        return {"bytes": n * (512 + 160 + 512), "flops": n * 256 * 5}
    if case["op"] == "read":
        n = sum(lens) * case["hkv"]
        return {"bytes": n * (160 + 512), "flops": n * 256 * 2}
    rows = case["batch"] * case["hq"] * 128
    new = case["batch"] * case["hkv"] * (512 + 160 + 512) if case["op"] == "step" else 0
    return {"bytes": sum(lens) * case["hkv"] * 160 + 4 * rows + new, "flops": 4 * sum(lens) * case["hq"] * 128}


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _pool(g, pages, hkv):
    """A pool whose every group stands for values of about unit spread: uniform codes, scales near 0.2."""
    pool = torch.randint(0, 256, (pages, hkv, HEAD_BYTES), generator=g, device="cuda", dtype=torch.uint8)
    s = 0.2 * torch.exp(0.25 * torch.randn(pages, hkv, 64, generator=g, device="cuda"))
    m = -s * (7.5 + 0.5 * torch.randn(pages, hkv, 64, generator=g, device="cuda"))
    pool[:, :, CODE_BYTES:] = torch.stack((s, m), -1).to(torch.bfloat16).view(torch.uint8).reshape(pages, hkv, 256)
    return pool.reshape(pages, hkv * HEAD_BYTES)


def _pages(g, lengths):
    """A page table of scattered pages, and how many pages the pool has."""
    counts = [-(-n // PAGE) for n in lengths]
    pages, most = sum(counts) + 7, max(1, max(counts))
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    counts = torch.tensor(counts, device="cuda")
    table = torch.full((len(lengths), most), -1, dtype=torch.int32, device="cuda")
    used = torch.arange(most, device="cuda")[None] < counts[:, None]
    table[used] = order[: int(counts.sum())]
    return table, pages


def _gain(g, dim):
    return (0.5 + torch.rand(dim, generator=g, device="cuda")).to(torch.bfloat16).float()


def _cumulative(lens):
    return _ints([sum(lens[:i]) for i in range(len(lens) + 1)])


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    state = dict(op=op)
    if op == "rope":
        rows, hq, hkv, dim, axes = (case[k] for k in ("rows", "hq", "hkv", "dim", "axes"))
        x = _normal(g, rows, hq + 2 * hkv, dim)  # the fused projection's rows
        q, k = x[:, :hq], x[:, hq:hq + hkv]
        if not case["fused"]:
            q, k = q.contiguous(), k.contiguous()
        # frames of 16 x 24 patches after a long text: time, height and width count on from the same place
        i = torch.arange(rows, device="cuda")
        first = int(torch.randint(0, 100000, (1,), generator=g, device="cuda"))
        positions = torch.stack((first + i // 384, first + i // 24 % 16, first + i % 24))[3 - axes:].to(torch.int32)
        state |= dict(q=q, k=k, positions=positions.contiguous(), q_gain=_gain(g, dim) if case["norm"] else None,
                      k_gain=_gain(g, dim) if case["norm"] else None)
        state["pair_axis"] = _pair_axis(_sections(axes, dim), case["interleaved"])
        return state
    hkv = case["hkv"]
    lens = _lengths(case)
    if op in ("write", "read"):
        past = _pasts(case)
        state["page_table"], pages = _pages(g, [a + b for a, b in zip(past, lens)])
        state |= dict(k_pages=_pool(g, pages, hkv), v_pages=_pool(g, pages, hkv), cu_seqlens=_cumulative(lens),
                      n_past=_ints(past), rows=sum(lens))
        if op == "write":
            # keys have a few dims of larger spread, values are even
            spread = 1 + 3 * (torch.rand(hkv, 128, generator=g, device="cuda") < 0.05)
            state["k"] = (torch.randn(sum(lens), hkv, 128, generator=g, device="cuda") * spread).to(torch.bfloat16)
            state["v"] = _normal(g, sum(lens), hkv, 128)
        return state
    batch, hq = case["batch"], case["hq"]
    state["page_table"], pages = _pages(g, lens)
    state |= dict(k_pages=_pool(g, pages, hkv), v_pages=_pool(g, pages, hkv), seq_lens=_ints(lens), longest=max(lens))
    state["q"] = (1.5 * torch.randn(batch, hq, 128, generator=g, device="cuda")).to(torch.bfloat16)
    if op == "step":
        state |= dict(k=_normal(g, batch, hkv, 128), v=_normal(g, batch, hkv, 128), q_gain=_gain(g, 128),
                      k_gain=_gain(g, 128), positions=None, pair_axis=None)
        state |= dict(last=state["seq_lens"] - 1, ones=_ints(list(range(batch + 1))))
        if case["axes"]:  # text after images: fewer positions than tokens, the same on each axis
            state["positions"] = (state["last"] // 2 + 5)[None].expand(3, batch).contiguous()
            state["pair_axis"] = _pair_axis(_sections(3, 128), True)
    return state


def _pair_axis(sections, interleaved):
    """The axis of each rotation pair: sections one after another, or taken in turn (the first axis where one has ended)."""
    n = len(sections)
    if not interleaved:
        return [a for a, count in enumerate(sections) for _ in range(count)]
    return [i % n if i < n * sections[i % n] else 0 for i in range(sum(sections))]


# ------------------------------------------------------------------ one pass

def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


def _qa():
    import paged_kv_gqa_attention_gb300 as qa

    return qa


def _kept(state, name, make):
    """A buffer that a serving program keeps: made on the first pass."""
    if name not in state:
        state[name] = make()
    return state[name]


def _own_rope(s):
    return _qa().qa_rope_rows(s["q"], s["k"], s["positions"], q_gain=s["q_gain"], k_gain=s["k_gain"], rms_eps=RMS_EPS,
                              rope_theta=ROPE_THETA, pair_axis=s["pair_axis"])


def _own_read(s):
    return _qa().qa_kvq_read(s["k_pages"], s["v_pages"], s["page_table"], s["cu_seqlens"], s["rows"], n_past=s["n_past"])


def _own_write(s):
    _qa().qa_kvq_write(s["k"], s["v"], s["cu_seqlens"], s["page_table"], s["k_pages"], s["v_pages"], n_past=s["n_past"])
    return _own_read(s)


def _workspace(s):
    batch, pages = s["page_table"].shape
    size = _qa().qa_kvq_decode_workspace_size(
        batch, 0, n_q_heads=s["q"].shape[1], n_kv_heads=s["k_pages"].shape[1] // HEAD_BYTES,
        num_pages=s["k_pages"].shape[0], max_pages_per_seq=pages)
    return torch.zeros(size, dtype=torch.uint8, device="cuda")


def _own_attn(s):
    return _qa().qa_kvq_decode_attn(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["seq_lens"],
                                    workspace=_kept(s, "workspace", lambda: _workspace(s)), stable_metadata=2)


def _own_step(s):
    qa = _qa()
    out = qa.qa_kvq_decode_step(s["q"], s["k"], s["v"], s["q_gain"], s["k_gain"], s["page_table"], s["seq_lens"],
                                s["k_pages"], s["v_pages"], positions=s["positions"], pair_axis=s["pair_axis"],
                                workspace=_kept(s, "workspace", lambda: _workspace(s)), rms_eps=RMS_EPS,
                                rope_theta=ROPE_THETA, stable_metadata=2)
    batch = s["page_table"].shape[0]
    k, v = qa.qa_kvq_read(s["k_pages"], s["v_pages"], s["page_table"], s["ones"], batch, n_past=s["last"])
    return out, k, v


_OWN = dict(rope=_own_rope, write=_own_write, read=_own_read, attn=_own_attn, step=_own_step)


# ------------------------------------------------------------------ plain forms

def _rotated(x, positions, gain, pair_axis):
    """bf16 rows [T, H, D] normed and rotated by positions [axes, T], in 32 bits, the angles in 64."""
    half = x.shape[-1] // 2
    y = x.float()
    if gain is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + RMS_EPS) * gain
    freq = ROPE_THETA ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    axis = torch.tensor(pair_axis or [0] * half, device="cuda")
    angle = positions.double()[axis].T * freq
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    a, b = y[..., :half], y[..., half:]
    return torch.cat((a * cos - b * sin, a * sin + b * cos), -1).to(torch.bfloat16)


def _plain_rope(s):
    return tuple(_rotated(s[n], s["positions"], s[n + "_gain"], s["pair_axis"]) for n in ("q", "k"))


def _quantised(x):
    """Codes [T, H, 4, 32] (int32) and (s, m) [T, H, 4, 2] (bf16) of bf16 rows [T, H, 128]."""
    x = x.float().reshape(*x.shape[:2], 4, GROUP)
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s = ((hi - lo) / torch.full_like(lo, 15)).to(torch.bfloat16).float()  # a tensor divisor: a true division
    r = torch.where(s >= torch.finfo(torch.float32).tiny, 1 / s, 0)
    n = torch.round((x - lo) * r).clamp(0, 15).to(torch.int32)
    return n, torch.cat((s, lo), -1).to(torch.bfloat16)


def _views(pool):
    """A pool's K codes, V codes and parameters as bytes of each token."""
    pool = pool.view(pool.shape[0], -1, HEAD_BYTES)
    codes, params = pool[..., :CODE_BYTES], pool[..., CODE_BYTES:]
    p, h = pool.shape[:2]
    return codes.view(p, h, PAGE, 64), codes.view(p, h, 2, 8, 4, 4, 2, 2), params.view(p, h, PAGE, 16)


def _places(s, rows):
    """The page and the slot in it of each packed row."""
    cu, past = s["cu_seqlens"].long(), s["n_past"].long()
    i = torch.arange(rows, device="cuda")
    r = torch.searchsorted(cu, i, right=True) - 1
    at = past[r] + i - cu[r]
    return s["page_table"][r, at // PAGE].long(), at % PAGE


def _put(s, k, v, page, slot):
    for name, x in (("k", k), ("v", v)):
        n, params = _quantised(x)
        k_codes, v_codes, p = _views(s[name + "_pages"])
        t, h = n.shape[:2]
        p[page, :, slot] = params.view(torch.uint8).reshape(t, h, 16)
        if name == "k":
            n = n.view(t, h, 4, 4, 4, 2).transpose(2, 3)  # [c][g] words of 8 dims, two a byte
            k_codes[page, :, slot] = (n[..., 0] | n[..., 1] << 4).to(torch.uint8).reshape(t, h, 64)
        else:
            n = n.view(t, h, 4, 8, 2, 2).transpose(2, 3)  # [r][g] words of 4 dims, two a byte
            v_codes[page, :, slot // 8, :, slot % 8 // 2, :, slot % 2] = (n[..., 0] | n[..., 1] << 4).to(torch.uint8)


def _nibbles(b):
    return torch.stack((b & 15, b >> 4), -1)


def _row_values(s, page, slot):
    """The values of rows at (page, slot): K and V, bf16 [T, H, 128]."""
    out = []
    for name in ("k", "v"):
        k_codes, v_codes, p = _views(s[name + "_pages"])
        p = p[page, :, slot].contiguous().view(torch.bfloat16).float()
        t, h = p.shape[:2]
        if name == "k":
            n = _nibbles(k_codes[page, :, slot].view(t, h, 4, 4, 4)).transpose(2, 3)
        else:
            n = _nibbles(v_codes[page, :, slot // 8, :, slot % 8 // 2, :, slot % 2]).transpose(2, 3)
        p = p.view(t, h, 4, 2, 1)
        out.append((p[:, :, :, 1] + p[:, :, :, 0] * n.reshape(t, h, 4, GROUP)).to(torch.bfloat16).view(t, h, 128))
    return tuple(out)


def _plain_write(s):
    page, slot = _places(s, s["rows"])
    _put(s, s["k"], s["v"], page, slot)
    return _row_values(s, page, slot)


def _plain_read(s):
    return _row_values(s, *_places(s, s["rows"]))


def _page_values(pool, table, is_k):
    """The values of whole page-table rows in 32 bits: [B, H, pages * 16, 128]."""
    pages = pool.view(pool.shape[0], -1, HEAD_BYTES)[table.clamp(min=0).long()]  # [B, pages, H, 1280]
    b, n_pages, h = pages.shape[:3]
    p = pages[..., CODE_BYTES:].contiguous().view(torch.bfloat16).float().view(b, n_pages, h, PAGE, 4, 2, 1)
    codes = pages[..., :CODE_BYTES]
    if is_k:  # [t][c][g][byte][nibble] -> [t][g][c][byte][nibble]
        n = _nibbles(codes.view(b, n_pages, h, PAGE, 4, 4, 4)).transpose(4, 5)
    else:  # [u][r][p][g][e][byte][nibble] -> [u][p][e][g][r][byte][nibble]
        n = _nibbles(codes.view(b, n_pages, h, 2, 8, 4, 4, 2, 2)).permute(0, 1, 2, 3, 5, 7, 6, 4, 8, 9)
    x = p[..., 1, :] + p[..., 0, :] * n.reshape(b, n_pages, h, PAGE, 4, GROUP)
    return x.view(b, n_pages, h, PAGE, 128).transpose(1, 2).reshape(b, h, n_pages * PAGE, 128)


def _attended(q, s):
    b, hq, d = q.shape
    hkv = s["k_pages"].shape[1] // HEAD_BYTES
    q = q.float().view(b, hkv, hq // hkv, d)
    score = q @ _page_values(s["k_pages"], s["page_table"], True).transpose(-1, -2) / math.sqrt(d)
    t = torch.arange(score.shape[-1], device="cuda")
    score = score.masked_fill(t >= s["seq_lens"].view(b, 1, 1, 1), -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    out = (p @ _page_values(s["v_pages"], s["page_table"], False)) / p.sum(-1, keepdim=True)
    return out.view(b, hq, d).to(torch.bfloat16)


def _plain_attn(s):
    return _attended(s["q"], s)


def _plain_step(s):
    positions = s["last"][None] if s["positions"] is None else s["positions"]
    q, k = (_rotated(s[n], positions, s[n + "_gain"], s["pair_axis"]) for n in ("q", "k"))
    last = s["last"].long()
    page, slot = s["page_table"][torch.arange(len(last), device="cuda"), last // PAGE].long(), last % PAGE
    _put(s, k, s["v"], page, slot)
    return (_attended(q, s), *_row_values(s, page, slot))


_PLAIN = dict(rope=_plain_rope, write=_plain_write, read=_plain_read, attn=_plain_attn, step=_plain_step)


# ------------------------------------------------------------------ 64 bits

def _exact_rope(x, positions, gain, pair_axis):
    x = x.double()
    dim = x.shape[-1]
    if gain is not None:
        x = x / torch.sqrt(torch.sum(x ** 2, -1, keepdim=True) / dim + RMS_EPS) * gain.double()
    out = torch.empty_like(x)
    for i in range(dim // 2):
        a = (positions[pair_axis[i] if pair_axis else 0].double() * ROPE_THETA ** (-2.0 * i / dim))[:, None]
        u, w = x[..., i], x[..., i + dim // 2]
        out[..., i], out[..., i + dim // 2] = u * torch.cos(a) - w * torch.sin(a), u * torch.sin(a) + w * torch.cos(a)
    return out


def _to_bf16(x):
    return x.to(torch.float32).to(torch.bfloat16)


def _exact_quantised(x):
    """The values that rows [T, H, 128] stand for once quantised; the definition's roundings, each from 64 bits."""
    x = x.double()
    out = torch.empty_like(x)
    for g in range(0, 128, GROUP):
        y = x[..., g:g + GROUP]
        lo, hi = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
        s = _to_bf16(((hi - lo).float().double() / 15)).double()
        r = torch.where(s > 0, 1 / s, torch.zeros_like(s)).float().double()
        n = torch.round(((y - lo).float().double() * r).float().double()).clamp(0, 15)
        out[..., g:g + GROUP] = lo + s * n
    return out


def _exact_rows(pool, table, n, is_k):
    """The values of a request's first n positions: [H, n, 128]."""
    t, d = torch.meshgrid(torch.arange(PAGE, device="cuda"), torch.arange(128, device="cuda"), indexing="ij")
    g = d // GROUP
    if is_k:
        nibble = d % 8
        at = 64 * t + 16 * (d % GROUP // 8) + 4 * g + nibble // 2
    else:
        nibble = d % 4
        at = 512 * (t // 8) + 64 * (d % GROUP // 4) + 16 * (t % 8 // 2) + 4 * g + 2 * (t % 2) + nibble // 2
    pages = pool.view(pool.shape[0], -1, HEAD_BYTES)[table[: -(-n // PAGE)].long()]
    code = (pages[:, :, at] >> (4 * (nibble % 2)).to(torch.uint8)) & 15
    p = pages[:, :, CODE_BYTES:].contiguous().view(torch.bfloat16).double()
    value = p[:, :, 8 * t + 2 * g + 1] + p[:, :, 8 * t + 2 * g] * code
    return value.transpose(0, 1).reshape(pages.shape[1], -1, 128)[:, :n]


def _exact_attended(q, s, lens, new=None):
    """Attention of each request over its cache; `new`: K and V values that take the place of the last position's."""
    hkv = s["k_pages"].shape[1] // HEAD_BYTES
    out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        k, v = (_exact_rows(s[name], s["page_table"][b], n, name == "k_pages") for name in ("k_pages", "v_pages"))
        if new is not None:
            k[:, -1], v[:, -1] = new[0][b], new[1][b]
        x = q[b].double().view(hkv, -1, 128)
        p = torch.softmax(torch.einsum("hgd,htd->hgt", x, k) / math.sqrt(128.0), -1)
        out[b] = torch.einsum("hgt,htd->hgd", p, v).reshape(-1, 128)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return tuple(_exact_rope(s[n], s["positions"], s[n + "_gain"], s["pair_axis"]) for n in ("q", "k"))
    lens = _lengths(case)
    if op == "write":
        return _exact_quantised(s["k"]), _exact_quantised(s["v"])
    if op == "read":
        rows = [(s["page_table"][b], a, a + n) for b, (a, n) in enumerate(zip(_pasts(case), lens))]
        return tuple(torch.cat([_exact_rows(s[name], table, end, name == "k_pages")[:, first:] for table, first, end in rows],
                               1).transpose(0, 1) for name in ("k_pages", "v_pages"))
    if op == "attn":
        return _exact_attended(s["q"], s, lens)
    positions = s["last"][None] if s["positions"] is None else s["positions"]
    q, k = (_to_bf16(_exact_rope(s[n], positions, s[n + "_gain"], s["pair_axis"])) for n in ("q", "k"))
    new = _exact_quantised(k), _exact_quantised(s["v"])
    return (_exact_attended(q, s, lens, new), *new)
