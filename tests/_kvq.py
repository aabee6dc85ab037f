"""Plain numpy definitions of the rotary positions and the 4-bit cache, for
the tests: the quantiser in the exact order of its fp32 roundings, the page
format byte by byte, attention and rotation in 64 bits."""
import numpy as np

import workloads as wl

GROUP, HEAD_BYTES, CODE_BYTES, PAGE = 32, 1280, 1024, 16


def bf16(x):
    """Rounds float32 to bf16, as float32 (NaN stays NaN)."""
    x = np.asarray(x, np.float32)
    y = (wl.bf16_bits(x).astype(np.uint32) << np.uint32(16)).view(np.float32).reshape(x.shape)
    return np.where(np.isnan(x), np.float32(np.nan), y)


def f32(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << np.uint32(16)).view(np.float32)


def quantise(bits):
    """bf16 bit patterns [..., 128] -> codes [..., 128] (uint8) and parameter
    bits [..., 4, 2] (uint16: s, m)."""
    with np.errstate(all="ignore"):
        x = f32(bits).reshape(*bits.shape[:-1], 4, GROUP)
        lo, hi = x.min(-1), x.max(-1)
        d = hi - lo
        s = bf16(d / np.float32(15))
        s = np.where(s >= np.finfo(np.float32).tiny, s, np.float32(0))
        r = np.where(s > 0, np.float32(1) / s, np.float32(0))
        n = np.rint((x - lo[..., None]) * r[..., None])
        bad = ~np.isfinite(d)
        n = np.where(bad[..., None], 0, n)
    assert ((n >= 0) & (n <= 15)).all()
    nan = np.uint16(0x7FC0)
    sm = np.stack((np.where(bad, nan, wl.bf16_bits(np.where(bad, 0, s))), np.where(bad, nan, wl.bf16_bits(np.where(bad, 0, lo)))), -1)
    return n.reshape(bits.shape).astype(np.uint8), sm.astype(np.uint16)


def code_places(is_k):
    """Byte offset in a head's part of a page and nibble (0 low, 1 high) of
    token t's dim d: two arrays [16, 128]."""
    at, nib = np.zeros((PAGE, 128), np.int64), np.zeros((PAGE, 128), np.int64)
    for t in range(PAGE):
        for d in range(128):
            g = d // 32
            if is_k:
                c, j = d % 32 // 8, d % 8
                at[t, d], nib[t, d] = 64 * t + 16 * c + 4 * g + j // 2, j % 2
            else:
                r, i = d % 32 // 4, d % 4
                u, p, e = t // 8, t % 8 // 2, t % 2
                at[t, d], nib[t, d] = 512 * u + 64 * r + 16 * p + 4 * g + 2 * e + i // 2, i % 2
    return at, nib


PLACES = {True: code_places(True), False: code_places(False)}


def put_rows(pool, table_row, first, bits, is_k):
    """Writes rows bits [n, H, 128] at positions first.. of one request into
    pool [P, H * 1280] (uint8, in place)."""
    at, nib = PLACES[is_k]
    codes, sm = quantise(bits)
    heads = pool.reshape(pool.shape[0], -1, HEAD_BYTES)
    for i in range(len(bits)):
        page, t = table_row[(first + i) // PAGE], (first + i) % PAGE
        for h in range(heads.shape[1]):
            head = heads[page, h]
            for half in (0, 1):
                sel = nib[t] == half
                keep = 0xF0 if half == 0 else 0x0F
                head[at[t][sel]] = (head[at[t][sel]] & keep) | (codes[i, h][sel] << (4 * half))
            head[CODE_BYTES + 16 * t:CODE_BYTES + 16 * t + 16] = sm[i, h].reshape(-1).view(np.uint8)


def rows(pool, table_row, first, n, is_k):
    """s, m and codes as float64 of positions [first, first + n): each [H, n, 128]."""
    at, nib = PLACES[is_k]
    pos = np.arange(first, first + n)
    pages, t = np.asarray(table_row)[pos // PAGE], pos % PAGE
    heads = pool.reshape(pool.shape[0], -1, HEAD_BYTES)[pages]  # [n, H, 1280]
    codes = np.take_along_axis(heads, np.broadcast_to(at[t][:, None], (n, heads.shape[1], 128)), -1)
    codes = (codes >> (4 * nib[t][:, None])) & 15
    params = np.ascontiguousarray(heads[..., CODE_BYTES:]).view(np.uint16).reshape(n, heads.shape[1], PAGE, 4, 2)
    params = f32(params[np.arange(n), :, t]).astype(np.float64)  # [n, H, 4, 2]
    s, m = (np.repeat(params[..., i], GROUP, -1).transpose(1, 0, 2) for i in (0, 1))
    return s, m, codes.transpose(1, 0, 2).astype(np.float64)


def decode(q, k_pool, v_pool, table, lens, scale=None):
    """Attention in 64 bits over the 4-bit cache, and a bound on a kernel's
    error.  q float64 [B, Hq, 128]; returns out, bound [B, Hq, 128].

    The bound: probabilities times scales are rounded to fp16 for the product
    with the codes, 2^-11 of themselves (half a step), and act on n; the
    result is rounded once to bf16, 2^-8 of itself; and 2^-10 of the weighted
    values for the fp32 scores: sums over 128 dims of |q| (|m| + 15 s), about
    128 x 1.5 x 9 for these inputs, times 1/sqrt(128) and a few roundings of
    2^-23 each, are 2^-15 to 2^-13 absolute (up to 2^-10 for queries of 12),
    and move p by that much relatively."""
    B, Hq, D = q.shape
    H = k_pool.shape[1] // HEAD_BYTES
    scale = D ** -0.5 if scale is None else scale
    out, bound = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    for b, n in enumerate(lens):
        if n <= 0:
            continue
        ks, km, kn = rows(k_pool, table[b], 0, n, True)
        vs, vm, vn = rows(v_pool, table[b], 0, n, False)
        x = q[b].reshape(H, Hq // H, D)
        sc = np.einsum("hgd,htd->hgt", x, km + ks * kn) * scale
        p = np.exp(sc - sc.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        v = vm + vs * vn
        o = np.einsum("hgt,htd->hgd", p, v)
        out[b] = o.reshape(Hq, D)
        bound[b] = (2.0 ** -11 * np.einsum("hgt,htd->hgd", p, vs * vn) + 2.0 ** -8 * np.abs(o)
                    + 2.0 ** -10 * np.einsum("hgt,htd->hgd", p, np.abs(v))).reshape(Hq, D)
    return out, bound


def rope(x, positions, gain, pair_axis, eps=wl.RMS_EPS, theta=wl.ROPE_THETA):
    """x float64 [T, H, D] normed and rotated in 64 bits; also |y_i| + |y_{i + D/2}|
    of each element (the size of what its result is a difference of)."""
    D = x.shape[-1]
    y = x if gain is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(gain, np.float64)
    positions = np.atleast_2d(positions)
    axis = np.zeros(D // 2, int) if pair_axis is None else np.asarray(pair_axis)
    a = positions[axis].T.astype(np.float64) * theta ** (-2.0 * np.arange(D // 2) / D)
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    u, w = y[..., :D // 2], y[..., D // 2:]
    size = np.abs(u) + np.abs(w)
    return np.concatenate((u * c - w * s, u * s + w * c), -1), np.concatenate((size, size), -1)


def random_pool(rng, pages, heads):
    """Every byte random; group parameters as of values of unit spread."""
    pool = rng.integers(0, 256, size=(pages, heads, HEAD_BYTES), dtype=np.uint8)
    s = 0.2 * np.exp(0.25 * rng.standard_normal((pages, heads, 64)))
    m = -s * (7.5 + 0.5 * rng.standard_normal((pages, heads, 64)))
    sm = wl.bf16_bits(np.stack((s, m), -1).astype(np.float32))
    pool[..., CODE_BYTES:] = np.ascontiguousarray(sm).view(np.uint8).reshape(pages, heads, 256)
    return pool.reshape(pages, heads * HEAD_BYTES)


def poison_after(pool, table, lens):
    """NaN parameters and 0xff codes in every slot past each request's length."""
    heads = pool.reshape(pool.shape[0], -1, HEAD_BYTES)
    nan = np.full(8, 0x7FC0, np.uint16).view(np.uint8)
    for b, n in enumerate(lens):
        for pos in range(max(n, 0), -(-max(n, 0) // PAGE) * PAGE):
            heads[table[b][pos // PAGE], :, CODE_BYTES + 16 * (pos % PAGE):][:, :16] = nan


def page_table(rng, lens, spare=3, width=None):
    counts = [-(-int(n) // PAGE) for n in lens]
    pages = sum(counts) + spare
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), width or max(1, max(counts))), -1, np.int32)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    return table, pages
