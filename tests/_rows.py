"""Plain numpy definitions of drafted rows over a paged bf16 cache and of
cross attention, in 64 bits, and inputs for their tests."""
import numpy as np

import _kvq
import workloads as wl

PAGE = 16


def tree(rng, n, back=None):
    """Parents of a random tree of n rows; back: how far behind a parent may lie."""
    return np.array([-1 if i == 0 else rng.integers(max(0, i - (back or i)), i) for i in range(n)], np.int32)


def depths(parents):
    d = []
    for p in parents:
        d.append(0 if p < 0 else d[p] + 1)
    return np.array(d, np.int64)


def seen(parents):
    """[n, n]: row i sees row j."""
    n = len(parents)
    out = np.zeros((n, n), bool)
    for i in range(n):
        j = i
        while j >= 0:
            out[i, j] = True
            j = parents[j]
    return out


def cumulative(counts):
    return np.concatenate(([0], np.cumsum(counts))).astype(np.int32)


def places(table, n_past, rows):
    """Page and slot of every packed row."""
    at = [(b, p + i) for b, (p, n) in enumerate(zip(n_past, rows)) for i in range(n)]
    return (np.array([table[b, x // PAGE] for b, x in at], np.int64), np.array([x % PAGE for _, x in at], np.int64))


def attention(q, k_pool, v_pool, table, rows, keys, visible, scale=None):
    """q float64 [T, Hq, 128]; pools float64 [P, 16, H, 128]; keys: positions of
    each request; visible[b]: bool [rows, keys] or None.  Returns out and a
    bound on a kernel's error, both [T, Hq, 128].

    The bound: the result is rounded once to bf16, 2^-8 of itself.  A
    probability enters the product as p_hi + p_lo, p_hi truncated to bf16 and
    the rest, below 2^-7 of p, rounded to bf16: 2^-15 of p.  Scores are sums
    over 128 dims in fp32, whose terms' roundings and the tensor core's own
    (each at most 2^-23 of the largest partial sum, 16 terms at a time) stay
    below 2^-20 of sum |q k|; with the scale that moves p by as much
    relatively, in it and in the sum.  The running sums of p v take a rounding
    of 2^-23 each 16 keys, and the merge a few more."""
    T, Hq, D = q.shape
    H = k_pool.shape[2]
    scale = D ** -0.5 if scale is None else scale
    out, bound, first = np.zeros(q.shape), np.zeros(q.shape), 0
    for b, (n, m) in enumerate(zip(rows, keys)):
        if n == 0:
            continue
        if m > 0:
            pages = table[b, :-(-m // PAGE)]
            k, v = (p[pages].reshape(-1, H, D)[:m] for p in (k_pool, v_pool))
            x = q[first:first + n].reshape(n, H, Hq // H, D)
            vis = np.ones((n, m), bool) if visible is None else visible[b]
            hide = ~vis[:, None, None, :]
            with np.errstate(invalid="ignore"):
                sc = np.where(hide, -np.inf, np.einsum("nhgd,thd->nhgt", x, k) * scale)
                size = np.where(hide, 0, np.einsum("nhgd,thd->nhgt", np.abs(x), np.abs(k)) * scale).max(-1, keepdims=True)
            top = sc.max(-1, keepdims=True)
            p = np.exp(sc - np.where(np.isfinite(top), top, 0))
            p /= np.where(p.sum(-1, keepdims=True) > 0, p.sum(-1, keepdims=True), 1)
            # a hidden value takes no part, whatever it holds
            o, mass = np.zeros((n, H, Hq // H, D)), np.zeros((n, H, Hq // H, D))
            for i in range(n):
                j = np.nonzero(vis[i])[0]
                o[i] = np.einsum("hgt,thd->hgd", p[i][..., j], v[j])
                mass[i] = np.einsum("hgt,thd->hgd", p[i][..., j], np.abs(v[j]))
            out[first:first + n] = o.reshape(n, Hq, D)
            share = 2.0 ** -15 + 2 * 2.0 ** -20 * size + (m / 16 + 64) * 2.0 ** -23
            bound[first:first + n] = (2.0 ** -8 * np.abs(o) + share * mass + 1e-30).reshape(n, Hq, D)
        first += n
    return out, bound


def tree_visible(parents, rows, n_past):
    """visible for attention(): every cached position, and a row's ancestors."""
    out, first = [], 0
    for n, past in zip(rows, n_past):
        t = np.arange(n) - 1 if parents is None else parents[first:first + n]
        out.append(np.concatenate((np.ones((n, past), bool), seen(t)), 1))
        first += n
    return out


def accept(draft, target, parents, rows):
    """Paths (lists of row numbers) and the token after each (None without rows)."""
    paths, tokens, first = [], [], 0
    for n in rows:
        t = np.arange(n) - 1 if parents is None else parents[first:first + n]
        path, token = ([0] if n else []), None
        while path:
            token = target[first + path[-1]]
            nxt = [c for c in range(n) if t[c] == path[-1] and draft[first + c] == token]
            if not nxt:
                break
            path.append(nxt[0])
        paths.append(path)
        tokens.append(token)
        first += n
    return paths, tokens


def pool(rng, pages, heads):
    return wl.normal_bf16(rng, (pages, PAGE, heads, 128))


def poison(bits_pool, table, keys):
    """NaN in every slot that holds no key: unused pages, and slots past each request's keys."""
    used = np.zeros(bits_pool.shape[:2], bool)
    for b, m in enumerate(keys):
        for j in range(-(-m // PAGE)):
            used[table[b, j], :min(PAGE, m - j * PAGE)] = True
    bits_pool[~used] = wl.bf16_bits(np.array([np.nan], np.float32))[0]


page_table = _kvq.page_table
