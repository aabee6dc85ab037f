"""Cases, plain forms and exact results of the operators that verify drafted tokens over a paged cache, and of cross attention.

A serving program drafts a tree of tokens for each request, checks all of them in one forward and keeps a path:

    append  key and value rows written to their pages, normed and rotated on the way (drafted rows, prompt chunks, or the
            plain rows of an encoder's states), with the rotated queries
    tree    attention of a tree of drafted tokens over the cache: every cached position, and a token's ancestors
    cross   attention of packed rows to paged states of another length, without an order between them
    settle  the end of a checked step: every layer's drafted rows appended, the accepted path found and its rows moved
            to where a plain continuation would have put them

``run`` computes them with elementary torch operations, or, where ``own`` is true, with the calls a serving program
makes of the package.  ``exact`` has each result in 64 bits, written from the operators' definitions.

A tree is one array: parents[i] is the row, counted within its request, that row i continues, -1 for a row that
continues the cache, and always less than i.  Row i of a request lies at position n_past + i of the cache; its rotary
position is n_past + its depth.
"""
import math
import random

import torch

own = False

PAGE = 16
DIM = 128
ROPE_THETA = 1.0e6
RMS_EPS = 1.0e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the drafted trees of a full batch, in the fused projection's rows
        dict(name="append drafts", op="append", batch=64, lo=5, hi=33, past=4000, hq=16, hkv=8, kind="tree", fused=True, len_seed=1),
        # a packed bucket of prompt chunks with images in them: three axes
        dict(name="append chunks", op="append", batch=16, lo=200, hi=2000, past=3000, hq=16, hkv=8, kind="axes", fused=True, len_seed=2),
        # an encoder's states laid into pages, as the projections leave them
        dict(name="append states", op="append", batch=8, lo=130, hi=15600, past=0, hq=8, hkv=8, kind="states", fused=True, len_seed=3),
        # one caller's small tree over a short cache: latency
        dict(name="tree single", op="tree", batch=1, rows_lo=8, rows_hi=8, lo=257, hi=257, hq=16, hkv=8, chain=False, len_seed=4),
        # the ordinary decode batch, each request with a tree of up to 16
        dict(name="tree batch", op="tree", batch=32, rows_lo=9, rows_hi=16, lo=200, hi=2000, hq=16, hkv=8, chain=False, len_seed=5),
        # large trees
        dict(name="tree wide", op="tree", batch=24, rows_lo=33, rows_hi=64, lo=500, hi=8000, hq=16, hkv=8, chain=False, len_seed=6),
        # the long-context batch with a few drafted tokens in a line
        dict(name="tree long", op="tree", batch=64, rows_lo=4, rows_hi=8, lo=2000, hi=16000, hq=16, hkv=8, chain=True, len_seed=7),
        # a decoder's prefix tokens over short audio
        dict(name="cross few", op="cross", batch=5, rows_lo=1, rows_hi=4, lo=13, hi=390, hq=8, hkv=8, len_seed=8),
        # prompts over two minutes of audio
        dict(name="cross prompts", op="cross", batch=8, rows_lo=40, rows_hi=448, lo=1170, hi=1560, hq=16, hkv=8, len_seed=9),
        # prompts over up to twenty minutes
        dict(name="cross long", op="cross", batch=8, rows_lo=100, rows_hi=448, lo=2000, hi=15600, hq=16, hkv=8, len_seed=10),
        # a single caller's step settled in four layers
        dict(name="settle one", op="settle", batch=1, lo=8, hi=8, past=300, layers=4, hkv=8, len_seed=11),
        # a full batch's
        dict(name="settle batch", op="settle", batch=64, lo=16, hi=64, past=1000, layers=4, hkv=8, len_seed=12),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["append", "tree", "tree", "cross", "settle"])
    hkv = rng.choice([1, 2, 4, 5, 8, 8, 8, 8])
    case = dict(op=op, hkv=hkv, len_seed=rng.randrange(1 << 20))
    if op != "settle":
        case["hq"] = hkv * rng.choice([1, 2, 2])
    if op == "append":
        kind = rng.choice(["tree", "tree", "line", "axes", "states"])
        batch = _spread(rng, 1, 128)
        hi = _spread(rng, 1, 64 if kind == "tree" else 30000 // batch)
        return case | dict(batch=batch, lo=_spread(rng, 1, hi), hi=hi, past=rng.choice([0, _spread(rng, 1, 4000)]), kind=kind,
                           fused=rng.random() < 0.5)
    if op == "settle":
        hi = _spread(rng, 1, 64)
        return case | dict(batch=_spread(rng, 1, 128), lo=_spread(rng, 1, hi), hi=hi, past=_spread(rng, 1, 2000),
                           layers=rng.randint(1, 4))
    if op == "tree":
        batch = _spread(rng, 1, 128)
        rows = _spread(rng, 1, 64)
        hi = _spread(rng, 1, min(16000, (500000 if rows <= 8 else 150000) // batch))
        return case | dict(batch=batch, rows_lo=_spread(rng, 1, rows), rows_hi=rows, lo=_spread(rng, 1, hi), hi=hi,
                           chain=rng.random() < 0.3)
    batch = _spread(rng, 1, 32)
    rows = _spread(rng, 1, 448)
    hi = _spread(rng, 1, min(15600, 30000000 // (batch * rows)))
    return case | dict(batch=batch, rows_lo=_spread(rng, 1, rows), rows_hi=rows, lo=_spread(rng, 1, hi), hi=hi)


def _whole(case, salt, lo, hi):
    rng = random.Random(case["len_seed"] * 7 + salt)
    return [rng.randint(lo, hi) for _ in range(case["batch"])]


def _rows(case):
    """Rows of each request."""
    return _whole(case, 0, case.get("rows_lo", case.get("lo")), case.get("rows_hi", case.get("hi")))


def _past(case):
    """Cached positions of each request (of a cross attention: its states)."""
    if case["op"] in ("tree", "cross"):
        return _whole(case, 1, case["lo"], case["hi"])
    if case.get("kind") == "states":
        return [0] * case["batch"]
    return _whole(case, 1, case["past"] // 4, case["past"])


def _trees(case):
    """A tree for each request: some parents close behind, some anywhere before."""
    rng = random.Random(case["len_seed"] * 7 + 2)
    chain = case.get("chain", False)
    return [[i - 1 if chain or i == 0 else rng.randint(max(0, i - 4), i - 1) if rng.random() < 0.5 else rng.randint(0, i - 1)
             for i in range(n)] for n in _rows(case)]


def _depth(tree):
    out = []
    for p in tree:
        out.append(0 if p < 0 else out[p] + 1)
    return out


def work(case):
    rows, hkv = _rows(case), case["hkv"]
    row = hkv * DIM * 2  # bytes of one row of K or V
    if case["op"] == "append":
        q = 0 if case["kind"] == "states" else 2 * case["hq"] * DIM * 2
        return {"bytes": sum(rows) * (4 * row + q), "flops": sum(rows) * (q // 4 + row // 2) * 6}
    if case["op"] == "settle":  # the rows read and written once each; what is accepted is a few of them
        return {"bytes": case["layers"] * sum(rows) * 4 * row, "flops": case["layers"] * sum(rows) * row // 2 * 6}
    hq, past = case["hq"], _past(case)
    if case["op"] == "cross":
        seen, held = sum(n * m for n, m in zip(rows, past)), sum(past)
    else:
        trees = _trees(case)
        seen = sum(n * m for n, m in zip(rows, past)) + sum(sum(_depth(t)) + len(t) for t in trees)
        held = sum(past) + sum(rows)
    return {"bytes": held * 2 * row + sum(rows) * hq * DIM * 4, "flops": 4 * DIM * hq * seen}


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, size=1.0):
    return (size * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


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


def _gain(g):
    return (0.5 + torch.rand(DIM, generator=g, device="cuda")).to(torch.bfloat16).float()


def _cumulative(counts):
    return _ints([sum(counts[:i]) for i in range(len(counts) + 1)])


def _tokens(case, seed):
    """Drafted tokens, and what the model answers at each: often one of the drafted continuations."""
    rng = random.Random(seed)
    draft, target = [], []
    for tree in _trees(case):
        d = [rng.randrange(40) for _ in tree]
        for i in range(len(tree)):
            children = [c for c, p in enumerate(tree) if p == i]
            target.append(d[rng.choice(children)] if children and rng.random() < 0.85 else rng.randrange(40))
        draft += d
    return _ints(draft), _ints(target)


def prepare(case, seed):
    g = _generator(seed)
    op, hkv = case["op"], case["hkv"]
    rows, past = _rows(case), _past(case)
    total = sum(rows)
    held = past if op == "cross" else [a + b for a, b in zip(past, rows)]
    state = dict(op=op, rows=rows, past=past, total=total, max_rows=max(rows), cu_seqlens=_cumulative(rows))
    state["page_table"], pages = _pages(g, held)
    layers = case.get("layers", 1)
    state["k_pages"] = [_normal(g, pages, PAGE, hkv, DIM) for _ in range(layers)]
    state["v_pages"] = [_normal(g, pages, PAGE, hkv, DIM) for _ in range(layers)]
    state["n_past"] = _ints(past)  # of a cross attention: the states' lengths
    if op in ("tree", "cross"):
        state["q"] = _normal(g, total, case["hq"], DIM, size=1.5)
    if op in ("tree", "settle") or case.get("kind") == "tree":
        flat = [p for tree in _trees(case) for p in tree]
        state["parents"] = None if case.get("chain") else _ints(flat)
    if op == "append":
        kind, hq = case["kind"], case["hq"]
        state |= dict(kind=kind, parents=state.get("parents"), positions=None, pair_axis=None, q_gain=None, k_gain=None)
        x = _normal(g, total, (0 if kind == "states" else hq) + 2 * hkv, DIM)  # the fused projection's rows
        at = x.shape[1] - 2 * hkv
        q, k, v = x[:, :at], x[:, at:at + hkv], x[:, at + hkv:]
        if not case["fused"]:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        state |= dict(q=None if kind == "states" else q, k=k, v=v)
        if kind != "states":
            state |= dict(q_gain=_gain(g), k_gain=_gain(g))
        if kind == "axes":  # frames of 16 x 24 patches after a long text
            i = torch.arange(total, device="cuda")
            first = int(torch.randint(0, 100000, (1,), generator=g, device="cuda"))
            state["positions"] = torch.stack((first + i // 384, first + i // 24 % 16, first + i % 24)).to(torch.int32)
            state["pair_axis"] = [i % 3 if i < 60 else 0 for i in range(64)]
    if op == "settle":
        state["k"] = [_normal(g, total, hkv, DIM) for _ in range(layers)]
        state["v"] = [_normal(g, total, hkv, DIM) for _ in range(layers)]
        state |= dict(k_gain=_gain(g), draft=None, target=None)
        state["q_gain"] = state["k_gain"]
        state["draft"], state["target"] = _tokens(case, seed)
    return state


# ------------------------------------------------------------------ one pass

def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


def _qa():
    import paged_kv_gqa_attention_gb300 as qa

    return qa


def _own_append(s):
    args = dict(n_past=s["n_past"], parents=s["parents"])
    if s["kind"] == "states":
        args = dict(rotate=False)
    else:
        args |= dict(positions=s["positions"], pair_axis=s["pair_axis"], q_gain=s["q_gain"], k_gain=s["k_gain"],
                     rms_eps=RMS_EPS, rope_theta=ROPE_THETA)
    q = _qa().qa_append_rows(s["q"], s["k"], s["v"], s["cu_seqlens"], s["page_table"], s["k_pages"][0], s["v_pages"][0], **args)
    return (s["k_pages"][0], s["v_pages"][0]) + (() if q is None else (q,))


def _workspace(s):
    """Kept by a serving program from call to call."""
    if "workspace" not in s:
        size = _qa().qa_rows_attn_workspace_size(s["max_rows"], n_q_heads=s["q"].shape[1], n_kv_heads=s["k_pages"][0].shape[2])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _own_tree(s):
    return _qa().qa_tree_attn(s["q"], s["cu_seqlens"], s["n_past"], s["page_table"], s["k_pages"][0], s["v_pages"][0],
                              s["max_rows"], parents=s["parents"], workspace=_workspace(s), stable_metadata=1)


def _own_cross(s):
    return _qa().qa_cross_attn(s["q"], s["cu_seqlens"], s["n_past"], s["page_table"], s["k_pages"][0], s["v_pages"][0],
                               s["max_rows"], workspace=_workspace(s), stable_metadata=1)


def _own_settle(s):
    qa = _qa()
    for k, v, k_pages, v_pages in zip(s["k"], s["v"], s["k_pages"], s["v_pages"]):
        qa.qa_append_rows(None, k, v, s["cu_seqlens"], s["page_table"], k_pages, v_pages, n_past=s["n_past"],
                          parents=s["parents"], q_gain=s["q_gain"], k_gain=s["k_gain"], rms_eps=RMS_EPS, rope_theta=ROPE_THETA)
    found = qa.qa_tree_accept(s["draft"], s["target"], s["parents"], s["cu_seqlens"], s["n_past"], s["page_table"],
                              s["k_pages"], s["v_pages"], s["max_rows"])
    return (*found, *s["k_pages"], *s["v_pages"])


_OWN = dict(append=_own_append, tree=_own_tree, cross=_own_cross, settle=_own_settle)


# ------------------------------------------------------------------ plain forms

def _places(s):
    """The request of each packed row, and the row's number in it."""
    cu = s["cu_seqlens"].long()
    i = torch.arange(s["total"], device="cuda")
    r = torch.searchsorted(cu, i, right=True) - 1
    return r, i - cu[r]


def _slots(s, r, at):
    return s["page_table"][r, at // PAGE].long(), at % PAGE


def _depths(s, r, i):
    """How many ancestors each row has."""
    if s["parents"] is None:
        return i
    first = s["cu_seqlens"].long()[r]
    parent = s["parents"].long()
    up = torch.where(parent < 0, parent, parent + first)
    node, depth = up, torch.zeros_like(i)
    for _ in range(s["max_rows"] - 1):
        depth = depth + (node >= 0)
        node = torch.where(node >= 0, up[node.clamp(min=0)], node)
    return depth


def _rotated(x, positions, gain, pair_axis):
    """bf16 rows [T, H, D] normed and rotated by positions [axes, T], in 32 bits, the angles in 64."""
    half = DIM // 2
    y = x.float()
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + RMS_EPS) * gain
    freq = ROPE_THETA ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    axis = torch.tensor(pair_axis or [0] * half, device="cuda")
    angle = positions.double()[axis].T * freq
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    a, b = y[..., :half], y[..., half:]
    return torch.cat((a * cos - b * sin, a * sin + b * cos), -1).to(torch.bfloat16)


def _plain_append(s):
    r, i = _places(s)
    past = s["n_past"].long()[r]
    page, slot = _slots(s, r, past + i)
    k, out = s["k"], ()
    if s["kind"] != "states":
        positions = (past + _depths(s, r, i))[None] if s["positions"] is None else s["positions"]
        k = _rotated(k, positions, s["k_gain"], s["pair_axis"])
        out = (_rotated(s["q"], positions, s["q_gain"], s["pair_axis"]),)
    s["k_pages"][0][page, slot] = k
    s["v_pages"][0][page, slot] = s["v"]
    return (s["k_pages"][0], s["v_pages"][0]) + out


def _plain_rows(s, b, n):
    """A request's first n positions of K and V, in 32 bits: [H, n, D] each."""
    table = s["page_table"][b, : -(-n // PAGE)].long()
    return tuple(s[name][0][table].reshape(-1, *s[name][0].shape[2:])[:n].float().transpose(0, 1)
                 for name in ("k_pages", "v_pages"))


def _plain_attended(s, b, first, n_rows, n_keys, visible):
    hkv = s["k_pages"][0].shape[2]
    q = s["q"][first:first + n_rows].float()
    q = q.view(n_rows, hkv, -1, DIM).permute(1, 2, 0, 3)  # [H, group, rows, D]
    k, v = _plain_rows(s, b, n_keys)
    score = q @ k.transpose(-1, -2)[:, None] / math.sqrt(DIM)
    if visible is not None:
        score = score.masked_fill(~visible, -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    out = (p @ v[:, None]) / p.sum(-1, keepdim=True)
    return out.permute(2, 0, 1, 3).reshape(n_rows, -1, DIM).to(torch.bfloat16)


def _plain_tree(s):
    out, first = [], 0
    for b, (n, past) in enumerate(zip(s["rows"], s["past"])):
        i = torch.arange(n, device="cuda")
        if s["parents"] is None:
            visible = i[None] <= i[:, None]
        else:  # a row sees itself and what its parent sees; parents come first
            parent = s["parents"][first:first + n].long()
            visible = torch.eye(n, dtype=torch.bool, device="cuda")
            node = parent
            for _ in range(n - 1):
                visible = visible | (i[None] == node[:, None])
                node = torch.where(node >= 0, parent[node.clamp(min=0)], node)
        visible = torch.cat((torch.ones(n, past, dtype=torch.bool, device="cuda"), visible), 1)
        out.append(_plain_attended(s, b, first, n, past + n, visible))
        first += n
    return torch.cat(out)


def _plain_cross(s):
    out, first = [], 0
    for b, (n, held) in enumerate(zip(s["rows"], s["past"])):
        out.append(_plain_attended(s, b, first, n, held, None))
        first += n
    return torch.cat(out)


def _plain_settle(s):
    r, i = _places(s)
    past = s["n_past"].long()
    page, slot = _slots(s, r, past[r] + i)
    positions = (past[r] + _depths(s, r, i))[None]
    for k, v, k_pages, v_pages in zip(s["k"], s["v"], s["k_pages"], s["v_pages"]):
        k_pages[page, slot] = _rotated(k, positions, s["k_gain"], None)
        v_pages[page, slot] = v
    batch, most = len(s["rows"]), s["max_rows"]
    b = torch.arange(batch, device="cuda")
    padded = {}
    for name in ("draft", "target", "parents"):
        padded[name] = torch.full((batch, most), -2, dtype=torch.int64, device="cuda")
        padded[name][r, i] = s[name].long()
    path = torch.full((batch, most), -1, dtype=torch.int64, device="cuda")
    node = path[:, 0] = torch.zeros_like(b)
    found = torch.ones_like(b, dtype=torch.bool)
    for step in range(1, most):
        answer = padded["target"][b, node]
        fits = (padded["parents"] == node[:, None]) & (padded["draft"] == answer[:, None])
        found = found & fits.any(-1)
        child = fits.to(torch.int32).argmax(-1)
        node = torch.where(found, child, node)
        path[:, step] = torch.where(found, child, -1)
    count = (path >= 0).sum(-1)
    answer = padded["target"][b, node]
    # every row is read before one is written; past the path a row is written to where it was
    to = torch.where(path >= 0, torch.arange(most, device="cuda"), 0)
    source, place = past[:, None] + path.clamp(min=0), past[:, None] + to
    everyone = b[:, None].expand(batch, most)
    from_page, from_slot = _slots(s, everyone, source)
    page, slot = _slots(s, everyone, place)
    for pool in (*s["k_pages"], *s["v_pages"]):
        pool[page, slot] = pool[from_page, from_slot]
    return (count.to(torch.int32), path.to(torch.int32), answer.to(torch.int32), *s["k_pages"], *s["v_pages"])


_PLAIN = dict(append=_plain_append, tree=_plain_tree, cross=_plain_cross, settle=_plain_settle)


# ------------------------------------------------------------------ 64 bits

def _exact_rope(x, positions, gain, pair_axis):
    x = x.double()
    x = x / torch.sqrt(torch.sum(x ** 2, -1, keepdim=True) / DIM + RMS_EPS) * gain.double()
    out = torch.empty_like(x)
    for i in range(DIM // 2):
        a = (positions[pair_axis[i] if pair_axis else 0].double() * ROPE_THETA ** (-2.0 * i / DIM))[:, None]
        u, w = x[..., i], x[..., i + DIM // 2]
        out[..., i], out[..., i + DIM // 2] = u * torch.cos(a) - w * torch.sin(a), u * torch.sin(a) + w * torch.cos(a)
    return out


def _exact_positions(case):
    """The cache position and the rotary position of each row, as lists."""
    at, turn = [], []
    trees = _trees(case) if case["op"] == "settle" or case["kind"] == "tree" else None
    for b, (n, past) in enumerate(zip(_rows(case), _past(case))):
        at.append([past + i for i in range(n)])
        turn += [past + d for d in (_depth(trees[b]) if trees else range(n))]
    return at, turn


def _exact_put(pool, table, at, rows):
    first = 0
    for b, positions in enumerate(at):
        t = torch.tensor(positions, device="cuda")
        pool[table[b][t // PAGE].long(), t % PAGE] = rows[first:first + len(positions)]
        first += len(positions)


def exact(case, seed):
    s = prepare(case, seed)
    op, table = case["op"], s["page_table"]
    if op == "append":
        if case["kind"] == "states":
            at, turn = [list(range(n)) for n in s["rows"]], None
        else:
            at, turn = _exact_positions(case)
            turn = torch.tensor(turn, device="cuda")[None] if s["positions"] is None else s["positions"]
        k_pages, v_pages = s["k_pages"][0].double(), s["v_pages"][0].double()
        k = s["k"].double() if turn is None else _exact_rope(s["k"], turn, s["k_gain"], s["pair_axis"])
        _exact_put(k_pages, table, at, k)
        _exact_put(v_pages, table, at, s["v"].double())
        return (k_pages, v_pages) + (() if turn is None else (_exact_rope(s["q"], turn, s["q_gain"], s["pair_axis"]),))
    if op == "settle":
        at, turn = _exact_positions(case)
        turn = torch.tensor(turn, device="cuda")[None]
        draft, target = s["draft"].tolist(), s["target"].tolist()
        first, paths, answers = 0, [], []
        for tree in _trees(case):
            path = [0]
            while True:
                answer = target[first + path[-1]]
                child = next((c for c, p in enumerate(tree) if p == path[-1] and draft[first + c] == answer), None)
                if child is None:
                    break
                path.append(child)
            paths.append(path)
            answers.append(answer)
            first += len(tree)
        pools = [p.double() for p in (*s["k_pages"], *s["v_pages"])]
        for layer in range(case["layers"]):
            _exact_put(pools[layer], table, at, _exact_rope(s["k"][layer], turn, s["k_gain"], None))
            _exact_put(pools[case["layers"] + layer], table, at, s["v"][layer].double())
        for pool in pools:
            for b, path in enumerate(paths):
                a = torch.tensor([s["past"][b] + i for i in path], device="cuda")
                rows = pool[table[b][a // PAGE].long(), a % PAGE].clone()
                a = s["past"][b] + torch.arange(len(path), device="cuda")
                pool[table[b][a // PAGE].long(), a % PAGE] = rows
        return (_ints([len(p) for p in paths]), _ints([p + [-1] * (s["max_rows"] - len(p)) for p in paths]), _ints(answers), *pools)
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    hkv, first = case["hkv"], 0
    trees = _trees(case) if op == "tree" else None
    for b, (n, past) in enumerate(zip(s["rows"], s["past"])):
        held = past + n if trees else past
        if trees:
            hidden = [[True] * n for _ in range(n)]
            for i in range(n):
                j = i
                while j >= 0:
                    hidden[i][j] = False
                    j = trees[b][j]
            hidden = torch.tensor(hidden, device="cuda")
        pages = table[b, : -(-held // PAGE)].long()
        k, v = (s[name][0][pages].double().reshape(-1, hkv, DIM)[:held] for name in ("k_pages", "v_pages"))
        for h in range(hkv):
            x = s["q"][first:first + n].double().reshape(n, hkv, -1, DIM)[:, h]  # [n, group, D]
            score = torch.einsum("ngd,td->ngt", x, k[:, h]) / math.sqrt(float(DIM))
            if trees:
                score[:, :, past:] = score[:, :, past:].masked_fill(hidden[:, None], -math.inf)
            out[first:first + n].view(n, hkv, -1, DIM)[:, h] = torch.einsum("ngt,td->ngd", torch.softmax(score, -1), v[:, h])
        first += n
    return out
