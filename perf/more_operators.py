"""Rotary positions and a sliding window beside the paged cache: what is measured.

A model with rotary positions rotates its new keys on their way into the cache and its queries beside them
(spec_kv_append_rope), or rows without a cache, by positions of several axes (spec_rope); a layer with a sliding window
attends over the latest positions and the first few (spec_kv_attend_window). `own` chooses between these calls and their
plain form in torch operations.

Shapes come from the verify workloads: 64 sequences with 8 drafts and lengths 512..4096, ragged 1..8 drafts with lengths
128..32768, trees of branching 4, 2, 2 (29 nodes), pages of 16 tokens; heads (8 key-value heads of 128), windows and image
grids are generic.
"""
import math

import torch

own = False

E4M3_MAX = 448.0


def _case(name, op, **kw):
    c = dict(name=name, op=op, batch=64, t_lo=1, t_hi=1, len_lo=512, len_hi=4096, q_heads=32, kv_heads=8, head_dim=128,
             block=16, dtype="bf16", tree="", order="nhd", window=0, sinks=0, rotary=128, adjacent=False, axes=1,
             alternating=False, grid="")
    c.update(kw)
    return c


def listed():
    return [
        # one new token of one sequence past its window: what a single user waits for
        _case("window_one_1", "window", batch=1, len_lo=32768, len_hi=32768, window=4096, sinks=4),
        # one new token of each sequence of a batch, an 8-bit cache, some contexts shorter than the window
        _case("window_one_64_e4m3", "window", dtype="e4m3", len_lo=128, len_hi=32768, window=1024, sinks=4),
        # the verify pass of the headline workload in a layer with a short window
        _case("window_chain_64", "window", t_lo=9, t_hi=9, window=1024, sinks=4),
        # the ragged workload over an 8-bit cache, 8 query heads to a key-value head, a long window
        _case("window_chain_ragged", "window", t_lo=2, t_hi=9, len_lo=128, len_hi=32768, q_heads=64, dtype="e4m3",
              window=4096, sinks=16),
        # the verify pass of a token tree
        _case("window_tree_64", "window", tree="4,2,2", len_lo=128, len_hi=32768, window=2000, sinks=4),
        # few sequences with long contexts and a window that is itself long
        _case("window_long_2", "window", batch=2, t_lo=9, t_hi=9, len_lo=131071, len_hi=131071, window=65536, sinks=128),
        # one new token of one sequence, with its queries
        _case("append_one_1", "append", batch=1, len_lo=4110, len_hi=4110),
        # the new tokens of a verify round into an 8-bit cache, with their queries
        _case("append_round_64_e4m3", "append", t_lo=9, t_hi=9, dtype="e4m3"),
        # token trees, positions by depth, a quarter of each head rotated in adjacent pairs
        _case("append_tree_64", "append", tree="4,2,2", rotary=32, adjacent=True),
        # prompts of uneven lengths, with their queries
        _case("append_prompt_64", "append", t_lo=1, t_hi=4095, len_lo=0, len_hi=0),
        # the queries of a verify round of a model that reads images: positions of three axes
        _case("rope_round_64", "rope", t_lo=9, t_hi=9, axes=3),
        # the queries of a video prompt: frames, rows and columns, a pair's axis alternating
        _case("rope_video_8", "rope", batch=8, grid="16,32,32", axes=3, alternating=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window"] * 4 + ["append"] * 2 + ["rope"])
    kv_heads = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 96, 128, 128, 128])
    c = _case("", op, batch=_log_int(rng, 1, 96), kv_heads=kv_heads, q_heads=kv_heads * rng.choice([1, 2, 4, 5, 7, 8]),
              head_dim=d, block=rng.choice([16, 16, 32, 64, 128, 24]), dtype=rng.choice(["bf16", "e4m3"]),
              order=rng.choice(["nhd", "hnd"]), rotary=rng.choice([d, d, d // 2, 32]), adjacent=rng.random() < 0.3)
    del c["name"]
    if op == "rope":
        c["axes"] = rng.choice([1, 3, 3, 2])
        c["alternating"] = c["axes"] > 1 and rng.random() < 0.5
        if c["axes"] == 3 and rng.random() < 0.5:
            c["batch"] = min(c["batch"], 8)
            c["grid"] = ",".join(str(_log_int(rng, 1, n)) for n in (16, 32, 32))
        else:
            c["t_hi"] = _log_int(rng, 1, 1000)
            c["t_lo"] = rng.randint(1, c["t_hi"])
        return c
    kind = rng.choice(["one", "chain", "ragged", "tree"])
    if kind == "tree":
        c["tree"] = rng.choice(["4,2,2", "3,2,2,1", "5,3", "2,2,2"])
    elif kind != "one":
        c["t_hi"] = rng.randint(2, rng.choice([9, 17, 65]))
        c["t_lo"] = c["t_hi"] if kind == "chain" else rng.randint(1, c["t_hi"])
    if op == "append":
        if kind == "ragged":
            c["t_hi"] = _log_int(rng, 1, 60 if c["dtype"] == "e4m3" else min(2000, 100000 // c["batch"]))
            c["t_lo"] = rng.randint(1, c["t_hi"])
        c["len_lo"], c["len_hi"] = 0, _log_int(rng, 1, 1000)  # what is in the cache before the new tokens
        return c
    # bytes and operations stay under the largest listed case's
    c["window"] = _log_int(rng, 5, 16384)
    c["sinks"] = rng.choice([0, 1, 4, 4, 16, 100])
    most = min(40000, 500000 // c["batch"])
    c["window"] = max(5, min(c["window"], int(5.5e10 / (4 * c["q_heads"] * d * max(_tokens(c)) * c["batch"])) - 200))
    c["len_hi"] = _log_int(rng, 64, most)
    c["len_lo"] = rng.randint(32, c["len_hi"])
    return c


# ------------------------------------------------------------------ sizes
def _tree(text):
    """Parents of a tree with the given number of children per level, node 0 the root, in level order."""
    parent, level = [-1], [0]
    for n in (int(x) for x in text.split(",")):
        start = len(parent)
        parent += [u for u in level for _ in range(n)]
        level = list(range(start, len(parent)))
    return parent


def _depths(case, t):
    """How far below a sequence's first new token each of its t new tokens lies."""
    if not case["tree"]:
        return list(range(t))
    depth = []
    for p in _tree(case["tree"]):
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return depth


def _spread(lo, hi, n, step=0.6180339887498949, at=0.37):
    """n whole numbers spread evenly over [lo, hi], in no particular order."""
    return [lo + min(hi - lo, int(((at + step * b) % 1.0) * (hi - lo + 1))) for b in range(n)]


def _tokens(case):
    """New tokens of each sequence."""
    if case["grid"]:
        return [math.prod(int(x) for x in case["grid"].split(","))] * case["batch"]
    if case["tree"]:
        return [len(_tree(case["tree"]))] * case["batch"]
    return _spread(case["t_lo"], case["t_hi"], case["batch"], at=0.81)


def _lengths(case):
    """Cache length of each sequence, its new tokens included."""
    lens, t = _spread(case["len_lo"], case["len_hi"], case["batch"]), _tokens(case)
    return [a + b for a, b in zip(lens, t)] if case["op"] == "append" else [max(a, b) for a, b in zip(lens, t)]


def _sections(case):
    """Pairs of each axis; the first has what the others leave."""
    pairs, n = case["rotary"] // 2, case["axes"]
    rest = [pairs * 3 // 8 if not case["alternating"] and n == 3 else pairs // n] * (n - 1)
    return [pairs - sum(rest)] + rest


def work(case):
    t, lens = _tokens(case), _lengths(case)
    h, hq, d = case["kv_heads"], case["q_heads"], case["head_dim"]
    entry = 2 * h * (d * (1 if case["dtype"] == "e4m3" else 2) + (4 if case["dtype"] == "e4m3" else 0))  # K and V of a token
    rows = sum(t)
    if case["op"] == "rope":
        return {"bytes": rows * (2 * hq * d * 2 + 4 * case["axes"]), "flops": 0}
    if case["op"] == "append":
        return {"bytes": rows * (2 * h * d * 2 + entry + 2 * hq * d * 2), "flops": 0}
    read = seen = 0
    for k, n in zip(t, lens):
        c = n - k
        lo = max(0, c + 1 - case["window"])  # the earliest position in the first token's window
        read += min(case["sinks"], lo) + n - lo
        for x in _depths(case, k):
            at = min(c, max(0, c + x + 1 - case["window"]))
            seen += min(case["sinks"], at) + c - at + min(x + 1, case["window"])
    return {"bytes": read * entry + 2 * rows * hq * d * 2 + 4 * (read // case["block"]), "flops": 4 * hq * d * seen}


# ------------------------------------------------------------------ inputs
class State:
    pass


def _offsets(counts, dev):
    return torch.tensor([0] + counts, dtype=torch.int64).cumsum(0).to(dev)


def _positions(case, gen, dev):
    """int32 [axes, rows]: the places in a grid after a text of some length, or a text's own, the same on every axis."""
    axes, t = case["axes"], _tokens(case)
    start = torch.randint(0, 4096, (case["batch"],), generator=gen, device=dev)
    if case["grid"]:
        f, y, x = (torch.arange(int(n), device=dev) for n in case["grid"].split(","))
        place = torch.stack([g.reshape(-1) for g in torch.meshgrid(f, y, x, indexing="ij")])
        return (place[:, None] + start[None, :, None]).reshape(3, -1).to(torch.int32).contiguous()
    seq = torch.repeat_interleave(torch.arange(case["batch"], device=dev), torch.tensor(t, device=dev))
    off = _offsets(t, dev)
    at = start[seq] + torch.arange(sum(t), device=dev) - off[seq]
    return at.to(torch.int32).repeat(axes, 1)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    s = State()
    s.case = case
    b, h, hq, d, bs = case["batch"], case["kv_heads"], case["q_heads"], case["head_dim"], case["block"]
    t, lens = _tokens(case), _lengths(case)
    s.t_max, s.rows, s.len_max = max(t), sum(t), max(lens)
    # scores with a spread of a few units: some tokens matter much more than others
    s.q = torch.randn((s.rows, hq, d), generator=gen, device=dev).mul_(3).to(torch.bfloat16)
    s.out = torch.empty_like(s.q)
    if case["op"] != "window":
        pairs = case["rotary"] // 2
        s.inv_freq = (10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float().to(dev)
    if case["op"] == "rope":
        s.positions = _positions(case, gen, dev)
    else:
        s.row_off = _offsets(t, dev)
        s.kv_lens = torch.tensor(lens, dtype=torch.int32, device=dev)
        s.parent = torch.tensor(_tree(case["tree"]) * b, dtype=torch.int32, device=dev) if case["tree"] else None
        # the page table: each sequence's pages lie anywhere in the pool; pages that no token sees any more are gone
        first = [max(0, n - k + 1 - case["window"]) // bs if case["window"] else 0 for k, n in zip(t, lens)]
        keep = [[j for j in range(-(-n // bs)) if j >= f or j * bs < case["sinks"]] for f, n in zip(first, lens)]
        pages = sum(map(len, keep)) + 3
        order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
        s.table = torch.full((b, max(k[-1] for k in keep) + 1), -1, dtype=torch.int32)
        where = torch.tensor([i * s.table.shape[1] + j for i, k in enumerate(keep) for j in k])
        s.table = s.table.to(dev)
        s.table.view(-1)[where.to(dev)] = order[:len(where)]
        shape = (1, pages, bs, h, d) if case["order"] == "nhd" else (1, pages, h, bs, d)

        def pool():
            x = torch.empty(shape, dtype=torch.bfloat16 if case["dtype"] == "bf16" else torch.float8_e4m3fn, device=dev)
            scale = None
            if case["dtype"] == "e4m3":
                scale = torch.exp2(torch.randn((1, pages, h, bs), generator=gen, device=dev) * 0.5 - 6)
                codes = torch.randn(shape[1:], generator=gen, device=dev, dtype=torch.bfloat16) * 96
                x[0] = codes.clamp(-448, 448).to(x.dtype)  # codes up to the format's largest
            else:
                x.normal_(generator=gen)
            return (x if case["order"] == "nhd" else x.transpose(2, 3)), scale

        s.k, s.k_scale = pool()
        s.v, s.v_scale = pool()
    if case["op"] == "append":
        s.k_new = torch.randn((s.rows, h, d), generator=gen, device=dev, dtype=torch.bfloat16)
        s.v_new = torch.randn((s.rows, h, d), generator=gen, device=dev, dtype=torch.bfloat16)
    if own:
        import speculative_decoding_verification_38_gb300 as sv

        s.sv = sv
        if case["op"] != "window":
            s.rope = sv.Rope(s.inv_freq, adjacent=case["adjacent"], sections=_sections(case) if case["axes"] > 1 else None,
                             alternating=case["alternating"])
        if case["op"] != "rope":
            s.cache = sv.KVCache(s.k, s.v, s.table, k_scale=s.k_scale, v_scale=s.v_scale)
        if case["op"] == "window":
            s.args = sv.AttendArgs(cache=s.cache, q=s.q, out=s.out, kv_lens=s.kv_lens, row_off=s.row_off, t_max=s.t_max,
                                   scale=1 / math.sqrt(d), parent=s.parent)
            s.args.set_workspace(sv.Workspace.for_attend(s.args))
    return s


# ------------------------------------------------------------------ plain forms
def _raw(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _read(pool, scale, page, slot):
    """Entries [..., H, D] at (page, slot), as numbers."""
    x = _raw(pool[0])[page, slot]
    if scale is None:
        return x.float()
    return x.view(torch.float8_e4m3fn).float() * scale[0].transpose(1, 2)[page, slot].unsqueeze(-1)


def _reach(s):
    """Whether a tree's node is another or lies below it [T, T], and the nodes' depths [T]."""
    n, dev = s.t_max, s.q.device
    if s.parent is None:
        at = torch.arange(n, device=dev)
        return at[:, None] >= at[None, :], at
    up = torch.zeros((n, n), dtype=torch.float32, device=dev)
    up[torch.arange(1, n, device=dev), s.parent[1:n].long()] = 1
    reach = torch.linalg.matrix_power(up + torch.eye(n, device=dev), 16) > 0
    return reach, reach.sum(1) - 1


def _window(s):
    """Over the sinks and the window's positions, gathered for each sequence."""
    c, dev = s.case, s.q.device
    b, hq, h, d, w, bs = c["batch"], c["q_heads"], c["kv_heads"], c["head_dim"], c["window"], c["block"]
    lens = s.kv_lens.long()[:, None]
    ctx = lens - (s.row_off[1:] - s.row_off[:-1])[:, None]
    lo = (ctx + 1 - w).clamp(min=0)
    span = min(w + s.t_max - 1, s.len_max)
    pos = torch.cat([torch.arange(c["sinks"], device=dev).expand(b, -1), lo + torch.arange(span, device=dev)], 1)
    there = torch.cat([torch.arange(c["sinks"], device=dev).expand(b, -1) < torch.minimum(lo, lens),
                       lo + torch.arange(span, device=dev) < lens], 1)
    n = pos.shape[1]
    page = torch.gather(s.table.long(), 1, torch.where(there, pos, lens - 1) // bs)
    slot = torch.where(there, pos, lens - 1) % bs
    reach, depth = _reach(s)
    node = pos - ctx  # of a new token; below zero before them
    inside = node.clamp(0, s.t_max - 1)
    late = torch.where(node < 0, node, depth[inside])[:, None]  # its position, from the first new token's
    near = (depth[None, :, None] - late < w) | (pos < c["sinks"])[:, None]
    seen = there[:, None] & near & ((node < 0)[:, None] | reach[:, inside].permute(1, 0, 2))
    rows = (s.row_off[:-1, None] + torch.arange(s.t_max, device=dev)).clamp(max=s.rows - 1)
    q = s.q[rows].float().view(b, s.t_max, h, hq // h, d).permute(0, 2, 3, 1, 4).reshape(b, h, -1, d)
    score = torch.matmul(q, _read(s.k, s.k_scale, page, slot).permute(0, 2, 3, 1)).mul_(1 / math.sqrt(d))
    score = score.view(b, h, hq // h, s.t_max, n).masked_fill_(~seen[:, None, None], -math.inf)
    p = torch.exp_(score.sub_(score.amax(-1, keepdim=True).clamp(min=-1e30)))
    total = p.sum(-1, keepdim=True)
    v = _read(s.v, s.v_scale, page, slot).permute(0, 2, 1, 3)
    o = torch.matmul(p.view(b, h, -1, n), v).view(b, h, hq // h, s.t_max, d) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(b, s.t_max, hq, d)
    at = torch.arange(s.rows, device=dev)
    seq = torch.searchsorted(s.row_off, at, right=True) - 1
    return o[seq, at - s.row_off[seq]].to(torch.bfloat16)


def _axis_of_pair(case):
    """The axis that each pair turns by."""
    pairs, parts = case["rotary"] // 2, _sections(case)
    if case["alternating"]:
        n = case["axes"]
        return [i % n if i < n * parts[i % n] else 0 for i in range(pairs)]
    return [a for a, k in enumerate(parts) for _ in range(k)]


def _turns(s, positions):
    """Cosines and sines [rows, 1, pairs] of positions [axes, rows], the angles in 64 bits."""
    axis = torch.tensor(_axis_of_pair(s.case), device=positions.device)
    angle = positions.double()[axis].t() * s.inv_freq.double()
    return angle.cos().float().unsqueeze(1), angle.sin().float().unsqueeze(1)


def _rotate(s, x, cos, sin):
    r = s.case["rotary"]
    x = x.float()
    y = x.clone()
    first, second = (slice(0, r, 2), slice(1, r, 2)) if s.case["adjacent"] else (slice(0, r // 2), slice(r // 2, r))
    a, b = x[..., first], x[..., second]
    y[..., first] = a * cos - b * sin
    y[..., second] = b * cos + a * sin
    return y


def _quantise(x):
    """Codes and scale: the smallest power of two that brings the largest value to 448 or less."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m > 0.875, e - 8, e - 9)
    scale = torch.where(m == 0, torch.ones_like(m), torch.exp2(e.clamp(min=-126).float()))
    return (x / scale.unsqueeze(-1)).to(torch.float8_e4m3fn), scale


def _append(s):
    at = torch.arange(s.rows, device=s.q.device)
    seq = torch.searchsorted(s.row_off, at, right=True) - 1
    t = at - s.row_off[seq]
    ctx = s.kv_lens.long()[seq] - (s.row_off[seq + 1] - s.row_off[seq])
    place = ctx + (t if s.parent is None else _reach(s)[1][t])
    cos, sin = _turns(s, place[None])
    k = _rotate(s, s.k_new, cos, sin)
    page, slot = s.table.long()[seq, (ctx + t) // s.case["block"]], (ctx + t) % s.case["block"]
    kc, ks = _quantise(k) if s.k_scale is not None else (k.to(torch.bfloat16), None)
    vc, vs = _quantise(s.v_new) if s.v_scale is not None else (s.v_new, None)
    _raw(s.k[0])[page, slot] = _raw(kc)
    _raw(s.v[0])[page, slot] = _raw(vc)
    if ks is not None:
        s.k_scale[0].transpose(1, 2)[page, slot] = ks
        s.v_scale[0].transpose(1, 2)[page, slot] = vs
    s.out.copy_(_rotate(s, s.q, cos, sin))


def _outputs(s):
    if s.case["op"] != "append":
        return s.out
    r = {"k": s.k, "v": s.v, "q": s.out}
    if s.k_scale is not None:
        r |= {"k_scale": s.k_scale, "v_scale": s.v_scale}
    return r


def run(s):
    op = s.case["op"]
    if not own:
        if op == "window":
            return _window(s)
        if op == "append":
            _append(s)
        else:
            s.out.copy_(_rotate(s, s.q, *_turns(s, s.positions)))
    elif op == "window":
        s.sv.check(s.sv.spec_kv_attend_window(s.args, s.case["window"], s.case["sinks"]), "spec_kv_attend_window")
    elif op == "append":
        s.sv.check(s.sv.spec_kv_append_rope(s.cache, s.rope, s.k_new, s.v_new, s.kv_lens, row_off=s.row_off, t_max=s.t_max,
                                            parent=s.parent, q=s.q, q_out=s.out), "spec_kv_append_rope")
    else:
        s.sv.check(s.sv.spec_rope(s.rope, s.q, s.out, s.positions), "spec_rope")
    return _outputs(s)


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_turn(case, s.inv_freq, s.q, s.positions)
    if case["op"] == "append":
        return _exact_append(s)
    hq, h, d, bs, w = case["q_heads"], case["kv_heads"], case["head_dim"], case["block"], case["window"]
    out = torch.zeros((s.rows, hq, d), dtype=torch.float64, device=s.q.device)
    off, lens = s.row_off.tolist(), s.kv_lens.tolist()
    for i in range(case["batch"]):
        n, t = lens[i], off[i + 1] - off[i]
        c, depth = n - t, _depths(case, t)
        above = [p if case["tree"] else u - 1 for u, p in enumerate(_tree(case["tree"]) if case["tree"] else range(t))]
        lo = max(0, c + 1 - w)
        j = torch.cat([torch.arange(min(case["sinks"], lo)), torch.arange(lo, n)])  # what any of them sees
        see = torch.zeros((t, len(j)), dtype=torch.bool)
        for u in range(t):
            see[u] = (j < c) & ((j < case["sinks"]) | (j > c + depth[u] - w))
            a = u
            while a >= 0:  # itself and what it follows
                if depth[u] - depth[a] < w or c + a < case["sinks"]:
                    see[u] |= j == c + a
                a = above[a]
        j, see = j.to(s.q.device), see.to(s.q.device)
        page, slot = s.table[i, j // bs].long(), j % bs
        for g in range(h):
            k, v = (_one_head(p, sc, page, slot, g) for p, sc in ((s.k, s.k_scale), (s.v, s.v_scale)))
            q = s.q[off[i]:off[i + 1], g * (hq // h):(g + 1) * (hq // h)].double()
            x = torch.einsum("tgd,nd->gtn", q, k) / math.sqrt(d)
            a = torch.softmax(torch.where(see, x, torch.full_like(x, -math.inf)), -1)
            out[off[i]:off[i + 1], g * (hq // h):(g + 1) * (hq // h)] = torch.einsum("gtn,nd->tgd", a, v)
    return out


def _one_head(pool, scale, page, slot, g):
    x = _raw(pool[0])[page, slot, g]
    if scale is None:
        return x.double()
    return x.view(torch.float8_e4m3fn).double() * scale[0, page, g, slot].double()[:, None]


def _exact_turn(case, inv_freq, x, positions):
    """Pairs as complex numbers, each times e^(i angle)."""
    r, parts = case["rotary"], _sections(case)
    angle = torch.empty((x.shape[0], r // 2), dtype=torch.float64, device=x.device)
    used = [0] * case["axes"]
    for i in range(r // 2):
        a = i % case["axes"] if case["alternating"] else next(k for k in range(case["axes"]) if used[k] < parts[k])
        a = a if used[a] < parts[a] else 0
        used[a] += 1
        angle[:, i] = positions[a].double() * inv_freq[i].double()
    y = x.double()
    z = y[..., :r].reshape(*y.shape[:-1], r // 2, 2) if case["adjacent"] else y[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2)
    z = torch.view_as_complex(z.contiguous()) * torch.polar(torch.ones_like(angle), angle)[:, None]
    z = torch.view_as_real(z)
    y[..., :r] = z.flatten(-2) if case["adjacent"] else z.transpose(-1, -2).flatten(-2)
    return y


def _exact_append(s):
    """One sequence after another, in 64 bits."""
    c, dev = s.case, s.q.device
    if s.k.numel() > 600_000_000:
        return None
    off, lens, bs = s.row_off.tolist(), s.kv_lens.tolist(), c["block"]
    out = {"k": s.k.double(), "v": s.v.double(), "q": torch.empty(s.q.shape, dtype=torch.float64, device=dev)}
    if s.k_scale is not None:
        out |= {"k_scale": s.k_scale.double(), "v_scale": s.v_scale.double()}
    for i, n in enumerate(lens):
        t, rows = off[i + 1] - off[i], slice(off[i], off[i + 1])
        place = (n - t + torch.tensor(_depths(c, t), device=dev))[None]
        out["q"][rows] = _exact_turn(c, s.inv_freq, s.q[rows], place)
        j = torch.arange(n - t, n, device=dev)
        page, slot = s.table[i, j // bs].long(), j % bs
        for name, x in (("k", _exact_turn(c, s.inv_freq, s.k_new[rows], place)), ("v", s.v_new[rows].double())):
            if s.k_scale is not None:
                top = x.abs().amax(-1)
                sc = torch.where(top > 0, torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX)).clamp(min=-126)), 1.0)
                out[name + "_scale"][0].transpose(1, 2)[page, slot] = sc
                x = x / sc[..., None]
            out[name][0, page, slot] = x
    return out
