"""The paged key-value cache next to the verify step: what is measured.

A verify round writes its new tokens' keys and values into a paged cache (spec_kv_append), attends from those tokens over
the cache (spec_kv_attend), and after a tree verify keeps the accepted path's entries (spec_kv_compact); spec_kv_gather
reads a cache back as contiguous rows. `own` chooses between these calls and their plain form in torch operations.

Shapes come from the verify workloads: 64 sequences with 8 drafts and lengths 512..4096, ragged 1..8 drafts with lengths
128..32768, trees of branching 4, 2, 2 (29 nodes), pages of 16 tokens; the heads (8 key-value heads of 128) are generic.
"""
import math

import torch

own = False

E4M3_MAX = 448.0


def _case(name, op, **kw):
    c = dict(name=name, op=op, batch=64, t_lo=1, t_hi=1, len_lo=512, len_hi=4096, q_heads=32, kv_heads=8, head_dim=128,
             block=16, dtype="bf16", tree="", layers=1, order="nhd")
    c.update(kw)
    return c


def listed():
    return [
        # one new token of one sequence: what a single user waits for
        _case("attend_one_1", "attend", batch=1, len_lo=4111, len_hi=4111),
        # one new token of each sequence of a batch, the cache in 8 bits: decoding without drafts
        _case("attend_one_64_e4m3", "attend", dtype="e4m3"),
        # the verify pass of the headline workload: 8 drafts and the token before them
        _case("attend_chain_64", "attend", t_lo=9, t_hi=9),
        # the ragged workload's lengths and drafts over an 8-bit cache, 8 query heads to a key-value head
        _case("attend_chain_ragged", "attend", t_lo=2, t_hi=9, len_lo=128, len_hi=32768, q_heads=64, dtype="e4m3"),
        # the verify pass of a token tree
        _case("attend_tree_64", "attend", tree="4,2,2"),
        # few sequences with long contexts: the cache's length has to be split to fill the GPU
        _case("attend_long_2", "attend", batch=2, t_lo=9, t_hi=9, len_lo=131071, len_hi=131071),
        # the new tokens of a verify round into an 8-bit cache
        _case("append_round_64", "append", t_lo=9, t_hi=9, dtype="e4m3"),
        # prompts of uneven lengths into an 8-bit cache
        _case("append_prompt_64", "append", t_lo=1, t_hi=4095, len_lo=0, len_hi=0, dtype="e4m3"),
        # one short cache read back
        _case("gather_1", "gather", batch=1, len_lo=777, len_hi=777),
        # a batch's 8-bit caches read back
        _case("gather_64_e4m3", "gather", dtype="e4m3"),
        # the accepted paths of a few trees in one layer
        _case("compact_tree_4", "compact", batch=4, tree="4,2,2", len_lo=40, len_hi=200),
        # the accepted paths of a batch of trees in all layers
        _case("compact_tree_64", "compact", tree="4,2,2", layers=32, len_lo=40, len_hi=200),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend"] * 5 + ["append", "gather", "compact"])
    kv_heads = rng.choice([1, 2, 4, 8])
    c = _case("", op, batch=_log_int(rng, 1, 96), kv_heads=kv_heads, q_heads=kv_heads * rng.choice([1, 2, 4, 5, 7, 8]),
              head_dim=rng.choice([64, 128, 128, 128]), block=rng.choice([16, 16, 32, 64, 128, 24]),
              dtype=rng.choice(["bf16", "e4m3"]), order=rng.choice(["nhd", "hnd"]))
    del c["name"]
    if op == "append":
        c["t_hi"] = _log_int(rng, 1, 4000)
        c["t_lo"] = rng.randint(1, c["t_hi"])
        c["len_lo"], c["len_hi"] = 0, _log_int(rng, 1, 1000)  # what is in the cache before the new tokens
        return c
    if op == "compact":
        c["tree"] = rng.choice(["4,2,2", "3,2,2,1", "5,3", "2,2,2"])
        c["layers"] = _log_int(rng, 1, 32)
        c["len_lo"], c["len_hi"] = 64, 64 + _log_int(rng, 1, 400)
        return c
    if op == "attend":
        kind = rng.choice(["one", "chain", "ragged", "tree"])
        if kind == "tree":
            c["tree"] = rng.choice(["4,2,2", "3,2,2,1", "5,3", "2,2,2"])
        elif kind != "one":
            c["t_hi"] = rng.randint(2, rng.choice([9, 17, 65]))
            c["t_lo"] = c["t_hi"] if kind == "chain" else rng.randint(1, c["t_hi"])
    # bytes and operations stay under the largest listed case's
    most = min(40000, (250000 if op == "gather" else 500000) // c["batch"],
               int(1.6e11 / (4 * c["q_heads"] * c["head_dim"] * max(_tokens(c)) * c["batch"])))
    most = max(64, most)
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


def _spread(lo, hi, n, step=0.6180339887498949, at=0.37):
    """n whole numbers spread evenly over [lo, hi], in no particular order."""
    return [lo + min(hi - lo, int(((at + step * b) % 1.0) * (hi - lo + 1))) for b in range(n)]


def _tokens(case):
    """New tokens of each sequence."""
    if case["tree"]:
        return [len(_tree(case["tree"]))] * case["batch"]
    return _spread(case["t_lo"], case["t_hi"], case["batch"], at=0.81)


def _lengths(case):
    """Cache length of each sequence, its new tokens included."""
    lens, t = _spread(case["len_lo"], case["len_hi"], case["batch"]), _tokens(case)
    if case["op"] == "append":
        return [a + b for a, b in zip(lens, t)]
    return [max(a, b) for a, b in zip(lens, t)] if case["op"] != "gather" else lens


def _paths(case):
    """Accepted paths, one for each sequence: 0 nodes up to the tree's depth, through the first child of the root or its
    last one (whose slots the path's own entries never reach, so that a second pass over the same cache changes nothing)."""
    parent = _tree(case["tree"])
    kids = {}
    for v, p in enumerate(parent):
        kids.setdefault(p, []).append(v)
    depth = case["tree"].count(",") + 1
    paths = []
    for b in range(case["batch"]):
        path, u = [], 0
        for d in range(b % (depth + 1)):
            k = kids[u]
            u = k[-1] if d == 0 and len(k) >= depth and b % 2 else k[0] if d == 0 else k[(b // 3) % len(k)]
            path.append(u)
        paths.append(path if all(v == i + 1 or v > len(path) for i, v in enumerate(path)) else path[:1])
    return paths


def work(case):
    t, lens = _tokens(case), _lengths(case)
    h, d = case["kv_heads"], case["head_dim"]
    entry = 2 * h * (d * (1 if case["dtype"] == "e4m3" else 2) + (4 if case["dtype"] == "e4m3" else 0))  # K and V of a token
    pages = sum(-(-n // case["block"]) for n in lens)
    if case["op"] == "append":
        return {"bytes": sum(t) * (2 * h * d * 2 + entry), "flops": 0}
    if case["op"] == "gather":
        return {"bytes": sum(lens) * (entry + 2 * h * d * 2) + 4 * pages, "flops": 0}
    if case["op"] == "compact":
        moved = sum(sum(v != i + 1 for i, v in enumerate(p)) for p in _paths(case))
        return {"bytes": 2 * moved * entry * case["layers"] + 16 * case["batch"], "flops": 0}
    rows = sum(t)
    if case["tree"]:
        parent = _tree(case["tree"])
        depth = [0] * len(parent)
        for v in range(1, len(parent)):
            depth[v] = depth[parent[v]] + 1
        seen = sum(len(parent) * (n - len(parent)) + sum(depth) + len(parent) for n in lens)
    else:
        seen = sum(k * (n - k) + k * (k + 1) // 2 for k, n in zip(t, lens))
    return {"bytes": sum(lens) * entry + 2 * rows * case["q_heads"] * d * 2 + 4 * pages,
            "flops": 4 * case["q_heads"] * d * seen}


# ------------------------------------------------------------------ inputs
class State:
    pass


def _offsets(counts, dev):
    return torch.tensor([0] + counts, dtype=torch.int64).cumsum(0).to(dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    s = State()
    s.case = case
    b, h, d, bs, layers = case["batch"], case["kv_heads"], case["head_dim"], case["block"], case["layers"]
    t, lens = _tokens(case), _lengths(case)
    s.t_max, s.rows, s.len_max = max(t), sum(t), max(lens)
    s.row_off = _offsets(t, dev)
    s.kv_lens = torch.tensor(lens, dtype=torch.int32, device=dev)
    # the page table: each sequence's pages lie anywhere in the pool
    need = [-(-n // bs) for n in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    start = _offsets(need, dev)[:-1]
    s.table = order[(start[:, None] + torch.arange(max(1, max(need)), device=dev)).clamp(max=pages - 1)].contiguous()
    shape = (layers, pages, bs, h, d) if case["order"] == "nhd" else (layers, pages, h, bs, d)

    def pool():
        x = torch.empty(shape, dtype=torch.bfloat16 if case["dtype"] == "bf16" else torch.float8_e4m3fn, device=dev)
        scale = None
        if case["dtype"] == "e4m3":
            scale = torch.exp2(torch.randn((layers, pages, h, bs), generator=gen, device=dev) * 0.5 - 6)
            for i in range(layers):  # codes up to the format's largest
                x[i] = (torch.randn(shape[1:], generator=gen, device=dev, dtype=torch.bfloat16) * 96).clamp(-448, 448).to(x.dtype)
        else:
            x.normal_(generator=gen)
        return (x if case["order"] == "nhd" else x.transpose(2, 3)), scale

    s.k, s.k_scale = pool()
    s.v, s.v_scale = pool()
    if case["op"] == "attend":
        # scores with a spread of a few units: some tokens matter much more than others
        s.q = torch.randn((s.rows, case["q_heads"], d), generator=gen, device=dev).mul_(3).to(torch.bfloat16)
        s.scale = 1 / math.sqrt(d)
        s.out = torch.empty_like(s.q)
        s.parent = torch.tensor(_tree(case["tree"]) * b, dtype=torch.int32, device=dev) if case["tree"] else None
    elif case["op"] == "append":
        s.k_new = torch.randn((s.rows, h, d), generator=gen, device=dev, dtype=torch.bfloat16)
        s.v_new = torch.randn((s.rows, h, d), generator=gen, device=dev, dtype=torch.bfloat16)
    elif case["op"] == "gather":
        s.out_off = _offsets(lens, dev)
        s.k_out = torch.empty((sum(lens), h, d), dtype=torch.bfloat16, device=dev)
        s.v_out = torch.empty_like(s.k_out)
    else:
        paths = _paths(case)
        s.path = torch.tensor([p + [-1] * (n - len(p)) for p, n in zip(paths, t)], dtype=torch.int32, device=dev).reshape(-1)
        s.accepted = torch.tensor([len(p) for p in paths], dtype=torch.int32, device=dev)
        s.kv_out = torch.empty_like(s.kv_lens)
    if own:
        import speculative_decoding_verification_38_gb300 as sv

        s.sv = sv
        s.cache = sv.KVCache(s.k, s.v, s.table, k_scale=s.k_scale, v_scale=s.v_scale)
        if case["op"] == "attend":
            s.args = sv.AttendArgs(cache=s.cache, q=s.q, out=s.out, kv_lens=s.kv_lens, row_off=s.row_off, t_max=s.t_max,
                                   scale=s.scale, parent=s.parent)
            s.args.set_workspace(sv.Workspace.for_attend(s.args))
    return s


# ------------------------------------------------------------------ plain forms
def _entry_index(s, pos):
    """Page and slot of positions [B, n] of each sequence (positions past the table read its last page)."""
    page = (pos // s.case["block"]).clamp(max=s.table.shape[1] - 1)
    return torch.gather(s.table.long(), 1, page), pos % s.case["block"]


def _raw(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _read(pool, scale, page, slot, out_dtype=torch.float32):
    """Entries [..., H, D] of layer 0 at (page, slot), as numbers."""
    x = _raw(pool[0])[page, slot]
    if scale is None:
        return x.to(out_dtype)
    return x.view(torch.float8_e4m3fn).to(out_dtype) * scale[0].transpose(1, 2)[page, slot].to(out_dtype).unsqueeze(-1)


def _visible(s, pos, dtype=torch.float32):
    """Whether query token t of sequence b sees position j: [B, T, L]."""
    lens = s.kv_lens.long()[:, None, None]
    t = (s.row_off[1:] - s.row_off[:-1])[:, None, None]
    q = torch.arange(s.t_max, device=pos.device)[None, :, None]
    j = pos[None, None, :]
    if s.parent is None:
        return (j <= lens - t + q) & (j < lens)
    n = s.t_max
    up = torch.zeros((n, n), dtype=dtype, device=pos.device)
    up[torch.arange(1, n, device=pos.device), s.parent[1:n].long()] = 1
    reach = torch.linalg.matrix_power(up + torch.eye(n, dtype=dtype, device=pos.device), 16) > 0
    node = (j - (lens - t)).expand(-1, n, -1)
    return (node < 0) | ((node < n) & reach[q.expand_as(node), node.clamp(0, n - 1)])


def _attend(s):
    c = s.case
    b, hq, h, d = c["batch"], c["q_heads"], c["kv_heads"], c["head_dim"]
    pos = torch.arange(s.len_max, device=s.q.device)
    page, slot = _entry_index(s, pos[None].expand(b, -1))
    rows = (s.row_off[:-1, None] + torch.arange(s.t_max, device=s.q.device)).clamp(max=s.rows - 1)
    q = s.q[rows].float().view(b, s.t_max, h, hq // h, d).permute(0, 2, 3, 1, 4).reshape(b, h, -1, d)
    k = _read(s.k, s.k_scale, page, slot).permute(0, 2, 3, 1)
    score = torch.matmul(q, k).mul_(s.scale)
    del k
    seen = _visible(s, pos)
    score = score.view(b, h, hq // h, s.t_max, s.len_max).masked_fill_(~seen[:, None, None], -math.inf)
    p = torch.exp_(score.sub_(score.amax(-1, keepdim=True).clamp(min=-1e30)))
    total = p.sum(-1, keepdim=True)
    v = _read(s.v, s.v_scale, page, slot).permute(0, 2, 1, 3)
    o = torch.matmul(p.view(b, h, -1, s.len_max), v).view(b, h, hq // h, s.t_max, d) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(b, s.t_max, hq, d)
    at = torch.arange(s.rows, device=o.device)
    seq = torch.searchsorted(s.row_off, at, right=True) - 1
    return o[seq, at - s.row_off[seq]].to(torch.bfloat16)


def _quantise(x):
    """Codes and scale: the smallest power of two that brings the largest value to 448 or less."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m > 0.875, e - 8, e - 9)
    scale = torch.where(m == 0, torch.ones_like(m), torch.exp2(e.clamp(min=-126).float()))
    return (x / scale.unsqueeze(-1)).to(torch.float8_e4m3fn), scale


def _append(s):
    at = torch.arange(s.rows, device=s.k_new.device)
    seq = torch.searchsorted(s.row_off, at, right=True) - 1
    pos = s.kv_lens.long()[seq] - s.row_off[seq + 1] + at
    page, slot = s.table.long()[seq, pos // s.case["block"]], pos % s.case["block"]
    kc, ks = _quantise(s.k_new) if s.k_scale is not None else (s.k_new, None)
    vc, vs = _quantise(s.v_new) if s.v_scale is not None else (s.v_new, None)
    _raw(s.k[0])[page, slot] = _raw(kc)
    _raw(s.v[0])[page, slot] = _raw(vc)
    if ks is not None:
        s.k_scale[0].transpose(1, 2)[page, slot] = ks
        s.v_scale[0].transpose(1, 2)[page, slot] = vs


def _gather(s):
    at = torch.arange(s.k_out.shape[0], device=s.k_out.device)
    seq = torch.searchsorted(s.out_off, at, right=True) - 1
    pos = at - s.out_off[seq]
    page, slot = s.table.long()[seq, pos // s.case["block"]], pos % s.case["block"]
    s.k_out.copy_(_read(s.k, s.k_scale, page, slot))
    s.v_out.copy_(_read(s.v, s.v_scale, page, slot))


def _compact(s):
    b, n = s.case["batch"], s.t_max
    i = torch.arange(n - 1, device=s.path.device)[None].expand(b, -1)
    path = s.path.view(b, n)[:, :-1].long()
    base = (s.kv_lens.long() - n)[:, None]
    live = i < s.accepted[:, None]
    src = _entry_index(s, base + torch.where(live, path, i + 1))
    dst = _entry_index(s, base + 1 + i)
    _raw(s.k)[:, dst[0], dst[1]] = _raw(s.k)[:, src[0], src[1]]
    _raw(s.v)[:, dst[0], dst[1]] = _raw(s.v)[:, src[0], src[1]]
    if s.k_scale is not None:
        ks, vs = s.k_scale.transpose(2, 3), s.v_scale.transpose(2, 3)
        ks[:, dst[0], dst[1]] = ks[:, src[0], src[1]]
        vs[:, dst[0], dst[1]] = vs[:, src[0], src[1]]
    s.kv_out.copy_(s.kv_lens - (n - 1 - s.accepted))


def _outputs(s):
    if s.case["op"] == "gather":
        return {"k": s.k_out, "v": s.v_out}
    r = {"k": s.k, "v": s.v}
    if s.k_scale is not None:
        r |= {"k_scale": s.k_scale, "v_scale": s.v_scale}
    if s.case["op"] == "compact":
        r["kv_out"] = s.kv_out
    return r


def run(s):
    op = s.case["op"]
    if not own:
        if op == "attend":
            return _attend(s)
        {"append": _append, "gather": _gather, "compact": _compact}[op](s)
        return _outputs(s)
    sv = s.sv
    if op == "attend":
        sv.check(sv.spec_kv_attend(s.args), "spec_kv_attend")
        return s.out
    if op == "append":
        sv.check(sv.spec_kv_append(s.cache, s.k_new, s.v_new, s.kv_lens, row_off=s.row_off, t_max=s.t_max), "spec_kv_append")
    elif op == "gather":
        sv.check(sv.spec_kv_gather(s.cache, s.kv_lens, s.out_off, s.k_out, s.v_out), "spec_kv_gather")
    else:
        sv.check(sv.spec_kv_compact(s.cache, s.row_off, s.path, s.accepted, s.kv_lens, s.kv_out), "spec_kv_compact")
    return _outputs(s)


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("gather", "append", "compact"):
        return _exact_cache(s)
    b, hq, h, d, bs = case["batch"], case["q_heads"], case["kv_heads"], case["head_dim"], case["block"]
    out = torch.zeros((s.rows, hq, d), dtype=torch.float64, device=s.q.device)
    off, lens = s.row_off.tolist(), s.kv_lens.tolist()
    for i in range(b):
        n, t = lens[i], off[i + 1] - off[i]
        j = torch.arange(n, device=s.q.device)
        page, slot = s.table[i, j // bs].long(), j % bs
        see = torch.ones((t, n), dtype=torch.bool, device=s.q.device)
        see[:, n - t:] = False
        for u in range(t):
            a = u
            while a >= 0:  # itself and what it follows
                see[u, n - t + a] = True
                a = a - 1 if s.parent is None else int(_tree(case["tree"])[a])
        for g in range(h):
            k, v = (_one_head(p, sc, page, slot, g) for p, sc in ((s.k, s.k_scale), (s.v, s.v_scale)))
            q = s.q[off[i]:off[i + 1], g * (hq // h):(g + 1) * (hq // h)].double()
            x = torch.einsum("tgd,nd->gtn", q, k) / math.sqrt(d)
            w = torch.softmax(torch.where(see, x, torch.full_like(x, -math.inf)), -1)
            out[off[i]:off[i + 1], g * (hq // h):(g + 1) * (hq // h)] = torch.einsum("gtn,nd->tgd", w, v)
    return out


def _one_head(pool, scale, page, slot, g):
    x = _raw(pool[0])[page, slot, g]
    if scale is None:
        return x.double()
    return x.view(torch.float8_e4m3fn).double() * scale[0, page, g, slot].double()[:, None]


def _exact_cache(s):
    """Append, gather and compact, one sequence after another, in 64 bits."""
    c = s.case
    off, lens, bs = s.row_off.tolist(), s.kv_lens.tolist(), c["block"]
    if c["op"] == "gather":
        got = {"k": [], "v": []}
        for i, n in enumerate(lens):
            j = torch.arange(n, device=s.table.device)
            page, slot = s.table[i, j // bs].long(), j % bs
            for name, pool, scale in (("k", s.k, s.k_scale), ("v", s.v, s.v_scale)):
                got[name].append(torch.stack([_one_head(pool, scale, page, slot, g) for g in range(c["kv_heads"])], 1))
        return {name: torch.cat(x) for name, x in got.items()}
    if s.k.numel() > 600_000_000:
        return None
    out = {}
    if c["op"] == "compact":
        accepted = s.accepted.tolist()
        for name, pool, scale in (("k", s.k, s.k_scale), ("v", s.v, s.v_scale)):
            out[name] = pool.double()
            if scale is not None:
                out[name + "_scale"] = scale.double()
            for i, n in enumerate(lens):
                for a in range(accepted[i]):
                    src, dst = n - s.t_max + int(s.path[i * s.t_max + a]), n - s.t_max + 1 + a
                    (ps, pd), (ss, sd) = s.table[i, [src // bs, dst // bs]].tolist(), (src % bs, dst % bs)
                    out[name][:, pd, sd] = out[name][:, ps, ss]
                    if scale is not None:
                        out[name + "_scale"][:, pd, :, sd] = out[name + "_scale"][:, ps, :, ss]
        out["kv_out"] = None
        return out
    for name, pool, scale, new in (("k", s.k, s.k_scale, s.k_new), ("v", s.v, s.v_scale, s.v_new)):
        whole = pool.double()
        scales = None if scale is None else scale.double()
        for i, n in enumerate(lens):
            t = off[i + 1] - off[i]
            j = torch.arange(n - t, n, device=s.table.device)
            page, slot = s.table[i, j // bs].long(), j % bs
            x = new[off[i]:off[i + 1]].double()
            if scales is not None:
                top = x.abs().amax(-1)
                sc = torch.where(top > 0, torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX)).clamp(min=-126)), 1.0)
                scales[0].transpose(1, 2)[page, slot] = sc
                x = x / sc[..., None]
            whole[0, page, slot] = x
        out[name] = whole
        if scales is not None:
            out[name + "_scale"] = scales
    return out
