"""The paged cache's operators on the GPU against the float64 oracle (oracle/kv.py); the bounds are derived in
tests/kv_cases.py from the kernels' roundings."""
import numpy as np
import pytest
import torch

from oracle import kv as okv
from tests.kv_cases import Case, random_tree, tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_38_gb300 as sv

    sv.build()
    return sv


def _append(sv, c, new_dtype=torch.bfloat16, offsets=True, seed=5, edit=None):
    g = torch.Generator().manual_seed(seed)
    c.to_device(sv)
    new = [(torch.randn((c.rows, c.H, c.D), generator=g) * torch.exp(torch.randn((c.rows, c.H, 1), generator=g) * 3))
           .to(new_dtype) for _ in range(2)]
    if edit:
        edit(new)
    status = torch.full((c.B,), -7, dtype=torch.int32, device=c.device)
    sv.check(sv.spec_kv_append(c.cache, new[0].to(c.device), new[1].to(c.device), c.dlens,
                               row_off=c.doff if offsets else None, t_max=c.t_max, layer=c.layer, seq_status=status),
             "spec_kv_append")
    k, v, ks, vs = c.host()
    held16 = [x.to(torch.bfloat16) if c.dtype == "bf16" else x for x in new]
    okv.append(k, v, ks, vs, c.table, c.layer, held16[0].double().numpy(), held16[1].double().numpy(), c.row_off, c.lens)
    return status, (k, v, ks, vs)


def _same_cache(c, want):
    k, v, ks, vs = want
    np.testing.assert_array_equal(c.raw(c.dk), k)
    np.testing.assert_array_equal(c.raw(c.dv), v)
    if ks is not None:
        np.testing.assert_array_equal(c.dks.cpu().numpy(), ks)
        np.testing.assert_array_equal(c.dvs.cpu().numpy(), vs)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("new_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,D,bs,order,pad", [(2, 64, 16, "nhd", 0), (3, 128, 5, "hnd", 16), (1, 96, 1, "nhd", 32),
                                              (8, 256, 32, "hnd", 0), (5, 16, 24, "nhd", 0)])
def test_append(sv, dtype, new_dtype, H, D, bs, order, pad):
    """Codes, scales and untouched slots, exactly: ragged new tokens, none at all, lengths equal to the new tokens'."""
    c = Case(lens=[9, 40, 1, 17, 3, 64], tokens=[9, 3, 1, 0, 3, 33], H=H, D=D, bs=bs, dtype=dtype, order=order, pad=pad,
             layers=2, layer=1)
    status, want = _append(sv, c, new_dtype)
    assert status.tolist() == [0] * c.B
    _same_cache(c, want)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_append_equal_tokens_without_offsets(sv, dtype):
    c = Case(lens=[5, 77, 6], tokens=[5, 5, 5], H=2, D=64, dtype=dtype)
    status, want = _append(sv, c, offsets=False)
    assert status.tolist() == [0, 0, 0]
    _same_cache(c, want)


def test_append_extreme_values(sv):
    """Zeros, one value at the border of a scale, subnormals, the largest floats, NaN and infinities."""
    c = Case(lens=[12], tokens=[12], H=1, D=16, dtype="e4m3")

    def edit(new):
        for x in new:
            x[0] = 0
            x[1] = 0
            x[1, 0, 3] = 448.0
            x[2] = 0
            x[2, 0, 3] = 448.0 * (1 + 2**-20)
            x[3] = 1e-41
            x[4, 0, 0] = 3.4e38
            x[5, 0, 1] = float("nan")
            x[6, 0, 2] = float("inf")
            x[7] = -float("inf")
            x[8] = -0.0
            x[9] = 2.0**-126
            x[10, 0] = torch.tensor([1 + 1 / 16, 1 + 3 / 16, -1 - 1 / 16, 448 / 256, 464 / 256, 2.0**-9, 2.0**-10, 3 * 2.0**-11]
                                    * 2)

    status, want = _append(sv, c, torch.float32, edit=edit)
    assert status.tolist() == [0]
    _same_cache(c, want)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_append_statuses(sv, dtype):
    c = Case(lens=[20, 20, 20, 20, 20], tokens=[4, 4, 4, 4, 4], H=2, D=32, dtype=dtype, bs=4)
    c.to_device(sv)
    before = c.raw(c.dk), c.raw(c.dv)
    c.dlens.copy_(torch.tensor([20, 3, 21, 20, 20], dtype=torch.int32))
    c.dtable[3, 4] = 10**6
    c.dtable[4, 4] = -1
    new = torch.randn((c.rows, 2, 32)).to(torch.bfloat16).cuda()
    status = torch.full((5,), -7, dtype=torch.int32, device="cuda")
    sv.check(sv.spec_kv_append(c.cache, new, new, c.dlens, row_off=c.doff, seq_status=status), "append")
    assert status.tolist() == [0, 2, 2, 4, 4]
    after = c.raw(c.dk), c.raw(c.dv)
    mine = np.zeros(c.held.shape, dtype=bool)
    for j in range(16, 20):
        mine[c.table[0, j // 4], j % 4] = True
    for x, y in zip(before, after):
        np.testing.assert_array_equal(x[:, ~mine], y[:, ~mine])
    bad = c.doff.clone()
    bad[2] = 3  # falls: sequence 1 ends before it starts
    bad[5] = 10**9
    c.dlens.fill_(20)
    sv.check(sv.spec_kv_append(c.cache, new, new, c.dlens, row_off=bad, seq_status=status), "append")
    assert status.tolist()[1] == 4 and status.tolist()[4] == 4


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,D,bs,order,pad", [(2, 64, 16, "nhd", 0), (3, 128, 5, "hnd", 16), (1, 96, 1, "nhd", 32),
                                              (8, 256, 32, "hnd", 0), (5, 16, 24, "nhd", 0)])
def test_gather(sv, dtype, out_dtype, H, D, bs, order, pad):
    """Every entry, rounded once; empty sequences; nothing past the last row."""
    c = Case(lens=[9, 0, 40, 0, 0, 1, 131, 64], tokens=[0] * 8, H=H, D=D, bs=bs, dtype=dtype, order=order, pad=pad,
             layers=2, layer=1)
    c.to_device(sv)
    off = np.concatenate([[0], np.cumsum(c.lens)]).astype(np.int64)
    rows = int(off[-1])
    out = [torch.full((rows + 3, H, D), 7.0, dtype=out_dtype, device="cuda") for _ in range(2)]
    status = torch.full((c.B,), -7, dtype=torch.int32, device="cuda")
    sv.check(sv.spec_kv_gather(c.cache, c.dlens, torch.from_numpy(off).cuda(), out[0], out[1], layer=1,
                               seq_status=status), "gather")
    assert status.tolist() == [0] * c.B
    k, v, ks, vs = c.host()
    for pool, sc, got in ((k, ks, out[0]), (v, vs, out[1])):
        assert (got[rows:] == 7).all()
        for b in range(c.B):
            for h in range(H):
                want = okv.entries(pool, sc, c.table[b], 1, h, c.lens[b])
                seg = got[off[b]:off[b + 1], h].double().cpu().numpy()
                # a product of 4 and 24 bits rounded to float32, then to the output's type
                lim = (2.0**-24 + (2.0**-8 if out_dtype == torch.bfloat16 else 0)) * np.abs(want) if sc is not None else 0
                assert (np.abs(seg - want) <= lim).all()


def test_gather_statuses(sv):
    c = Case(lens=[8, 8, 8, 8], tokens=[0] * 4, H=1, D=32, bs=4)
    c.to_device(sv)
    c.dlens.copy_(torch.tensor([8, 7, -1, 8], dtype=torch.int32))
    c.dtable[3, 1] = 999
    off = torch.tensor([0, 8, 16, 24, 32], dtype=torch.int64, device="cuda")
    out = [torch.full((32, 1, 32), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    status = torch.full((4,), -7, dtype=torch.int32, device="cuda")
    sv.check(sv.spec_kv_gather(c.cache, c.dlens, off, *out, seq_status=status), "gather")
    assert status.tolist() == [0, 4, 4, 4]
    for x in out:
        assert (x[8:24] == 7).all() and (x[28:] == 0).all() and not (x[24:28] == 0).any()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,D,bs,order", [(2, 64, 16, "nhd"), (3, 128, 5, "hnd"), (1, 32, 1, "nhd")])
def test_compact(sv, dtype, H, D, bs, order):
    """Paths that overlap their targets, whole trees, chains, nothing accepted, all layers."""
    n = [29, 29, 1, 12, 40, 29, 7, 20]
    path = [[2, 3, 4], [4, 16, 28], [], list(range(1, 12)), list(range(2, 40, 2)), [], [1, 2, 6], [1, 2, 3, 4, 9, 11, 12, 13, 14, 15, 16, 19]]
    c = Case(lens=[29, 100, 1, 77, 40, 64, 9, 33], tokens=n, H=H, D=D, bs=bs, dtype=dtype, order=order, layers=3)
    c.to_device(sv)
    off = c.row_off
    flat = np.full(c.rows, -1, np.int32)
    for b, p in enumerate(path):
        flat[off[b]:off[b] + len(p)] = p
    acc = np.array([len(p) for p in path], np.int32)
    out = torch.full((c.B,), -7, dtype=torch.int32, device="cuda")
    blocks, status = out.clone(), out.clone()
    sv.check(sv.spec_kv_compact(c.cache, c.doff, torch.from_numpy(flat).cuda(), torch.from_numpy(acc).cuda(), c.dlens,
                                out, out_num_blocks=blocks, seq_status=status), "compact")
    k, v, ks, vs = c.host()
    want = okv.compact((k, v), (ks, vs), c.table, off, flat, acc, c.lens)
    assert status.tolist() == [0] * c.B
    assert out.tolist() == want.tolist() and blocks.tolist() == [-(-x // bs) for x in want.tolist()]
    _same_cache(c, (k, v, ks, vs))


def test_compact_statuses_leave_the_cache(sv):
    c = Case(lens=[20] * 8, tokens=[6] * 8, H=2, D=32, bs=4, layers=2)
    c.to_device(sv)
    before = c.raw(c.dk), c.raw(c.dv)
    path = torch.tensor([[2, 2, -1, -1, -1, -1], [3, 6, -1, -1, -1, -1], [0, 1, -1, -1, -1, -1], [2, 3, 4, 5, 5, 5],
                         [2, 4, -1, -1, -1, -1], [2, 4, -1, -1, -1, -1], [2, 4, -1, -1, -1, -1], [3, 2, -1, -1, -1, -1]],
                        dtype=torch.int32, device="cuda").reshape(-1)
    acc = torch.tensor([2, 2, 2, 6, -1, 2, 2, 2], dtype=torch.int32, device="cuda")
    c.dlens[5] = 5
    c.dtable[6, 4] = 10**8
    out, status = (torch.full((8,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    sv.check(sv.spec_kv_compact(c.cache, c.doff, path, acc, c.dlens, out, seq_status=status), "compact")
    assert status.tolist() == [4, 4, 4, 4, 4, 2, 4, 4]
    assert out.tolist() == c.dlens.tolist()
    np.testing.assert_array_equal(before[0], c.raw(c.dk))
    np.testing.assert_array_equal(before[1], c.raw(c.dv))


# ------------------------------------------------------------------ attention
SHAPES = [  # H, G, D, bs, order, pad
    (2, 4, 128, 16, "nhd", 0),
    (1, 1, 64, 16, "hnd", 0),
    (3, 5, 128, 5, "nhd", 16),
    (2, 8, 64, 1, "hnd", 32),
    (1, 7, 96, 24, "nhd", 0),
    (2, 2, 16, 128, "hnd", 0),
    (1, 3, 256, 32, "nhd", 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,G,D,bs,order,pad", SHAPES)
def test_attend_one_token(sv, dtype, H, G, D, bs, order, pad):
    """Single tokens, lengths from one up, around a tile's and a page's end, and none at all."""
    c = Case(lens=[1, 2, 16, 17, 127, 128, 129, 0, 300, 1025], tokens=[1, 1, 1, 1, 1, 1, 1, 0, 1, 1], H=H, G=G, D=D, bs=bs,
             dtype=dtype, order=order, pad=pad, layers=2, layer=1, q_scale=2.0)
    c.attend(sv)
    assert c.status.tolist() == [0] * c.B
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,G,D,bs,order,pad", SHAPES)
def test_attend_chain(sv, dtype, H, G, D, bs, order, pad):
    """Ragged chains: the new tokens alone, across a tile's end, more than a tile of them."""
    c = Case(lens=[9, 140, 128, 3, 260, 640, 128], tokens=[9, 17, 5, 3, 65, 1, 128], H=H, G=G, D=D, bs=bs, dtype=dtype,
             order=order, pad=pad, q_scale=2.0)
    c.attend(sv)
    assert c.status.tolist() == [0] * c.B
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,G,D,bs,order,pad", SHAPES[:5])
def test_attend_tree(sv, dtype, H, G, D, bs, order, pad):
    trees = [tree([4, 2, 2]), [-1], random_tree(40, 1), random_tree(128, 2), tree([64]), list(range(-1, 30))]
    c = Case(lens=[29, 300, 140, 200, 65, 129], tokens=[len(t) for t in trees], H=H, G=G, D=D, bs=bs, dtype=dtype,
             order=order, pad=pad, parent=sum(trees, []), q_scale=2.0)
    c.attend(sv)
    assert c.status.tolist() == [0] * c.B
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_attend_long(sv, dtype):
    """Few sequences over many tiles: the length is split, and joined."""
    c = Case(lens=[20011, 7], tokens=[3, 2], H=1, G=4, D=128, bs=16, dtype=dtype, q_scale=3.0)
    c.attend(sv)
    c.check()
    first = c.out.clone()
    c.attend(sv)
    assert torch.equal(first, c.out)  # the same call twice: the same bits


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("G,D,t", [(1, 64, 1), (4, 128, 1), (4, 128, 5), (4, 64, 9), (8, 128, 9), (4, 128, 29), (8, 128, 17)])
def test_attend_many_tiles_to_a_processor(sv, dtype, G, D, t):
    """More tiles than 152 processors take at once: runs of several tiles over several sequences and heads, every
    size of row tile, groups of rows with nothing to do."""
    lens = [int(x) for x in np.random.default_rng(3).integers(t, 1500, 24)]
    c = Case(lens=lens, tokens=[max(1, t - b % 3) for b in range(24)], H=8, G=G, D=D, dtype=dtype, q_scale=2.0)
    c.attend(sv)
    assert c.status.tolist() == [0] * c.B
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("G,D,t", [(1, 128, 1), (2, 64, 9), (4, 128, 9), (8, 128, 9), (4, 128, 29)])
def test_attend_many_short_sequences(sv, dtype, G, D, t):
    """Many sequences of a tile or less, so that each processor has more entries than tiles in flight; some empty."""
    B = 300
    tokens = [0 if b % 7 == 3 else 1 + (b * 5) % t for b in range(B)]
    lens = [max(tokens[b], (b * 37) % 150) for b in range(B)]
    c = Case(lens=lens, tokens=tokens, H=4, G=G, D=D, dtype=dtype, q_scale=2.0)
    c.attend(sv)
    assert c.status.tolist() == [0] * c.B
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("G,D,t", [(4, 128, 4), (8, 64, 4), (3, 96, 15), (5, 128, 16), (4, 128, 32), (2, 64, 64)])
def test_attend_one_entry_over_many_processors(sv, dtype, G, D, t):
    """Every size of row tile with an entry in 40 parts and one in a few: groups of parts, and groups of groups."""
    c = Case(lens=[5003, 390], tokens=[t, t], H=1, G=G, D=D, dtype=dtype, q_scale=2.0)
    c.attend(sv)
    assert c.status.tolist() == [0, 0]
    c.check()
    first = c.out.clone()
    for _ in range(3):
        c.attend(sv)
        assert torch.equal(first, c.out)  # whoever joins them: the same bits


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_attend_growing_scores(sv, dtype):
    """Scores that rise along the cache (every tile a new maximum), then fall."""
    for sign in (1, -1):
        c = Case(lens=[1500], tokens=[2], H=1, G=2, D=64, dtype=dtype)
        ramp = torch.linspace(0.1, 4.0, 1500)
        for j in range(1500):
            g, i = okv.slot_of(c.table[0], j, c.bs)
            x = torch.full((64,), float(ramp[j] if sign > 0 else ramp[-1 - j]))
            row = c.k[0, g, i, 0]
            row.copy_(x.to(torch.bfloat16) if dtype == "bf16" else (x * 64).to(torch.float8_e4m3fn).view(torch.uint8))
            if dtype == "e4m3":
                c.ks[0, g, 0, i] = 2.0**-6
        c.q = torch.full_like(c.q, 2.0)
        c.attend(sv)
        c.check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_attend_queries_of_wide_range(sv, dtype, D):
    """An element far above a row's others takes nothing from them: keys are zero where it stands, so that the scores
    are the small ones' alone, and the bound counts those."""
    c = Case(lens=[150, 40], tokens=[9, 3], H=2, G=4, D=D, dtype=dtype)
    spike = torch.randint(D, (c.rows, 8), generator=c.g)
    c.q.scatter_(2, spike[..., None], torch.full((c.rows, 8, 1), 2.0**16, dtype=torch.bfloat16))
    for row in range(c.rows):
        for head in range(8):
            c.k[..., head // 4, spike[row, head]] = 0
    c.attend(sv)
    assert c.status.tolist() == [0, 0]
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_attend_query_that_is_not_finite(sv, dtype, value):
    """Its own row is NaN, and no other."""
    make = lambda: Case(lens=[150, 40], tokens=[9, 3], H=2, G=4, D=128, dtype=dtype, q_scale=2.0)  # noqa: E731
    clean, c = make(), make()
    c.q[4, 5, 77] = value
    c.attend(sv)
    out, lse, av, mag, spread = clean.expected()
    got = c.out.double().cpu().numpy()
    keep = np.ones(got.shape[:2], dtype=bool)
    keep[4, 5] = False
    assert np.isnan(got[4, 5]).all()
    assert (np.abs(got - out) <= clean.bound(out, av, mag, spread))[keep].all()


def _unseen_values(c, value):
    """`value` in the keys and values of the last new token of every sequence (which only it sees)."""
    code = 127 if c.dtype == "e4m3" else value
    for b in range(c.B):
        if c.tokens[b] > 1:
            g, i = okv.slot_of(c.table[b], c.lens[b] - 1, c.bs)
            c.k[c.layer, g, i] = code
            c.v[c.layer, g, i] = code


@pytest.mark.parametrize("dtype,value", [("bf16", float("nan")), ("bf16", float("inf")), ("bf16", -float("inf")),
                                         ("e4m3", float("nan"))])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("as_tree", [False, True])
def test_attend_unseen_nan_and_infinity(sv, dtype, value, D, as_tree):
    """What a token does not see has no effect on it."""
    lens, tokens = [5, 130, 257, 300], [5, 4, 2, 9]
    parent = sum(([-1] + [0] * (t - 1) for t in tokens), []) if as_tree else None
    make = lambda: Case(lens=lens, tokens=tokens, H=2, G=4, D=D, dtype=dtype, parent=parent, q_scale=2.0)  # noqa: E731
    clean, c = make(), make()
    _unseen_values(c, value)
    c.attend(sv)
    out, lse, av, mag, spread = clean.expected()
    got = c.out.double().cpu().numpy()
    last = c.row_off[1:] - 1
    keep = np.ones(c.rows, dtype=bool)
    keep[last] = False
    far = np.abs(got - out) - c.bound(out, av, mag, spread)
    assert (far[keep] <= 0).all()
    assert not np.isfinite(got[last]).all(-1).any()  # and the token that sees it is not finite


def test_attend_infinite_value_that_is_seen(sv):
    """An infinity of the values is seen by some rows only: those get it, the others do not."""
    c = Case(lens=[40], tokens=[6], H=1, G=2, D=64, q_scale=1.0)
    g, i = okv.slot_of(c.table[0], 36, c.bs)  # new token 2: rows 2.. see it
    c.v[0, g, i, 0, 5] = float("inf")
    c.attend(sv)
    got = c.out.float().cpu()
    assert torch.isinf(got[2:, :, 5]).all() and torch.isfinite(got[:2]).all()
    other = torch.ones(64, dtype=torch.bool)
    other[5] = False
    assert torch.isfinite(got[:, :, other]).all()


def test_attend_scores_of_minus_infinity(sv):
    """A position whose score is -inf weighs nothing; a token with nothing else gets zeros and lse -inf."""
    c = Case(lens=[1, 30], tokens=[1, 1], H=1, G=1, D=64)
    c.q.fill_(1.0)
    g, i = okv.slot_of(c.table[0], 0, c.bs)
    c.k[0, g, i] = -float("inf")
    g, i = okv.slot_of(c.table[1], 12, c.bs)
    c.k[0, g, i, 0, 0] = -float("inf")
    c.attend(sv)
    assert (c.out[0] == 0).all() and c.lse[0, 0] == -float("inf")
    assert torch.isfinite(c.out[1].float()).all() and torch.isfinite(c.lse[1]).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("big", [1e-3, 1e3])
def test_attend_large_and_small_queries(sv, dtype, big):
    """Queries of very different sizes in one call, elements far below their row's largest."""
    c = Case(lens=[200, 90], tokens=[4, 2], H=2, G=4, D=128, dtype=dtype)
    w = torch.exp(torch.randn((c.rows, 8, 1), generator=c.g) * 2) * big
    c.q = (c.q.float() * w).to(torch.bfloat16)
    c.q[:, :, ::3] *= 2.0**-12
    c.scale /= big
    c.attend(sv)
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [128, 256])
def test_attend_equal_tokens_strided_queries_and_no_lse(sv, dtype, D):
    """row_off None, q a slice of a fused projection, no lse, no statuses."""
    c = Case(lens=[33, 200, 3], tokens=[3, 3, 3], H=2, G=2, D=D, dtype=dtype)
    fused = torch.randn((9, 12, D)).to(torch.bfloat16)
    fused[:, :4] = c.q
    c.attend(sv, offsets=False, lse=False, status=False, q=fused.cuda()[:, :4])
    c.check()


@pytest.mark.parametrize("D", [128, 256])
def test_attend_statuses(sv, D):
    """Errors stay with their sequence: zeros for it, the others as they are."""
    par = [[-1, 0, 1, 1]] * 6
    par[3] = [-1, 0, 2, 1]  # node 2 its own parent
    par[4] = [0, 0, 1, 1]
    c = Case(lens=[40] * 6, tokens=[4] * 6, H=2, G=4, D=D, bs=4, parent=sum(par, []))
    good = Case(lens=[40] * 6, tokens=[4] * 6, H=2, G=4, D=D, bs=4, parent=[-1, 0, 1, 1] * 6)
    c.to_device(sv)
    c.dlens.copy_(torch.tensor([40, 3, 41, 40, 40, 40], dtype=torch.int32))
    c.dtable[5, 2] = c.held.shape[0]
    c.attend(sv)
    assert c.status.tolist() == [0, 2, 2, 4, 4, 4]
    assert (c.out[4:20] == 0).all() and (c.lse[4:20] == -float("inf")).all()
    out, lse, av, mag, spread = good.expected()
    got = c.out.double().cpu().numpy()
    assert (np.abs(got - out)[:4] <= good.bound(out, av, mag, spread)[:4]).all()
    assert torch.isfinite(c.out[20:].float()).all() and (c.out[20:] != 0).any()


@pytest.mark.parametrize("D", [128, 256])
def test_attend_bad_offsets_write_nothing(sv, D):
    c = Case(lens=[40] * 3, tokens=[4] * 3, H=1, G=1, D=D, bs=4)
    c.to_device(sv)
    c.doff.copy_(torch.tensor([0, 4, 2, 100], dtype=torch.int64))
    c.attend(sv)
    assert c.status.tolist() == [0, 4, 4]
    assert (c.out[4:] == 7).all() and (c.lse[4:] == 7).all()


def test_operators_on_another_stream(sv):
    """append, attend and gather queued on a stream of their own."""
    c = Case(lens=[33, 200], tokens=[5, 9], H=2, G=4, D=128, dtype="e4m3")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        status, want = _append(sv, c)
        c.attend(sv)
    s.synchronize()
    _same_cache(c, want)
    c.k, c.v = (torch.from_numpy(x) for x in want[:2])
    c.ks, c.vs = (torch.from_numpy(x) for x in want[2:])
    c.raw = lambda x: x.numpy()
    c.check()


def test_attend_in_a_graph(sv):
    """Captured once, replayed on changed inputs and lengths."""
    c = Case(lens=[33, 700], tokens=[5, 9], H=2, G=4, D=128)
    args = c.attend(sv)
    first = c.out.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.check(sv.spec_kv_attend(args), "spec_kv_attend")
    c.out.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, c.out)
    c.lens = [20, 699]
    c.dlens.copy_(torch.tensor(c.lens, dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    c.check()
