"""Attention with a sliding window and sinks on the GPU against the float64 oracle (oracle/kv.py); the bounds are derived
in tests/kv_cases.py. In every case here what no token sees is NaN, and the table's entries of pages that no token sees
lie far outside the pool."""
import numpy as np
import pytest
import torch

from oracle import kv as okv
from tests.kv_cases import random_tree, tree
from tests.window_cases import WindowCase

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_38_gb300 as sv

    sv.build()
    return sv


SHAPES = [  # H, G, D, bs, order, pad
    (2, 4, 128, 16, "nhd", 0),
    (1, 1, 64, 16, "hnd", 0),
    (3, 5, 128, 5, "nhd", 16),
    (2, 8, 64, 1, "hnd", 32),
    (1, 7, 96, 24, "nhd", 0),
    (2, 2, 16, 128, "hnd", 0),
    (1, 3, 256, 32, "nhd", 0),
]
WINDOWS = [(1, 0), (1, 1), (7, 3), (16, 16), (100, 4), (128, 0), (129, 130), (1000, 17), (2**31 - 1, 2**31 - 1)]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("H,G,D,bs,order,pad", SHAPES)
def test_one_token(sv, dtype, window, sinks, H, G, D, bs, order, pad):
    c = WindowCase(lens=[1, 2, 16, 17, 127, 128, 129, 0, 300, 1025], tokens=[1, 1, 1, 1, 1, 1, 1, 0, 1, 1], H=H, G=G, D=D,
                   bs=bs, dtype=dtype, order=order, pad=pad, layers=2, layer=1, q_scale=2.0, window=window, sinks=sinks)
    c.attend(sv)
    assert c.status.tolist() == [0] * c.B
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("H,G,D,bs,order,pad", SHAPES)
def test_chain(sv, dtype, window, sinks, H, G, D, bs, order, pad):
    """Ragged chains: windows shorter than the chain, that end inside it, within a tile, past the start."""
    c = WindowCase(lens=[9, 140, 128, 3, 260, 640, 128], tokens=[9, 17, 5, 3, 65, 1, 128], H=H, G=G, D=D, bs=bs, dtype=dtype,
                   order=order, pad=pad, q_scale=2.0, window=window, sinks=sinks)
    c.attend(sv)
    assert c.status.tolist() == [0] * c.B
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (3, 0), (20, 5), (40, 0), (130, 4), (5000, 3)])
@pytest.mark.parametrize("H,G,D,bs,order,pad", SHAPES[:5] + SHAPES[6:])
def test_tree(sv, dtype, window, sinks, H, G, D, bs, order, pad):
    """Windows by depth, down to a token's own position; sinks that reach into the tree."""
    trees = [tree([4, 2, 2]), [-1], random_tree(40, 1), random_tree(128, 2), tree([64]), list(range(-1, 30))]
    c = WindowCase(lens=[29, 300, 140, 200, 65, 129], tokens=[len(t) for t in trees], H=H, G=G, D=D, bs=bs, dtype=dtype,
                   order=order, pad=pad, parent=sum(trees, []), q_scale=2.0, window=window, sinks=sinks)
    c.attend(sv)
    assert c.status.tolist() == [0] * c.B
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("G,D,t", [(1, 64, 1), (4, 128, 1), (4, 128, 5), (4, 64, 9), (8, 128, 9), (4, 128, 29), (8, 128, 17)])
def test_many_tiles_to_a_processor(sv, dtype, G, D, t):
    """More tiles than 152 processors take at once, every size of row tile; half the batch as trees."""
    lens = [int(x) for x in np.random.default_rng(3).integers(t, 1800, 14)]
    tokens = [max(1, t - b % 3) for b in range(14)]
    for parent in (None, sum((random_tree(n, b) for b, n in enumerate(tokens)), [])):
        c = WindowCase(lens=lens, tokens=tokens, H=8, G=G, D=D, dtype=dtype, q_scale=2.0, window=900, sinks=5, parent=parent)
        c.attend(sv)
        assert c.status.tolist() == [0] * c.B
        c.check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("G,D,t", [(1, 128, 1), (2, 64, 9), (4, 128, 9), (8, 128, 9), (4, 128, 29)])
def test_many_short_sequences(sv, dtype, G, D, t):
    B = 300
    tokens = [0 if b % 7 == 3 else 1 + (b * 5) % t for b in range(B)]
    lens = [max(tokens[b], (b * 37) % 150) for b in range(B)]
    c = WindowCase(lens=lens, tokens=tokens, H=4, G=G, D=D, dtype=dtype, q_scale=2.0, window=33, sinks=2)
    c.attend(sv)
    assert c.status.tolist() == [0] * c.B
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("G,D,t", [(4, 128, 4), (8, 64, 4), (3, 96, 15), (5, 128, 16), (4, 128, 32), (2, 64, 64)])
def test_one_entry_over_many_processors(sv, dtype, G, D, t):
    """Every size of row tile with a window in 40 parts; the same call twice gives the same bits."""
    c = WindowCase(lens=[9003, 390], tokens=[t, t], H=1, G=G, D=D, dtype=dtype, q_scale=2.0, window=5003, sinks=20)
    c.attend(sv)
    assert c.status.tolist() == [0, 0]
    c.check()
    first = c.out.clone()
    for _ in range(3):
        c.attend(sv)
        assert torch.equal(first, c.out)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("as_tree", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_window_past_every_length_is_none(sv, dtype, as_tree, D):
    tokens = [9, 17, 1, 40]
    parent = sum((random_tree(n, b) for b, n in enumerate(tokens)), []) if as_tree else None
    kw = dict(lens=[9, 700, 300, 1500], tokens=tokens, H=2, G=2, D=D, dtype=dtype, parent=parent, q_scale=2.0, hide=False)
    plain, c = (WindowCase(window=1500, sinks=n, **kw) for n in (0, 0))
    c.attend(sv)
    c.check()
    args = c.args
    again = torch.empty_like(c.out)
    args.struct.out = again.data_ptr()
    sv.check(sv.spec_kv_attend(args), "spec_kv_attend")
    out, lse, av, mag, spread = plain.expected()
    c.check(again)
    assert (np.abs((again.double() - c.out.double()).cpu().numpy()) <= 2 * c.bound(out, av, mag, spread)).all()


def _parted(c, b):
    """Positions that some tokens of sequence b see and others do not."""
    see = c.seen(b)
    return np.flatnonzero(see.any(0) & ~see.all(0))


@pytest.mark.parametrize("dtype,value", [("bf16", float("nan")), ("bf16", float("inf")), ("bf16", -float("inf")),
                                         ("e4m3", float("nan"))])
@pytest.mark.parametrize("window,sinks", [(3, 0), (40, 4), (130, 0), (300, 20)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("as_tree", [False, True])
def test_values_that_only_some_rows_see(sv, dtype, value, window, sinks, D, as_tree):
    """A NaN or an infinity at the window's end, or in a new token, reaches the rows that see it and no other."""
    tokens = [5, 4, 2, 9, 33]
    parent = sum((random_tree(n, 7 + b) for b, n in enumerate(tokens)), []) if as_tree else None
    make = lambda: WindowCase(lens=[5, 130, 257, 300, 700], tokens=tokens, H=2, G=4, D=D, dtype=dtype, parent=parent,  # noqa: E731
                              q_scale=2.0, window=window, sinks=sinks)
    for pick in (0, -1):
        clean, c = make(), make()
        hit = np.zeros(c.rows, dtype=bool)
        for b in range(c.B):
            p = _parted(c, b)
            if len(p):
                c.fill(b, p[pick], value)
                hit[c.row_off[b]:c.row_off[b + 1]] |= c.seen(b)[:, p[pick]]
        c.attend(sv)
        out, lse, av, mag, spread = clean.expected()
        got = c.out.double().cpu().numpy()
        assert hit.any() and (~hit).any()
        assert (np.abs(got - out) <= clean.bound(out, av, mag, spread))[~hit].all()
        if value != value:
            assert np.isnan(got[hit]).all()
        # the values alone, their keys as they were: weighted sums of theirs
        c = make()
        for b in range(c.B):
            p = _parted(c, b)
            if len(p):
                c.fill(b, p[pick], value, "v")
        c.attend(sv)
        got = c.out.double().cpu().numpy()
        assert (np.abs(got - out) <= clean.bound(out, av, mag, spread))[~hit].all()
        assert not np.isfinite(got[hit]).any()


@pytest.mark.parametrize("value", [2.0**20, 2.0**40, 2.0**100, float("inf"), float("nan")])
@pytest.mark.parametrize("as_tree", [False, True])
@pytest.mark.parametrize("H,G,D,t", [(2, 1, 64, 5), (1, 4, 128, 8), (2, 4, 128, 9), (1, 8, 64, 9), (1, 4, 128, 29), (1, 2, 256, 4)])
def test_value_scales_that_only_some_rows_see(sv, value, as_tree, H, G, D, t):
    """The e4m3 scale of a position at the window's end leaves no trace in the rows past it, tiles that every row sees
    before and after it."""
    parent = sum((random_tree(t, b) for b in range(3)), []) if as_tree else None
    make = lambda: WindowCase(lens=[600, 1300, 250], tokens=[t] * 3, H=H, G=G, D=D, dtype="e4m3", parent=parent, q_scale=2.0,  # noqa: E731
                              window=200, sinks=140)
    clean, c = make(), make()
    hit = np.zeros(c.rows, dtype=bool)
    for b in range(c.B):
        p = _parted(c, b)[0]
        g, i = c.pages_of[b, p // c.bs], p % c.bs
        c.vs[c.layer, g, :, i] = value
        hit[c.row_off[b]:c.row_off[b + 1]] |= c.seen(b)[:, p]
    c.attend(sv)
    out, lse, av, mag, spread = clean.expected()
    got = c.out.double().cpu().numpy()
    assert hit.any() and (~hit).any()
    assert (np.abs(got - out) <= clean.bound(out, av, mag, spread))[~hit].all()
    if np.isfinite(value) and value < 2.0**60:
        out, lse, av, mag, spread = c.expected()
        assert (np.abs(got - out) <= c.bound(out, av, mag, spread)).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_scores_of_minus_infinity(sv, dtype):
    """Rows whose every score is -inf: zeros and lse -inf, beside rows that see more."""
    c = WindowCase(lens=[200], tokens=[3], H=1, G=2, D=64, dtype=dtype, window=2, sinks=0)
    c.q.fill_(1.0)
    for j in (197, 198):  # what rows 0 and 1 see of the window; row 1 and 2 see 198, row 2 sees 199
        if dtype == "bf16":
            c.fill(0, j, -float("inf"), "k")
        else:
            g, i = okv.slot_of(c.pages_of[0], j, c.bs)
            c.ks[0, g, :, i] = float("inf")
            c.k[0, g, i] = 0x80 | 0x38
    g, i = okv.slot_of(c.pages_of[0], 196, c.bs)
    c.k[0, g, i] = c.k[0, c.pages_of[0, 197 // 16], 197 % 16]
    if dtype == "e4m3":
        c.ks[0, g, :, i] = float("inf")
    c.attend(sv)
    assert (c.out[:2] == 0).all() and (c.lse[:2] == -float("inf")).all()
    g, i = okv.slot_of(c.pages_of[0], 199, c.bs)
    want = c.v[0, g, i, 0].double() if dtype == "bf16" else torch.from_numpy(
        okv.E4M3[c.v[0, g, i, 0].numpy()] * float(c.vs[0, g, 0, i]))
    assert torch.allclose(c.out[2].double().cpu(), want.expand(2, -1), rtol=2.0**-8, atol=0)


@pytest.mark.parametrize("D", [64, 256])
def test_statuses(sv, D):
    """Errors of length and offsets, a page outside the pool that is seen (its positions are left out), and ones that are
    not seen (no error)."""
    c = WindowCase(lens=[200] * 6, tokens=[4] * 6, H=2, G=2, D=D, window=40, sinks=20, dtype="bf16", seed=3)
    c.to_device(sv)
    c.dlens[1] = 3
    c.dlens[2] = 10**6
    c.dtable[3, 0] = 10**8      # the sinks'
    c.dtable[4, 12] = -1        # the new tokens'
    c.attend(sv)
    assert c.status.tolist() == [0, 2, 2, 4, 4, 0]
    out, lse, av, mag, spread = c.expected()
    ok = np.zeros(c.rows, dtype=bool)
    ok[:4] = ok[20:] = True
    got = c.out.double().cpu().numpy()
    assert (np.abs(got - out) <= c.bound(out, av, mag, spread))[ok].all()
    assert (got[4:12] == 0).all() and (c.lse[4:12] == -float("inf")).all()
    # without the sinks' first page: what is left of them, and the window
    left = okv.sight(4, 200, None, 40, 20)
    left[:, :16] = False
    k, v, ks, vs = c.host()
    for t in range(4):
        for h in range(4):
            kk, vv = (okv.entries(p, None, c.pages_of[3], 0, h // 2, 200, left[t])[left[t]] for p in (k, v))
            s = c.scale * kk @ c.q[12 + t, h].double().numpy()
            w = np.exp(s - s.max())
            assert np.abs(got[12 + t, h] - w @ vv / w.sum()).max() <= 2.0**-7 * np.abs(vv).max()


def test_bad_parent(sv):
    trees = [tree([2, 2]), [-1, 0, 2, 1], [0, 0]]
    c = WindowCase(lens=[100, 100, 100], tokens=[7, 4, 2], H=2, G=4, D=64, window=30, sinks=4, hide=False)
    c.parent = np.asarray(sum(trees, []), np.int32)
    c.attend(sv)
    assert c.status.tolist() == [0, 4, 4]
    assert (c.out[7:] == 0).all() and (c.lse[7:] == -float("inf")).all() and not (c.out[:7] == 0).all((1, 2)).any()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("as_tree", [False, True])
def test_captured_and_replayed(sv, dtype, as_tree):
    """A graph of the call follows lengths that change between its replays."""
    t = 9
    parent = random_tree(t, 1) + random_tree(t, 2) if as_tree else None
    lens = [[700, 300], [40, 9], [699, 131]]
    c = WindowCase(lens=lens[0], tokens=[t, t], H=2, G=4, D=64, dtype=dtype, window=60, sinks=4, hide=False, parent=parent)
    c.attend(sv)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.check(sv.spec_kv_attend_window(c.args, 60, 4), "spec_kv_attend_window")
    for n in lens:
        c.lens = n
        c.dlens.copy_(torch.tensor(n, dtype=torch.int32))
        c.out.fill_(7.0)
        graph.replay()
        c.check()


def test_one_workspace_serves_windows_and_none(sv):
    """Calls in turn, with and without a window, on one workspace; row tiles of every size."""
    for t in (1, 5, 9, 17, 29):
        c = WindowCase(lens=[500, 900], tokens=[t, t], H=2, G=4, D=128, window=100, sinks=4, hide=False, q_scale=2.0)
        c.attend(sv)
        first = c.out.clone()
        for _ in range(2):
            sv.check(sv.spec_kv_attend(c.args), "spec_kv_attend")
            sv.check(sv.spec_kv_attend_window(c.args, 100, 4), "spec_kv_attend_window")
        assert torch.equal(first, c.out)
        c.check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,G,D", [(641, 2, 64), (1300, 4, 128)])
def test_many_sequences(sv, dtype, B, G, D):
    r = np.random.default_rng(B)
    tokens = [int(x) for x in r.integers(0, 6, B)]
    lens = [t + int(x) if t else 0 for t, x in zip(tokens, r.integers(0, 200, B))]
    c = WindowCase(lens=lens, tokens=tokens, H=1, G=G, D=D, dtype=dtype, window=50, sinks=3, q_scale=2.0)
    c.attend(sv)
    assert c.status.tolist() == [0] * B
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 256])
def test_batch_without_new_tokens(sv, dtype, D):
    c = WindowCase(lens=[30, 0, 7], tokens=[0, 0, 0], H=2, G=2, D=D, dtype=dtype, window=5, sinks=1)
    c.attend(sv)
    assert c.status.tolist() == [0, 0, 0]


# ------------------------------------------------------------------ up to 16 rows to a key-value head
FEW = [  # G, t, D, bs, order
    (1, 16, 128, 16, "nhd"), (2, 8, 64, 16, "hnd"), (4, 4, 128, 5, "nhd"), (8, 2, 96, 16, "nhd"), (3, 5, 128, 24, "hnd"),
    (16, 1, 64, 1, "nhd"), (1, 9, 32, 128, "hnd"), (2, 4, 128, 16, "hnd"), (1, 8, 16, 16, "nhd"),
]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("as_tree", [False, True])
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (5, 7), (16, 16), (40, 3), (200, 0), (2**31 - 1, 5)])
@pytest.mark.parametrize("G,t,D,bs,order", FEW)
def test_few_rows(sv, dtype, as_tree, window, sinks, G, t, D, bs, order):
    """Ragged chains and trees of few rows: windows shorter than the tree is deep, sinks among the new tokens."""
    tokens = [t, max(1, t - 1), 1, t, 0, t]
    lens = [t, 33, 17, 400, 9, 131]
    parent = sum((random_tree(n, b) if n else [] for b, n in enumerate(tokens)), []) if as_tree else None
    c = WindowCase(lens=lens, tokens=tokens, H=2, G=G, D=D, bs=bs, dtype=dtype, order=order, parent=parent, q_scale=2.0,
                   window=window, sinks=sinks)
    c.attend(sv)
    assert c.status.tolist() == [0] * c.B
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,H", [(1, 1), (3, 2), (19, 8), (25, 8), (40, 8), (101, 8)])
@pytest.mark.parametrize("G,t,D", [(4, 1, 64), (4, 4, 64)])
def test_few_rows_of_many_entries(sv, dtype, B, H, G, t, D):
    """Entries in pieces, and by eight, four and two warps; more of them than fit at once. The same call twice: the same bits."""
    r = np.random.default_rng(B)
    tokens = [int(x) for x in r.integers(1, t + 1, B)]
    lens = [n + int(x) for n, x in zip(tokens, r.integers(0, 700, B))]
    c = WindowCase(lens=lens, tokens=tokens, H=H, G=G, D=D, dtype=dtype, window=500, sinks=9, q_scale=2.0)
    c.attend(sv)
    assert c.status.tolist() == [0] * B
    c.check()
    first = c.out.clone()
    for _ in range(3):
        c.attend(sv)
        assert torch.equal(first, c.out)


@pytest.mark.parametrize("dtype,value", [("bf16", float("nan")), ("bf16", float("inf")), ("bf16", -float("inf")),
                                         ("e4m3", float("nan"))])
@pytest.mark.parametrize("window,sinks", [(3, 0), (12, 4), (130, 0)])
@pytest.mark.parametrize("G,t,D", [(1, 16, 128), (4, 4, 64), (2, 4, 96)])
@pytest.mark.parametrize("as_tree", [False, True])
def test_values_that_only_some_of_few_rows_see(sv, dtype, value, window, sinks, G, t, D, as_tree):
    lens = [t, 130, 257, 500]
    parent = sum((random_tree(t, 7 + b) for b in range(4)), []) if as_tree else None
    make = lambda: WindowCase(lens=lens, tokens=[t] * 4, H=2, G=G, D=D, dtype=dtype, parent=parent, q_scale=2.0,  # noqa: E731
                              window=window, sinks=sinks)
    clean = make()
    out, lse, av, mag, spread = clean.expected()
    for what in ("kv", "v"):
        c = make()
        hit = np.zeros(c.rows, dtype=bool)
        for b in range(c.B):
            p = _parted(c, b)
            for at in ((p[0], p[-1]) if len(p) else ()):
                c.fill(b, at, value, what)
                hit[c.row_off[b]:c.row_off[b + 1]] |= c.seen(b)[:, at]
        c.attend(sv)
        got = c.out.double().cpu().numpy()
        assert hit.any() and (~hit).any()
        assert (np.abs(got - out) <= clean.bound(out, av, mag, spread))[~hit].all()
        if what == "v" or value != value:
            assert not np.isfinite(got[hit]).any()


@pytest.mark.parametrize("value", [2.0**20, 2.0**100, float("inf"), float("nan")])
@pytest.mark.parametrize("as_tree", [False, True])
@pytest.mark.parametrize("G,t,D", [(1, 16, 128), (4, 4, 64), (2, 4, 128)])
def test_value_scales_that_only_some_of_few_rows_see(sv, value, as_tree, G, t, D):
    parent = sum((random_tree(t, b) for b in range(3)), []) if as_tree else None
    make = lambda: WindowCase(lens=[600, 1300, 250], tokens=[t] * 3, H=2, G=G, D=D, dtype="e4m3", parent=parent, q_scale=2.0,  # noqa: E731
                              window=200, sinks=140)
    clean, c = make(), make()
    hit = np.zeros(c.rows, dtype=bool)
    for b in range(c.B):
        p = _parted(c, b)[0]
        g, i = c.pages_of[b, p // c.bs], p % c.bs
        c.vs[c.layer, g, :, i] = value
        hit[c.row_off[b]:c.row_off[b + 1]] |= c.seen(b)[:, p]
    c.attend(sv)
    out, lse, av, mag, spread = clean.expected()
    got = c.out.double().cpu().numpy()
    assert hit.any() and (~hit).any()
    assert (np.abs(got - out) <= clean.bound(out, av, mag, spread))[~hit].all()
    if value == 2.0**20:
        out, lse, av, mag, spread = c.expected()
        assert (np.abs(got - out) <= c.bound(out, av, mag, spread)).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("power", [10, 33, 60, 110])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("G,t,D", [(8, 1, 64), (4, 4, 128), (8, 9, 64)])
def test_scores_far_from_zero(sv, dtype, power, sign, G, t, D):
    """All scores about sign * 2^power: equal keys, so that the weights are equal and a row's output is a mean of values."""
    c = WindowCase(lens=[300, 40], tokens=[t, t], H=1, G=G, D=D, dtype=dtype, window=100, sinks=5)
    half = power // 2
    for b in range(2):
        for j in range(c.lens[b]):
            g, i = c.pages_of[b, j // c.bs], j % c.bs
            if not c.seen(b)[:, j].any():
                continue
            if dtype == "bf16":
                c.k[0, g, i, 0] = sign * 2.0**(power - half)
            else:
                c.k[0, g, i, 0] = 0x38 | (0x80 if sign < 0 else 0)
                c.ks[0, g, 0, i] = 2.0**(power - half)
    c.q.fill_(2.0**half)
    c.attend(sv)
    k, v, ks, vs = c.host()
    got = c.out.double().cpu().numpy()
    for b in range(2):
        see = c.seen(b)
        vv = okv.entries(v, vs, c.table[b], 0, 0, c.lens[b], see.any(0))
        for u in range(t):
            want, mean = vv[see[u]].mean(0), np.abs(vv[see[u]]).mean(0)
            row = got[c.row_off[b] + u]
            assert (np.abs(row - want) <= 2.0**-8 * np.abs(want) + 2.0**-10 * mean).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("G,t", [(4, 3), (4, 9)])
def test_query_that_is_not_finite(sv, dtype, value, G, t):
    """Its own row is NaN, and no other."""
    make = lambda: WindowCase(lens=[150, 40], tokens=[t, 2], H=2, G=G, D=128, dtype=dtype, q_scale=2.0, window=60, sinks=2)  # noqa: E731
    clean, c = make(), make()
    c.q[1, 5, 77] = value
    c.attend(sv)
    out, lse, av, mag, spread = clean.expected()
    got = c.out.double().cpu().numpy()
    keep = np.ones(got.shape[:2], dtype=bool)
    keep[1, 5] = False
    assert np.isnan(got[1, 5]).all()
    assert (np.abs(got - out) <= clean.bound(out, av, mag, spread))[keep].all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("G,t", [(2, 1), (4, 4), (4, 9)])
def test_growing_scores(sv, dtype, G, t):
    """Scores that rise along the window (every run a new maximum), then fall."""
    for sign in (1, -1):
        c = WindowCase(lens=[1500], tokens=[t], H=1, G=G, D=64, dtype=dtype, window=1200, sinks=30)
        ramp = torch.linspace(0.1, 4.0, 1500)
        for j in range(1500):
            if not c.seen(0)[:, j].any():
                continue
            g, i = c.pages_of[0, j // c.bs], j % c.bs
            x = torch.full((64,), float(ramp[j] if sign > 0 else ramp[-1 - j]))
            c.k[0, g, i, 0].copy_(x.to(torch.bfloat16) if dtype == "bf16" else (x * 64).to(torch.float8_e4m3fn).view(torch.uint8))
            if dtype == "e4m3":
                c.ks[0, g, 0, i] = 2.0**-6
        c.q = torch.full_like(c.q, 2.0)
        c.attend(sv)
        c.check()


def test_layers_of_a_cache_by_one_argument_struct(sv):
    """set_layer between calls, strided queries, outputs without lse and statuses, on a stream of its own."""
    c = WindowCase(lens=[70, 300], tokens=[2, 2], H=2, G=2, D=64, layers=3, layer=2, window=50, sinks=2, hide=False)
    wide = torch.randn((c.rows, 8, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    c.q = wide[:, 2:6].cpu()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.attend(sv, lse=False, status=False, q=wide[:, 2:6], stream=s)
        c.args.set_layer(0)
        sv.check(sv.spec_kv_attend_window(c.args, 50, 2, stream=s), "window")
        c.args.set_layer(2)
        sv.check(sv.spec_kv_attend_window(c.args, 50, 2, stream=s), "window")
    s.synchronize()
    c.check()


@pytest.mark.parametrize("G", [2, 8])
def test_offsets_past_32_bits(sv, G):
    """Pages two gigabytes apart: rotating append and windowed attention as in a cache whose pages lie together."""
    H, D, bs, t = 2, 64, 16, 4
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([45], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    near = [torch.randn((1, 3, bs, H, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    far = []
    for x in near:
        room = torch.empty(2 * 2**30 + bs * H * D, dtype=torch.bfloat16, device="cuda")
        view = room.as_strided((1, 3, bs, H, D), (0, 2**30, H * D, D, 1))
        view.copy_(x)
        far.append(view)
    k, v = (torch.randn((t, H, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn((t, H * G, D), generator=g, device="cuda").to(torch.bfloat16)
    rope = sv.Rope(torch.logspace(0, -4, 32, device="cuda"))
    got = []
    for pools in (near, far):
        cache = sv.KVCache(*pools, table)
        turned, out = torch.empty_like(q), torch.empty_like(q)
        sv.check(sv.spec_kv_append_rope(cache, rope, k, v, lens, t_max=t, q=q, q_out=turned), "append")
        args = sv.AttendArgs(cache=cache, q=turned, out=out, kv_lens=lens, t_max=t, scale=0.125)
        args.set_workspace(sv.Workspace.for_attend(args))
        sv.check(sv.spec_kv_attend_window(args, 30, 3), "window")
        got.append((turned, out, pools[0].clone(), pools[1].clone()))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_a_workspace_without_a_window_may_be_smaller(sv):
    """spec_kv_attend's own need has not grown: the size function names what serves both calls."""
    c = WindowCase(lens=[300, 40], tokens=[2, 2], H=2, G=4, D=128, window=50, sinks=2, hide=False)
    c.attend(sv)
    need = sv.spec_kv_attend_workspace_size(c.args)
    c.args.struct.workspace_bytes = need - 256
    assert sv.spec_kv_attend_window(c.args, 50, 2) == sv.SPEC_ERR_WORKSPACE
    sv.check(sv.spec_kv_attend(c.args), "attend")
    torch.cuda.synchronize()
