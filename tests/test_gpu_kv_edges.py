"""The paged cache's operators where they could go wrong and the other GPU tests do not reach, against the float64 oracle
(oracle/kv.py); bounds from tests/kv_cases.py."""
import math

import numpy as np
import pytest
import torch

from oracle import kv as okv
from tests.kv_cases import Case, random_tree, tree  # noqa: F401
from tests.test_gpu_kv import _append, _same_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_38_gb300 as sv

    sv.build()
    return sv


# ------------------------------------------------------------------ compaction
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("in_place", [True, False])
def test_compact_lengths_in_place_with_more_ctas_than_are_resident(sv, dtype, in_place):
    """kv_lens_out is kv_lens_in: every CTA of a sequence has to take the old length. 256 trees of 7 nodes in 32 layers
    are 2,048 (bf16) CTAs and more, several waves of them."""
    B, N = 256, 7
    paths = [[6], [2, 6], [], [1, 3, 5], [4], [3, 4, 5, 6], [1, 2], [5, 6]]
    paths = [paths[b % 8] for b in range(B)]
    c = Case(lens=[N + (5 * b) % 11 for b in range(B)], tokens=[N] * B, H=4, D=64 if dtype == "bf16" else 112, bs=4,
             dtype=dtype, layers=32)
    c.to_device(sv)
    flat = np.full(c.rows, -1, np.int32)
    for b, p in enumerate(paths):
        flat[b * N:b * N + len(p)] = p
    acc = np.array([len(p) for p in paths], np.int32)
    lens = c.dlens.clone()
    out = lens if in_place else torch.full_like(lens, -7)
    blocks, status = (torch.full((B,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    sv.check(sv.spec_kv_compact(c.cache, c.doff, torch.from_numpy(flat).cuda(), torch.from_numpy(acc).cuda(), lens, out,
                                out_num_blocks=blocks, seq_status=status), "compact")
    k, v, ks, vs = c.host()
    want = okv.compact((k, v), (ks, vs), c.table, c.row_off, flat, acc, c.lens)
    assert status.tolist() == [0] * B
    assert out.tolist() == want.tolist() and blocks.tolist() == [-(-x // 4) for x in want.tolist()]
    _same_cache(c, (k, v, ks, vs))


def test_compact_in_place_keeps_the_length_of_a_bad_sequence(sv):
    """Statuses and lengths of the second launch: a path that does not rise, a length too short, a page outside the pool."""
    c = Case(lens=[20] * 5, tokens=[6] * 5, H=4, D=64, bs=4, layers=16)
    c.to_device(sv)
    before = c.raw(c.dk), c.raw(c.dv)
    path = torch.tensor([[2, 2], [2, 4], [2, 4], [1, 2], [2, 9]], dtype=torch.int32, device="cuda")
    path = torch.cat([path, torch.full((5, 4), -1, dtype=torch.int32, device="cuda")], 1).reshape(-1)
    acc = torch.full((5,), 2, dtype=torch.int32, device="cuda")
    lens = c.dlens.clone()
    lens[1] = 5
    c.dtable[2, 4] = 10**8
    status = torch.full((5,), -7, dtype=torch.int32, device="cuda")
    sv.check(sv.spec_kv_compact(c.cache, c.doff, path, acc, lens, lens, seq_status=status), "compact")
    assert status.tolist() == [4, 2, 4, 0, 4]
    assert lens.tolist() == [20, 5, 20, 17, 20]
    np.testing.assert_array_equal(before[0], c.raw(c.dk))
    np.testing.assert_array_equal(before[1], c.raw(c.dv))


# ------------------------------------------------------------------ attention: scales of what a row does not see
def _last_token_scale(c, value):
    """V's scale of each sequence's last new token, in every head."""
    for b in range(c.B):
        j = c.lens[b] - 1
        c.vs[c.layer, int(c.table[b, j // c.bs]), :, j % c.bs] = value


def _sees_last(c):
    """Rows whose token is a sequence's last: a chain's or a tree's last token is seen by itself alone."""
    return np.isin(np.arange(c.rows), c.row_off[1:] - 1)


@pytest.mark.parametrize("value", [2.0**20, 2.0**31, 2.0**40, 2.0**100, float("inf"), float("nan")])
@pytest.mark.parametrize("as_tree", [False, True])
@pytest.mark.parametrize("H,G,D,t", [(2, 1, 64, 5), (1, 4, 128, 8), (2, 4, 128, 9), (1, 8, 64, 9), (1, 4, 128, 29),
                                     (1, 2, 256, 6)])
def test_attend_unseen_value_scale(sv, value, as_tree, H, G, D, t):
    """A large or non-finite V scale leaves no trace in rows that do not see its token: at the front of a tile, inside
    one, alone in the last one, after many. Its own row has the entry's value, or is not finite; every lse stays right."""
    lens = [t, t + 3, 128 + t, 128 + t - 1, 129, 300, 1025, 2000]
    trees = [random_tree(t, 7 + b) for b in range(len(lens))]
    c = Case(lens=lens, tokens=[t] * len(lens), H=H, G=G, D=D, dtype="e4m3", q_scale=2.0,
             parent=sum(trees, []) if as_tree else None)
    _last_token_scale(c, value)
    c.attend(sv)
    assert c.status.tolist() == [0] * c.B
    with np.errstate(invalid="ignore"):
        out, lse, av, mag, spread = c.expected()
    got, mine = c.out.double().cpu().numpy(), _sees_last(c)
    if np.isfinite(value):
        c.check()
        return
    assert not np.isfinite(got[mine]).any()
    with np.errstate(invalid="ignore"):
        far = np.abs(got - out) - c.bound(out, av, mag, spread)
    assert np.isfinite(got[~mine]).all() and (far[~mine] <= 0).all(), np.nanmax(far[~mine])
    es = 2.0**-23 * (D + 8) * mag + 2.0**-20  # as in Case.check
    assert (np.abs(c.lse.double().cpu().numpy() - lse) <= es + 2.0**-21 * (1 + np.abs(lse)) + max(lens) * 2.0**-24).all()


@pytest.mark.parametrize("G,t", [(1, 4), (8, 9), (4, 32)])
def test_attend_value_scales_of_a_wide_range(sv, G, t):
    """Scales from 2^-60 to 2^60 all over the cache, new tokens among them: a row's unit goes by what it sees, tile after
    tile."""
    c = Case(lens=[t, 40 + t, 260, 1500, 3000], tokens=[t] * 5, H=2, G=G, D=128, dtype="e4m3", q_scale=2.0)
    c.vs[:] = torch.exp2(torch.randint(-60, 61, c.vs.shape, generator=c.g).float())
    c.attend(sv)
    assert c.status.tolist() == [0] * 5
    c.check()


@pytest.mark.parametrize("G,D,t", [(1, 64, 1), (4, 128, 9), (8, 128, 9), (4, 64, 29)])
def test_attend_weightless_token_with_a_large_scale(sv, G, D, t):
    """V scales of 2^-100 and, on new tokens whose weight is zero in float32, of 2^30: the product of a row's unit with
    the latter is not finite before the unit moves, and zero times it must stay zero. 160 (sequence, head) pairs, so
    that a processor comes to the new tokens' tile after others."""
    c = Case(lens=[t + 1, t + 40] + [900, 1025] * 19, tokens=[t] * 40, H=4, G=G, D=D, dtype="e4m3")
    c.vs[:] = 2.0**-100
    c.ks[:] = 1.0
    c.q = torch.ones_like(c.q)
    k = torch.zeros(c.held.shape)
    for b in range(c.B):
        for j in range(c.lens[b] - t, c.lens[b]):
            g, i = int(c.table[b, j // c.bs]), j % c.bs
            k[g, i] = -448.0  # a score of -448 sqrt(D)
            c.vs[0, g, :, i] = 2.0**30
    c.k.copy_(k[None, :, :, None, None].expand(c.k.shape).to(torch.float8_e4m3fn).view(torch.uint8))
    c.attend(sv)
    assert c.status.tolist() == [0] * 40
    c.check()


# ------------------------------------------------------------------ attention: scores far from zero
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("power", [10, 33, 60, 110, 112])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("G,D,t", [(8, 64, 1), (8, 64, 3), (8, 128, 5), (8, 64, 12), (8, 256, 3)])
def test_attend_scores_far_from_zero(sv, dtype, power, sign, G, D, t):
    """Equal scores of up to 2^117 either side of zero, and others twice as far below: a row is the mean of the values
    that share its largest score."""
    lens = [t, t + 1, 127 + t, 300, 1100]
    c = Case(lens=lens, tokens=[t] * len(lens), H=1, G=G, D=D, dtype=dtype)
    r = np.random.default_rng(3)
    half = 2.0 ** (power // 2 if dtype == "bf16" else 0)  # k's magnitude; the rest lies with q (e4m3: K's scales too)
    rest = 2.0**power / half / (1 if dtype == "bf16" else 2.0 ** (power // 2))
    far = torch.from_numpy(r.random(c.held.shape) < 0.3)  # positions whose score lies further down (page, slot)
    for b in range(c.B):
        far[int(c.table[b, 0]), 0] = False  # every token sees position 0
    k = torch.where(far, -2.0 if sign > 0 else 2.0, 1.0)[None, :, :, None, None].expand(c.k.shape) * half
    c.k.copy_(k.to(torch.bfloat16) if dtype == "bf16" else k.to(torch.float8_e4m3fn).view(torch.uint8))
    if dtype == "e4m3":
        c.ks[:] = 2.0 ** (power // 2)
    q = sign * rest * torch.from_numpy(1 + r.random((c.rows, G, 1))).expand(c.rows, G, D)
    c.q = q.to(torch.bfloat16)
    c.attend(sv)
    assert c.status.tolist() == [0] * c.B
    got, lse = c.out.double().cpu().numpy(), c.lse.double().cpu().numpy()
    _, v, _, vs = c.host()
    s = c.q.double().numpy().sum(-1) * c.scale * half * (1 if dtype == "bf16" else 2.0 ** (power // 2))
    for b in range(c.B):
        vv = okv.entries(v, vs, c.table[b], 0, 0, lens[b])
        near = np.array([not far[int(c.table[b, j // c.bs]), j % c.bs] for j in range(lens[b])])
        for i in range(t):
            seen = near & (np.arange(lens[b]) <= lens[b] - t + i)
            row = int(c.row_off[b]) + i
            want, mean = vv[seen].mean(0), np.abs(vv[seen]).mean(0)
            # an output's rounding, weights of 11 bits and more, float32 sums (tests/kv_cases.py)
            bound = 2.0**-8 * np.abs(want) + (2.0**-10 + lens[b] * 2.0**-23) * mean + 1e-30
            assert (np.abs(got[row] - want) <= bound).all(), (b, i, np.abs(got[row] - want).max())
            assert (np.abs(lse[row] - s[row] - np.log(seen.sum())) <= 2.0**-23 * (D + 8) * (np.abs(s[row]) + 10)).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("G,D,t", [(1, 64, 1), (2, 128, 9), (4, 128, 9), (8, 128, 9), (8, 64, 12), (2, 256, 3)])
def test_attend_large_values_under_rising_scores(sv, dtype, G, D, t):
    """Values of about 2^100 with scores that rise by up to 2^58 in the weights from one tile to a later one of the same
    processor (and team of its warps): the sums stay finite. 160 (sequence, head) pairs, so that one has several tiles."""
    c = Case(lens=[t, 300 + t] + [900, 1300] * 19, tokens=[t] * 40, H=4, G=G, D=D, dtype=dtype)
    rise = np.array([0, 12, 3, 1, 40, 50, 58, 30, 96, 70, 100, 60])  # log2 of the weights, by tile
    unit = math.log(2) / (c.scale * D) / (1.0 if dtype == "bf16" else 2.0**-3)
    k = torch.zeros(c.held.shape)
    for b in range(c.B):
        for j in range(c.lens[b]):
            k[int(c.table[b, j // c.bs]), j % c.bs] = float(rise[j // 128])
    k = (k * unit)[None, :, :, None, None].expand(c.k.shape)
    if dtype == "bf16":
        c.k.copy_(k.to(torch.bfloat16))
        c.v.mul_(2.0**100)
    else:
        c.k.copy_(k.to(torch.float8_e4m3fn).view(torch.uint8))
        c.ks[:] = 2.0**-3
        c.vs.mul_(2.0**98)
    c.q = torch.ones_like(c.q)
    c.attend(sv)
    assert c.status.tolist() == [0] * 40
    c.check()


# ------------------------------------------------------------------ large batches
def _lens(B, most, seed):
    """Lengths and new tokens of a batch, empty sequences among them."""
    r = np.random.default_rng(seed)
    tokens = r.integers(0, 6, B)
    tokens[r.random(B) < 0.3] = 0
    return (tokens + r.integers(0, most, B) * (r.random(B) < 0.8)).tolist(), tokens.tolist()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("B", [33, 300, 1100, 2100])
def test_append_and_gather_of_many_sequences(sv, dtype, B):
    """A row's sequence is found in steps of 32: one to three of them, sequences without rows between."""
    lens, tokens = _lens(B, 20, B)
    c = Case(lens=lens, tokens=tokens, H=2, D=32, bs=4, dtype=dtype)
    status, want = _append(sv, c)
    assert status.tolist() == [0] * B
    _same_cache(c, want)
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    got = [torch.full((int(off[-1]), 2, 32), 7.0, device="cuda") for _ in range(2)]
    status.fill_(-7)
    sv.check(sv.spec_kv_gather(c.cache, c.dlens, torch.from_numpy(off).cuda(), *got, seq_status=status), "gather")
    assert status.tolist() == [0] * B
    k, v, ks, vs = want
    for pool, sc, x in ((k, ks, got[0]), (v, vs, got[1])):
        x = x.cpu().numpy()
        for b in range(B):
            for h in range(2):
                e = okv.entries(pool, sc, c.table[b], 0, h, lens[b]).astype(np.float32)
                np.testing.assert_array_equal(x[off[b]:off[b + 1], h], e)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,G,D", [(641, 2, 64), (1300, 4, 128), (2700, 1, 64)])
@pytest.mark.parametrize("as_tree", [False, True])
def test_attend_many_sequences(sv, dtype, B, G, D, as_tree):
    """More sequences than a CTA has threads: each counts several. A bad one and empty ones among them."""
    lens, tokens = _lens(B, 200 if B < 1000 else 24, B + 1)
    lens[B // 2], tokens[B // 2] = 9, 4
    parent = sum((random_tree(t, b) for b, t in enumerate(tokens) if t), []) if as_tree else None
    c = Case(lens=lens, tokens=tokens, H=1, G=G, D=D, bs=8, dtype=dtype, parent=parent)
    c.attend(sv)
    assert c.status.tolist() == [0] * B
    c.check()
    c.dlens[B // 2] = 3  # shorter than its new tokens
    c.attend(sv)
    assert c.status.tolist() == [2 if b == B // 2 else 0 for b in range(B)]
    lo, hi = int(c.row_off[B // 2]), int(c.row_off[B // 2 + 1])
    assert (c.out[lo:hi] == 0).all() and torch.isneginf(c.lse[lo:hi]).all()
    keep = np.r_[0:lo, hi:c.rows]
    out, lse, av, mag, spread = c.expected()
    far = np.abs(c.out.double().cpu().numpy() - out) - c.bound(out, av, mag, spread)
    assert (far[keep] <= 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 256])
def test_batch_without_new_tokens(sv, dtype, D):
    """No rows at all: statuses only, nothing else touched."""
    c = Case(lens=[0, 5, 300], tokens=[0, 0, 0], H=2, G=2, D=D, dtype=dtype)
    c.attend(sv)
    assert c.status.tolist() == [0, 0, 0]
    before = c.raw(c.dk), c.raw(c.dv)
    new = torch.zeros((0, 2, D), dtype=torch.bfloat16, device="cuda")
    c.status.fill_(-7)
    sv.check(sv.spec_kv_append(c.cache, new, new, c.dlens, row_off=c.doff, seq_status=c.status), "append")
    assert c.status.tolist() == [0, 0, 0]
    np.testing.assert_array_equal(before[0], c.raw(c.dk))
    np.testing.assert_array_equal(before[1], c.raw(c.dv))


# ------------------------------------------------------------------ refusals
def test_types_are_refused_by_their_own_names(sv):
    c = Case(lens=[9], tokens=[3], H=2, D=32)
    c.to_device(sv)
    x = torch.zeros((3, 2, 32), dtype=torch.float16, device="cuda")
    with pytest.raises(TypeError, match="^k_new must be float32 or bfloat16"):
        sv.spec_kv_append(c.cache, x, x, c.dlens, row_off=c.doff)
    with pytest.raises(TypeError, match="^k_out must be float32 or bfloat16"):
        y = torch.zeros((9, 2, 32), dtype=torch.float16, device="cuda")
        sv.spec_kv_gather(c.cache, c.dlens, torch.tensor([0, 9], device="cuda"), y, y)
