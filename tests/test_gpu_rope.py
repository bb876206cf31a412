"""Rotary positions on the GPU against the float64 oracle (oracle/kv.py): rows without a cache, and new keys on their way
into the cache with the queries beside them. The bounds are derived in tests/window_cases.py."""
import numpy as np
import pytest
import torch

from oracle import kv as okv
from tests.kv_cases import Case, random_tree, tree
from tests.window_cases import check_e4m3, rope_bound, rotary, rounding

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_38_gb300 as sv

    sv.build()
    return sv


def _near(got, x, pos, inv, dtype, adjacent=False, factor=1.0, **how):
    """got against the rotation of x, both tensors [rows, heads, D]; dtype: what got was rounded to (None: float32)."""
    half = len(inv)
    y = okv.rope(x.double().cpu().numpy(), pos, inv.cpu().numpy(), adjacent=adjacent, factor=factor, **how)
    off = rope_bound(x.double().cpu().numpy(), half, adjacent, factor) + rounding(y, dtype) + 2.0**-24 * np.abs(y)
    far = np.abs(got.double().cpu().numpy() - y) - off
    assert (far <= 0).all(), (float(far.max()), np.unravel_index(far.argmax(), far.shape))
    still = slice(2 * half, None)
    assert torch.equal(got[..., still].cpu(), x[..., still].cpu().to(got.dtype))


SHAPES = [  # rows, heads, D, half, adjacent
    (1, 1, 128, 64, False), (5, 3, 64, 32, False), (7, 32, 128, 64, True), (300, 5, 128, 16, False), (33, 2, 256, 128, False),
    (9, 7, 256, 128, True), (12, 4, 80, 16, True), (12, 4, 80, 20, False), (5, 3, 40, 20, True), (6, 1, 8, 1, False),
    (6, 2, 8, 4, True), (20, 3, 96, 24, False), (20, 3, 96, 48, False), (17, 3, 24, 11, True), (17, 3, 24, 11, False),
    (4097, 1, 64, 32, False),
]


@pytest.mark.parametrize("dtype,out_dtype", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("rows,heads,D,half,adjacent", SHAPES)
def test_rows(sv, dtype, out_dtype, rows, heads, D, half, adjacent):
    g = torch.Generator().manual_seed(rows + D)
    x = torch.randn((rows, heads, D), generator=g).to(dtype)
    pos = torch.randint(0, 100000, (rows,), generator=g).to(torch.int32)
    inv = rotary(half).cuda()
    out = torch.full((rows, heads, D), 7.0, dtype=out_dtype, device="cuda")
    sv.check(sv.spec_rope(sv.Rope(inv, adjacent=adjacent), x.cuda(), out, pos.cuda()), "spec_rope")
    _near(out, x, [pos.tolist()], inv, out_dtype if out_dtype == BF else None, adjacent)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,heads,D,half,adjacent", SHAPES)
def test_rows_in_place_are_the_same(sv, dtype, rows, heads, D, half, adjacent):
    """In place, and rows that lie apart as a slice of a fused projection: what lies between them stays."""
    x = torch.randn((rows, heads + 2, D), generator=torch.Generator().manual_seed(rows)).to(dtype).cuda()
    pos = torch.arange(rows, dtype=torch.int32, device="cuda") * 3
    rope = sv.Rope(rotary(half).cuda(), adjacent=adjacent, factor=0.75)
    before = x.clone()
    out = torch.empty((rows, heads, D), dtype=dtype, device="cuda")
    sv.check(sv.spec_rope(rope, x[:, 1:1 + heads], out, pos), "spec_rope")
    assert torch.equal(x, before)
    sv.check(sv.spec_rope(rope, x[:, 1:1 + heads], x[:, 1:1 + heads], pos), "spec_rope")
    assert torch.equal(x[:, 1:1 + heads], out)
    assert torch.equal(x[:, 0], before[:, 0]) and torch.equal(x[:, 1 + heads], before[:, 1 + heads])


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("D,half,sections,alternating", [
    (128, 64, (16, 24, 24), False), (128, 64, (22, 21, 21), True), (64, 32, (0, 32), False), (64, 32, (32, 0), False),
    (64, 32, (16, 16), True), (64, 32, (29, 0, 1, 2), True), (80, 20, (1, 2, 3, 14), False), (256, 128, (44, 42, 42), True),
    (256, 128, (1, 1, 125, 1), False), (40, 20, (8, 6, 6), True),
])
def test_axes(sv, adjacent, D, half, sections, alternating):
    g = torch.Generator().manual_seed(D)
    rows = 37
    x = torch.randn((rows, 3, D), generator=g)
    pos = torch.randint(0, 5000, (len(sections), rows), generator=g).to(torch.int32)
    inv = rotary(half).cuda()
    out = torch.empty_like(x, device="cuda")
    rope = sv.Rope(inv, adjacent=adjacent, sections=sections, alternating=alternating)
    sv.check(sv.spec_rope(rope, x.cuda(), out, pos.cuda()), "spec_rope")
    _near(out, x, pos.tolist(), inv, None, adjacent, sections=sections, alternating=alternating)


@pytest.mark.parametrize("position", [0, 1, -1, 65535, 2**20 + 1, -(2**24) - 1, 2**30, 2**31 - 1, -(2**31)])
def test_far_positions(sv, position):
    """An angle counts its whole turns exactly, whatever the position; frequencies from the fastest to 2^-60."""
    inv = torch.cat([rotary(32, 1e6), 2.0 ** -torch.arange(29).float() * 1.9, torch.tensor([2.0**-60, 0.0, 1e-45])]).cuda()
    x = torch.randn((3, 2, 128), generator=torch.Generator().manual_seed(1))
    out = torch.empty_like(x, device="cuda")
    pos = torch.full((3,), position, dtype=torch.int32)
    sv.check(sv.spec_rope(sv.Rope(inv), x.cuda(), out, pos.cuda()), "spec_rope")
    _near(out, x, [pos.tolist()], inv, None)


def test_unusual_frequencies(sv):
    """Negative ones turn back; larger than the limit or not finite: NaN in their pairs alone."""
    inv = rotary(32)
    inv[3], inv[7], inv[9], inv[12], inv[20] = -0.5, float("nan"), float("inf"), 2.0**21, 100.0
    x = torch.randn((5, 2, 64), generator=torch.Generator().manual_seed(2))
    out = torch.empty_like(x, device="cuda")
    pos = torch.arange(1, 6, dtype=torch.int32)
    sv.check(sv.spec_rope(sv.Rope(inv.cuda()), x.cuda(), out, pos.cuda()), "spec_rope")
    lost = [7, 9, 12, 39, 41, 44]
    assert out[..., lost].isnan().all()
    keep = [i for i in range(64) if i not in lost]
    known = inv.clone()
    known[[7, 9, 12]] = 0
    y = okv.rope(x.double().numpy(), [pos.tolist()], known.numpy())
    off = rope_bound(x.double().numpy(), 32, False, 1.0)
    assert (np.abs(out.double().cpu().numpy() - y) <= off)[..., keep].all()


def test_values_that_are_not_finite_stay_in_their_pair(sv):
    x = torch.randn((4, 3, 64), generator=torch.Generator().manual_seed(3))
    bad = x.clone()
    bad[1, 2, 5], bad[2, 0, 40] = float("nan"), float("inf")
    rope = sv.Rope(rotary(32).cuda())
    pos = torch.arange(4, dtype=torch.int32, device="cuda") + 9
    out = [torch.empty_like(x, device="cuda") for _ in range(2)]
    for o, y in zip(out, (x, bad)):
        sv.check(sv.spec_rope(rope, y.cuda(), o, pos), "spec_rope")
    touched = torch.zeros_like(x, dtype=torch.bool)
    touched[1, 2, [5, 37]] = touched[2, 0, [8, 40]] = True
    same = out[0] == out[1]
    assert same[~touched.cuda()].all() and not out[1][touched.cuda()].isfinite().any()


def test_a_row_read_many_times(sv):
    """A broadcast input (row stride 0) turned by each row's own position; one row alone in place, whatever its stride."""
    x = torch.randn((1, 3, 64), generator=torch.Generator().manual_seed(5)).to(BF).cuda()
    pos = torch.arange(70, dtype=torch.int32, device="cuda") * 11
    rope = sv.Rope(rotary(32).cuda())
    got, want = (torch.empty((70, 3, 64), dtype=BF, device="cuda") for _ in range(2))
    sv.check(sv.spec_rope(rope, x.expand(70, 3, 64), got, pos), "spec_rope")
    sv.check(sv.spec_rope(rope, x.repeat(70, 1, 1), want, pos), "spec_rope")
    assert torch.equal(got, want)
    y = x.expand(70, 3, 64)
    before = x.clone()
    assert sv.spec_rope(rope, y, y, pos) == sv.SPEC_ERR_INVALID_ARG
    assert torch.equal(x, before)
    one = y[:1]
    sv.check(sv.spec_rope(rope, one, one, pos[5:6]), "spec_rope")
    assert torch.equal(x[0], want[5])


@pytest.mark.parametrize("sections", [(2**32 + 16, 16), (-1, 33), (33, 0)])
def test_sections_that_no_head_has(sv, sections):
    with pytest.raises(ValueError):
        sv.Rope(rotary(32).cuda(), sections=sections)


def test_no_rows(sv):
    x = torch.zeros((0, 2, 64), dtype=BF, device="cuda")
    pos = torch.zeros(0, dtype=torch.int32, device="cuda")
    sv.check(sv.spec_rope(sv.Rope(rotary(32).cuda()), x, x, pos), "spec_rope")


# ------------------------------------------------------------------ into the cache
def _places(c, positions=None, axes=1):
    if positions is not None:
        return positions.reshape(axes, -1).tolist()
    out = []
    for b in range(c.B):
        lo, T = int(c.row_off[b]), c.tokens[b]
        d = np.arange(T) if c.parent is None else okv.depths(c.parent[lo:lo + T])
        out += (c.lens[b] - T + d).tolist()
    return [out] * axes


def _append(sv, c, *, half, new_dtype=BF, q_heads=4, adjacent=False, positions=None, in_place=False, offsets=True,
            how=None, factor=1.0, seed=5, stream=None):
    """Calls spec_kv_append_rope on the case and checks everything that it writes, and that the rest stays."""
    how = how or {}
    g = torch.Generator().manual_seed(seed)
    c.to_device(sv)
    k0, v0 = c.raw(c.dk), c.raw(c.dv)
    s0 = None if c.dks is None else (c.dks.cpu().numpy().copy(), c.dvs.cpu().numpy().copy())
    k, v = ((torch.randn((c.rows, c.H, c.D), generator=g) * torch.exp(torch.randn((c.rows, c.H, 1), generator=g) * 2))
            .to(new_dtype) for _ in range(2))
    q = torch.randn((c.rows, q_heads, c.D), generator=g).to(new_dtype) if q_heads else None
    dq = q.cuda() if q_heads else None
    q_out = dq if in_place else torch.full((c.rows, q_heads, c.D), 7.0, dtype=BF, device="cuda") if q_heads else None
    inv = rotary(half).cuda()
    rope = sv.Rope(inv, adjacent=adjacent, factor=factor, **how)
    status = torch.full((c.B,), -7, dtype=torch.int32, device="cuda")
    parent = None if c.parent is None else torch.from_numpy(c.parent).cuda()
    sv.check(sv.spec_kv_append_rope(c.cache, rope, k.cuda(), v.cuda(), c.dlens, row_off=c.doff if offsets else None, t_max=c.t_max,
                                    parent=parent, positions=None if positions is None else positions.cuda(), q=dq, q_out=q_out,
                                    layer=c.layer, seq_status=status, stream=stream), "spec_kv_append_rope")
    if stream is not None:
        stream.synchronize()
    assert status.tolist() == [0] * c.B
    pos = _places(c, positions, len(how["sections"]) if "sections" in how else 1)
    if q_heads:
        _near(q_out, q, pos, inv, BF, adjacent, factor, **how)
    x = k.double().numpy()
    y = okv.rope(x, pos, inv.cpu().numpy(), adjacent=adjacent, factor=factor, **how)
    off = rope_bound(x, half, adjacent, factor)
    k1, v1 = c.raw(c.dk), c.raw(c.dv)
    ks1, vs1 = (None, None) if s0 is None else (c.dks.cpu().numpy(), c.dvs.cpu().numpy())
    for b in range(c.B):
        for t in range(c.tokens[b]):
            r = c.row_off[b] + t
            p, i = okv.slot_of(c.table[b], c.lens[b] - c.tokens[b] + t, c.bs)
            if c.dtype == "bf16":
                assert (np.abs(k1[c.layer, p, i] - y[r]) <= off[r] + rounding(y[r], BF)).all()
                assert np.array_equal(v1[c.layer, p, i], v[r].to(BF).double().numpy())
            else:
                check_e4m3(k1[c.layer, p, i], ks1[c.layer, p, :, i], y[r], off[r])
                for h in range(c.H):
                    code, s = okv.quantise(v[r, h].double().numpy())
                    assert np.array_equal(v1[c.layer, p, i, h], code) and vs1[c.layer, p, h, i] == s
            for now, was in ((k1, k0), (v1, v0)):
                was[c.layer, p, i] = now[c.layer, p, i]
            if s0 is not None:
                s0[0][c.layer, p, :, i], s0[1][c.layer, p, :, i] = ks1[c.layer, p, :, i], vs1[c.layer, p, :, i]
    np.testing.assert_array_equal(k1, k0)  # the rest of the cache
    np.testing.assert_array_equal(v1, v0)
    if s0 is not None:
        np.testing.assert_array_equal(ks1, s0[0])
        np.testing.assert_array_equal(vs1, s0[1])


CACHES = [  # H, D, bs, order, pad, half, adjacent, q_heads
    (2, 64, 16, "nhd", 0, 32, False, 8), (3, 128, 5, "hnd", 16, 64, True, 3), (1, 96, 1, "nhd", 32, 24, False, 7),
    (8, 256, 32, "hnd", 0, 128, False, 8), (5, 16, 24, "nhd", 0, 8, True, 0), (2, 80, 16, "hnd", 0, 20, False, 2),
    (1, 48, 8, "nhd", 0, 11, True, 5),
]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("new_dtype", [BF, F32])
@pytest.mark.parametrize("H,D,bs,order,pad,half,adjacent,q_heads", CACHES)
def test_append_chain(sv, dtype, new_dtype, H, D, bs, order, pad, half, adjacent, q_heads):
    """Ragged new tokens, none at all, lengths equal to the new tokens'; one layer of two."""
    c = Case(lens=[9, 40, 1, 17, 3, 64], tokens=[9, 3, 1, 0, 3, 33], H=H, D=D, bs=bs, dtype=dtype, order=order, pad=pad,
             layers=2, layer=1)
    _append(sv, c, half=half, new_dtype=new_dtype, adjacent=adjacent, q_heads=q_heads)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,D,bs,order,pad,half,adjacent,q_heads", CACHES[:3])
def test_append_trees(sv, dtype, H, D, bs, order, pad, half, adjacent, q_heads):
    """A node's position is its depth's."""
    trees = [tree([4, 2, 2]), [-1], random_tree(40, 1), tree([64]), list(range(-1, 30))]
    c = Case(lens=[29, 300, 140, 65, 129], tokens=[len(t) for t in trees], H=H, D=D, bs=bs, dtype=dtype, order=order, pad=pad,
             parent=sum(trees, []))
    _append(sv, c, half=half, adjacent=adjacent, q_heads=q_heads)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("how", [{}, dict(sections=(8, 12, 12)), dict(sections=(12, 10, 10), alternating=True)])
def test_append_with_given_positions(sv, dtype, how):
    c = Case(lens=[19, 40, 1], tokens=[9, 3, 1], H=2, D=64, dtype=dtype)
    axes = len(how.get("sections", (1,)))
    pos = torch.randint(-5, 3000, (axes, c.rows), generator=torch.Generator().manual_seed(4)).to(torch.int32)
    _append(sv, c, half=32, positions=pos if axes > 1 else pos[0], how=how, factor=1.25)


def test_append_axes_without_positions_are_the_caches(sv):
    c = Case(lens=[19, 40, 1], tokens=[9, 3, 1], H=2, D=64)
    _append(sv, c, half=32, how=dict(sections=(8, 12, 12)))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("half", [32, 20])
def test_append_queries_in_place_and_equal_tokens(sv, dtype, half):
    c = Case(lens=[5, 77, 6], tokens=[5, 5, 5], H=2, D=64, dtype=dtype)
    _append(sv, c, half=half, in_place=True, offsets=False, q_heads=6)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_append_on_another_stream(sv, dtype):
    s = torch.cuda.Stream()
    c = Case(lens=[40, 9], tokens=[3, 9], H=2, D=64, dtype=dtype)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _append(sv, c, half=32, stream=s)


def _same_as_apart(sv, c, half, q_heads, new_dtype, **how):
    """The one call against spec_rope into float32 and spec_kv_append: the same bits everywhere."""
    g = torch.Generator(device="cuda").manual_seed(8)
    c.to_device(sv)
    k, v = (torch.randn((c.rows, c.H, c.D), generator=g, device="cuda").to(new_dtype) for _ in range(2))
    q = torch.randn((c.rows, q_heads, c.D), generator=g, device="cuda").to(new_dtype)
    rope = sv.Rope(rotary(half).cuda(), **how)
    pos = torch.tensor(_places(c)[0], dtype=torch.int32, device="cuda")
    turned, want_q = torch.empty(k.shape, device="cuda"), torch.empty(q.shape, dtype=BF, device="cuda")
    sv.check(sv.spec_rope(rope, k, turned, pos), "spec_rope")
    sv.check(sv.spec_rope(rope, q, want_q, pos), "spec_rope")
    kept = [None if t is None else t.clone() for t in (c.dk, c.dv, c.dks, c.dvs)]
    sv.check(sv.spec_kv_append(c.cache, turned, v.float(), c.dlens, c.doff, c.t_max, layer=c.layer), "spec_kv_append")
    want = [None if t is None else t.clone() for t in (c.dk, c.dv, c.dks, c.dvs)]
    for t, old in zip((c.dk, c.dv, c.dks, c.dvs), kept):
        if t is not None:
            t.copy_(old)
    q_out = torch.empty_like(want_q)
    parent = None if c.parent is None else torch.from_numpy(c.parent).cuda()
    sv.check(sv.spec_kv_append_rope(c.cache, rope, k, v, c.dlens, row_off=c.doff, t_max=c.t_max, parent=parent, q=q, q_out=q_out,
                                    layer=c.layer), "spec_kv_append_rope")
    raw = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
    assert torch.equal(q_out, want_q)
    for got, w in zip((c.dk, c.dv, c.dks, c.dvs), want):
        assert got is None or torch.equal(raw(got), raw(w))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("new_dtype", [BF, F32])
@pytest.mark.parametrize("D,half,adjacent", [(128, 64, False), (64, 16, True), (96, 11, False)])
def test_append_of_prompts_is_rotate_then_append(sv, dtype, new_dtype, D, half, adjacent):
    """Many rows, so that a CTA takes several tokens, across sequences' ends and over empty ones."""
    tokens = [0, 700, 1, 0, 0, 2049, 3, 1500, 0, 4000, 9000, 0, 777, 0]
    c = Case(lens=[t + (13 * b if t else 0) for b, t in enumerate(tokens)], tokens=tokens, H=2, D=D, bs=16, dtype=dtype)
    _same_as_apart(sv, c, half, 5, new_dtype, adjacent=adjacent)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("B", [33, 300, 2100])
def test_append_of_many_sequences(sv, dtype, B):
    r = np.random.default_rng(B)
    trees = [random_tree(int(r.integers(1, 12)), b) if b % 5 else [] for b in range(B)]
    c = Case(lens=[len(t) + int(r.integers(0, 40)) for t in trees], tokens=[len(t) for t in trees], H=1, D=32, dtype=dtype,
             parent=sum(trees, []))
    _same_as_apart(sv, c, 16, 2, BF)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_append_statuses(sv, dtype):
    """What a sequence with an error may write: nothing; past a bad page, its queries; under a bad parent, nothing."""
    parent = sum(([-1, 0, 1, 1] for _ in range(8)), [])
    parent[4 * 5 + 2] = 2  # its own parent: token 2 of sequence 5
    parent[4 * 6] = 0      # a root that is none
    parent[4 * 7 + 1] = -1
    c = Case(lens=[20] * 8, tokens=[4] * 8, H=2, D=32, dtype=dtype, bs=4)
    c.to_device(sv)
    before = c.raw(c.dk), c.raw(c.dv)
    c.dlens.copy_(torch.tensor([20, 3, 21, 20, 20, 20, 20, 20], dtype=torch.int32))
    c.dtable[3, 4] = 10**6
    c.dtable[4, 4] = -1
    new = torch.randn((c.rows, 2, 32)).to(BF).cuda()
    q = torch.randn((c.rows, 2, 32)).to(BF).cuda()
    out = torch.full_like(q, 7.0)
    status = torch.full((8,), -7, dtype=torch.int32, device="cuda")
    rope = sv.Rope(rotary(16).cuda())
    sv.check(sv.spec_kv_append_rope(c.cache, rope, new, new, c.dlens, row_off=c.doff, t_max=4,
                                    parent=torch.tensor(parent, dtype=torch.int32).cuda(), q=q, q_out=out, seq_status=status), "append")
    assert status.tolist() == [0, 2, 2, 4, 4, 4, 4, 4]
    wrote = (out != 7).flatten(1).any(1).view(8, 4).tolist()
    assert wrote == [[True] * 4, [False] * 4, [False] * 4, [True] * 4, [True] * 4, [True, True, False, True], [False] * 4,
                     [True, False, False, False]]
    mine = np.zeros(c.held.shape, dtype=bool)
    for b, ts in ((0, range(4)), (5, (0, 1, 3)), (7, (0,))):
        for t in ts:
            mine[c.table[b, 4], t] = True
    for x, y in zip(before, (c.raw(c.dk), c.raw(c.dv))):
        np.testing.assert_array_equal(x[:, ~mine], y[:, ~mine])
        assert not (x[:, mine] == y[:, mine]).all((2, 3)).any()
    bad = c.doff.clone()
    bad[2], bad[8] = 3, 10**9  # falls; past the rows
    c.dlens.fill_(20)
    out.fill_(7.0)
    sv.check(sv.spec_kv_append_rope(c.cache, rope, new, new, c.dlens, row_off=bad, t_max=4, q=q, q_out=out, seq_status=status), "append")
    assert status.tolist()[1] == 4 and status.tolist()[7] == 4
    assert (out[28:] == 7).all()


def test_append_leaves_rows_behind_the_last_sequence(sv):
    c = Case(lens=[20, 9], tokens=[4, 2], H=2, D=32)
    c.to_device(sv)
    new = torch.randn((30, 2, 32)).to(BF).cuda()
    out = torch.full_like(new, 7.0)
    before = c.raw(c.dk)
    sv.check(sv.spec_kv_append_rope(c.cache, sv.Rope(rotary(16).cuda()), new, new, c.dlens, row_off=c.doff, t_max=4, q=new, q_out=out),
             "append")
    assert (out[6:] == 7).all() and not (out[:6] == 7).any()
    after = c.raw(c.dk)
    assert ((after != before) & ~(np.isnan(after) & np.isnan(before))).any((0, 3, 4)).sum() == 6


def test_append_captured_and_replayed(sv):
    """A graph of the call follows lengths that change between its replays."""
    c = Case(lens=[40, 9], tokens=[3, 2], H=2, D=64)
    c.to_device(sv)
    rope = sv.Rope(rotary(32).cuda())
    k, q = (torch.randn((5, h, 64), generator=torch.Generator().manual_seed(h)).to(BF).cuda() for h in (2, 6))
    out = torch.empty_like(q)
    call = lambda: sv.check(sv.spec_kv_append_rope(c.cache, rope, k, k, c.dlens, row_off=c.doff, t_max=3, q=q, q_out=out), "append")  # noqa: E731
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([40, 9], [30, 2], [5, 7]):
        c.dlens.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(7.0)
        graph.replay()
        c.lens = lens
        _near(out, q.cpu(), _places(c), rope.inv_freq, BF)
