"""Rotary positions and the sliding window without a GPU: the oracle against torch, the struct layouts, the rule by which
the tiles hold what is seen, and the host's refusals, which come before any CUDA call."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import kv as okv
from tests.kv_cases import random_tree, tree
from tests.test_abi import sv, test_struct_layout_matches_header as _layout  # noqa: F401
from tests.test_kv_host import CACHE_REFUSALS, FAKE, _attend, _cache
from tests.window_cases import WindowCase, rotary


@pytest.mark.parametrize("cname,pyname", [("spec_rope_t", "SpecRope"), ("spec_kv_append_rope_args_t", "SpecKvAppendRopeArgs")])
def test_struct_layout(sv, cname, pyname):  # noqa: F811
    _layout(sv, cname, pyname)


# ------------------------------------------------------------------ oracle
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("how", [{}, dict(sections=(6, 5, 5)), dict(sections=(6, 5, 5), alternating=True),
                                 dict(sections=(0, 16)), dict(factor=0.8)])
def test_oracle_rotation_matches_torch(adjacent, how):
    g = torch.Generator().manual_seed(1)
    x = torch.randn((7, 3, 40), generator=g, dtype=torch.float64)
    pos = torch.randint(-50, 40000, (3, 7), generator=g)
    inv = rotary(16)
    got = okv.rope(x.numpy(), pos.tolist(), inv.numpy(), adjacent=adjacent, **how)
    want = x.clone()
    for i in range(16):
        a = 0
        if "sections" in how:
            s = how["sections"]
            a = (i % 3 if i < 3 * s[i % 3] else 0) if how.get("alternating") else next(
                k for k in range(len(s)) if i < sum(s[:k + 1]))
        t = pos[a].double() * inv[i].double()
        p, q = (2 * i, 2 * i + 1) if adjacent else (i, i + 16)
        f = how.get("factor", 1.0)
        c, s_ = f * torch.cos(t)[:, None], f * torch.sin(t)[:, None]
        want[..., p], want[..., q] = x[..., p] * c - x[..., q] * s_, x[..., q] * c + x[..., p] * s_
    np.testing.assert_allclose(got, want.numpy(), rtol=0, atol=1e-10)
    assert np.array_equal(got[..., 32:], x[..., 32:].numpy())


def test_oracle_rotation_of_far_positions():
    """An angle of 2^31 - 1 radians, by its remainder in whole numbers."""
    got = okv.rope(np.array([[[1.0, 0.0]]]), [[2**31 - 1]], np.array([1.0], np.float32))
    assert abs(got[0, 0, 0] - math.cos(2**31 - 1)) < 1e-12 and abs(got[0, 0, 1] - math.sin(2**31 - 1)) < 1e-12


@pytest.mark.parametrize("parent", [None, tree([3, 2]), random_tree(10, 3), [-1]])
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (4, 3), (11, 0), (500, 30)])
def test_oracle_sight(parent, window, sinks):
    T = 10 if parent is None else len(parent)
    for L in (T, T + 1, T + 25):
        see = okv.sight(T, L, parent, window, sinks)
        for t in range(T):
            up, way = t, []
            while up >= 0:
                way.append(up)
                up = up - 1 if parent is None else parent[up]
            place = L - T + len(way) - 1
            for j in range(L):
                if j < L - T:
                    want = j < sinks or place - j < window
                else:
                    want = j - (L - T) in way and (j < sinks or way.index(j - (L - T)) < window)
                assert see[t, j] == want, (t, j)


# ------------------------------------------------------------------ the order in which tiles hold positions
def _sight(T, L, window, sinks, box):
    """The kernel's own rule (struct Sight): places s1, i1, offsets di, de, end, first position, first place that parts."""
    up = lambda x: -(-x // box) * box  # noqa: E731
    ctx = L - T
    lo = max(0, ctx + 1 - window)
    first = min(sinks, L)
    s1 = first // box * box if lo < up(first) else up(first)
    last, e0 = up(L), max(s1, lo // box * box)
    i0 = min(max(up(max(0, ctx + T - window)), e0), last)
    di, i1 = i0 - s1, last - (i0 - s1)
    return s1, i1, di, e0 - i1, i1 + i0 - e0, lo, ctx if ctx < s1 else s1 if ctx < i0 else ctx - di


@pytest.mark.parametrize("box", [1, 8, 16])
def test_places_hold_what_is_seen_once(box):
    r = np.random.default_rng(box)
    for _ in range(3000):
        T = int(r.integers(1, 129))
        L = T + int(r.integers(0, 600))
        window = int(r.integers(1, 700)) if r.random() < 0.8 else int(r.integers(1, 10))
        sinks = int(r.choice([0, 0, 1, 4, 16, 17, 100, 900]))
        s1, i1, di, de, end, lo, tail = _sight(T, L, window, sinks, box)
        place = np.arange(end)
        pos = np.where(place < s1, place, np.where(place < i1, place + di, place + de))
        assert 0 <= s1 <= i1 <= end and (pos >= 0).all() and len(set(pos.tolist())) == end
        assert (pos[::box] % box == 0).all() and end % box == 0  # whole boxes, as they lie
        see = okv.sight(T, L, None, window, sinks)
        seen = see.any(0)
        where = np.full(-(-L // box) * box, -1)
        where[pos] = place
        assert (where[:L][seen] >= 0).all()  # nothing seen is left out
        boxes = pos.reshape(-1, box)
        assert all(seen[b[b < L]].any() for b in boxes)  # and no box is loaded for nothing
        inside = pos < L
        assert np.array_equal(seen[pos[inside]], ((pos < sinks) | (pos >= lo))[inside])
        assert all(seen[p] for p in pos[s1:i1] if p < L)  # (a whole tile of these is not looked at position by position)
        # before `tail`, a position is seen by every row or by none
        for p in pos[:tail]:
            assert p >= L or see[:, p].all() or not see[:, p].any()


# ------------------------------------------------------------------ refusals
def _rope(sv, **kw):  # noqa: F811
    r = sv.SpecRope()
    r.struct_size = ctypes.sizeof(sv.SpecRope)
    r.rotary_dim, r.axes, r.factor, r.inv_freq = 64, 1, 1.0, FAKE
    for name, x in kw.items():
        if name == "sections":
            for i, n in enumerate(x):
                r.sections[i] = n
        else:
            setattr(r, name, x)
    return r


def _append(sv, **kw):  # noqa: F811
    a = sv.SpecKvAppendRopeArgs()
    a.struct_size = ctypes.sizeof(sv.SpecKvAppendRopeArgs)
    a.new_dtype, a.t_max, a.rows, a.q_heads = 1, 9, 36, 8
    a.row_off = a.kv_lens = a.k_new = a.v_new = a.q = FAKE
    a.q_out = FAKE + 4096
    a.new_token_stride, a.q_token_stride, a.q_out_token_stride = 128, 512, 512
    for name, x in kw.items():
        setattr(a, name, x)
    return a


ROPE_REFUSALS = [
    (dict(struct_size=8), 1), (dict(rotary_dim=0), 1), (dict(rotary_dim=-2), 1), (dict(rotary_dim=33), 1),
    (dict(rotary_dim=66), 1), (dict(adjacent=2), 1), (dict(adjacent=-1), 1), (dict(alternating=2), 1), (dict(axes=0), 1),
    (dict(axes=5), 1), (dict(factor=float("nan")), 1), (dict(factor=float("inf")), 1), (dict(factor=-float("inf")), 1),
    (dict(inv_freq=None), 1), (dict(inv_freq=FAKE + 2), 2), (dict(axes=3, sections=(10, 10, 10)), 1),
    (dict(axes=3, sections=(40, -4, -4)), 1), (dict(axes=2, sections=(33, 0)), 1),
    (dict(axes=3, sections=(10, 11, 11), alternating=1), 1), (dict(axes=2, sections=(0, 32), alternating=1), 1),
    (dict(axes=3, sections=(2**31 - 1, 2**31 - 1, 34)), 1),
]


@pytest.mark.parametrize("kw,status", ROPE_REFUSALS)
def test_rope_refusals(sv, kw, status):  # noqa: F811
    L, r = sv.lib(), _rope(sv, **kw)
    assert L.spec_rope(ctypes.byref(r), FAKE, 1, 128, FAKE, 1, 128, 36, 2, 64, FAKE, None) == status
    assert L.spec_kv_append_rope(ctypes.byref(_cache(sv)), ctypes.byref(r), ctypes.byref(_append(sv)), None) == status


@pytest.mark.parametrize("at,value,status", [
    (0, None, 1), (1, None, 1), (2, 2, 1), (2, -1, 1), (3, -128, 1), (4, None, 1), (5, 3, 1), (6, -8, 1), (7, -1, 1),
    (8, 0, 1), (9, 0, 1), (10, None, 1),
    (1, FAKE + 8, 2), (4, FAKE + 8, 2), (3, 132, 2), (6, 4, 2), (10, FAKE + 2, 2), (9, 68, 2), (8, 65536, 5), (9, 264, 5),
    (7, 1 << 31, 5),
])
def test_rope_rows_refusals(sv, at, value, status):  # noqa: F811
    a = [ctypes.byref(_rope(sv)), FAKE, 1, 128, FAKE + 4096, 1, 128, 36, 2, 64, FAKE, None]
    a[at] = value
    assert sv.lib().spec_rope(*a) == status


@pytest.mark.parametrize("at,value", [(2, 0), (5, 0), (3, 136), (6, 136)])
def test_rope_in_place_needs_one_type_and_stride(sv, at, value):  # noqa: F811
    a = [ctypes.byref(_rope(sv)), FAKE, 1, 128, FAKE, 1, 128, 36, 2, 64, FAKE, None]
    a[at] = value
    assert sv.lib().spec_rope(*a) == 1


@pytest.mark.parametrize("x,stride", [(FAKE, 0), (FAKE, 120), (FAKE + 4096, 0), (FAKE + 4096, 120)])
def test_rows_that_overlap_are_not_written(sv, x, stride):  # noqa: F811
    """Rows of a broadcast tensor may be read, but not turned in place or written to: two would be one row of memory."""
    a = [ctypes.byref(_rope(sv)), x, 1, stride, FAKE, 1, stride, 36, 2, 64, FAKE, None]
    assert sv.lib().spec_rope(*a) == 1
    a = _append(sv, q=x, q_out=FAKE, q_token_stride=stride, q_out_token_stride=stride)
    assert sv.lib().spec_kv_append_rope(ctypes.byref(_cache(sv)), ctypes.byref(_rope(sv)), ctypes.byref(a), None) == 1


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS)
def test_append_rope_refuses_a_cache(sv, kw, status):  # noqa: F811
    c = _cache(sv, **kw)
    assert sv.lib().spec_kv_append_rope(ctypes.byref(c), ctypes.byref(_rope(sv)), ctypes.byref(_append(sv)), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(struct_size=8), 1), (dict(layer=2), 1), (dict(layer=-1), 1), (dict(new_dtype=2), 1), (dict(rows=-1), 1),
    (dict(row_off=None, rows=35), 1), (dict(row_off=None, rows=0, t_max=0), 1), (dict(kv_lens=None), 1), (dict(k_new=None), 1),
    (dict(v_new=None), 1), (dict(new_token_stride=-128), 1), (dict(q_heads=-1), 1), (dict(q=None), 1), (dict(q_out=None), 1),
    (dict(parent=FAKE, positions=FAKE), 1), (dict(q_token_stride=-8), 1), (dict(q_out_token_stride=-8), 1),
    (dict(q_out=FAKE, q_out_token_stride=1024), 1), (dict(new_dtype=0, q_out=FAKE), 1),
    (dict(k_new=FAKE + 8), 2), (dict(v_new=FAKE + 8), 2), (dict(new_token_stride=132), 2), (dict(row_off=FAKE + 4), 2),
    (dict(kv_lens=FAKE + 2), 2), (dict(parent=FAKE + 2), 2), (dict(positions=FAKE + 2), 2), (dict(q=FAKE + 8), 2),
    (dict(q_out=FAKE + 8), 2), (dict(q_token_stride=516), 2), (dict(q_out_token_stride=516), 2), (dict(seq_status=FAKE + 1), 2),
    (dict(rows=1 << 31), 5), (dict(q_heads=65536), 5), (dict(rows=1 << 28, q_heads=16), 5),
])
def test_append_rope_refusals(sv, kw, status):  # noqa: F811
    a = _append(sv, **kw)
    assert sv.lib().spec_kv_append_rope(ctypes.byref(_cache(sv)), ctypes.byref(_rope(sv)), ctypes.byref(a), None) == status


def test_null_structs(sv):  # noqa: F811
    L = sv.lib()
    c, r, a = ctypes.byref(_cache(sv)), ctypes.byref(_rope(sv)), ctypes.byref(_append(sv))
    assert L.spec_kv_append_rope(None, r, a, None) == L.spec_kv_append_rope(c, None, a, None) == 1
    assert L.spec_kv_append_rope(c, r, None, None) == 1
    assert L.spec_kv_attend_window(None, None, 4, 0, None) == L.spec_kv_attend_window(c, None, 4, 0, None) == 1


@pytest.mark.parametrize("window,sinks", [(0, 0), (-1, 0), (4, -1), (-2**31, 0)])
def test_window_refusals(sv, window, sinks):  # noqa: F811
    assert sv.lib().spec_kv_attend_window(ctypes.byref(_cache(sv)), ctypes.byref(_attend(sv)), window, sinks, None) == 1


@pytest.mark.parametrize("kw,status", [(dict(t_max=129, rows=36), 5), (dict(q=FAKE + 8), 2), (dict(workspace=None), 3),
                                       (dict(workspace_bytes=1024), 3), (dict(scale=0.0), 1)])
def test_window_refuses_what_the_attention_refuses(sv, kw, status):  # noqa: F811
    a = _attend(sv, **kw)
    assert sv.lib().spec_kv_attend_window(ctypes.byref(_cache(sv)), ctypes.byref(a), 16, 4, None) == status


@pytest.mark.parametrize("window,sinks,want", [
    (16, 4, (16, 4)), (2**31 - 1, 2**31 - 1, (2**31 - 1, 2**31 - 1)), (2**31, 0, (2**31 - 1, 0)), (2**32 + 5, 3, (2**31 - 1, 3)),
    (7, 2**32 + 1, (7, 2**31 - 1)), (5 - 2**32, 0, (-1, 0)), (5, 1 - 2**32, (5, -1)), (-2**31 - 1, 2**40, (-1, 2**31 - 1)),
])
def test_binding_passes_no_window_by_its_low_bits(monkeypatch, window, sinks, want):
    """A window past 32 bits is the largest one, and one below them stays a refusal."""
    import types

    import speculative_decoding_verification_38_gb300 as sv

    called = []
    fake = types.SimpleNamespace(spec_kv_attend_window=lambda *a: called.append(a[2:4]) or 0)
    monkeypatch.setattr(sv, "_lib", fake)
    args = types.SimpleNamespace(cache=types.SimpleNamespace(ref=None), ref=None)
    sv.spec_kv_attend_window(args, window, sinks, stream=0)
    assert called == [want]


def test_binding_refuses_before_the_library():
    import speculative_decoding_verification_38_gb300 as sv

    with pytest.raises(ValueError):
        sv.Rope(torch.zeros(32))  # not on a GPU
    with pytest.raises(ValueError):
        sv.spec_rope(None, torch.zeros((3, 2, 64)), torch.zeros((3, 2, 64)), None)


def test_case_hides_what_no_token_sees():
    c = WindowCase(lens=[200, 40, 3], tokens=[5, 1, 3], window=20, sinks=3, bs=16, device="cpu")
    assert (c.table[0, 1:11] == np.array([(10**8, -1, -10**9)[p % 3] for p in range(1, 11)])).all()
    assert c.table[0, 0] >= 0 and (c.table[0, 11:13] >= 0).all() and (c.table[2, 0] >= 0).all()
    out, lse = c.expected()[:2]
    assert np.isfinite(out).all() and np.isfinite(lse).all()
