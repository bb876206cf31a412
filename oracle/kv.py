"""Float64 oracle of the paged key-value cache's operators (test infrastructure).

Plain numpy, one sequence, token and head after another; it shares no code with the CUDA path. Arrays: a cache is
k, v [layers, pages, slots, heads, dim] (float64 values of bf16 caches, uint8 codes of e4m3 ones), scales
[layers, pages, heads, slots] or None, table [B, max_blocks].
"""
from __future__ import annotations

import numpy as np


def _e4m3_table() -> np.ndarray:
    """The value of every 8-bit code: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7F and 0xFF are NaN."""
    t = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m / 8 * 2.0**-6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        t[c] = np.nan if (c & 127) == 127 else (-x if c & 128 else x)
    return t


E4M3 = _e4m3_table()


def e4m3_encode(x: np.ndarray) -> np.ndarray:
    """Nearest code, ties to the even mantissa, values past 448 to 448, NaN to 0x7F; signs kept."""
    x = np.asarray(x, dtype=np.float64)
    mag = E4M3[:127]  # 0 .. 448, rising
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(mag, np.nan_to_num(a)), 1, 126)
    lo = hi - 1
    dl, dh = a - mag[lo], mag[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi))).astype(np.uint8)
    code = np.where(np.signbit(x), code | 128, code).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(127), code)


def quantise(x: np.ndarray):
    """One entry [D] -> (codes, scale): the smallest power of two (not below 2^-126) that brings the largest finite
    value to 448 or less; NaN and infinities become NaN."""
    x = np.asarray(x, dtype=np.float64)
    fin = np.isfinite(x)
    top = np.max(np.abs(x[fin]), initial=0.0)
    e = 0
    if top > 0:
        e = -126
        while top / 2.0**e > 448:
            e += 1
    return e4m3_encode(np.where(fin, x, np.nan) / 2.0**e), np.float32(2.0**e)


def slot_of(table_row, pos: int, bs: int):
    return int(table_row[pos // bs]), pos % bs


def append(k, v, ks, vs, table, layer, k_new, v_new, row_off, kv_lens):
    """In place; k_new, v_new float64 [rows, H, D] (already rounded to the cache's 16-bit type where it has one)."""
    bs = k.shape[2]
    for b in range(len(kv_lens)):
        T = int(row_off[b + 1] - row_off[b])
        for t in range(T):
            g, i = slot_of(table[b], int(kv_lens[b]) - T + t, bs)
            for pool, sc, new in ((k, ks, k_new), (v, vs, v_new)):
                for h in range(k.shape[3]):
                    x = new[row_off[b] + t, h]
                    if sc is None:
                        pool[layer, g, i, h] = x
                    else:
                        pool[layer, g, i, h], sc[layer, g, h, i] = quantise(x)


def entries(pool, sc, table_row, layer, h, n: int, wanted=None) -> np.ndarray:
    """Positions 0..n-1 of one head as float64 values [n, D]; zeros for those that are not wanted (a bool each)."""
    bs = pool.shape[2]
    out = np.zeros((n, pool.shape[4]))
    for j in range(n) if wanted is None else np.flatnonzero(wanted):
        g, i = slot_of(table_row, j, bs)
        out[j] = pool[layer, g, i, h] if sc is None else E4M3[pool[layer, g, i, h]] * float(sc[layer, g, h, i])
    return out


def ancestors(parent) -> np.ndarray:
    """[T, T]: whether token u is token t itself or an ancestor of it."""
    T = len(parent)
    see = np.zeros((T, T), dtype=bool)
    for t in range(T):
        u = t
        while u >= 0:
            see[t, u] = True
            u = int(parent[u])
    return see


def sight(T: int, L: int, parent=None, window: int = 0, sinks: int = 0) -> np.ndarray:
    """[T, L]: what each of the last T of L positions sees. window > 0: of that, what lies less than `window` before its
    own position (L - T and its place in the chain, or its depth in the tree), and the first `sinks`."""
    see = np.ones((T, L), dtype=bool)
    see[:, L - T:] = np.tril(np.ones((T, T), dtype=bool)) if parent is None else ancestors(parent)
    if window > 0:
        depth = np.arange(T) if parent is None else ancestors(parent).sum(1) - 1
        place = np.concatenate([np.arange(L - T), L - T + depth])
        see &= (place[None, L - T:].T - place[None, :] < window) | (np.arange(L) < sinks)
    return see


def attend(q, k, v, ks, vs, table, layer, row_off, kv_lens, scale, parent=None, window=0, sinks=0):
    """out [rows, Hq, D], lse [rows, Hq] and, for error bounds: the weighted mean of |v| (same shape as out), the
    largest |s| with its sum of |q k| terms [rows, Hq], and max |v| over the seen positions divided by the sum of the
    weights relative to the largest [rows, Hq]."""
    rows, Hq, D = q.shape
    H = k.shape[3]
    G = Hq // H
    out = np.zeros((rows, Hq, D))
    lse = np.full((rows, Hq), -np.inf)
    av = np.zeros((rows, Hq, D))
    mag = np.zeros((rows, Hq))
    spread = np.zeros((rows, Hq))
    for b in range(len(kv_lens)):
        lo, T, L = int(row_off[b]), int(row_off[b + 1] - row_off[b]), int(kv_lens[b])
        if T == 0:
            continue
        see = sight(T, L, None if parent is None else parent[lo:lo + T], window, sinks)
        for h in range(H):
            kk, vv = (entries(p, sc, table[b], layer, h, L, see.any(0)) for p, sc in ((k, ks), (v, vs)))
            for g in range(G):
                for t in range(T):
                    ok = see[t]
                    qq = q[lo + t, h * G + g]
                    s = scale * (kk[ok] @ qq)
                    m = s.max()
                    if m == -np.inf:
                        continue
                    w = np.exp(s - m)
                    r, c = lo + t, h * G + g
                    out[r, c] = (w @ vv[ok]) / w.sum()
                    lse[r, c] = m + np.log(w.sum())
                    av[r, c] = (w @ np.abs(vv[ok])) / w.sum()
                    mag[r, c] = scale * (np.abs(kk[ok]) @ np.abs(qq)).max()
                    spread[r, c] = np.abs(vv[ok]).max() * ok.sum() / w.sum()
    return out, lse, av, mag, spread


def compact(pools, scales, table, node_off, path, accepted, kv_lens):
    """In place over k and v pools (and scales); returns the new lengths."""
    bs = pools[0].shape[2]
    new = np.array(kv_lens, dtype=np.int32)
    for b in range(len(kv_lens)):
        N = int(node_off[b + 1] - node_off[b])
        base = int(kv_lens[b]) - N
        for i in range(int(accepted[b])):
            (gs, ss), (gd, sd) = (slot_of(table[b], base + n, bs) for n in (int(path[node_off[b] + i]), 1 + i))
            for p in pools:
                p[:, gd, sd] = p[:, gs, ss]
            for s in scales:
                if s is not None:
                    s[:, gd, :, sd] = s[:, gs, :, ss]
        new[b] = kv_lens[b] - (N - 1 - int(accepted[b]))
    return new


def depths(parent) -> np.ndarray:
    return ancestors(parent).sum(1) - 1


def axis_of_pair(half: int, sections=None, alternating=False) -> np.ndarray:
    """The axis each pair turns by: sections in blocks, or in turn as long as each lasts, the rest by axis 0."""
    if sections is None:
        return np.zeros(half, dtype=int)
    if not alternating:
        return np.repeat(np.arange(len(sections)), sections)
    n = len(sections)
    return np.array([i % n if i // n < sections[i % n] else 0 for i in range(half)])


def rope(x, positions, inv_freq, *, adjacent=False, sections=None, alternating=False, factor=1.0):
    """x [rows, heads, D] float64, positions [axes, rows], inv_freq [half] as float32 values: the pairs as complex
    numbers, each times factor e^(i angle). The angle's turns are taken in 128-bit whole numbers, so that they are good
    for any position."""
    half = len(inv_freq)
    axis = axis_of_pair(half, sections, alternating)
    num, den = 2 * 2646693125139304345, 842468587426513207  # 2 pi, to 36 digits
    turn = np.empty((x.shape[0], half))
    for i in range(half):
        m, e = np.frexp(np.float64(inv_freq[i]))
        whole, shift = int(m * 2**24), int(24 - e)  # inv_freq = whole / 2^shift, exactly
        for r in range(x.shape[0]):
            up = int(positions[axis[i]][r]) * whole * den
            down = num << shift if shift >= 0 else num
            up = up if shift >= 0 else up << -shift
            turn[r, i] = (up % down) / down
    z = np.exp(2j * np.pi * turn)[:, None, :] * factor
    y = np.array(x, dtype=np.float64)
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if adjacent else (slice(0, half), slice(half, 2 * half))
    w = (y[..., a] + 1j * y[..., b]) * z
    y[..., a], y[..., b] = w.real, w.imag
    return y
