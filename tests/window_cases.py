"""Inputs of the tests of the sliding window and of rotary positions."""
import numpy as np
import torch

from oracle import kv as okv
from tests.kv_cases import Case, half_step


class WindowCase(Case):
    """A Case whose tokens see `window` positions and the first `sinks`. Where no token of a sequence sees a position,
    there is NaN in the cache, and the table's entries of pages without one that is seen lie far outside the pool."""

    def __init__(self, *, window, sinks=0, hide=True, **kw):
        super().__init__(**kw)
        self.window, self.sinks = window, sinks
        self.pages_of = self.table.copy()
        if not hide:
            return
        for b in range(self.B):
            if not self.tokens[b]:
                continue
            seen = self.seen(b).any(0)
            for j in np.flatnonzero(~seen):
                self.fill(b, j, float("nan"))
            for p in range(-(-self.lens[b] // self.bs)):
                if not seen[p * self.bs:(p + 1) * self.bs].any():
                    self.table[b, p] = (10**8, -1, -10**9)[p % 3]

    def seen(self, b):
        lo, T = self.row_off[b], self.tokens[b]
        return okv.sight(T, self.lens[b], None if self.parent is None else self.parent[lo:lo + T], self.window, self.sinks)

    def fill(self, b, j, value, what="kv"):
        """Position j of sequence b, all of its elements."""
        g, i = self.pages_of[b, j // self.bs], j % self.bs
        for name in what:
            getattr(self, name)[self.layer, g, i] = (127 if value != value else int(value)) if self.dtype == "e4m3" else value

    def expected(self):
        k, v, ks, vs = self.host()
        return okv.attend(self.q.double().numpy(), k, v, ks, vs, self.table, self.layer, self.row_off, self.lens,
                          self.scale, self.parent, self.window, self.sinks)

    def attend(self, sv, **kw):
        call = sv.spec_kv_attend

        class Windowed:  # the same call site, with the window
            def __getattr__(_, name):
                return getattr(sv, name)

            @staticmethod
            def spec_kv_attend(args, stream=None):
                assert call is sv.spec_kv_attend
                return sv.spec_kv_attend_window(args, self.window, self.sinks, stream)

        return super().attend(Windowed(), **kw)


def pair_sum(x, half, adjacent):
    """|x_a| + |x_b| of each element's pair; zero past the rotary part."""
    s = np.zeros_like(x)
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if adjacent else (slice(0, half), slice(half, 2 * half))
    s[..., a] = s[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return s


def rope_bound(x, half, adjacent, factor):
    """How far a rotated element may be from the formula's before its rounding: sine and cosine are off by 2^-23 each,
    times the factor (2^-24), a product and a fused one round by 2^-24 each; of |x_a| + |x_b| all together less than
    2^-22."""
    return 2.0**-22 * abs(factor) * pair_sum(x, half, adjacent)


def rounding(y, dtype):
    return 0.0 if dtype is None else half_step(dtype) * np.abs(y) + 2.0**-149


def check_e4m3(codes, scale, y, off):
    """Codes and scales [..., D], [...] against values y known to within `off`: the scale is the smallest power of two
    that brings the largest value to 448 or less, for some values that near, and each code the nearest of its value."""
    top, slack = np.abs(y).max(-1), off.max(-1)
    s = scale.astype(np.float64)
    assert (np.log2(s) == np.round(np.log2(s))).all()
    assert (top - slack <= 448 * s).all() and ((top + slack > 224 * s) | (s == 2.0**-126) | (top + slack == 0)).all()
    got = okv.E4M3[codes] * s[..., None]
    step = np.maximum(2.0**-4 * np.abs(y), 2.0**-10 * s[..., None])  # half a step, normal or not
    assert (np.abs(got - y) <= step + off).all(), float((np.abs(got - y) - step - off).max())


def rotary(half, base=10000.0):
    return (base ** (-torch.arange(half, dtype=torch.float64) / half)).float()
