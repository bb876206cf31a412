"""Scores that rise along a window of many tiles to a processor: references that move past the tiles which find their maxima
first, and that stay where a weight is the most that its format takes; values near float32's range."""
import math

import numpy as np
import pytest
import torch

from oracle import kv as okv
from tests.test_gpu_window import sv  # noqa: F401
from tests.window_cases import WindowCase

pytestmark = pytest.mark.gpu

# log2 of the weights, four tiles each (as many as teams take in turn, and the first two groups are those that find their
# maxima first): up to 2^9.75 a reference stays, past that it moves
RISE = [0, 1, 10.7, 10.8, 3, 20.5, 40, 49.7, 20, 49.8, 70, 30, 79.7, 100]


class Rising(WindowCase):
    """A chain, of which every 19th sequence is looked at."""

    step = 19

    def check(self):
        for b in range(self.B):
            if b % self.step:
                self.out[self.row_off[b]:self.row_off[b + 1]] = 0
                self.lse[self.row_off[b]:self.row_off[b + 1]] = 0
        super().check()

    def expected(self):
        """okv.attend of this case, all positions of a sequence at once; zeros for those that are not looked at."""
        k, v, ks, vs = self.host()
        shape = (self.rows, self.H * self.G, self.D)
        out, av = np.zeros(shape), np.zeros(shape)
        lse, mag, spread = (np.zeros(shape[:2]) for _ in range(3))
        q = self.q.double().numpy()
        for b in range(0, self.B, self.step):
            see, j = self.seen(b), np.arange(self.lens[b])
            see, j = see[:, see.any(0)], j[see.any(0)]
            p, i = self.pages_of[b, j // self.bs], j % self.bs
            rows = slice(self.row_off[b], self.row_off[b + 1])
            for h in range(self.H):
                kk, vv = ((pool[self.layer, p, i, h] if sc is None else
                           okv.E4M3[pool[self.layer, p, i, h]] * sc[self.layer, p, h, i][:, None].astype(np.float64))
                          for pool, sc in ((k, ks), (v, vs)))
                for c in range(h * self.G, (h + 1) * self.G):
                    s = np.where(see, self.scale * (q[rows, c] @ kk.T), -np.inf)
                    m = s.max(1, keepdims=True)
                    w = np.exp(s - m)
                    n = w.sum(1, keepdims=True)
                    out[rows, c], av[rows, c] = w @ vv / n, w @ np.abs(vv) / n
                    lse[rows, c] = (m + np.log(n))[:, 0]
                    mag[rows, c] = self.scale * np.where(see, np.abs(q[rows, c]) @ np.abs(kk).T, 0).max(1)
                    spread[rows, c] = np.where(see, np.abs(vv).max(1), 0).max(1) * see.sum(1) / n[:, 0]
        return out, lse, av, mag, spread


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("G,D,t,falling", [(4, 128, 2, False), (2, 64, 9, False), (4, 128, 9, False), (8, 64, 9, False),
                                           (8, 128, 14, False), (4, 128, 9, True)])
def test_rising_scores(sv, dtype, G, D, t, falling):  # noqa: F811
    """152 sequences of one head, so that each is one processor's."""
    n = 128 * 4 * len(RISE)
    c = Rising(lens=[n - 3 * (b % 7) for b in range(152)], tokens=[t] * 152, H=1, G=G, D=D, dtype=dtype, window=n - 200, sinks=5,
               hide=False)
    rise = np.repeat(RISE[::-1] if falling else RISE, 512)
    want = torch.zeros(c.held.shape, dtype=torch.float64)  # a key's every element, so that its score is rise * ln 2
    for b in range(c.B):
        j = np.arange(c.lens[b])
        want[c.table[b, j // c.bs], j % c.bs] = torch.from_numpy(rise[:c.lens[b]] * math.log(2) / (c.scale * D))
    if dtype == "bf16":
        c.k.copy_(want[None, :, :, None, None].expand(c.k.shape))
        c.v.mul_(2.0**100)
    else:
        c.k.fill_(0x38)  # one
        c.ks.copy_(want[None, :, None, :].expand(c.ks.shape))
        # a scale that fills its unit, and ones below it
        even = torch.zeros(c.held.shape[0], dtype=torch.bool)
        even[torch.from_numpy(c.table[::2][c.table[::2] >= 0]).long()] = True
        c.vs[:, even] = 2.0**98
        c.vs[:, ~even] *= 2.0**97
    c.q = torch.ones_like(c.q)
    c.to_device(sv)
    # (a table that could hold more: with few rows, the kernel of many tiles too)
    c.dtable = torch.cat([c.dtable, torch.full((c.B, 600), -5, dtype=torch.int32, device="cuda")], 1)
    c.cache = sv.KVCache(c.dk, c.dv, c.dtable, k_scale=c.dks, v_scale=c.dvs)
    for window in (c.window, 2**30):
        c.window = window
        c.attend(sv)
        assert c.status.tolist() == [0] * c.B and c.out.isfinite().all()
        c.check()
