"""Up to 16 query rows to a key-value head through windows too long for one processor to go through an entry alone: against
the float64 oracle (bounds: tests/kv_cases.py), and shared out over the processors whatever the lengths. As in
tests/test_gpu_window.py, what no token sees is NaN and its pages' table entries lie outside the pool."""
import numpy as np
import pytest
import torch

from tests.kv_cases import random_tree
from tests.test_gpu_window import sv  # noqa: F401
from tests.window_cases import WindowCase

pytestmark = pytest.mark.gpu

# one sequence past the window, one as long as it, others short or without new tokens: 80 entries, one to a piece
B = 80


def _case(dtype, G, D, t, *, bs=16, order="nhd", sinks=5, as_tree=False, H=1, **kw):
    window = 8300 if dtype == "bf16" else 16500
    tokens = [t, t] + [0 if b % 9 == 4 else max(1, t - b % 3) for b in range(B // H - 2)]
    lens = [window + 700, window] + [n + (b * 37) % 150 if n else 0 for b, n in enumerate(tokens[2:])]
    parent = sum((random_tree(n, b) if n else [] for b, n in enumerate(tokens)), []) if as_tree else None
    return WindowCase(lens=lens, tokens=tokens, H=H, G=G, D=D, bs=bs, dtype=dtype, order=order, parent=parent, q_scale=2.0,
                      window=window, sinks=sinks, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("as_tree", [False, True])
@pytest.mark.parametrize("G,D,t,bs,order,sinks", [(1, 64, 1, 16, "nhd", 5), (4, 128, 1, 16, "nhd", 0), (4, 128, 4, 5, "hnd", 17),
                                                  (1, 96, 16, 16, "nhd", 130), (5, 16, 3, 128, "nhd", 1)])
def test_long_windows(sv, dtype, as_tree, G, D, t, bs, order, sinks):  # noqa: F811
    """Ragged chains and trees; the same call twice gives the same bits."""
    c = _case(dtype, G, D, t, bs=bs, order=order, sinks=sinks, as_tree=as_tree)
    c.attend(sv)
    assert c.status.tolist() == [0] * c.B
    c.check()
    first = c.out.clone()
    c.attend(sv)
    assert torch.equal(first, c.out)


@pytest.mark.parametrize("dtype,value", [("bf16", float("nan")), ("bf16", float("inf")), ("e4m3", float("nan"))])
@pytest.mark.parametrize("as_tree", [False, True])
def test_values_that_only_some_rows_see(sv, dtype, value, as_tree):  # noqa: F811
    """At the window's end and in a new token: into the rows that see it and no other."""
    make = lambda: _case(dtype, 4, 64, 4, as_tree=as_tree)  # noqa: E731
    clean = make()
    out, lse, av, mag, spread = clean.expected()
    c = make()
    hit = np.zeros(c.rows, dtype=bool)
    for b in (0, 1):
        see = c.seen(b)
        part = np.flatnonzero(see.any(0) & ~see.all(0))
        for at in (part[0], part[-1]):
            c.fill(b, at, value, "v")
            hit[c.row_off[b]:c.row_off[b + 1]] |= see[:, at]
    c.attend(sv)
    got = c.out.double().cpu().numpy()
    assert hit.any() and not hit[c.row_off[0]:c.row_off[2]].all()
    assert (np.abs(got - out) <= clean.bound(out, av, mag, spread))[~hit].all()
    assert not np.isfinite(got[hit]).any()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_statuses_and_replays(sv, dtype):  # noqa: F811
    """Errors beside sound sequences; a graph of the call follows the lengths; a workspace that served short windows."""
    c = _case(dtype, 4, 64, 2, hide=False)
    c.attend(sv)
    c.check()
    window, c.window = c.window, 40
    sv.check(sv.spec_kv_attend_window(c.args, 40, c.sinks), "short")
    c.check()
    c.window = window
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.check(sv.spec_kv_attend_window(c.args, c.window, c.sinks), "long")
    c.lens = [300, 17] + c.lens[2:]
    c.dlens.copy_(torch.tensor(c.lens, dtype=torch.int32))
    c.out.fill_(7.0)
    graph.replay()
    c.check()
    c.dlens[0] = 1
    c.dtable[1, 0] = -1
    graph.replay()
    assert c.status.tolist()[:3] == [2, 4, 0] and c.status.tolist()[3:] == [0] * (c.B - 3)
    assert (c.out[:2] == 0).all() and (c.lse[:2] == -float("inf")).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_one_long_sequence_among_short_ones(sv, dtype):  # noqa: F811
    """The long one is every processor's work: no slower than three times the same call without a window (one processor to
    each of its heads took 8 to 14 times as long)."""
    c = WindowCase(lens=[131072] + [64] * 151, tokens=[1] * 152, H=1, G=4, D=128, dtype=dtype, window=131072, hide=False)
    c.attend(sv)

    def us(call):
        call()
        best = 1e9
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(10):
                call()
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b) * 100)
        return best

    whole = us(lambda: sv.check(sv.spec_kv_attend(c.args), "attend"))
    through = us(lambda: sv.check(sv.spec_kv_attend_window(c.args, 131072, 0), "window"))
    assert through <= 3 * whole, (through, whole)
