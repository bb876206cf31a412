"""What the size function asks for, and what each call takes: with up to 16 rows to a key-value head a caller without a window
pays for one no more than its trees' depths."""
import ctypes

import pytest

from tests.test_abi import sv  # noqa: F401
from tests.test_kv_host import _attend, _cache

PARTS, DEPTHS = 2 * 160, 160 * 128  # two parts for each of 160 CTAs at most; a byte for each of a CTA's tree's nodes


def _need(sv, **kw):  # noqa: F811
    """Of the size function, for head_dim 128 less what every workspace has (head_dim 256 needs no more than that)."""
    size = [sv.lib().spec_kv_attend_workspace_size(ctypes.byref(_cache(sv, head_dim=d, **kw.get("cache", {}))),
                                                   ctypes.byref(_attend(sv, **kw.get("args", {})))) for d in (128, 256)]
    return size[0] - size[1]


@pytest.mark.parametrize("q_heads,t_max", [(2, 1), (8, 1), (8, 2), (2, 9), (16, 2), (8, 4), (32, 1)])
@pytest.mark.parametrize("batch", [1, 4, 76, 2000])
def test_few_rows_need_their_tiles_parts(sv, q_heads, t_max, batch):  # noqa: F811
    assert q_heads // 2 * t_max <= 16
    need = _need(sv, args=dict(q_heads=q_heads, t_max=t_max, row_off=1 << 20, rows=1), cache=dict(batch=batch))
    assert need == PARTS * 16 * (128 * 4 + 8) + DEPTHS


@pytest.mark.gpu
@pytest.mark.parametrize("G,t,tile", [(1, 1, 16), (4, 4, 16), (4, 5, 32), (4, 9, 48), (8, 9, 80), (4, 29, 128)])
def test_each_call_takes_what_it_needs(sv, G, t, tile):  # noqa: F811
    """spec_kv_attend the parts of its own tiles and no more; a byte less is refused, by either call."""
    import torch

    from tests.window_cases import WindowCase

    c = WindowCase(lens=[300, 40], tokens=[t, t], H=2, G=G, D=128, window=50, sinks=2, hide=False)
    c.attend(sv)
    size = sv.spec_kv_attend_workspace_size(c.args)
    header = size - _need(sv, args=dict(q_heads=2 * G, t_max=t, row_off=1 << 20, rows=1))
    alone = header + -(-PARTS * tile * (128 * 4 + 8) // 256) * 256
    for need, call in ((alone, sv.spec_kv_attend), (size, lambda a: sv.spec_kv_attend_window(a, 50, 2))):
        c.args.struct.workspace_bytes = need - 1
        assert call(c.args) == sv.SPEC_ERR_WORKSPACE
        c.args.struct.workspace_bytes = need
        sv.check(call(c.args), "attend")
    torch.cuda.synchronize()
    c.check()
