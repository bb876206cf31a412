"""Layers and numbers of tokens that no 32-bit number holds: refused by the cache's calls, not taken by their low bits."""
import pytest
import torch

from tests.kv_cases import Case
from tests.test_gpu_rope import BF, sv  # noqa: F401
from tests.window_cases import rotary

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layer", [2**32, 2**32 + 1, -(2**32), 2**31, 2**63])
def test_layers_past_32_bits(sv, layer):  # noqa: F811
    c = Case(lens=[20, 9], tokens=[4, 2], H=2, D=32, layers=2)
    c.to_device(sv)
    before = c.raw(c.dk), c.raw(c.dv)
    new = torch.randn((6, 2, 32)).to(BF).cuda()
    out = torch.full((32, 2, 32), 7.0, dtype=BF, device="cuda")
    q = torch.full_like(new, 1.0)
    rope = sv.Rope(rotary(16).cuda())
    off = torch.tensor([0, 20, 29], device="cuda")
    args = sv.AttendArgs(cache=c.cache, q=q, out=torch.full_like(q, 7.0), kv_lens=c.dlens, row_off=c.doff, t_max=4, scale=1.0,
                         layer=layer)
    args.set_workspace(torch.zeros(sv.spec_kv_attend_workspace_size(args), dtype=torch.uint8, device="cuda"))
    again = sv.AttendArgs(cache=c.cache, q=q, out=torch.full_like(q, 7.0), kv_lens=c.dlens, row_off=c.doff, t_max=4, scale=1.0)
    again.set_workspace(args.workspace)
    again.set_layer(layer)
    for status in (sv.spec_kv_append(c.cache, new, new, c.dlens, c.doff, 4, layer),
                   sv.spec_kv_append_rope(c.cache, rope, new, new, c.dlens, row_off=c.doff, t_max=4, q=q, q_out=q, layer=layer),
                   sv.spec_kv_gather(c.cache, c.dlens, off, out[:29], out[:29].clone(), layer),
                   sv.spec_kv_attend(args), sv.spec_kv_attend_window(args, 5, 1), sv.spec_kv_attend(again)):
        assert status == sv.SPEC_ERR_INVALID_ARG
    torch.cuda.synchronize()
    for was, now in zip(before, (c.raw(c.dk), c.raw(c.dv))):
        assert ((was == now) | ((was != was) & (now != now))).all()
    assert (q == 1).all() and (out == 7).all()


def test_tokens_past_32_bits(sv):  # noqa: F811
    c = Case(lens=[20, 9], tokens=[3, 3], H=2, D=32)
    c.to_device(sv)
    new = torch.randn((6, 2, 32)).to(BF).cuda()
    rope = sv.Rope(rotary(16).cuda())
    for t in (2**32 + 3, 3 - 2**32):
        assert sv.spec_kv_append(c.cache, new, new, c.dlens, t_max=t) == sv.SPEC_ERR_INVALID_ARG
        assert sv.spec_kv_append_rope(c.cache, rope, new, new, c.dlens, t_max=t) == sv.SPEC_ERR_INVALID_ARG
    args = sv.AttendArgs(cache=c.cache, q=new, out=torch.empty_like(new), kv_lens=c.dlens, t_max=2**32 + 3, scale=1.0)
    args.set_workspace(torch.zeros(1 << 24, dtype=torch.uint8, device="cuda"))
    assert sv.spec_kv_attend(args) == sv.SPEC_ERR_UNSUPPORTED  # as any more than SPEC_KV_MAX_QUERIES
    assert sv.spec_kv_attend_window(args, 5, 1) == sv.SPEC_ERR_UNSUPPORTED
