"""How far below the root a tree's node may lie in the rotating append: as far as the attention takes new tokens."""
import numpy as np
import pytest
import torch

from oracle import kv as okv
from tests.kv_cases import Case, tree
from tests.test_gpu_rope import BF, sv  # noqa: F401
from tests.window_cases import rope_bound, rotary, rounding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_nodes_too_deep_are_refused(sv, dtype):  # noqa: F811
    """128 nodes in a chain, then longer ones; many nodes that are not deep; a long way beside a short one."""
    chain = lambda n: list(range(-1, n - 1))  # noqa: E731
    trees = [chain(128), chain(129), tree([40, 20]), chain(300), chain(100) + [0] * 150, [-1], chain(128) + [127]]
    c = Case(lens=[len(t) + 5 * b for b, t in enumerate(trees)], tokens=[len(t) for t in trees], H=1, D=64, dtype=dtype,
             parent=sum(trees, []))
    c.to_device(sv)
    g = torch.Generator().manual_seed(3)
    k, q = ((torch.randn((c.rows, h, 64), generator=g)).to(BF) for h in (1, 2))
    out = torch.full((c.rows, 2, 64), 7.0, dtype=BF, device="cuda")
    status = torch.full((c.B,), -7, dtype=torch.int32, device="cuda")
    before = c.raw(c.dk)
    inv = rotary(32).cuda()
    sv.check(sv.spec_kv_append_rope(c.cache, sv.Rope(inv), k.cuda(), k.cuda(), c.dlens, row_off=c.doff, t_max=c.t_max,
                                    parent=torch.from_numpy(c.parent).cuda(), q=q.cuda(), q_out=out, seq_status=status), "append")
    assert status.tolist() == [0, 4, 0, 4, 0, 0, 4]
    depth = []
    for t in trees:
        at = []
        for p in t:
            at.append(at[p] + 1 if p >= 0 else 0)
        depth += at
    depth = np.array(depth)
    base = np.repeat([n - len(t) for n, t in zip(c.lens, trees)], [len(t) for t in trees])
    taken = depth < sv.SPEC_KV_MAX_QUERIES
    got = out.double().cpu().numpy()
    assert (got[~taken] == 7).all() and (~taken).sum() == 1 + 172 + 1
    x = q.double().numpy()
    want = okv.rope(x, [(base + depth).tolist()], inv.cpu().numpy())
    assert (np.abs(got - want) <= rope_bound(x, 32, False, 1.0) + rounding(want, BF))[taken].all()
    after = c.raw(c.dk)
    for b in range(c.B):
        for t in range(c.tokens[b]):
            r = c.row_off[b] + t
            p, i = okv.slot_of(c.table[b], c.lens[b] - c.tokens[b] + t, c.bs)
            same = np.array_equal(after[0, p, i], before[0, p, i], equal_nan=True)
            assert same != taken[r], (b, t)
