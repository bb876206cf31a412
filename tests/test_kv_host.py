"""The paged cache without a GPU: the oracle against torch, the struct layouts, and the host's refusals, which come
before any CUDA call."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import kv as okv
from tests.kv_cases import Case, random_tree, tree
from tests.test_abi import sv, test_struct_layout_matches_header as _layout  # noqa: F401


@pytest.mark.parametrize("cname,pyname", [("spec_kv_cache_t", "SpecKvCache"), ("spec_kv_attend_args_t", "SpecKvAttendArgs")])
def test_struct_layout(sv, cname, pyname):  # noqa: F811
    _layout(sv, cname, pyname)


# ------------------------------------------------------------------ oracle
def test_oracle_codes_match_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    np.testing.assert_array_equal(okv.E4M3, codes.view(torch.float8_e4m3fn).double().numpy())
    g = torch.Generator().manual_seed(1)
    x = torch.cat([torch.randn(20000, generator=g) * torch.exp(torch.randn(20000, generator=g) * 3),
                   torch.from_numpy(okv.E4M3[:127]).float(), -torch.from_numpy(okv.E4M3[:127]).float(),
                   torch.from_numpy((okv.E4M3[:126] + okv.E4M3[1:127]) / 2).float()]).clamp(-448, 448)
    np.testing.assert_array_equal(okv.e4m3_encode(x.numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_oracle_scale_is_the_smallest_power_of_two():
    for top in (448.0, 448.1, 1.0, 1.75, 1.7500001, 3e38, 2.0**-126, 1e-45):
        codes, s = okv.quantise(np.array([top, -top / 3]))
        assert top / float(s) <= 448 and math.log2(s) == round(math.log2(s))
        assert top / (float(s) / 2) > 448 or float(s) == 2.0**-126
    assert okv.quantise(np.zeros(4))[1] == 1.0
    codes, s = okv.quantise(np.array([np.nan, np.inf, 2.0]))
    assert s == 2.0**-7 and (codes[:2] == 127).all() and okv.E4M3[codes[2]] == 256


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("as_tree", [False, True])
def test_oracle_attention_matches_torch(dtype, as_tree):
    t = [random_tree(9, 4), tree([2, 2]), [-1]]
    c = Case(lens=[30, 7, 12], tokens=[len(x) for x in t], H=2, G=3, D=32, bs=5, dtype=dtype, device="cpu",
             parent=sum(t, []) if as_tree else None)
    out, lse = c.expected()[:2]
    k, v, ks, vs = c.host()
    for b in range(3):
        T, L, lo = c.tokens[b], c.lens[b], c.row_off[b]
        for hq in range(6):
            kk, vv = (torch.from_numpy(okv.entries(p, s, c.table[b], 0, hq // 3, L)) for p, s in ((k, ks), (v, vs)))
            x = c.q[lo:lo + T, hq].double() @ kk.T * c.scale
            see = torch.ones((T, L), dtype=torch.bool)
            for i in range(T):
                for j in range(T):
                    u = i
                    while as_tree and u > j:
                        u = t[b][u]
                    see[i, L - T + j] = u == j if as_tree else j <= i
            x = x.masked_fill(~see, -math.inf)
            np.testing.assert_allclose(out[lo:lo + T, hq], (torch.softmax(x, -1) @ vv).numpy(), rtol=1e-12, atol=1e-13)
            np.testing.assert_allclose(lse[lo:lo + T, hq], torch.logsumexp(x, -1).numpy(), rtol=1e-13)


def test_oracle_append_then_read_and_compact():
    c = Case(lens=[20, 9], tokens=[6, 9], H=2, D=16, bs=4, device="cpu")
    k, v, ks, vs = c.host()
    new = np.random.default_rng(0).normal(size=(15, 2, 16))
    okv.append(k, v, ks, vs, c.table, 0, new, 2 * new, c.row_off, c.lens)
    for b in range(2):
        for h in range(2):
            got = okv.entries(k, ks, c.table[b], 0, h, c.lens[b])[c.lens[b] - c.tokens[b]:]
            np.testing.assert_array_equal(got, new[c.row_off[b]:c.row_off[b + 1], h])
    path = np.full(15, -1, np.int32)
    path[:3] = [2, 3, 5]
    lens = okv.compact((k, v), (None, None), c.table, c.row_off, path, [3, 0], c.lens)
    assert lens.tolist() == [18, 1]
    np.testing.assert_array_equal(okv.entries(v, vs, c.table[0], 0, 1, 18)[14:], 2 * new[[0, 2, 3, 5], 1])


# ------------------------------------------------------------------ refusals
FAKE = 1 << 20  # never dereferenced: validation fails before any launch


def _cache(sv, **kw):  # noqa: F811
    c = sv.SpecKvCache()
    c.struct_size = ctypes.sizeof(sv.SpecKvCache)
    c.batch, c.kv_heads, c.head_dim, c.block_size = 4, 2, 64, 16
    c.num_blocks, c.max_blocks, c.layers, c.dtype = 100, 10, 2, sv.SPEC_BF16
    c.k = c.v = c.block_table = FAKE
    c.layer_stride, c.block_stride, c.token_stride, c.head_stride = 100 * 2048, 2048, 128, 64
    for name, x in kw.items():
        setattr(c, name, x)
    return c


def _attend(sv, **kw):  # noqa: F811
    a = sv.SpecKvAttendArgs()
    a.struct_size = ctypes.sizeof(sv.SpecKvAttendArgs)
    a.layer, a.q_heads, a.t_max, a.rows = 0, 8, 9, 36
    a.row_off = a.kv_lens = a.q = a.out = a.workspace = FAKE
    a.q_token_stride, a.scale, a.workspace_bytes = 512, 0.125, 1 << 34
    for name, x in kw.items():
        setattr(a, name, x)
    return a


CACHE_REFUSALS = [
    (dict(struct_size=8), 1), (dict(batch=0), 1), (dict(batch=65537), 1), (dict(kv_heads=0), 1), (dict(head_dim=0), 1),
    (dict(block_size=0), 1), (dict(num_blocks=0), 1), (dict(max_blocks=0), 1), (dict(layers=0), 1), (dict(dtype=0), 1),
    (dict(dtype=3), 1), (dict(k=0), 1), (dict(v=0), 1), (dict(block_table=0), 1), (dict(dtype=2), 1),  # no scales
    (dict(token_stride=-64), 1), (dict(head_dim=512), 5), (dict(kv_heads=65536), 5), (dict(block_size=65537), 5),
    (dict(max_blocks=1 << 27), 5), (dict(k=FAKE + 8), 2), (dict(v=FAKE + 2), 2), (dict(block_table=FAKE + 2), 2),
    (dict(head_dim=60), 2), (dict(token_stride=132), 2), (dict(head_stride=4), 2), (dict(block_stride=1), 2),
    (dict(layer_stride=12), 2), (dict(dtype=2, k_scale=FAKE + 2, v_scale=FAKE), 2),
    (dict(dtype=2, k_scale=FAKE, v_scale=FAKE, head_dim=72), 2),
]


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS)
def test_cache_refusals(sv, kw, status):  # noqa: F811
    L = sv.lib()
    c = _cache(sv, **kw)
    p = ctypes.byref(c)
    assert L.spec_kv_append(p, 0, FAKE, FAKE, 1, 128, 36, FAKE, 9, FAKE, None, None) == status
    assert L.spec_kv_gather(p, 0, FAKE, FAKE, 36, FAKE, FAKE, 1, None, None) == status
    assert L.spec_kv_compact(p, FAKE, 36, FAKE, FAKE, FAKE, FAKE, None, None, None) == status
    # the attention also checks its head counts, which a wrong kv_heads upsets first
    assert L.spec_kv_attend(p, ctypes.byref(_attend(sv)), None) in ((status,) if "kv_heads" not in kw else (status, 1))


def test_null_structs(sv):  # noqa: F811
    L = sv.lib()
    assert L.spec_kv_append(None, 0, FAKE, FAKE, 1, 128, 36, FAKE, 9, FAKE, None, None) == 1
    assert L.spec_kv_gather(None, 0, FAKE, FAKE, 36, FAKE, FAKE, 1, None, None) == 1
    assert L.spec_kv_compact(None, FAKE, 36, FAKE, FAKE, FAKE, FAKE, None, None, None) == 1
    assert L.spec_kv_attend(None, None, None) == 1
    assert L.spec_kv_attend(ctypes.byref(_cache(sv)), None, None) == 1
    assert L.spec_kv_attend_workspace_size(None, None) == 0


@pytest.mark.parametrize("at,value,status", [
    (1, 2, 1), (1, -1, 1), (2, None, 1), (3, None, 1), (4, 2, 1), (5, -128, 1), (6, -1, 1), (9, None, 1),
    (2, FAKE + 8, 2), (3, FAKE + 4, 2), (5, 4, 2), (7, FAKE + 4, 2), (9, FAKE + 2, 2), (10, FAKE + 1, 2), (6, 1 << 31, 5),
])
def test_append_refusals(sv, at, value, status):  # noqa: F811
    a = [ctypes.byref(_cache(sv)), 0, FAKE, FAKE, 1, 128, 36, FAKE, 9, FAKE, None, None]
    a[at] = value
    assert sv.lib().spec_kv_append(*a) == status


def test_append_without_offsets_needs_equal_tokens(sv):  # noqa: F811
    p = ctypes.byref(_cache(sv))
    assert sv.lib().spec_kv_append(p, 0, FAKE, FAKE, 1, 128, 35, None, 9, FAKE, None, None) == 1
    assert sv.lib().spec_kv_append(p, 0, FAKE, FAKE, 1, 128, 0, None, 0, FAKE, None, None) == 1


@pytest.mark.parametrize("at,value,status", [
    (1, 2, 1), (2, None, 1), (3, None, 1), (4, -1, 1), (5, None, 1), (6, None, 1), (7, 2, 1), (5, FAKE + 4, 2),
    (6, FAKE + 8, 2), (3, FAKE + 4, 2), (2, FAKE + 1, 2), (8, FAKE + 2, 2), (4, 1 << 31, 5),
])
def test_gather_refusals(sv, at, value, status):  # noqa: F811
    a = [ctypes.byref(_cache(sv)), 0, FAKE, FAKE, 36, FAKE, FAKE, 1, None, None]
    a[at] = value
    assert sv.lib().spec_kv_gather(*a) == status


@pytest.mark.parametrize("at,value,status", [
    (1, None, 1), (2, 3, 1), (2, 1 << 31, 1), (3, None, 1), (4, None, 1), (5, None, 1), (6, None, 1), (1, FAKE + 4, 2),
    (3, FAKE + 2, 2), (4, FAKE + 2, 2), (5, FAKE + 2, 2), (6, FAKE + 2, 2), (7, FAKE + 2, 2), (8, FAKE + 2, 2),
])
def test_compact_refusals(sv, at, value, status):  # noqa: F811
    a = [ctypes.byref(_cache(sv)), FAKE, 36, FAKE, FAKE, FAKE, FAKE, None, None, None]
    a[at] = value
    assert sv.lib().spec_kv_compact(*a) == status


@pytest.mark.parametrize("kw,columns", [
    (dict(head_dim=256), 32), (dict(head_dim=8), 1), (dict(head_dim=256, dtype=2, k_scale=FAKE, v_scale=FAKE), 17),
    (dict(head_dim=16, dtype=2, k_scale=FAKE, v_scale=FAKE), 2),
])
def test_compact_refuses_more_columns_than_a_launch_has(sv, kw, columns):  # noqa: F811
    """A launch has 65535 CTAs of 256 threads for a sequence, one thread for each column of K and V, layer and head."""
    most = 65535 * 256 // (2 * columns)
    L = sv.lib()
    for layers, heads in ((most + 1, 1), (most // 4 + 1, 4), (1 << 18, 65535)):
        c = _cache(sv, layers=layers, kv_heads=heads, **kw)
        assert L.spec_kv_compact(ctypes.byref(c), FAKE, 36, FAKE, FAKE, FAKE, FAKE, None, None, None) == 5


@pytest.mark.parametrize("kw,status", [
    (dict(struct_size=8), 1), (dict(layer=2), 1), (dict(layer=-1), 1), (dict(q_heads=0), 1), (dict(q_heads=7), 1),
    (dict(t_max=0), 1), (dict(rows=37), 1), (dict(rows=-1), 1), (dict(row_off=None, rows=35), 1), (dict(kv_lens=None), 1),
    (dict(q=None), 1), (dict(out=None), 1), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(scale=-1.0), 1), (dict(q_token_stride=-512), 1), (dict(t_max=129, rows=36), 5),
    (dict(q=FAKE + 8), 2), (dict(q_token_stride=516), 2), (dict(out=FAKE + 8), 2), (dict(row_off=FAKE + 4), 2),
    (dict(kv_lens=FAKE + 2), 2), (dict(parent=FAKE + 1), 2), (dict(lse=FAKE + 2), 2), (dict(seq_status=FAKE + 3), 2),
    (dict(workspace=None), 3), (dict(workspace=FAKE + 16), 3), (dict(workspace_bytes=1024), 3),
])
def test_attend_refusals(sv, kw, status):  # noqa: F811
    c, a = _cache(sv), _attend(sv, **kw)
    assert sv.lib().spec_kv_attend(ctypes.byref(c), ctypes.byref(a), None) == status


def test_attend_workspace_is_host_arithmetic(sv):  # noqa: F811
    c = _cache(sv)
    n = sv.lib().spec_kv_attend_workspace_size(ctypes.byref(c), ctypes.byref(_attend(sv)))
    assert n > 0 and n % 256 == 0
    long = _cache(sv, max_blocks=1 << 20, num_blocks=1 << 24)
    assert sv.lib().spec_kv_attend_workspace_size(ctypes.byref(long), ctypes.byref(_attend(sv))) == n
    assert sv.lib().spec_kv_attend_workspace_size(ctypes.byref(c), ctypes.byref(_attend(sv, t_max=0))) == 0


def test_binding_refuses_before_the_library():
    import speculative_decoding_verification_38_gb300 as sv

    pool = torch.zeros((3, 4, 2, 64), dtype=torch.bfloat16)
    table = torch.zeros((1, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        sv.KVCache(pool, pool, table)  # not on a GPU
    with pytest.raises(ValueError):
        sv.KVCache(pool, pool[:2], table)
    with pytest.raises(TypeError):
        sv.KVCache(pool.float(), pool.float(), table)
