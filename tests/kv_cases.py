"""Inputs of the cache tests and the float64 side of their comparison."""
import math

import numpy as np
import torch

from oracle import kv as okv


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


class Case:
    """A paged cache with each sequence's pages anywhere in the pool, NaN (or the NaN code) in every slot that holds
    no position, and new tokens at the end of each sequence."""

    def __init__(self, *, lens, tokens, H=2, G=1, D=64, bs=16, dtype="bf16", order="nhd", layers=1, layer=0, seed=0,
                 parent=None, pad=0, q_scale=1.0, spare=2, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.g, self.H, self.G, self.D, self.bs, self.dtype, self.layers, self.layer = g, H, G, D, bs, dtype, layers, layer
        self.lens, self.tokens, self.B = list(lens), list(tokens), len(lens)
        self.rows = sum(self.tokens)
        self.t_max = max(1, max(self.tokens))
        self.row_off = np.concatenate([[0], np.cumsum(self.tokens)]).astype(np.int64)
        need = [-(-n // bs) for n in self.lens]
        pages = sum(need) + spare
        perm = torch.randperm(pages, generator=g).numpy().astype(np.int32)
        self.max_blocks = max(1, max(need))
        self.table = np.full((self.B, self.max_blocks), -5, np.int32)  # past the last page: never read
        at = 0
        held = np.zeros((pages, bs), dtype=bool)
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
            for j in range(self.lens[b]):
                held[self.table[b, j // bs], j % bs] = True
        self.held = held
        shape = (layers, pages, bs, H, D)
        self.k, self.v = (self._pool(shape, order, pad) for _ in range(2))
        self.ks = self.vs = None
        if dtype == "e4m3":
            self.ks, self.vs = (torch.exp2(torch.randn((layers, pages, H, bs), generator=g) - 4) for _ in range(2))
        self.q = (torch.randn((self.rows, H * G, D), generator=g) * q_scale).to(torch.bfloat16)
        self.parent = None if parent is None else np.asarray(parent, np.int32)
        self.scale = 1 / math.sqrt(D)
        self.device = device

    def _pool(self, shape, order, pad):
        layers, pages, bs, H, D = shape
        x = torch.randn(shape, generator=self.g)
        if self.dtype == "e4m3":
            x = (x * 90).clamp(-448, 448)
        x[:, torch.from_numpy(~self.held)] = float("nan")
        x = x.to(torch.bfloat16 if self.dtype == "bf16" else torch.float8_e4m3fn)
        # the wanted axis order, with `pad` elements between a row and the next
        room = torch.zeros((layers, pages, bs, H, D + pad) if order == "nhd" else (layers, pages, H, bs, D + pad),
                           dtype=torch.uint8 if self.dtype == "e4m3" else x.dtype)
        view = (room if order == "nhd" else room.transpose(2, 3))[..., :D]
        view.copy_(x.view(torch.uint8) if self.dtype == "e4m3" else x)
        self._rooms = getattr(self, "_rooms", []) + [(room, order, D)]
        return view

    # ---- the CUDA side
    def device_pool(self, i):
        room, order, D = self._rooms[i]
        room = room.to(self.device)
        if self.dtype == "e4m3":
            room = room.view(torch.float8_e4m3fn)
        return (room if order == "nhd" else room.transpose(2, 3))[..., :D]

    def to_device(self, sv):
        dev = self.device
        self.dk, self.dv = self.device_pool(0), self.device_pool(1)
        self.dks = None if self.ks is None else self.ks.to(dev)
        self.dvs = None if self.vs is None else self.vs.to(dev)
        self.dtable = torch.from_numpy(self.table).to(dev)
        self.dlens = torch.tensor(self.lens, dtype=torch.int32, device=dev)
        self.doff = torch.from_numpy(self.row_off).to(dev)
        self.cache = sv.KVCache(self.dk, self.dv, self.dtable, k_scale=self.dks, v_scale=self.dvs)
        return self.cache

    # ---- the float64 side
    def raw(self, x):
        """A pool as the oracle takes it: uint8 codes or float64 values."""
        return np.ascontiguousarray(x.cpu().view(torch.uint8).numpy() if self.dtype == "e4m3" else x.cpu().double().numpy())

    def host(self):
        return (self.raw(self.k), self.raw(self.v), None if self.ks is None else self.ks.numpy().copy(),
                None if self.vs is None else self.vs.numpy().copy())

    def expected(self):
        k, v, ks, vs = self.host()
        return okv.attend(self.q.double().numpy(), k, v, ks, vs, self.table, self.layer, self.row_off, self.lens,
                          self.scale, self.parent)

    def attend(self, sv, *, offsets=True, lse=True, q=None, status=True, stream=None):
        if not hasattr(self, "cache"):
            self.to_device(sv)
        dev = self.device
        q = self.q.to(dev) if q is None else q
        self.out = torch.full((self.rows, self.H * self.G, self.D), 7.0, dtype=torch.bfloat16, device=dev)
        self.lse = torch.full((self.rows, self.H * self.G), 7.0, dtype=torch.float32, device=dev) if lse else None
        self.status = torch.full((self.B,), -7, dtype=torch.int32, device=dev) if status else None
        parent = None if self.parent is None else torch.from_numpy(self.parent).to(dev)
        args = sv.AttendArgs(cache=self.cache, q=q, out=self.out, kv_lens=self.dlens,
                             row_off=self.doff if offsets else None, t_max=self.t_max, scale=self.scale, parent=parent,
                             lse=self.lse, layer=self.layer, seq_status=self.status)
        args.set_workspace(sv.Workspace.for_attend(args, stream=stream))
        self.args = args
        sv.check(sv.spec_kv_attend(args, stream), "spec_kv_attend")
        return args

    def bound(self, out, av, mag, spread):
        """How far an output may be from the float64 one, from the kernels' roundings:
        - the output's rounding to bf16: half a step of it;
        - a score's float32 sum of D products, its scaling and the exponential: a relative error of the weight of
          at most es = 2^-23 (D + 8) * (the largest sum of |q k| terms) + 2^-20, in numerator and denominator;
        - a weight held in 16 bits or as two parts of 8 (a half step of fp16 is 2^-11, relative) and float32 sums over
          the positions: (2^-11 + L 2^-23) of the mean |v|;
        - weights below fp16's range: at most 2^-30 of the largest weight each.
        """
        es = 2.0**-23 * (self.D + 8) * mag + 2.0**-20
        L = max(self.lens)
        return (half_step(torch.bfloat16) * np.abs(out) + (2 * es[..., None] + 2.0**-11 + L * 2.0**-23) * av
                + 2.0**-30 * spread[..., None] + 1e-30)

    def check(self, got=None):
        out, lse, av, mag, spread = self.expected()
        got = self.out if got is None else got
        g = got.double().cpu().numpy()
        far = np.abs(g - out) - self.bound(out, av, mag, spread)
        assert not np.isnan(g).any() or np.isnan(out).any(), "NaN where none is due"
        assert (far <= 0).all(), (float(far.max()), np.unravel_index(np.nanargmax(far), far.shape))
        if self.lse is not None:
            gl = self.lse.double().cpu().numpy()
            assert np.array_equal(np.isinf(gl), np.isinf(lse))
            fin = np.isfinite(lse)
            es = 2.0**-23 * (self.D + 8) * mag + 2.0**-20
            assert (np.abs(gl - lse)[fin] <= (es + 2.0**-21 * (1 + np.abs(lse)) + max(self.lens) * 2.0**-24)[fin]).all()


def tree(branching):
    """Parents in level order."""
    parent, level = [-1], [0]
    for n in branching:
        start = len(parent)
        parent += [u for u in level for _ in range(n)]
        level = list(range(start, len(parent)))
    return parent


def random_tree(n, seed):
    r = np.random.default_rng(seed)
    return [-1] + [int(r.integers(0, v)) for v in range(1, n)]
