"""Greedy decoding with token trees over the paged cache, every call of a round together.

A small random transformer (plain matrix products) decodes a batch. A round
per step: the drafter hangs a tree of candidates on each sequence's last
token; spec_kv_append writes the tree's keys and values, spec_kv_attend lets
each node see the cache and its ancestors, spec_tree_verify walks the tree on
the logits, and spec_kv_compact keeps the accepted path's entries and lengths.
With --rotary the keys are rotated on their way into the cache, the queries
beside them (spec_kv_append_rope), and with --window a token sees the latest
positions and the first few only (spec_kv_attend_window). What comes out is
what one token at a time gives, in fewer steps.

    python examples/tree_decode.py --cache e4m3 --batch 16 --tokens 128
    python examples/tree_decode.py --rotary --window 64 --sinks 4
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_38_gb300 as sv  # noqa: E402


class Model:
    """Random weights; the attention is the caller's."""

    def __init__(self, *, vocab=512, layers=2, q_heads=8, kv_heads=2, head_dim=64, seed=0, device="cuda", rotary=False):
        self.vocab, self.layers, self.q_heads, self.kv_heads, self.head_dim = vocab, layers, q_heads, kv_heads, head_dim
        width = q_heads * head_dim
        gen = torch.Generator().manual_seed(seed)
        new = lambda *shape: torch.randn(*shape, generator=gen).to(device)  # noqa: E731
        self.embed = new(vocab, width)
        self.qkv = [new(width, (q_heads + 2 * kv_heads) * head_dim) / width**0.5 for _ in range(layers)]
        self.out = [new(width, width) / width**0.5 for _ in range(layers)]
        self.freq = torch.exp(-torch.arange(0, width, 2, device=device) * (5.0 / width))
        # rotary: positions turn keys and queries; else they are added to the tokens
        self.rope = sv.Rope(10000.0 ** (-torch.arange(0, head_dim, 2, device=device) / head_dim)) if rotary else None

    def logits(self, tokens, positions, attend):
        """attend(layer, q [rows, q_heads, head_dim], k, v [rows, kv_heads, head_dim]) gives q's shape."""
        x = self.embed[tokens]
        if self.rope is None:
            angle = positions[:, None] * self.freq
            x = x + torch.cat([angle.sin(), angle.cos()], 1)
        D = self.head_dim
        for i in range(self.layers):
            y = (self._norm(x) @ self.qkv[i]).to(torch.bfloat16).view(len(x), -1, D)  # q, k and v stay one tensor
            q, k, v = y.split([self.q_heads, self.kv_heads, self.kv_heads], 1)
            x = x + attend(i, q, k, v).flatten(1).float() @ self.out[i]
        return self._norm(x) @ self.embed.t() / x.shape[1]**0.5

    @staticmethod
    def _norm(x):
        return x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)


class Decoder:
    """A batch of sequences and their cache."""

    def __init__(self, model, batch, max_len, *, quantised=False, block_size=16, seed=0, window=0, sinks=0):
        m, dev = model, model.embed.device
        self.model, self.batch, self.window, self.sinks = model, batch, window, sinks
        per = -(-max_len // block_size)
        shape = (m.layers, batch * per, block_size, m.kv_heads, m.head_dim)
        pages = torch.randperm(batch * per, generator=torch.Generator().manual_seed(seed))  # in no order
        scale = lambda: torch.empty(m.layers, batch * per, m.kv_heads, block_size, device=dev) if quantised else None  # noqa: E731
        kind = torch.float8_e4m3fn if quantised else torch.bfloat16
        self.cache = sv.KVCache(torch.empty(shape, dtype=kind, device=dev), torch.empty(shape, dtype=kind, device=dev),
                                pages.view(batch, per).to(torch.int32).to(dev), scale(), scale())
        self.lens = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.workspace = {}

    def step(self, tokens, row_off, t_max, depth, parent=None):
        """Logits of new tokens (rows of row_off) after the cache's; their entries are in the cache, self.lens is as it was."""
        m, dev = self.model, tokens.device
        counts = (row_off[1:] - row_off[:-1]).to(torch.int32)
        lens = self.lens + counts
        start = torch.repeat_interleave(self.lens, counts.long())
        out = torch.empty(len(tokens), m.q_heads, m.head_dim, dtype=torch.bfloat16, device=dev)

        def attend(layer, q, k, v):
            if m.rope is None:
                sv.check(sv.spec_kv_append(self.cache, k, v, lens, row_off, t_max, layer), "append")
            else:  # positions are the cache's own, a node's by its depth
                turned = torch.empty_like(out)
                sv.check(sv.spec_kv_append_rope(self.cache, m.rope, k, v, lens, row_off, t_max, parent=parent, q=q, q_out=turned,
                                                layer=layer), "append")
                q = turned
            args = sv.AttendArgs(cache=self.cache, q=q, out=out, kv_lens=lens, row_off=row_off, t_max=t_max,
                                 scale=m.head_dim**-0.5, parent=parent, layer=layer)
            if t_max not in self.workspace:  # one for each shape, kept
                self.workspace[t_max] = sv.Workspace.for_attend(args)
            args.set_workspace(self.workspace[t_max])
            if self.window:
                sv.check(sv.spec_kv_attend_window(args, self.window, self.sinks), "attend")
            else:
                sv.check(sv.spec_kv_attend(args), "attend")
            return out

        return m.logits(tokens, start + depth, attend), lens

    def prompt(self, tokens):
        """tokens [batch, n], in runs of what a call takes; the last position's logits."""
        for chunk in tokens.split(sv.SPEC_KV_MAX_QUERIES, 1):
            n, dev = chunk.shape[1], tokens.device
            off = torch.arange(self.batch + 1, device=dev) * n
            logits, self.lens = self.step(chunk.reshape(-1), off, n, torch.arange(n, device=dev).repeat(self.batch))
        return logits[off[1:] - 1]


def one_at_a_time(model, prompt, n, **how):
    """[batch, n] tokens, and by how much each one's logit led the next best's."""
    d = Decoder(model, len(prompt), prompt.shape[1] + n, **how)
    off = torch.arange(len(prompt) + 1, device=prompt.device)
    logits, tokens, lead = d.prompt(prompt), [], []
    for _ in range(n):
        best = logits.topk(2).values
        tokens.append(logits.argmax(1))
        lead.append(best[:, 0] - best[:, 1])
        logits, d.lens = d.step(tokens[-1], off, 1, torch.zeros_like(tokens[-1]))
    return torch.stack(tokens, 1), torch.stack(lead, 1)


def level_order(branching):
    """Parents and depths of a tree in which every node of depth i has branching[i] children."""
    parent, depth, level = [-1], [0], [0]
    for i, n in enumerate(branching):
        level = [len(parent) + j for j in range(len(level) * n)]
        for j, node in enumerate(level):
            parent.append(level[0] - len(level) // n + j // n)
            depth.append(i + 1)
    return parent, depth


def with_trees(model, prompt, n, propose, branching=(3, 2, 1), **how):
    """The same tokens by rounds over trees: [batch] lists, and the rounds they took. propose(history, parent) fills a
    tree: a token for every node but the first, which is the sequence's last one."""
    parent, depth = level_order(branching)
    N, batch, dev = len(parent), len(prompt), prompt.device
    d = Decoder(model, batch, prompt.shape[1] + n + 2 * N, **how)
    off = torch.arange(batch + 1, device=dev) * N
    parents = torch.tensor(parent * batch, dtype=torch.int32, device=dev)
    depths = torch.tensor(depth * batch, device=dev)
    out, path, accepted = (torch.empty(k, dtype=torch.int32, device=dev) for k in (batch * N, batch * N, batch))
    said = [[int(t)] for t in d.prompt(prompt).argmax(1)]
    text = [p.tolist() for p in prompt]
    rounds = 0
    while min(map(len, said)) < n:
        tokens = [[s[-1]] + propose(b, text[b] + s, parent) for b, s in enumerate(said)]
        tokens = torch.tensor(tokens, device=dev).reshape(-1)
        logits, lens = d.step(tokens, off, N, depths, parents)
        args = sv.tree_args(node_off=off, parent=parents, tokens=tokens.to(torch.int32), target=logits, out_tokens=out,
                            out_accepted=accepted, out_path=path)
        sv.check(sv.spec_tree_verify(args, greedy=True), "tree verify")
        sv.check(sv.spec_kv_compact(d.cache, off, path, accepted, lens, d.lens), "compact")
        rounds += 1
        for b, (row, k) in enumerate(zip(out.view(batch, N).tolist(), accepted.tolist())):
            if len(said[b]) < n:
                said[b] += row[:k + 1]
            else:  # done: its entries are not read again
                d.lens[b] = prompt.shape[1] + n
    return [s[:n] for s in said], rounds


def successors(vocab, seed=0):
    """A drafter: what followed a token before, the latest first, then anything."""
    gen = torch.Generator().manual_seed(seed)

    def propose(_, history, parent):
        after = {}
        for a, b in zip(history, history[1:]):
            after.setdefault(a, {}).pop(b, None)
            after[a][b] = True
        tokens, used = [history[-1]], {}
        for node in range(1, len(parent)):
            p, known = parent[node], list(reversed(after.get(tokens[parent[node]], {})))
            i = used[p] = used.get(p, -1) + 1
            tokens.append(known[i] if i < len(known) else int(torch.randint(vocab, (), generator=gen)))
        return tokens[1:]

    return propose


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--cache", choices=["bf16", "e4m3"], default="bf16")
    ap.add_argument("--batch", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--tokens", type=int, default=128)
    ap.add_argument("--rotary", action="store_true")
    ap.add_argument("--window", type=int, default=0, help="positions that a token sees (0: all)")
    ap.add_argument("--sinks", type=int, default=4, help="first positions that stay visible with a window")
    o = ap.parse_args()
    model = Model(rotary=o.rotary)
    prompt = torch.randint(model.vocab, (o.batch, o.prompt), generator=torch.Generator().manual_seed(1)).cuda()
    how = dict(quantised=o.cache == "e4m3", window=o.window, sinks=o.sinks)
    want, lead = one_at_a_time(model, prompt, o.tokens, **how)
    torch.cuda.synchronize()
    t = time.perf_counter()
    said, rounds = with_trees(model, prompt, o.tokens, successors(model.vocab), **how)
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    same = sum(s == w for s, w in zip(said, want.tolist()))
    print(f"{o.batch} sequences of {o.tokens} tokens in {rounds} rounds ({o.tokens / rounds:.2f} tokens a round, "
          f"{t / rounds * 1e3:.2f} ms a round); {same} of them equal to one token at a time (others part at a near tie)")


if __name__ == "__main__":
    main()
