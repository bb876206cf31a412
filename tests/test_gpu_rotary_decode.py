"""A round of a model with rotary positions and a sliding window, every call together: rotating append, windowed attention,
tree verify, compaction (examples/tree_decode.py), against the same model in float64 and against one token at a time."""
import pytest

torch = pytest.importorskip("torch")
from tests.test_gpu_tree_decode import example  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def _plain(model, tokens, window, sinks):
    """Logits of every position of tokens [n], float64 but for the keys', values' and queries' rounding to bfloat16."""
    n, D, pos = len(tokens), model.head_dim, torch.arange(len(tokens), device="cuda")
    angle = pos.double()[:, None] * model.rope.inv_freq.double()
    z = torch.polar(torch.ones_like(angle), angle)[:, None]

    def turn(x):
        y = torch.view_as_complex(x.double().unflatten(-1, (2, D // 2)).transpose(-1, -2).contiguous()) * z
        return torch.view_as_real(y).transpose(-1, -2).flatten(-2).to(torch.bfloat16).double()

    see = (pos[None] <= pos[:, None]) & ((pos[:, None] - pos[None] < window) | (pos[None] < sinks))

    def attend(_, q, k, v):
        q, k, v = turn(q), turn(k).repeat_interleave(4, 1), v.double().repeat_interleave(4, 1)
        s = torch.einsum("thd,nhd->htn", q, k) * D**-0.5
        w = torch.softmax(s.masked_fill(~see, -float("inf")), -1)
        return torch.einsum("htn,nhd->thd", w, v).to(torch.bfloat16)

    return model.logits(tokens, pos, attend)


def test_one_token_at_a_time_follows_the_formula(example):  # noqa: F811
    """The decoder's next tokens are the formula's, up to where two logits nearly tie."""
    model, n, window, sinks = example.Model(rotary=True), 24, 40, 4
    prompt = torch.randint(model.vocab, (3, 150), generator=torch.Generator().manual_seed(1)).cuda()
    tokens, lead = example.one_at_a_time(model, prompt, n, window=window, sinks=sinks)
    for b in range(3):
        logits = _plain(model, torch.cat([prompt[b], tokens[b]]), window, sinks)[len(prompt[b]) - 1:-1]
        top = logits.argmax(1)
        other = (top != tokens[b]).nonzero().flatten().tolist()
        # a logit is off by a few half steps (2^-8) of outputs of its own size
        assert all(lead[b, i] < 16 * 2.0**-8 for i in other)
        assert len(other) < n // 4


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("window", [40, 1000])
def test_tree_rounds_equal_single_tokens(example, quantised, window):  # noqa: F811
    """Equal up to the first place where two tokens' logits nearly tie (as without rotation and window)."""
    model, n = example.Model(rotary=True), 40
    prompt = torch.randint(model.vocab, (5, 150), generator=torch.Generator().manual_seed(1)).cuda()
    how = dict(quantised=quantised, window=window, sinks=4)
    want, lead = (x.tolist() for x in example.one_at_a_time(model, prompt, n, **how))
    gen = torch.Generator().manual_seed(2)

    def propose(b, history, parent):
        """The true continuation on a path of the tree, up to where it is left; the rest at random."""
        at = len(history) - prompt.shape[1]
        tokens, true = [history[-1]], {0: 0}  # nodes on the true path: their depth
        for node in range(1, len(parent)):
            p = parent[node]
            token = int(torch.randint(model.vocab, (), generator=gen))
            if p in true and p not in [parent[k] for k in true if k] and at + true[p] < n and token % 4:
                true[node] = true[p] + 1
                token = want[b][at + true[p]]
            tokens.append(token)
        return tokens[1:]

    said, rounds = example.with_trees(model, prompt, n, propose, **how)
    assert rounds < n - 6  # trees were accepted
    for b in range(len(said)):
        part = next((i for i in range(n) if said[b][i] != want[b][i]), n)
        assert part == n or lead[b][part] < 16 * 2.0**-8, (b, part, lead[b][part])
