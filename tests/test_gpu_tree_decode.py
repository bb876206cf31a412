"""examples/tree_decode.py: append, attend, tree verify and compact together give what one token at a time gives."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "tree_decode.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("tree_decode", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_trees_in_level_order(example):
    assert example.level_order([3, 2, 1]) == ([-1, 0, 0, 0, 1, 1, 2, 2, 3, 3, 4, 5, 6, 7, 8, 9],
                                              [0, 1, 1, 1, 2, 2, 2, 2, 2, 2, 3, 3, 3, 3, 3, 3])
    assert example.level_order([]) == ([-1], [0])


def test_drafter_fills_a_tree(example):
    parent, _ = example.level_order([2, 1])
    assert example.successors(10)(0, [5, 1, 5, 2, 7, 5], parent) [:2] == [2, 1]  # 2 followed 5 last, 1 before it
    assert example.successors(10)(0, [5, 1, 5, 2, 7, 5], parent)[2:] == [7, 5]


@pytest.mark.gpu
@pytest.mark.parametrize("quantised", [False, True])
def test_tree_rounds_equal_single_tokens(example, quantised):
    """Equal up to the first place where two tokens' logits nearly tie: the two ways round the attention's outputs
    (bf16, half a step 2^-8) and e4m3 weights differently, so logits differ by a few such steps of their own size."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    model, n = example.Model(), 48
    prompt = torch.randint(model.vocab, (5, 150), generator=torch.Generator().manual_seed(1)).cuda()
    want, lead = example.one_at_a_time(model, prompt, n, quantised=quantised)
    want, lead = want.tolist(), lead.tolist()
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

    said, rounds = example.with_trees(model, prompt, n, propose, quantised=quantised)
    assert rounds < n - 8  # trees were accepted
    for b in range(len(said)):
        part = next((i for i in range(n) if said[b][i] != want[b][i]), n)
        assert part == n or lead[b][part] < 16 * 2.0**-8, (b, part, lead[b][part])
