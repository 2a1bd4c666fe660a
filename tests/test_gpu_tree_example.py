"""The operators together: the example's drafted trees give the text of decoding token by token."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("beams,depth", [(4, 3), (2, 6), (10, 3), (1, 5)])
def test_trees_give_greedy_text(beams, depth):
    """Every token is the largest logit of the text before it, read as one chain without a cache, up to the rounding of
    the activations: some 16 roundings to bf16 of half a step, 2^-8, each."""
    import draft_tree as E

    model = E.Target(seed=1)
    texts, lens = E.generate(seed=1, rounds=12, beams=beams, depth=depth, model=model)
    for t, n in zip(texts, lens):
        short, size = E.shortfalls(model, t)
        assert max(short) <= 16 * 2.0 ** -8 * size
        assert n == len(t) - 1          # all but the last token are in the cache
    assert sum(len(t) - 1 for t in texts) > 12 * len(texts)  # some drafts were accepted


def test_single_steps_give_greedy_text():
    import draft_tree as E

    model = E.Target(seed=3)
    texts, lens = E.generate(seed=3, rounds=30, drafts=False, model=model)
    for t, n in zip(texts, lens):
        short, size = E.shortfalls(model, t)
        assert max(short) <= 16 * 2.0 ** -8 * size and n == len(t) - 1 == 30


def test_eviction_bounds_the_caches():
    import draft_tree as E

    text, lens = E.generate(seed=2, rounds=30, keep=32)
    assert all(n <= 32 + 16 + 4 for n in lens) and all(len(t) > 30 for t in text)
