"""The served batch's prefill (no GPU): which tokens enter the cache, and where."""
import importlib.util
import os
import sys

import pytest

FOLDER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, FOLDER)
    spec = importlib.util.spec_from_file_location("served_batch", os.path.join(FOLDER, "served_batch.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("share", [True, False])
@pytest.mark.parametrize("system,prompts", [
    (100, [3, 2, 10]), (100, [1, 0, 5]), (96, [3, 1, 2]), (96, [0, 2, 4]), (96, [2, 0, 0]), (32, [0]), (16, [0, 0]),
    (5, [1, 2]), (5, [0, 40]), (0, [1, 3])])
def test_every_token_but_the_last_enters_once(example, system, prompts, share):
    fed = []

    class Batch(example.ServedBatch):
        def _layer(self, rows, lens):
            for b, (r, n) in enumerate(zip(rows, lens)):
                fed.extend((b, n - len(r) + i, t) for i, t in enumerate(r))

    words = list(range(1000, 1000 + system))
    model = example.ServedDecoder(device="cpu")
    g = Batch(model, words, [list(range(100 * b, 100 * b + n)) for b, n in enumerate(prompts)], [0] * len(prompts),
              share=share, drafts=1)
    assert g.cached == [len(t) - 1 for t in g.tokens]
    places = {}
    for b, at, token in fed:
        assert at < len(g.tokens[b]) - 1 and g.tokens[b][at] == token
        slot = (int(g.cache.table[b, at // 16]), at % 16)
        assert slot not in places  # no token twice, no two in one place
        places[slot] = token
    for b, t in enumerate(g.tokens):
        for at, token in enumerate(t[:-1]):
            assert places[int(g.cache.table[b, at // 16]), at % 16] == token
