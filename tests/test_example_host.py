"""The example's limits (no GPU): sequences end where their pages do."""
import importlib.util
import os

import pytest

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "verify_step.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("verify_step", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.fixture(scope="module")
def model(example):
    return example.Decoder(device="cpu")


def test_prompts_longer_than_the_pages_are_refused(example, model):
    with pytest.raises(ValueError, match="sequence 1 has pages for 32 tokens"):
        example.Generation(model, [[1], list(range(33))], 3, longest=20)


def test_a_step_without_a_place_for_its_token_is_refused(example, model):
    g = example.Generation(model, [[1], [2]], 3, longest=16)
    g.tokens[1], g.cached[1] = list(range(17)), 16
    before = [list(t) for t in g.tokens], list(g.cached)
    g._layer = lambda rows, lens: pytest.fail("the step was taken")
    with pytest.raises(ValueError, match="sequence 1 has pages for 16 tokens"):
        g.step()
    assert before == (g.tokens, g.cached)


def test_drafts_end_with_the_pages(example, model):
    class Taken(Exception):
        pass

    def layer(rows, lens):
        seen.append((rows, lens))
        raise Taken

    for cached, drafts in ((12, 3), (13, 2), (14, 1), (15, 0)):
        seen = []
        g = example.Generation(model, [[1]], 3, longest=16)
        g.tokens[0], g.cached[0] = [7] * (cached + 1), cached
        g._draft = lambda t: [7, 7, 7]
        g._layer = layer
        with pytest.raises(Taken):
            g.step()
        assert seen == [([[7] * (drafts + 1)], [cached + drafts + 1])]
