"""The verify step's operators together, as the example runs them."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "verify_step.py")


@pytest.fixture(scope="module")
def example(require_gpu):
    spec = importlib.util.spec_from_file_location("verify_step", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


PROMPTS = [[1, 2, 3], [70, 80], list(range(100, 140))]


@pytest.mark.parametrize("cache,window", [(torch.bfloat16, 0), (torch.bfloat16, 40), (torch.float8_e4m3fn, 0)])
def test_drafts_change_the_speed_and_not_the_text(example, cache, window):
    """At a low temperature the text is the model's own, whatever is drafted:
    its output layer's peaks stand far above what rounding moves."""
    m = example.Decoder()
    with_drafts = example.Generation(m, PROMPTS, 3, cache, window, min(window, 4))
    alone = example.Generation(m, PROMPTS, 0, cache, window, min(window, 4))
    gained = [with_drafts.step() for _ in range(60)]
    while any(len(a) < len(b) for a, b in zip(alone.tokens, with_drafts.tokens)):
        assert alone.step() == [1, 1, 1]
    for a, b in zip(alone.tokens, with_drafts.tokens):
        assert a[:len(b)] == b
    assert all(1 <= n <= 4 for s in gained for n in s)
    assert sum(map(sum, gained)) > 1.5 * 3 * 60  # the text repeats itself, and drafts are taken


def test_the_cache_holds_the_accepted_tokens(example):
    """After drafts were refused: every accepted token's key and value, as one
    product of its embedding gives them (rows of a product do not depend on the
    others of its call beyond the last bits: one bf16 step)."""
    m = example.Decoder(seed=3)
    g = example.Generation(m, PROMPTS, 4)
    g._draft = lambda t: [(7 * t[-1] + i) % m.V for i in range(4)]  # nearly all of them refused
    gained = [g.step() for _ in range(40)]
    assert any(n == 1 for s in gained for n in s)
    Hq = m.H * m.G
    for b, (tokens, n) in enumerate(zip(g.tokens, g.cached)):
        assert len(tokens) == n + 1
        table = g.cache.table[b].long()
        for j in range(0, n, 7):
            x = m.embedding[torch.tensor([tokens[j]], device="cuda")]
            qkv = m.product(m.qkv, x).view(1, Hq + 2 * m.H, m.D)[0]
            for pages, want in ((g.cache.k, qkv[Hq:Hq + m.H]), (g.cache.v, qkv[Hq + m.H:])):
                got = pages[table[j // 16], j % 16].float()
                assert ((got - want).abs() <= 2 * 2.0 ** -8 * want.abs() + 1e-6).all(), (b, j)
