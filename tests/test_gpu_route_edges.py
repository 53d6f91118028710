"""The routing captured and replayed, and logits of +inf."""
import numpy as np
import pytest
import torch

import oracle
from few_row_quantized_amd import qgemv as q

from test_gpu_step import check_route

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu(require_gpu):
    torch.cuda.init()
    yield


@pytest.mark.parametrize("T,E,kw", [
    (5, 128, dict()), (300, 256, dict(score="sigmoid", bias=True, groups=8, keep=4, best=2, scale=2.5)),
    (70, 96, dict(renormalise=False, groups=3, keep=2))])
def test_captured_and_replayed(T, E, kw):
    """Outputs that the call allocates stay the graph's: replays with other logits,
    with eager calls between them."""
    g = torch.Generator().manual_seed(E)
    kw = dict(kw)
    if kw.get("bias"):
        kw["bias"] = 0.1 * torch.randn(E, generator=g)
    dev = {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
    x = torch.randn((T, E), generator=g).cuda()
    q.route(x, 8, **dev)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        experts, weights = q.route(x, 8, **dev)
    for i in range(4):
        new = torch.randn((T, E), generator=g)
        new[i, ::3] = -INF
        x.copy_(new)
        experts.fill_(-7)
        weights.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check_route(new, 8, experts, weights, f"replay {i} {kw}", **kw)
        e, w = q.route(x, 8, **dev)
        assert torch.equal(e, experts) and torch.equal(w, weights)


@pytest.mark.parametrize("kw,chosen", [
    (dict(), True), (dict(renormalise=False), True), (dict(score="sigmoid"), True),
    (dict(bias=torch.zeros(40)), False), (dict(groups=4, keep=2, best=2), False),
    (dict(score="sigmoid", bias=torch.zeros(40)), True)])
def test_logits_of_plus_infinity(kw, chosen):
    """Where a softmax has no values: weights NaN where the logits themselves
    choose, no expert where the scores do.  A sigmoid of it is 1."""
    x = torch.randn((3, 40), generator=torch.Generator().manual_seed(1))
    x[1, 7] = x[1, 30] = INF
    dev = {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
    experts, weights = (t.cpu() for t in q.route(x.cuda(), 4, **dev))
    ref = {n: v.double().numpy() if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
    ref["softmax"] = ref.pop("score", "softmax") == "softmax"
    with np.errstate(invalid="ignore"):
        e, w = oracle.route_reference(x.double().numpy(), 4, **ref)
    assert np.array_equal(experts.numpy(), e)
    assert (experts[1, 0] == 7) == chosen and (experts[[0, 2]] >= 0).all()
    z = weights.double().numpy()
    assert np.array_equal(np.isnan(z), np.isnan(w)) and np.isnan(z[1]).all() == (ref["softmax"] and chosen)
    ok = ~np.isnan(w)
    assert (np.abs(z[ok] - w[ok]) <= (2.0 ** -24 + 1e-12) * np.abs(w[ok])).all()
