"""Attention over a shared prefix where scores have no sign or no size, queries
are not finite, and values that some rows see are not."""
import numpy as np
import pytest
import torch

from few_row_quantized_amd import qgemv as q

from kv_util import KvDevice
from test_gpu_shared import BF, F8, HF, TYPES, parity, problem, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu(require_gpu):
    torch.cuda.init()
    yield


SHAPES = [(BF, BF, 128), (HF, HF, 64), (BF, F8, 128), (HF, F8, 256), (BF, BF, 256), (BF, F8, 64)]


@pytest.mark.parametrize("qt,ct,D", SHAPES)
@pytest.mark.parametrize("scale", [-0.1, 0.0, -0.0, 1e-4, -2.0, 1.5])
def test_scales(qt, ct, D, scale):
    """Of either sign, none, small and large."""
    p = problem(160, [3, 4, 2], [300, 100, 170], H=2, G=3, D=D, page=16, q_dtype=qt, dtype=ct, seed=21)
    p.scale = scale
    parity(p, 160, f"scale={scale} {ct} D={D}")


@pytest.mark.parametrize("D", [64, 128])
def test_a_head_without_a_scale_and_one_of_the_other_sign(D):
    p = problem(160, [3, 4, 2], [300, 100, 170], H=3, G=2, D=D, page=16, dtype=F8, seed=22)
    p.k_scale[0], p.k_scale[2] = 0.0, -0.25
    parity(p, 160, f"k_scale D={D}")


def same_kind(got, want):
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(np.isposinf(got), np.isposinf(want)) and np.array_equal(np.isneginf(got), np.isneginf(want))


def check_the_finite(p, out, lse, ref, label):
    """The rows without strays have their usual bound."""
    ok = np.isfinite(ref["out"])
    clean = out.clone()
    clean[torch.from_numpy(~ok).cuda()] = 0
    for k in ("out", "mass"):
        ref[k][~ok] = 0
    ref["size"][~np.isfinite(ref["size"])] = 0
    z = lse.clone()
    none = torch.from_numpy(~np.isfinite(ref["lse"])).cuda()
    z[none] = 0
    ref["lse"][~np.isfinite(ref["lse"])] = 0
    ref["top"] = float(np.nanmax(np.abs(p.v.float().numpy()[np.isfinite(p.v.float().numpy())])))
    p.check(clean, z, ref, label)


@pytest.mark.parametrize("qt,ct,D", SHAPES)
@pytest.mark.parametrize("scale", [0.1, -0.1, 0.0])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_queries_that_are_not_finite(qt, ct, D, scale, value):
    """One head of a row each: of a sequence past the prefix, of one that ends
    within it (whose rows see common tokens alone) and of one right after it."""
    p = problem(160, [3, 4, 2], [300, 100, 161], H=2, G=3, D=D, page=16, q_dtype=qt, dtype=ct, seed=23)
    p.scale = scale
    for t, hq, d in ((1, 0, 5), (4, 4, D - 1), (7, 2, D // 2)):
        p.q[t, hq, d] = value
    with np.errstate(invalid="ignore"):
        ref = p.reference()
    d = KvDevice(p)
    out, lse = run(d, 160)
    assert np.isnan(ref["out"]).all(-1).sum() == 3
    same_kind(out.double().cpu().numpy(), ref["out"])
    same_kind(lse.double().cpu().numpy(), ref["lse"])
    check_the_finite(p, out, lse, ref, f"{value} {ct} D={D}")
    alone = q.attend(d.cache, d.q, d.start, d.len, p.M, scale=scale)
    assert torch.equal(alone.isnan(), out.isnan())


@pytest.mark.parametrize("qt,ct", TYPES)
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("window,sinks", [(60, 2), (0, 0)])
def test_values_that_only_some_rows_see(qt, ct, D, window, sinks):
    """NaNs and infinities in common tokens reach exactly the rows that see them:
    a window hides them from some, from others their sequence's end."""
    p = problem(192, [4, 1, 3, 2, 3], [230, 300, 245, 188, 150], H=2, G=3, D=D, page=16, q_dtype=qt, dtype=ct,
                window=window, sinks=sinks, seed=24)
    v = p.v.float()
    inf = float("nan") if ct == F8 else float("inf")
    for token, d, value in ((1, 1, inf), (148, 9, inf), (175, D - 1, float("nan")), (186, 17, inf), (187, 33, -inf), (190, 62, -inf)):
        v[int(p.table[0, token // 16]), token % 16, 1, d] = value
    p.v.copy_(v.to(p.v.dtype))
    with np.errstate(invalid="ignore"):
        ref = p.reference()
    out, lse = run(KvDevice(p), 192)
    assert (~np.isfinite(ref["out"])).any() and np.isfinite(ref["out"]).any()
    same_kind(out.double().cpu().numpy(), ref["out"])
    check_the_finite(p, out, lse, ref, f"strays {ct} D={D} window={window}")
