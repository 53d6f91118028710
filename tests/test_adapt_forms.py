"""The shapes of the adapters' GPU tests against the plan (no GPU)."""
import itertools

import torch

from few_row_quantized_amd import qgemv as q

from adapt_util import FORMS, whole_numbers
from kernel_config import adapt_plan
from kernel_objects import instances

CUS = 256  # of an MI355X


def planned():
    """Every form that a call can take, over sizes on both sides of each border."""
    rows = [1, 2, 5, 8, 12, 16, 17, 24, 31, 32, 33, 48, 63, 64, 65, 96, 100, 128, 130, 192, 200, 256, 320, 384, 448, 511, 512]
    adapters = [1, 2, 3, 4, 6, 7, 8, 10, 12, 16, 24, 32, 64, 100, 256, 257, 5000]
    columns = [1, 256, 1000, 4096, 6144, 8192, 11000, 16384, 17408, 27000, 44000, 65536, 131072, 1 << 22]
    return {adapt_plan(T, n, r, 4096, N, CUS)
            for T, n, r, N in itertools.product(rows, adapters, range(8, 257, 16), columns)}


def test_the_shapes_reach_every_form():
    """The first product's kernels (all but the last number) and the second's
    (all but the ranks of the first)."""
    want, got = planned(), {adapt_plan(*s, CUS) for s in FORMS}
    assert {p[:3] for p in want} == {p[:3] for p in got}
    assert {(p[0], p[1], p[3]) for p in want} == {(p[0], p[1], p[3]) for p in got}


def test_the_library_has_these_kernels_and_no_others():
    want = planned()
    for dtype in (0, 1):
        assert ({i[1:] for i in instances(q.LIB_PATH, "adapt_down_kernel") if i[0] == dtype}
                == {p[:3] for p in want})
        assert ({i[1:] for i in instances(q.LIB_PATH, "adapt_up_kernel") if i[0] == dtype}
                == {(p[0], p[1], p[3]) for p in want})


def test_two_parts_would_not_hold_the_sums():
    """That the GPU test of whole numbers sees a missing part: two parts of bf16
    have 16 to 18 bits of 24, one of fp16 11 to 12."""
    v = whole_numbers(20, 2, 16, 256, torch.bfloat16, 1)[-1].double()
    first = v.bfloat16().double()
    second = (v - first).bfloat16().double()
    third = (v - first - second).bfloat16().double()
    assert (first + second + third == v).all() and (first + second != v).double().mean() > 0.9
    scaled = v * 2.0 ** -10  # the largest between 2^13 and 2^14
    one = scaled.half().double()
    two = one + (scaled - one).half().double()
    assert ((scaled - two).abs() <= 2.0 ** -23 * scaled.amax(1, keepdim=True)).all()
    assert not ((scaled - one).abs() <= 2.0 ** -23 * scaled.amax(1, keepdim=True)).all()
