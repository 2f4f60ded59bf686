"""The attention half's operators on the GPU at values where a rounding, a
mask or a range can go wrong: NaN, infinities, numbers at both ends of fp32's
range, scales far apart, and entries that a call may not use."""

import math

import pytest
import torch

from tests import attn_reference as R
from tests.test_gpu_attn import DT, check_append, gen, i32, make_cache, make_table, make_weights, normal, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture(scope="module")
def m():
    import moe_decode_layer_sm_b200
    return moe_decode_layer_sm_b200


def bits(t):
    return t.view(torch.uint8) if t.dtype == R.FP8 else t


# --------------------------------------------------------------------- append

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rot", [None, (64, 0, False), (32, 32, False), (32, 0, True), (6, 10, False)])
@pytest.mark.parametrize("d,page", [(64, 16), (64, 128), (128, 128)])   # 1, 2 and 4 units of 16 values a thread
def test_append_nan_stays_nan(m, dtype, rot, d, page):
    """A NaN with no infinity beside it, in values, in keys that are rotated and
    in dimensions that are not; both signs; a head of nothing else."""
    rope = None if rot is None else m.Rope(rot[0], offset=rot[1], interleaved=rot[2])
    k, v = (normal((1, page, 4, d), DT[dtype], 300 + i) for i in (0, 1))
    for x in (k, v):
        x[0, 3, 0, 5] = math.nan
        x[0, page - 1, 1, d - 1], x[0, 0, 1, 40] = -math.nan, math.nan
        x[0, :, 2] = math.nan
    check_append(m, dtype, [page], [page], page, 4, d, page, rope, k=k, v=v)
