"""GPU parity of chunk attention at scales of either sign: signs are turned once for each part
of a tile, whether it lies in one workgroup, is cut among several, or goes on past the
16384 keys whose places are kept at a time; and at blocks' scales near the ends of
their range."""

import numpy as np
import pytest
import torch

from tests.test_gpu_chunk import Case
from tests.test_gpu_chunk_steps import check, one

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mqa_logits_amd  # noqa: F401


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "fp16")])
@pytest.mark.parametrize("scale", [-0.1, -0.02, 0.0])
@pytest.mark.parametrize("ctx,new", [([70, 1, 0, 200], [33, 1, 0, 60]), ([700, 2100], [90, 3]), ([17000], [2])])
def test_scale(ctx, new, scale, d, dtype):
    c = Case(ctx, new, 8, 2, d, 32, dtype, seed=sum(new))
    c.scale = scale
    c.check(f"scale {scale}")


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("unusual", [False, True])
def test_negative_scale_past_one_stretch(unusual, d, dtype):
    c = one(17000, 2, d, dtype, seed=d)
    c.scale = -0.05
    if unusual:                              # from a step of the first stretch on, and of the second
        for head, step in enumerate([0, 1, 100, 254, 255, 256, 257, 260]):
            page, at = c.slot(0, step * 64)
            c.vs[page, at, head, 0] = 139
    check(c, "negative scale")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("side,low,high,dtype", [("v", 200, 221, "bf16"), ("v", 0, 3, "bf16"), ("v", 0, 3, "fp16"),
                                                 ("k", 0, 3, "bf16"), ("k", 0, 3, "fp16")])
def test_blocks_scales_near_the_ends(side, low, high, dtype, d):
    c = Case([300, 1200], [70, 9], 10, 2, d, 32, dtype, seed=low + d)
    pool = c.ks if side == "k" else c.vs
    rng = np.random.default_rng(low)
    held = (pool <= 252) & (rng.random(pool.shape) < 0.3)
    pool[held] = rng.integers(low, high, held.sum())
    c.check(f"{side} scales from {low}")
