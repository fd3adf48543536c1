"""GPU parity of gathered weights where the keys are divided among workgroups: sequences
that a share crosses, more than a scan holds, without rows or with very many, units and
spans that follow one another, and scales of either sign."""

import numpy as np
import pytest
import torch

from tests.test_gpu_chunk import Case
from tests.test_gpu_gathered import check, gather, true_lse

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mqa_logits_amd  # noqa: F401


def ragged(batch, most, new, seed):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, most + 1, batch)
    ctx[rng.integers(0, batch, batch // 8)] = 0
    return ctx, np.minimum(ctx, rng.integers(0, new + 1, batch))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("batch,most,max_ctx,new,hq,hkv", [
    (64, 3000, None, 2, 8, 4),               # few rows, shares of several sequences
    (300, 600, 2000, 2, 8, 1),               # more sequences than threads
    (64, 900, 5000, 3, 6, 2),
    (300, 500, None, 10, 8, 1),              # many rows
    (40, 2500, None, 12, 16, 2),
])
def test_ragged(batch, most, max_ctx, new, hq, hkv, d, dtype):
    ctx, new = ragged(batch, most, new, seed=batch + d)
    check(Case(ctx, new, hq, hkv, d, 32, dtype, max_ctx=max_ctx, seed=batch), "ragged")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("ctx,new,hq,hkv", [
    ([100] * 10 + [700] + [50] * 9, [1] * 10 + [40] + [1] * 9, 8, 1),        # few rows but for one sequence
    ([4000] * 19 + [4100], [1] * 19 + [40], 8, 1),
    ([2500, 600, 90], [300, 0, 5], 8, 2),    # parts of 256 rows, of none
    ([700, 700], [700, 650], 4, 2),          # prompts
    ([700, 40], [700, 40], 6, 3),
    ([9000], [64], 16, 4),                   # several spans, rows cut up
    ([2600], [200], 5, 5),                   # 200 rows of five heads
    ([1500, 1400], [20, 33], 24, 8),         # heads that share a unit
])
def test_rows(ctx, new, hq, hkv, dtype):
    check(Case(ctx, new, hq, hkv, 128, 64, dtype, seed=sum(new)), "rows")


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("scale", [-0.1, -0.02, 0.0])
def test_scales(scale, new):
    c = Case([700, 300, 1000], [new] * 3, 8, 2, 64, 16, "bf16", seed=3)
    c.scale = scale
    check(c, f"scale {scale}")


@pytest.mark.parametrize("d", [64, 128])
def test_key_scales_outside_fp16_among_many_rows(d):
    c = Case([700, 2100], [80, 90], 8, 2, d, 16, "fp16", seed=4)
    c.ks[c.table[1, 60], :, 0] = 90          # some keys of one head, 64 of 2100
    c.ks[c.table[1, 3], 5, 1, 0] = 139
    check(c, "K's scales")


def test_the_same_again_and_wherever_it_lies():
    """A sequence's sums do not depend on what else is in the batch, where it has one unit."""
    ctx, new = [3000, 64, 1700, 2900], [3, 3, 3, 3]
    for hq, hkv in ((64, 1), (8, 1), (16, 4)):
        c = Case(ctx, new, hq, hkv, 128, 64, "bf16", seed=8)
        lse = true_lse(c).cuda()
        once, again = gather(c, lse), gather(c, lse)
        assert torch.equal(once, again)
        swapped = [3, 1, 2, 0]
        rows = np.concatenate([np.arange(c.offsets[b], c.offsets[b + 1]) for b in swapped])
        c.ctx, c.table, c.q = c.ctx[swapped], c.table[swapped], c.q[rows]
        other = gather(c, lse[torch.from_numpy(rows).cuda()])
        for at, b in enumerate(swapped):
            assert torch.equal(other[at], once[b])
