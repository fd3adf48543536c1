"""Seeded random calls of chunk attention, gathered weights and eviction against the 64-bit
oracle: lengths, new tokens (decoding, drafts, prompts, mixed), head layouts, types, block
sizes, bounds, rows that the buffer lacks or that nobody has, scales of either sign, blocks'
scales outside fp16 and NaN, free lists that end early, pools of any width."""

import os

import numpy as np
import pytest
import torch

from tests.test_gpu_chunk import Case
from tests.test_gpu_chunk_cut_rows import check as check_chunk
from tests.test_gpu_evict import POOLS, case as evict_case, check as check_evict
from tests.test_gpu_gathered import check as check_weights

pytestmark = pytest.mark.gpu
# more seeds for a longer sweep
SCALE = int(os.environ.get("MQA_RANDOM_CASES", "1"))


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mqa_logits_amd  # noqa: F401


def spread(rng, lo, hi):
    return int(round(np.exp(rng.uniform(np.log(lo), np.log(hi)))))


def draw(rng, most, pairs):
    """Contexts of up to `most` keys, up to `pairs` (row, head, key) triples."""
    while True:
        batch, size = spread(rng, 1, 40), spread(rng, 1 if rng.random() < 0.4 else 500, most)
        ctx = rng.integers(0, size + 1, batch)
        kind = rng.integers(4)
        new = [ctx, np.full(batch, rng.integers(1, 17)), rng.integers(0, 301, batch),
               np.where(rng.random(batch) < 0.2, rng.integers(1, 400, batch), 1)][kind]
        new = new if rng.random() < 0.1 else np.minimum(new, ctx)
        hkv, group = int(rng.choice([1, 1, 2, 3, 4, 8])), int(rng.choice([1, 2, 3, 4, 5, 8, 16, 33, 64]))
        if ctx.sum() <= 20000 and hkv * group <= 256 and new.sum() > 0 and (new * ctx).sum() * hkv * group <= pairs:
            break
    d, dtype = int(rng.choice([64, 128])), str(rng.choice(["bf16", "fp16"]))
    max_ctx = None if rng.random() < 0.6 else max(1, int(size * rng.uniform(0.3, 2)))
    c = Case(ctx, new, hkv * group, hkv, d, int(rng.choice([16, 32, 64])), dtype, max_ctx=max_ctx,
             seed=int(rng.integers(1 << 30)), q_size=1.0, pad=int(rng.integers(0, 5)) * (rng.random() < 0.3))
    if rng.random() < 0.3:
        c.q = c.q[:max(1, int(len(c.q) * rng.random()))].clone()
    if rng.random() < 0.3:
        c.scale = -c.scale
    if rng.random() < 0.4:
        for pool, values in ((c.vs, [100, 104, 137, 139, 140]), (c.ks, [60, 100, 104])):
            at = (pool <= 252) & (rng.random(pool.shape) < rng.choice([0.0, 0.001, 0.2]))
            pool[at] = rng.choice(values, at.sum())
    if rng.random() < 0.2:
        for pool in (c.vs, c.ks):
            at = (pool <= 252) & (rng.random(pool.shape) < 1e-4)
            pool[at] = rng.integers(253, 256, at.sum())
    return c


@pytest.mark.parametrize("seed", range(40 * SCALE))
def test_chunk(seed):
    check_chunk(draw(np.random.default_rng(seed), 9000, 1e9), f"random {seed}")


@pytest.mark.parametrize("seed", range(30 * SCALE))
def test_weights(seed):
    rng = np.random.default_rng(1000 + seed)
    check_weights(draw(rng, 6000, 1e7), f"random {seed}", before=rng.random() < 0.7)


@pytest.mark.parametrize("seed", range(30 * SCALE))
def test_evict(seed):
    rng = np.random.default_rng(2000 + seed)
    batch, size = spread(rng, 1, 200), spread(rng, 1, 60000)
    size = min(size, 150000 // batch)
    ctx, keep = rng.integers(0, size + 1, batch), spread(rng, 1, size)
    c = evict_case(ctx, keep, int(rng.integers(0, keep + 1)) if rng.random() < 0.8 else keep, int(rng.choice([16, 32, 64])),
                   str(rng.choice(list(POOLS))), max_ctx=None if rng.random() < 0.6 else max(1, int(size * rng.uniform(0.5, 2))),
                   seed=seed, free=None if rng.random() < 0.7 else int(rng.integers(0, batch * (keep // 16 + 1) + 1)))
    w = c["weights"]
    if rng.random() < 0.3:
        w[rng.random(w.shape) < 0.5] = -np.inf
    if rng.random() < 0.2:
        w[:] = rng.integers(0, 2 ** 32, w.shape, dtype=np.uint32).view(np.float32)
    check_evict(c)
