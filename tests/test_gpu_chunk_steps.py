"""GPU parity of chunk attention over stretches of many steps, against float64.

A workgroup keeps the places of 64 steps of 64 keys at a time, and of 16384 keys in LDS;
it leaves its usual loop for another at the first step with a scale outside what fp16
holds.  Here every workgroup has one whole tile (256 equal ones: 32 sequences of 8 KV
heads), whose first such step differs from KV head to KV head, around the borders of
those 64 steps.  All sequences are one sequence's: they have to agree bit for bit, and
the first one's rows with the 64-bit oracle within its bounds.
"""

import numpy as np
import pytest
import torch

from oracle import cache
from tests.gpu_helpers import dev, log
from tests.test_gpu_attention import assert_within
from tests.test_gpu_chunk import FLOOR, HALF, WEIGHTS, Case

pytestmark = pytest.mark.gpu

SEQUENCES, HEADS = 32, 8
FIRST_WINDOW = [60, 61, 62, 63, 64, 126, 127, None]      # a KV head's first unusual step
SECOND_STRETCH = [62, 255, 256, 317, 318, 319, 320, None]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mqa_logits_amd  # noqa: F401


def one(ctx, new, d, dtype, seed):
    return Case([ctx], [new], 2 * HEADS, HEADS, d, 64, dtype, seed=seed, q_size=1.0)


def mark(c, steps, side, scale):
    """The scale of one key of each step, a block of it, in the pool of `side`."""
    pool = {"k": c.ks, "v": c.vs}[side]
    for head, step in enumerate(steps):
        if step is not None:
            page, at = c.slot(0, step * 64 + 5 + 7 * head)
            pool[page, at, head, head % pool.shape[-1]] = scale


def check(c, what):
    import mqa_logits_amd as mq
    log(f"[chunk] {what} ctx={c.ctx[0]} rows={len(c.q)} D={c.q.shape[2]} {c.dtype}")
    n, ctx = len(c.q), np.repeat(c.ctx, SEQUENCES)
    q = c.q.repeat(SEQUENCES, 1, 1).cuda()
    out, lse = mq.paged_chunk_attention(
        "mxfp4", q, dev(c.k), dev(c.ks), dev(c.v), dev(c.vs), dev(ctx),
        dev(np.arange(SEQUENCES + 1, dtype=np.int32) * n), dev(np.repeat(c.table, SEQUENCES, 0)), c.max_ctx,
        scale=c.scale, return_lse=True)
    torch.cuda.synchronize()
    with np.errstate(all="ignore"):
        ref, ref_lse, tol, tol_lse = cache.attend_rows(
            c.q.double().numpy(), c.k, c.ks, c.v, c.vs, c.table, *c.rows(), c.scale, HALF[c.dtype], WEIGHTS,
            weight_floor=FLOOR)
    assert_within(out[:n].double().cpu().numpy(), ref, tol, what + " out")
    assert_within(lse[:n].double().cpu().numpy(), ref_lse, tol_lse, what + " lse")
    for x in (out, lse):
        x = x.unflatten(0, (SEQUENCES, n)).nan_to_num(nan=3e4)
        assert bool((x == x[:1]).all())
    return out[:n]


@pytest.mark.parametrize("ctx", [64, 4096, 4097, 4220, 8960])
@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16")])
def test_usual_scales(d, dtype, ctx):
    check(one(ctx, 5, d, dtype, seed=ctx), "usual scales")


# (a K scale that bf16 does not hold is NaN, and takes the whole row with it)
@pytest.mark.parametrize("d,dtype,side,scale", [
    (64, "fp16", "v", 139), (64, "bf16", "v", 140), (128, "fp16", "v", 100), (128, "bf16", "v", 139),
    (64, "fp16", "k", 90), (128, "fp16", "k", 100), (128, "bf16", "v", 255), (64, "fp16", "v", 254),
])
def test_first_unusual_step(d, dtype, side, scale):
    c = one(8960, 5, d, dtype, seed=scale + d)
    mark(c, FIRST_WINDOW, side, scale)
    assert torch.isnan(check(c, f"{side} scale {scale}")).any() == (scale > 252)


@pytest.mark.parametrize("d,dtype,side,scale", [(64, "fp16", "k", 90), (128, "bf16", "v", 139)])
def test_first_unusual_step_of_long_contexts(d, dtype, side, scale):
    c = one(20990, 2, d, dtype, seed=scale + d)
    mark(c, SECOND_STRETCH, side, scale)
    check(c, f"{side} scale {scale}")


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16")])
def test_few_keys_after_the_exit(d, dtype):
    """70 steps: the places of the last one stand in for those behind it."""
    c = one(4420, 5, d, dtype, seed=d)
    mark(c, [60, 61, 62, 63, 64, 67, 68, 69], "v", 139)
    check(c, "few keys after the exit")
