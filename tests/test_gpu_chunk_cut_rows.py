"""GPU parity of calls whose offsets go past the rows of q: paged_kv_slots lays out more new
tokens than the step's buffers hold, and the rows from their end on are passed over.

Contexts are long enough for tiles to be cut among workgroups, several KV heads make
workgroups go from one head's tiles to the next's.  Rows are compared with the 64-bit
oracle: those at the borders of tiles and of the cut, and some others.
"""

import numpy as np
import pytest
import torch

from oracle import cache
from tests.gpu_helpers import dev, log
from tests.test_gpu_attention import assert_within
from tests.test_gpu_chunk import FLOOR, HALF, WEIGHTS, Case
from tests.test_gpu_gathered import check as check_weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mqa_logits_amd  # noqa: F401


def some_rows(c):
    """First and last rows of sequences and of tiles, and every 41st."""
    sequence, _ = c.rows()
    per = 256 // min(c.q.shape[1] // c.k.shape[2], 256)
    rows = []
    for b in range(len(c.ctx)):
        mine = np.flatnonzero(sequence == b)
        for t in range(0, len(mine), per):
            rows += [mine[t], mine[min(t + per, len(mine)) - 1]]
        rows += mine[::41].tolist()
    return np.unique(rows)


def check(c, what):
    log(f"[chunk] {what} ctx={c.ctx[:4]}.. offsets={c.offsets[:5]}.. rows={len(c.q)} "
        f"heads={c.q.shape[1]}/{c.k.shape[2]} D={c.q.shape[2]} {c.dtype}")
    # rows behind what the call is given of the buffers stay as they are
    out = torch.full((len(c.q) + 2, *c.q.shape[1:]), 7.0, dtype=c.q.dtype, device="cuda")
    lse = torch.full(out.shape[:2], 9.0, device="cuda")
    c.run(out=out[:-2], lse=lse[:-2])
    torch.cuda.synchronize()
    assert bool((out[-2:] == 7.0).all()) and bool((lse[-2:] == 9.0).all())
    at = some_rows(c)
    sequence, seen = c.rows()
    with np.errstate(all="ignore"):
        ref, ref_lse, tol, tol_lse = cache.attend_rows(
            c.q[at].double().numpy(), c.k, c.ks, c.v, c.vs, c.table, sequence[at], seen[at], c.scale,
            HALF[c.dtype], WEIGHTS, weight_floor=FLOOR)
    assert_within(out[at].double().cpu().numpy(), ref, tol, what + " out")
    assert_within(lse[at].double().cpu().numpy(), ref_lse, tol_lse, what + " lse")


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("ctx,new,rows,hq,hkv", [
    ([2359], [219], 97, 64, 8),
    ([4000], [256], 130, 8, 8),              # one tile, half of it
    ([1500, 900, 2000], [100, 219, 300], 181, 16, 2),    # within the second; the third has none
    ([700, 3000], [0, 700], 1, 12, 4),
    ([5000, 5000], [64, 500], 64 + 500 - 1, 4, 4),
    ([200, 2000], [300, 900], 411, 8, 2),    # more new tokens than the context
])
def test_rows_behind_the_buffer(ctx, new, rows, hq, hkv, d, dtype):
    c = Case(ctx, new, hq, hkv, d, 32, dtype, seed=rows, max_ctx=max(ctx) - 150)
    c.q = c.q[:rows].clone()
    check(c, "cut off")
    c = Case(ctx, new, hq, hkv, d, 32, dtype, seed=rows)
    c.q = c.q[:rows].clone()
    check(c, "cut off, whole contexts")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_tokens_of_a_step_that_holds_fewer(dtype):
    """Offsets from paged_kv_slots, whose total passes max_tokens."""
    import mqa_logits_amd as mq
    c = Case([1800, 2100], [150, 250], 16, 4, 64, 16, dtype, seed=2)
    slots, offsets, _ = mq.paged_kv_slots(dev(c.ctx), dev(np.array([150, 250], np.int32)),
                                          dev(np.arange(c.nb, dtype=np.int32)), dev(c.table), c.nb, 16, c.max_ctx, 333)
    assert slots.shape[0] == 333 and offsets.tolist() == [0, 150, 400]
    c.q = c.q[:333].clone()
    check(c, "a step's tokens")


@pytest.mark.parametrize("new,rows", [([2, 4], 3), ([30, 90], 61)])
def test_weights(new, rows):
    c = Case([700, 2100], new, 8, 2, 64, 32, "fp16", seed=rows)
    c.q = c.q[:rows].clone()
    check_weights(c, "cut off")
