"""GPU parity of attention of token chunks over the paged MXFP4 cache, against float64.

Tolerances are the oracle's per-entry bounds (oracle.cache.attention): the
result's own rounding, the rounding of the weights in the second product, and
fp32 sums.  The results are divided by the sum of the rounded weights, so a weight's
rounding (2^-12, half a step of fp16) counts twice: once for itself, once for
the sum.  Weights end at fp16's least subnormal, 2^-24, where the row's largest
is 2^8 at least: half a step there is 2^-33 of the largest, twice as well.  Unread pool slots hold random codes under NaN scales, so a key
outside a row's range, or a wrong block, cannot pass.
"""

import numpy as np
import pytest
import torch

from oracle import cache
from tests.gpu_helpers import dev, log
from tests.test_gpu_attention import DTYPES, assert_within

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
WEIGHTS, FLOOR = 2.0 ** -11, 2.0 ** -32


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mqa_logits_amd  # noqa: F401


class Case:
    """Sequences of ctx tokens, the last `new` of them in q; `pad` rows of nobody behind."""

    def __init__(self, ctx, new, hq=8, hkv=1, d=128, bs=64, dtype="bf16", max_ctx=None, seed=0,
                 q_size=2.0, sf=(125, 130), pad=0, extra_cols=1):
        rng = np.random.default_rng(seed)
        self.ctx, new = np.asarray(ctx, np.int32), np.asarray(new, np.int32)
        self.bs, self.dtype = bs, dtype
        self.max_ctx = int(max(self.ctx.max(), 1)) if max_ctx is None else max_ctx
        self.offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        batch = len(self.ctx)
        length = np.clip(self.ctx, 0, self.max_ctx)
        need = -(-length // bs)
        self.nb = int(need.sum()) + 3
        ids = rng.permutation(self.nb).astype(np.int32)
        self.table = rng.integers(-5, self.nb + 5, (batch, -(-self.max_ctx // bs) + extra_cols)).astype(np.int32)
        held = np.zeros((self.nb, bs), bool)
        at = 0
        for b in range(batch):
            self.table[b, :need[b]] = ids[at:at + need[b]]
            for j in range(length[b]):
                held[ids[at + j // bs], j % bs] = True
            at += need[b]
        shape = (self.nb, bs, hkv)
        self.k, self.v = (rng.integers(0, 256, (*shape, d // 2), dtype=np.uint8) for _ in range(2))
        self.ks, self.vs = (rng.integers(*sf, (*shape, d // 32), dtype=np.uint8) for _ in range(2))
        for s in (self.ks, self.vs):
            s[~held] = rng.integers(253, 256, s[~held].shape)
        self.q = torch.from_numpy(rng.normal(size=(self.offsets[-1] + pad, hq, d)) * q_size).to(DTYPES[dtype])
        self.scale = d ** -0.5

    def slot(self, b, j):
        return self.table[b, j // self.bs], j % self.bs

    def run(self, **kw):
        import mqa_logits_amd as mq
        args = dict(q=self.q.cuda(), token_offsets=dev(self.offsets), return_lse=True)
        args.update(kw)
        return mq.paged_chunk_attention("mxfp4", args.pop("q"), dev(self.k), dev(self.ks), dev(self.v),
                                        dev(self.vs), dev(self.ctx), args.pop("token_offsets"), dev(self.table),
                                        self.max_ctx, scale=self.scale, **args)

    def rows(self):
        return cache.chunk_rows(self.ctx, self.offsets, len(self.q), self.max_ctx)

    def reference(self):
        with np.errstate(all="ignore"):
            return cache.attend_rows(self.q.double().numpy(), self.k, self.ks, self.v, self.vs,
                                     self.table, *self.rows(), self.scale, HALF[self.dtype], WEIGHTS, weight_floor=FLOOR)

    def check(self, what):
        log(f"[chunk] {what} ctx={self.ctx[:4]}.. offsets={self.offsets[:5]}.. rows={len(self.q)} "
            f"heads={self.q.shape[1]}/{self.k.shape[2]} D={self.q.shape[2]} bs={self.bs} {self.dtype} max_ctx={self.max_ctx}")
        out = torch.full_like(self.q, 7.0, device="cuda")
        lse = torch.full(self.q.shape[:2], 9.0, device="cuda")
        self.run(out=out, lse=lse)
        torch.cuda.synchronize()
        ref, ref_lse, tol, tol_lse = self.reference()
        nobody = self.rows()[0] < 0
        ref[nobody], ref_lse[nobody] = 7.0, 9.0          # left as they were
        got = out.double().cpu().numpy()
        if self.dtype == "fp16":
            # fp16 rounds magnitudes from 65520 on to infinity; within the bound of that either way
            over = 65520.0
            ref = np.where(np.abs(ref) >= over + tol, np.copysign(np.inf, ref), ref)
            ref = np.where((np.abs(np.abs(ref) - over) < tol) & np.isinf(got), np.copysign(np.inf, ref), ref)
        assert_within(got, ref, tol, what + " out")
        assert_within(lse.double().cpu().numpy(), ref_lse, tol_lse, what + " lse")
        return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(8, 1), (16, 2), (15, 3), (33, 1), (64, 1), (130, 1), (4, 4)])
def test_heads(hq, hkv, d, dtype):
    Case([70, 1, 0, 300, 129], [33, 1, 0, 40, 129], hq, hkv, d, 32, dtype, seed=hq + d).check("heads")


@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("ctx,new", [
    ([1], [1]), ([2], [1]), ([64], [64]), ([65], [65]), ([63], [5]), ([257], [256]), ([513], [17]),
    ([700, 513, 600], [1, 513, 90]), ([1500], [700]), ([0, 5, 0, 64], [0, 5, 0, 1]),
    ([4100, 3], [9, 3]), ([16500], [20]),
])
def test_lengths(ctx, new, bs):
    Case(ctx, new, 12, 2, 64, bs, "fp16", seed=sum(ctx) + bs, pad=3).check("lengths")
    Case(ctx, new, 16, 2, 128, bs, "bf16", seed=sum(ctx) + bs).check("lengths")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_many_sequences(dtype):
    rng = np.random.default_rng(3)
    ctx = rng.integers(0, 700, 300)
    new = np.minimum(ctx, rng.integers(0, 9, 300))
    Case(ctx, new, 6, 2, 64, 16, dtype, max_ctx=1000, seed=5, pad=2).check("many")
    Case(ctx % 200, new % 3, 6, 2, 128, 16, dtype, max_ctx=200, seed=6).check("many, short")


def test_limits_of_lengths():
    # contexts over max_context_len, below the new tokens, negative
    Case([900, 3, -4, 40], [20, 7, 2, 40], 8, 2, 128, 16, "bf16", max_ctx=600, seed=8).check("limits")
    Case([900, 3, -4, 40], [20, 7, 2, 40], 8, 2, 64, 16, "fp16", max_ctx=30, seed=9).check("limits, short")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sf", [(100, 116), (112, 137), (104, 141), (126, 146), (90, 165)])
def test_scales_of_any_size(sf, d, dtype):
    # K over this range would give scores of any size: its own stay usual
    c = Case([300, 130, 520], [70, 130, 9], 10, 2, d, 32, dtype, seed=sf[0] + d, sf=sf)
    rng = np.random.default_rng(1)
    held = c.ks <= 252
    c.ks[held] = rng.integers(124, 129, held.sum())
    c.check("V's scales")


@pytest.mark.parametrize("d", [64, 128])
def test_key_scales_outside_fp16(d):
    # small K in some blocks: exact for fp16 queries only if not held in fp16
    c = Case([300, 130], [70, 130], 10, 2, d, 32, "fp16", seed=d)
    rng = np.random.default_rng(2)
    held = (c.ks <= 252) & (rng.random(c.ks.shape) < 0.02)
    c.ks[held] = rng.integers(60, 104, held.sum())
    c.check("K's scales")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_nan_scales(dtype):
    c = Case([300, 130, 520], [70, 130, 9], 10, 2, 128, 32, dtype, seed=4)
    for b, j, side, block in [(0, 250, "k", 1), (1, 60, "v", 2), (2, 519, "v", 0), (2, 100, "v", 3), (1, 129, "k", 0)]:
        page, at = c.slot(b, j)
        (c.ks if side == "k" else c.vs)[page, at, 1, block] = 253 + j % 3
    out, lse = c.check("NaN scales")
    assert torch.isnan(out).any() and not torch.isnan(out).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_offsets_past_the_rows(dtype):
    import mqa_logits_amd as mq  # noqa: F401
    # more new tokens than rows (max_tokens cut them off), and none given
    c = Case([70, 300], [33, 40], 8, 2, 64, 32, dtype, seed=1)
    whole, lse = c.run()
    c.q = c.q[:50]
    c.check("cut off")
    out, part = c.run(q=c.q.cuda())
    assert torch.equal(out, whole[:50]) and torch.equal(part, lse[:50])
    c = Case([70, 300], [33, 33], 8, 2, 64, 32, dtype, seed=1)
    assert all(torch.equal(a, b) for a, b in zip(c.run(), c.run(token_offsets=None)))


@pytest.mark.parametrize("batch", [5, 70])
def test_small_contexts(batch):
    """Tiles that are never cut, known to their workgroups or found by the lengths."""
    rng = np.random.default_rng(batch)
    ctx = rng.integers(0, 500, batch)
    Case(ctx, np.minimum(ctx, rng.integers(0, 60, batch)), 16, 8, 64, 16, "fp16", max_ctx=500, seed=batch).check("small contexts")


def test_shortest_contexts():
    """Tiles that are never cut, more than the chip holds."""
    rng = np.random.default_rng(9)
    ctx = rng.integers(0, 257, 90)
    Case(ctx, np.minimum(ctx, rng.integers(0, 80, 90)), 24, 8, 128, 32, "bf16", max_ctx=256, seed=9).check("shortest contexts")
