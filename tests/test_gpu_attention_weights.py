"""GPU tests of attention's weights: how exactly they enter the result.

One element of a key decides its score, the first step's keys (the first tile of
every wave, whichever kernel runs) score 0 and the rest `gap` octaves more, with
gaps up to 8: the running maximum stays behind, so the weights of most keys are
not near 1 and none of them is a power of two.  With values that are all alike
the result is that value, whatever the scores' rounding, for the same weights
stand above and below the fraction: what remains is the weights' own rounding
(two bf16 parts: 2^-16) and fp32 sums of at most 700 terms, 2^-15 together.
The results are rounded to nearest, and the nearest border lies 2^-9 (bf16) or
2^-12 (fp16) away: they have to be the value itself.
"""

import math

import numpy as np
import pytest
import torch

from oracle import cache
from tests.test_gpu_attention import Case, assert_within

pytestmark = pytest.mark.gpu

BATCH = 1100        # so many that a workgroup's piece holds whole sequences
# hq, hkv, next_n, max_context_len, topk (0: whole contexts): each kernel
KERNELS = [(8, 1, 1, 512, 0), (30, 1, 1, 512, 0), (7, 3, 2, 512, 0), (128, 1, 1, 65536, 0), (40, 1, 4, 65536, 0),
           (16, 4, 1, 65536, 0), (16, 8, 3, 8192, 0), (8, 1, 1, 512, 512), (64, 1, 1, 512, 512),
           (8, 4, 1, 512, 1024), (130, 1, 1, 512, 1024)]
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mqa_logits_amd  # noqa: F401


def alike(hq, hkv, next_n, max_ctx, topk, d, dtype, code, byte, batch=BATCH, keys=400, low=128):
    """(arguments, gaps [rows, hq], keys that a row sees, of which `low` score 0)."""
    bs = 64
    q_heads = hq // hkv * hkv
    per = -(-keys // bs)
    rng = np.random.default_rng(hq * 7 + d)
    i32 = dict(dtype=torch.int32, device="cuda")
    k = torch.zeros(batch * per, bs, hkv, d // 2, dtype=torch.uint8, device="cuda")
    k.view(batch, per * bs, hkv, d // 2)[:, low:, :, 0] = 0x02           # element 0 is 1
    sf = torch.full((batch * per, bs, hkv, d // 32), 127, dtype=torch.uint8, device="cuda")
    v, vs = torch.full_like(k, code * 17), torch.full_like(sf, byte)
    table = torch.zeros(batch, max(per, -(-max_ctx // bs)), **i32)
    table[:, :per] = torch.arange(batch * per, **i32).view(batch, per)
    gaps = torch.from_numpy(rng.uniform(0.05, 7.99, (batch * next_n, q_heads))).to(dtype)
    q = torch.zeros(batch * next_n, q_heads, d, dtype=dtype)
    q[:, :, 0] = gaps
    seen = keys - next_n + 1 + torch.arange(next_n).repeat(batch)
    indices = None
    if topk:
        indices = torch.full((batch * next_n, topk), -1, **i32)
        indices[:, :keys] = torch.arange(keys, **i32)
    args = ("mxfp4", q.cuda(), k, sf, v, vs, torch.full((batch,), keys, **i32), table, next_n, max_ctx)
    return args, dict(scale=math.log(2.0), indices=indices, return_lse=True), gaps.double(), seen, low


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv,next_n,max_ctx,topk", KERNELS)
def test_values_all_alike(hq, hkv, next_n, max_ctx, topk, d, dtype):
    import mqa_logits_amd as mq
    print(f"[weights] {hq}/{hkv} next_n={next_n} max_ctx={max_ctx} topk={topk} D={d} {dtype}", flush=True)
    args, kw, gaps, seen, low = alike(hq, hkv, next_n, max_ctx, topk, d, dtype, code=2, byte=127)
    out, lse = mq.paged_attention(*args, **kw)
    torch.cuda.synchronize()
    off = (out.float() - 1).abs().max()
    print(f"   largest difference {float(off):.3g}", flush=True)
    assert bool((out == 1).all())
    # lse: scores of up to 8 octaves rounded to fp32 a few times (2^-20), a sum of up to 700 terms
    ref = torch.log(low + (seen[:, None] - low) * torch.exp2(gaps))
    assert float((lse.double().cpu() - ref).abs().max()) <= 2.0 ** -16


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv,next_n,max_ctx,topk", KERNELS)
def test_large_values_all_alike(hq, hkv, next_n, max_ctx, topk, d):
    # 400 keys of 6 * 2^116: their sum is 0.59 * 2^128, inside fp32 as the
    # fraction's own terms are, however far the maximum stays behind
    import mqa_logits_amd as mq
    print(f"[large] {hq}/{hkv} next_n={next_n} max_ctx={max_ctx} topk={topk} D={d}", flush=True)
    args, kw, *_ = alike(hq, hkv, next_n, max_ctx, topk, d, torch.bfloat16, code=7, byte=243)
    out, lse = mq.paged_attention(*args, **kw)
    torch.cuda.synchronize()
    assert bool((out == 6 * 2.0 ** 116).all()) and bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("hq,hkv,max_ctx", [(8, 1, 700), (30, 1, 700), (128, 1, 262144), (16, 4, 65536)])
@pytest.mark.parametrize("q_size", [0.1, 3.0])
def test_large_values_of_either_sign(hq, hkv, max_ctx, q_size):
    # up to 700 keys of up to 6 * 2^115
    c = Case([300, 0, 1, 700], next_n=1, hq=hq, hkv=hkv, bs=16, max_ctx=max_ctx, q_size=q_size, seed=hq)
    c.vs = np.where(c.vs < 253, c.vs + 112, c.vs).astype(np.uint8)      # 237 .. 241
    out, _ = c.check("large values")
    assert bool(torch.isfinite(out).all()) and float(out.abs().max()) > 2.0 ** 110


@pytest.mark.parametrize("hq,hkv,max_ctx", [(8, 1, 16), (30, 1, 16), (128, 1, 262144), (16, 4, 65536), (8, 2, 4096)])
def test_one_key_of_the_largest_scale(hq, hkv, max_ctx):
    # byte 252: up to 6 * 2^125, which the key alone has to give back exactly
    c = Case([1, 1], next_n=1, hq=hq, hkv=hkv, bs=16, max_ctx=max_ctx, seed=hq)
    c.vs = np.where(c.vs < 253, 252, c.vs).astype(np.uint8)
    out, _ = c.run()
    ref, *_ = c.reference()
    assert np.array_equal(out.double().cpu().numpy(), ref) and np.abs(ref).max() == 1.5 * 2.0 ** 127


@pytest.mark.parametrize("scale", [0.0, 1e-44, 1e-40, -1e-40, 4e-39, -2e-38])
@pytest.mark.parametrize("hq,hkv,next_n,max_ctx,topk", KERNELS)
def test_factors_near_zero(hq, hkv, next_n, max_ctx, topk, scale):
    # <q, k> is 2^126 for the later keys and 0 for the others: scores of at most
    # 2.5 octaves, and none under a factor of 0
    import mqa_logits_amd as mq
    print(f"[factor] {scale} {hq}/{hkv} next_n={next_n} max_ctx={max_ctx} topk={topk}", flush=True)
    args, kw, _, seen, low = alike(hq, hkv, next_n, max_ctx, topk, 64, torch.bfloat16, code=4, byte=127)
    q, sf, v = args[1], args[3], args[4]
    q[:, :, 0] = 2.0 ** 63
    sf.fill_(127 + 63)
    v.view(BATCH, -1, hkv, 32)[:, :low] = 0x22                       # 1 instead of 2
    kw["scale"] = scale
    out, lse = mq.paged_attention(*args, **kw)
    torch.cuda.synchronize()
    r, late = math.exp(float(np.float32(scale)) * 2.0 ** 126), (seen - low).double()[:, None]
    ref = (low + 2 * late * r) / (low + late * r)
    # the result's rounding; a factor below 2^-126 times log2(e) is rounded by 2^-150, 2^-24 of a score
    assert float((out.double().cpu() - ref[..., None]).abs().max()) <= 2 * 2.0 ** -8 + 2.0 ** -14
    assert float((lse.double().cpu() - torch.log(low + late * r)).abs().max()) <= 2.0 ** -16


INFINITE = [(8, 2, 1, 700, 0), (30, 1, 1, 700, 0), (128, 1, 1, 262144, 0), (16, 4, 1, 65536, 0), (30, 1, 1, 700, 90)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("hq,hkv,next_n,max_ctx,topk", INFINITE)
def test_infinite_queries(hq, hkv, next_n, max_ctx, topk, dtype):
    # Element 7 of every key is +1 (sequence 0), +1 or -1 (1), zero somewhere (2).
    # A score of +inf, or 0 * inf, makes the row NaN; one of -inf is a weight of 0,
    # and a row of nothing else has no weight at all: 0 and -inf.
    inf = float("inf")
    c = Case([300, 300, 300], next_n=next_n, hq=hq, hkv=hkv, bs=16, dtype=dtype, max_ctx=max_ctx,
             topk=topk, seed=3)
    print(f"[infinite] {hq}/{hkv} max_ctx={max_ctx} topk={topk} {dtype}", flush=True)
    at = c.kept()

    def set_key(b, j, code):
        byte = c.k[at(b, j)]
        byte[:, 3] = (byte[:, 3] & 0x0f) | code << 4
    listed = [range(300)] * 3 if not topk else [c.indices[b] for b in range(3)]
    for b in range(3):
        for n, j in enumerate(listed[b]):
            set_key(b, int(j), 2 if b != 1 or n % 3 else 10)
    for n in (0, 40, 80):
        set_key(2, int(listed[2][n]), 0)
    finite, finite_lse = c.run()
    for h, x in ((0, inf), (1, -inf), (hq - 1, -inf)):
        c.q[:, h, 7] = x
    out, lse = c.run()
    torch.cuda.synchronize()
    rest = [h for h in range(hq) if h not in (0, 1, hq - 1)]
    assert torch.equal(out[:, rest], finite[:, rest]) and torch.equal(lse[:, rest], finite_lse[:, rest])
    assert bool(torch.isnan(out[:, 0]).all()) and bool(torch.isnan(lse[:, 0]).all())
    for h in (1, hq - 1):
        assert bool((out[0, h] == 0).all()) and float(lse[0, h]) == -inf
        assert bool(torch.isnan(out[1:, h]).all()) and bool(torch.isnan(lse[1:, h]).all())


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hq,hkv,next_n,max_ctx,topk", KERNELS)
def test_scores_of_the_largest_size(hq, hkv, next_n, max_ctx, topk, dtype, sign):
    # The later keys score +-2^23 .. 2^24 octaves, under a factor that is no power of
    # two, the first 128 score 0: one side has all the weight.  Values are 1 and 2.
    import mqa_logits_amd as mq
    print(f"[scores] {sign} {hq}/{hkv} next_n={next_n} max_ctx={max_ctx} topk={topk} {dtype}", flush=True)
    args, kw, _, seen, low = alike(hq, hkv, next_n, max_ctx, topk, 64, dtype, code=4, byte=127)
    q, sf, v = args[1], args[3], args[4]
    size = torch.linspace(1.05, 1.95, q.shape[0] * q.shape[1]).view(q.shape[:2]) * 2.0 ** 11
    q[:, :, 0] = (sign * size).to(q)
    sf.fill_(127 + 15)                                               # <q, k> = q 2^15
    v.view(BATCH, -1, hkv, 32)[:, :low] = 0x22                       # 1 instead of 2
    kw["scale"] = scale = float(np.float32(0.0884))
    out, lse = mq.paged_attention(*args, **kw)
    torch.cuda.synchronize()
    score = scale * q[:, :, 0].double().cpu() * 2.0 ** 15
    octaves = score.abs() / math.log(2.0)
    assert 2.0 ** 22.9 < float(octaves.min()) and float(octaves.max()) < 2.0 ** 24
    assert bool((out == (2 if sign > 0 else 1)).all())
    if sign > 0:
        ref = score + torch.log((seen - low).double())[:, None]
    else:
        ref = torch.full_like(score, math.log(low))
    # the factor, its product, the maximum with the sum's logarithm, and ln 2: a rounding of 2^-24 each
    assert bool(((lse.double().cpu() - ref).abs() <= 2.0 ** -22 * ref.abs()).all())


@pytest.mark.parametrize("topk", [0, 200])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv,next_n,max_ctx", [(8, 1, 2, 700), (30, 1, 1, 700), (128, 1, 1, 262144), (24, 2, 4, 262144),
                                                   (16, 4, 1, 65536), (24, 8, 3, 65536)])
def test_bf16_against_64_bits(hq, hkv, next_n, max_ctx, d, topk):
    # the oracle's bound, with 2^-16 for the weights
    c = Case([0, 1, 33, 300, 700], next_n=next_n, hq=hq, hkv=hkv, d=d, bs=16, max_ctx=max_ctx, topk=topk, seed=hq + d)
    print(f"[64 bits] {hq}/{hkv} next_n={next_n} D={d} max_ctx={max_ctx} topk={topk}", flush=True)
    out, lse = c.run()
    torch.cuda.synchronize()
    ref, ref_lse, tol, tol_lse = cache.attention(
        c.q.double().numpy(), c.k, c.ks, c.v, c.vs, c.ctx, c.table, next_n, max_ctx, c.scale,
        HALF[torch.bfloat16], 2.0 ** -16, indices=c.indices)
    assert_within(out.double().cpu().numpy(), ref, tol, "out")
    assert_within(lse.double().cpu().numpy(), ref_lse, tol_lse, "lse")
