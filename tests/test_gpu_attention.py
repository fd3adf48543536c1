"""GPU parity of attention over the paged MXFP4 cache, against float64.

Tolerances are the oracle's per-entry bounds (oracle.cache.attention): the
result's own rounding, the rounding of the weights in the second product, and
fp32 sums.  Unread pool slots hold random codes under NaN scales, so a key
outside a row's range, or a wrong block, cannot pass.
"""

import numpy as np
import pytest
import torch

from oracle import cache
from oracle.reference import paged_row_ranges
from tests.gpu_helpers import dev, log

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
# the result's rounding, and the weights' (two bf16 parts for fp16: each part
# halves eight bits away)
STEPS = {"bf16": (2.0 ** -8, 2.0 ** -8), "fp16": (2.0 ** -11, 2.0 ** -16)}


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mqa_logits_amd  # noqa: F401


class Case:
    def __init__(self, ctx, next_n=1, hq=8, hkv=1, d=128, bs=64, dtype="bf16", max_ctx=None,
                 topk=0, seed=0, q_size=2.0, sf=(125, 130), extra_cols=1):
        rng = np.random.default_rng(seed)
        self.ctx = np.asarray(ctx, np.int32)
        self.next_n, self.bs, self.dtype, self.topk = next_n, bs, dtype, topk
        self.max_ctx = int(max(self.ctx.max(), 1)) if max_ctx is None else max_ctx
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
        self.q = torch.from_numpy(rng.normal(size=(batch * next_n, hq, d)) * q_size).to(DTYPES[dtype])
        self.scale = d ** -0.5
        self.indices = None
        if topk:
            _, seen = paged_row_ranges(self.ctx, next_n, self.max_ctx)
            self.indices = np.full((batch * next_n, topk), -1, np.int32)
            for r, n in enumerate(seen):
                pick = np.sort(rng.permutation(n)[:topk])
                self.indices[r, :len(pick)] = pick

    def kept(self):
        """Pool and index positions of one key of one sequence."""
        return lambda b, j: (self.table[b, j // self.bs], j % self.bs)

    def run(self, **kw):
        import mqa_logits_amd as mq
        return mq.paged_attention("mxfp4", kw.pop("q", self.q.cuda()), dev(self.k), dev(self.ks),
                                  dev(self.v), dev(self.vs), dev(self.ctx), dev(self.table),
                                  self.next_n, self.max_ctx, scale=self.scale,
                                  indices=dev(self.indices), return_lse=True, **kw)

    def reference(self):
        with np.errstate(all="ignore"):
            return cache.attention(self.q.double().numpy(), self.k, self.ks, self.v, self.vs,
                                   self.ctx, self.table, self.next_n, self.max_ctx, self.scale,
                                   *STEPS[self.dtype], indices=self.indices)

    def check(self, what):
        log(f"[attention] {what} batch={len(self.ctx)} next_n={self.next_n} "
            f"heads={self.q.shape[1]}/{self.k.shape[2]} D={self.q.shape[2]} bs={self.bs} "
            f"{self.dtype} max_ctx={self.max_ctx} topk={self.topk}")
        out, lse = self.run()
        torch.cuda.synchronize()
        ref, ref_lse, tol, tol_lse = self.reference()
        got = out.double().cpu().numpy()
        if self.dtype == "fp16":
            # fp16 rounds magnitudes from 65520 (half a step over its largest,
            # 65504) on to infinity; within the bound of that either way
            over = 65520.0
            ref = np.where(np.abs(ref) >= over + tol, np.copysign(np.inf, ref), ref)
            ref = np.where((np.abs(np.abs(ref) - over) < tol) & np.isinf(got),
                           np.copysign(np.inf, ref), ref)
        assert_within(got, ref, tol, what + " out")
        assert_within(lse.double().cpu().numpy(), ref_lse, tol_lse, what + " lse")
        return out, lse


def assert_within(got, ref, tol, what):
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaNs differ"
    same = got[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)]
    assert np.array_equal(*same), f"{what}: infinities differ"
    if fine.any():
        # rows without keys have a bound of 0 and a result of exactly 0
        ratio = np.abs(got[fine] - ref[fine]) / np.maximum(tol[fine], 1e-300)
        log(f"   {what}: max error/bound {ratio.max():.3g}")
        assert ratio.max() <= 1.0, f"{what}: error/bound {ratio.max():.3g}"


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64])
def test_lengths(bs, d, dtype):
    # zero, one, every edge of a half tile, a tile, a block and a wave's turn
    ctx = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300]
    Case(ctx, hq=8, hkv=2, d=d, bs=bs, dtype=dtype, seed=bs + d).check("lengths")


@pytest.mark.parametrize("hq,hkv", [(1, 1), (7, 1), (16, 1), (17, 1), (33, 1), (64, 1), (128, 1),
                                    (6, 3), (15, 3), (64, 8), (40, 40)])
def test_head_layouts(hq, hkv):
    Case([70, 1, 200], hq=hq, hkv=hkv, bs=16, seed=hq).check("heads")
    Case([70, 1, 200], next_n=3, hq=hq, hkv=hkv, d=64, bs=32, dtype="fp16", seed=hq).check("heads")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("next_n", [1, 2, 3, 4, 5, 8, 16])
def test_query_tokens(next_n, dtype):
    # rows that see nothing (contexts shorter than next_n), tails inside a tile
    Case([0, 1, next_n - 1, next_n, 31, 32, 40, 290, 256 + next_n], next_n=next_n, hq=10, hkv=2,
         bs=16, dtype=dtype, seed=next_n).check("next_n")


@pytest.mark.parametrize("batch,hkv,ctx", [(1, 1, 5000), (2, 2, 3111), (1, 4, 9000), (3, 1, 4097)])
def test_split_contexts(batch, hkv, ctx):
    # one long sequence beside short ones: several chunks, one chunk and none
    lens = [ctx, 100, 0][:batch]
    Case(lens, next_n=2, hq=8 * hkv, hkv=hkv, max_ctx=ctx, seed=ctx).check("split")
    Case(lens, next_n=1, hq=5 * hkv, hkv=hkv, d=64, bs=16, dtype="fp16", max_ctx=ctx + 500,
         seed=ctx).check("split")


def test_many_chunks():
    Case([66000], hq=2, hkv=1, seed=1).check("chunks")
    Case([66000], hq=2, hkv=1, d=64, dtype="fp16", seed=1).check("chunks")


def test_context_beyond_the_maximum():
    c = Case([500, 90], next_n=4, hq=8, hkv=2, bs=16, max_ctx=120, seed=3)
    c.check("clamped")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
def test_peaked_scores(d, dtype):
    # scores of some hundreds: a few keys take all the weight and the running
    # maximum moves late
    Case([600, 3000], hq=8, hkv=2, d=d, dtype=dtype, q_size=40.0, seed=9).check("peaked")


def test_negative_and_zero_scale():
    for scale in (-0.11, 0.0):
        c = Case([33, 400], hq=4, hkv=1, seed=4)
        c.scale = scale
        c.check("scale")


@pytest.mark.parametrize("topk", [1, 7, 31, 33, 64, 200, 513])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_selected_keys(topk, dtype):
    Case([0, 1, 5, 64, 100, 900], next_n=2, hq=16, hkv=2, bs=16, dtype=dtype, topk=topk,
         seed=topk).check("selected")
    Case([1000, 3], next_n=1, hq=64, hkv=1, d=64, bs=64, dtype=dtype, topk=topk,
         seed=topk).check("selected")


def test_selected_keys_split():
    Case([9000], next_n=1, hq=64, hkv=1, topk=2048, seed=6).check("selected, split")
    Case([9000, 40], next_n=2, hq=24, hkv=3, d=64, dtype="fp16", topk=1000, seed=6).check("selected, split")


def test_selected_keys_any_order_twice_and_out_of_range():
    c = Case([300, 50], next_n=2, hq=8, hkv=2, bs=16, topk=90, seed=8)
    rng = np.random.default_rng(0)
    c.indices = rng.integers(-20, 320, c.indices.shape).astype(np.int32)
    c.indices[:, 5] = c.indices[:, 6] = 3
    c.indices[1] = -1
    c.indices[2, :2] = [2 ** 31 - 1, -2 ** 31]
    c.check("any order")


def test_selecting_every_key_is_the_whole_context():
    whole = Case([333], next_n=1, hq=16, hkv=1, seed=2)
    out, lse = whole.run()
    whole.indices = np.arange(333, dtype=np.int32)[None]
    out2, lse2 = whole.run()
    ref, _, tol, tol_lse = whole.reference()
    assert_within(out2.double().cpu().numpy(), ref, tol, "every key")
    assert float((lse - lse2).abs().max()) <= 2 * tol_lse.max()


@pytest.mark.parametrize("d", [64, 128])
def test_nan_keys_and_values_reach_only_their_rows(d):
    # a NaN scale in the last keys: rows of earlier query tokens do not see them
    for side in ("k", "v"):
        c = Case([100, 260, 5], next_n=4, hq=6, hkv=2, d=d, bs=16, seed=d)
        at = c.kept()
        sf = c.ks if side == "k" else c.vs
        for b, j in ((0, 98), (1, 259), (2, 3)):
            sf[at(b, j)][1, d // 32 - 1] = 255
        out, lse = c.check("nan " + side)
        nan = torch.isnan(out)
        assert bool(nan[2, 3:].any()) and not bool(nan[:2].any()) and not bool(nan[:, :3].any())
        if side == "v":
            assert not bool(nan[..., :d - 32].any()) and not bool(torch.isnan(lse).any())


def test_nan_values_in_the_middle_and_selected():
    c = Case([400], next_n=2, hq=20, hkv=1, seed=5)
    c.vs[c.kept()(0, 70)][0, 2] = 253
    out, _ = c.check("nan in the middle")
    assert bool(torch.isnan(out[..., 64:96]).all()) and int(torch.isnan(out).sum()) == 2 * 20 * 32
    c.indices = np.array([[1, 70, 399, 5], [1, 71, 399, 5]], np.int32)
    out, _ = c.check("nan selected")
    assert bool(torch.isnan(out[0, :, 64:96]).all()) and not bool(torch.isnan(out[1]).any())


def test_nan_and_infinite_queries():
    c = Case([100, 100], next_n=1, hq=4, hkv=1, seed=5)
    c.q[0, 1, 7] = float("nan")
    out, lse = c.run()
    bad = torch.isnan(out).all(-1)
    assert bad.cpu().tolist() == [[False, True, False, False], [False] * 4]
    assert torch.isnan(lse).cpu().tolist() == bad.cpu().tolist()


def test_wide_and_extreme_scales():
    # block scales over forty octaves, where fp16 would overflow and underflow
    Case([150, 700], hq=4, hkv=1, dtype="fp16", sf=(107, 147), q_size=1e-5, seed=7).check("scales")
    Case([150, 700], hq=4, hkv=1, dtype="bf16", sf=(90, 160), q_size=1e-9, seed=7).check("scales")


def test_strided_queries_and_tables():
    c = Case([90, 300], next_n=2, hq=8, hkv=2, seed=12)
    wide = torch.randn(4, 3, 8, 128, device="cuda").to(torch.bfloat16)
    wide[:, 1] = c.q.cuda()
    a, b = c.run(q=wide[:, 1]), c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_outputs_workspace_and_guards():
    import mqa_logits_amd as mq
    c = Case([5000, 10], next_n=1, hq=8, hkv=1, seed=13)
    need = mq.paged_attention_workspace_size(2, 1, 8, 1, 128, c.max_ctx)
    assert need > 0
    ws = torch.full((need + 256,), 0xAB, dtype=torch.uint8, device="cuda")
    out = torch.full((3, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((3, 8), 5.0, device="cuda")
    got = c.run(workspace=ws[:need], out=out[:2], lse=lse[:2])
    assert got[0].data_ptr() == out.data_ptr() and bool((out[2] == 5).all()) and bool((lse[2] == 5).all())
    assert bool((ws[need:] == 0xAB).all())
    ref = c.run()
    assert torch.equal(ref[0], out[:2]) and torch.equal(ref[1], lse[:2])


def test_repeats_are_bitwise_equal():
    c = Case([4000, 77, 1500], next_n=2, hq=16, hkv=2, seed=14)
    a = c.run()
    for _ in range(5):
        b = c.run()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_streams_at_once():
    c, d = Case([4000, 77], hq=16, hkv=2, seed=15), Case([3500, 900], hq=16, hkv=2, seed=16)
    ref = c.run(), d.run()
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[], []]
    for _ in range(4):
        for i, (s, x) in enumerate(zip(streams, (c, d))):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got[i].append(x.run())
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in got[i]:
            assert torch.equal(out, ref[i][0]) and torch.equal(lse, ref[i][1])


@pytest.mark.parametrize("topk", [0, 700])
def test_step_captured_in_a_graph(topk):
    """slots -> write K and V -> (top-k ->) attention, one graph, replayed over a growing context,
    against the same calls made eagerly."""
    import mqa_logits_amd as mq
    torch.manual_seed(0)
    batch, next_n, hkv, group, d, bs, max_ctx = 3, 2, 2, 8, 128, 16, 2048
    start = torch.tensor([30, 0, 1200], dtype=torch.int32, device="cuda")
    nb = 200
    i32 = dict(dtype=torch.int32, device="cuda")

    class State:
        def __init__(self):
            g = torch.Generator(device="cuda").manual_seed(1)
            self.k, self.v = (torch.zeros(nb, bs, hkv, d // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
            self.ks, self.vs = (torch.full((nb, bs, hkv, d // 32), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
            self.table = torch.full((batch, max_ctx // bs), -1, **i32)
            self.free = torch.arange(nb, **i32)
            n = int(start.sum())
            slots, _, taken = mq.paged_kv_slots(start, start, self.free, self.table, nb, bs, max_ctx, n)
            x = torch.randn(2, n, hkv, d, generator=g, device="cuda").to(torch.bfloat16)
            mq.paged_kv_write("mxfp4", x[0], slots, self.k, self.ks)
            mq.paged_kv_write("mxfp4", x[1], slots, self.v, self.vs)
            self.free = self.free[int(taken):].clone()
            self.ctx, self.new = start.clone(), torch.full((batch,), next_n, **i32)
            self.q = torch.empty(batch * next_n, hkv * group, d, dtype=torch.bfloat16, device="cuda")
            self.x = torch.empty(2, batch * next_n, hkv, d, dtype=torch.bfloat16, device="cuda")
            self.logits = torch.empty(batch * next_n, max_ctx, device="cuda")

        def inputs(self, step):
            g = torch.Generator(device="cuda").manual_seed(100 + step)
            self.q.copy_(torch.randn(self.q.shape, generator=g, device="cuda"))
            self.x.copy_(torch.randn(self.x.shape, generator=g, device="cuda"))
            self.logits.copy_(torch.randn(self.logits.shape, generator=g, device="cuda"))

        def step(self):
            self.ctx += self.new
            slots, _, taken = mq.paged_kv_slots(self.ctx, self.new, self.free, self.table, nb, bs,
                                                max_ctx, batch * next_n)
            mq.paged_kv_write("mxfp4", self.x[0], slots, self.k, self.ks)
            mq.paged_kv_write("mxfp4", self.x[1], slots, self.v, self.vs)
            # the free list moves up by what was taken
            at = torch.arange(self.free.numel(), device="cuda") + taken
            self.free.copy_(self.free[at.clamp(max=self.free.numel() - 1)])
            indices = mq.mqa_logits_topk(self.logits, topk) if topk else None
            return mq.paged_attention("mxfp4", self.q, self.k, self.ks, self.v, self.vs, self.ctx,
                                      self.table, next_n, max_ctx, indices=indices, return_lse=True)

    eager, graphed, warm = State(), State(), State()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        warm.inputs(0)
        warm.step()
    torch.cuda.synchronize()
    graphed.inputs(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = graphed.step()
    for step in range(20):
        eager.inputs(step)
        graphed.inputs(step)
        ref = eager.step()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager.table, graphed.table) and torch.equal(eager.k, graphed.k)
        assert torch.equal(eager.vs, graphed.vs) and torch.equal(eager.free, graphed.free)
        assert torch.equal(ref[0], out) and torch.equal(ref[1], lse), f"step {step}"
        assert bool(torch.isfinite(out).all()) and bool(out.any())


def test_cache_beyond_32_bit_offsets():
    # a pool of 4.3 GB per side: the keys in its last blocks
    import mqa_logits_amd as mq
    bs, hkv, d = 64, 8, 128
    nb = (1 << 32) // (bs * hkv * d // 2) + 40
    c = Case([200, 64], next_n=1, hq=16, hkv=hkv, bs=bs, seed=20)
    ids = np.array([nb - 1, 3, nb - 2, nb - 17, nb - 30], np.int32)
    pools = []
    for p in (c.k, c.ks, c.v, c.vs):
        big = torch.zeros(nb, *p.shape[1:], dtype=torch.uint8, device="cuda")
        if p.shape[-1] == d // 32:
            big.fill_(255)
        pools.append(big)
    table = np.zeros((2, 4), np.int32)
    table[0], table[1, 0] = ids[:4], ids[4]
    old = np.concatenate([c.table[0, :4], c.table[1, :1]])
    for big, p in zip(pools, (c.k, c.ks, c.v, c.vs)):
        big[torch.from_numpy(ids.astype(np.int64)).cuda()] = dev(p[old])
    out, lse = mq.paged_attention("mxfp4", c.q.cuda(), pools[0], pools[1], pools[2], pools[3],
                                  dev(c.ctx), dev(table), 1, c.max_ctx, return_lse=True)
    same, same_lse = c.run()
    assert torch.equal(out, same) and torch.equal(lse, same_lse)
    # and a write there
    x = torch.randn(3, hkv, d, device="cuda").to(torch.bfloat16)
    slots = torch.tensor([nb * bs - 1, (nb - 2) * bs, nb * bs], device="cuda")
    small = torch.zeros(1, bs, hkv, d // 2, dtype=torch.uint8, device="cuda")
    small_sf = torch.zeros(1, bs, hkv, d // 32, dtype=torch.uint8, device="cuda")
    mq.paged_kv_write("mxfp4", x, slots, pools[0], pools[1])
    mq.paged_kv_write("mxfp4", x, torch.tensor([63, 0, -1], device="cuda"), small, small_sf)
    assert torch.equal(pools[0][nb - 1, 63], small[0, 63]) and torch.equal(pools[0][nb - 2, 0], small[0, 0])
    assert torch.equal(pools[1][nb - 1, 63], small_sf[0, 63])
