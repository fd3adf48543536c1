"""Chunk attention, gathered weights and eviction together, as a server runs them: new
tokens get slots and are written, attend, the cache is cut, decoding goes on with what
stayed; and captured into a graph, on another stream, with strided queries."""

import numpy as np
import pytest
import torch

from oracle import cache
from tests.gpu_helpers import dev, log
from tests.test_gpu_attention import assert_within
from tests.test_gpu_chunk import FLOOR, HALF, WEIGHTS, Case
from tests.test_gpu_evict import NAMES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mqa_logits_amd  # noqa: F401


class Server:
    BS, HQ, HKV, D, BATCH, MAX = 16, 8, 2, 64, 5, 400

    def __init__(self, dtype, seed):
        self.rng, self.dtype = np.random.default_rng(seed), dtype
        self.nb = 2 * self.BATCH * -(-self.MAX // self.BS)
        shape = (self.nb, self.BS, self.HKV)
        self.pools = [torch.zeros(*shape, n, dtype=torch.uint8, device="cuda")
                      for n in (self.D // 2, self.D // 32, self.D // 2, self.D // 32)]
        self.free = dev(self.rng.permutation(self.nb).astype(np.int32))
        self.table = torch.full((self.BATCH, -(-self.MAX // self.BS)), -1, dtype=torch.int32, device="cuda")
        self.ctx = torch.zeros(self.BATCH, dtype=torch.int32, device="cuda")
        self.sums = torch.zeros(self.BATCH, self.MAX, device="cuda")

    def random(self, *shape):
        return torch.from_numpy(self.rng.normal(size=shape)).to(self.dtype).cuda()

    def step(self, new):
        """New tokens in, out and lse; the sums follow."""
        import mqa_logits_amd as mq
        n = int(sum(new))
        new = dev(np.array(new, np.int32))
        self.ctx = self.ctx + new
        slots, offsets, taken = mq.paged_kv_slots(self.ctx, new, self.free, self.table, self.nb, self.BS, self.MAX, n)
        self.free = self.free[int(taken):].contiguous()
        k, v, q = (self.random(n, h, self.D) for h in (self.HKV, self.HKV, self.HQ))
        mq.paged_kv_write("mxfp4", k, slots, *self.pools[:2])
        mq.paged_kv_write("mxfp4", v, slots, *self.pools[2:])
        out, lse = mq.paged_chunk_attention("mxfp4", q, *self.pools, self.ctx, offsets, self.table, self.MAX, return_lse=True)
        mq.paged_attention_weights("mxfp4", q, lse, *self.pools[:2], self.ctx, offsets, self.table, self.MAX,
                                   weights=self.sums, out=self.sums)
        return q, out, lse, offsets

    def host(self):
        return [p.cpu().numpy() for p in self.pools]

    def cut(self, keep, recent):
        import mqa_logits_amd as mq
        before = dict(weights=self.sums.cpu().numpy(), context_lens=self.ctx.cpu().numpy(), block_table=self.table.cpu().numpy(),
                      free_blocks=self.free.cpu().numpy(), pools=self.host(), keep=keep, recent=recent, max_context_len=self.MAX)
        got = mq.paged_kv_evict(self.sums, self.ctx, self.table, self.free, self.pools, keep, recent, self.MAX)
        ref = cache.evict(**before)
        for name, g, r in zip(NAMES, got, ref):
            assert np.array_equal(g.cpu().numpy().view(np.int32), r.view(np.int32)), name
        for g, r in zip(self.host(), ref[-1]):
            assert np.array_equal(g, r)
        asked, back = got.counts.tolist()
        assert asked <= len(self.free)
        self.ctx, self.table, self.sums = got.context_lens, got.block_table, got.weights
        self.free = torch.cat([self.free[asked:], got.freed[:back]])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_run(dtype):
    import mqa_logits_amd as mq
    s, name = Server(dtype, 1), "bf16" if dtype == torch.bfloat16 else "fp16"
    steps = [[130, 0, 64, 17, 200], [1, 90, 1, 1, 1], [40, 40, 40, 40, 40], [1, 1, 1, 1, 1], [7, 0, 100, 0, 60]]
    for i, new in enumerate(steps):
        log(f"[run] step {i} {new} {dtype}")
        q, out, lse, offsets = s.step(new)
        rows = cache.chunk_rows(s.ctx.cpu().numpy(), offsets.cpu().numpy(), len(q), s.MAX)
        ref, ref_lse, tol, tol_lse = cache.attend_rows(q.double().cpu().numpy(), *s.host(), s.table.cpu().numpy(), *rows,
                                                       s.D ** -0.5, HALF[name], WEIGHTS, weight_floor=FLOOR)
        assert_within(out.double().cpu().numpy(), ref, tol, f"step {i} out")
        assert_within(lse.double().cpu().numpy(), ref_lse, tol_lse, f"step {i} lse")
        if max(new) == 1 and min(new) == 1:  # one token each: decoding's own attention agrees
            other = mq.paged_attention("mxfp4", q, *s.pools, s.ctx, s.table, 1, s.MAX)
            assert (other.double() - out.double()).abs().max() < 0.05 * out.double().abs().max()
        if i % 2:
            s.cut(100, 30)
            assert int(s.ctx.max()) <= 100


def calls(c, q, lse, sums, free, keep=100, ws=(None, None, None)):
    """What the graph tests capture: attention, sums, a cut."""
    import mqa_logits_amd as mq
    out = c.attend(q, ws[0])
    w = mq.paged_attention_weights("mxfp4", q, out[1], c.dk, c.dks, c.dctx, c.doff, c.dtable, c.max_ctx, scale=c.scale,
                                   weights=sums, workspace=ws[1])
    e = mq.paged_kv_evict(w, c.dctx, c.dtable, free, [c.dk, c.dks, c.dv, c.dvs], keep, 20, c.max_ctx, workspace=ws[2])
    return [*out, w, *e]


class Held(Case):
    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        self.dk, self.dks, self.dv, self.dvs = (dev(x) for x in (self.k, self.ks, self.v, self.vs))
        self.dctx, self.doff, self.dtable = dev(self.ctx), dev(self.offsets), dev(self.table)

    def attend(self, q, ws=None):
        import mqa_logits_amd as mq
        return mq.paged_chunk_attention("mxfp4", q, self.dk, self.dks, self.dv, self.dvs, self.dctx, self.doff, self.dtable,
                                        self.max_ctx, scale=self.scale, return_lse=True, workspace=ws)


def spare(c, n):
    """The case's pools with n free blocks behind, and their ids."""
    ids = torch.arange(c.nb, c.nb + n, dtype=torch.int32, device="cuda")
    for name in ("dk", "dks", "dv", "dvs"):
        p = getattr(c, name)
        setattr(c, name, torch.cat([p, torch.zeros(n, *p.shape[1:], dtype=p.dtype, device="cuda")]))
    return ids


@pytest.mark.parametrize("ctx,new,hq,hkv,d", [
    ([900, 300, 1500], [4, 4, 4], 64, 1, 128), ([900, 40000, 15], [3, 200, 15], 16, 2, 64), ([40, 20, 7], [1, 1, 1], 8, 8, 64)])
def test_captured_and_replayed(ctx, new, hq, hkv, d):
    c = Held(ctx, new, hq, hkv, d, 32, "bf16", seed=5)
    free = spare(c, 3 * 5)
    q, sums = c.q.cuda(), torch.rand(3, c.max_ctx, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(c, q, None, sums, free)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(c, q, None, sums, free)
    rng = np.random.default_rng(0)
    for i in range(6):
        log(f"[graph] replay {i} ctx={ctx} heads={hq}/{hkv} D={d}")
        lens = np.array(ctx if i in (0, 5) else [rng.integers(n, x + 1) for n, x in zip(new, ctx)], np.int32)
        c.dctx.copy_(dev(lens))
        q.copy_(torch.from_numpy(rng.normal(size=c.q.shape)).to(q.dtype))
        sums.copy_(torch.rand(3, c.max_ctx))
        want = [x.clone() for x in calls(c, q, None, sums, free)]
        pools = [x.clone() for x in (c.dk, c.dks, c.dv, c.dvs)]
        for x in (c.dk, c.dks, c.dv, c.dvs):
            x[c.nb:] = 0
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)
        for a, b in zip(pools, (c.dk, c.dks, c.dv, c.dvs)):
            assert torch.equal(a, b)


def test_another_stream_given_workspaces_and_strided_queries():
    import mqa_logits_amd as mq
    c = Held([900, 40000, 15], [3, 200, 15], 16, 2, 128, 64, "fp16", seed=6)
    free = spare(c, 3 * 2)
    q, sums = c.q.cuda(), torch.rand(3, c.max_ctx, device="cuda")
    want = calls(c, q, None, sums, free)
    n = len(q)
    sizes = (mq.paged_chunk_attention_workspace_size(3, n, 16, 2, 128, c.max_ctx),
             mq.paged_attention_weights_workspace_size(3, n, 16, 2, 128, c.max_ctx),
             mq.paged_kv_evict_workspace_size(3, c.max_ctx))
    wide = torch.full((n, 16 * 128 + 256), float("nan"), dtype=q.dtype, device="cuda")
    strided = wide[:, 64:64 + 16 * 128].unflatten(1, (16, 128))
    strided.copy_(q)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        # (what a workspace holds before does not matter)
        ws = [torch.full((max(s, 16),), 255, dtype=torch.uint8, device="cuda") for s in sizes]
        first = calls(c, strided, None, sums, free, ws=ws)
        again = calls(c, strided, None, sums, free, ws=ws)
    stream.synchronize()
    for a, b, x in zip(want, first, again):
        assert torch.equal(a, b) and torch.equal(a, x)


def test_two_streams_at_once():
    cases = [Held([900, 20000, 15], [3, 100, 15], 16, 2, 128, 64, "bf16", seed=i) for i in range(2)]
    frees = [spare(c, 3 * 2) for c in cases]
    qs, sums = [c.q.cuda() for c in cases], [torch.rand(3, c.max_ctx, device="cuda") for c in cases]
    want = [calls(c, q, None, s, f) for c, q, s, f in zip(cases, qs, sums, frees)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in cases], [None, None]
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = calls(cases[i], qs[i], None, sums[i], frees[i])
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for a, b in zip(w, g):
            assert torch.equal(a, b)


def test_beyond_32_bit_offsets():
    """A pool of 4.3 GB a side: keys in its last blocks, and free blocks there."""
    import mqa_logits_amd as mq
    bs, hkv, d = 64, 8, 128
    nb = (1 << 32) // (bs * hkv * d // 2) + 60
    c = Case([200, 64], [70, 64], 16, hkv, d, bs, seed=20)
    ids = np.array([nb - 1, 3, nb - 2, nb - 17, nb - 30], np.int32)
    old = np.concatenate([c.table[0, :4], c.table[1, :1]])
    pools = []
    for p in (c.k, c.ks, c.v, c.vs):
        big = torch.zeros(nb, *p.shape[1:], dtype=torch.uint8, device="cuda")
        if p.shape[-1] == d // 32:
            big.fill_(255)
        big[torch.from_numpy(ids).long().cuda()] = dev(p[old])
        pools.append(big)
    table = np.zeros((2, 4), np.int32)
    table[0], table[1, 0] = ids[:4], ids[4]
    q, off = c.q.cuda(), dev(c.offsets)
    want, want_lse = c.run()
    out, lse = mq.paged_chunk_attention("mxfp4", q, *pools, dev(c.ctx), off, dev(table), c.max_ctx, scale=c.scale, return_lse=True)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    ref = mq.paged_attention_weights("mxfp4", q, lse, dev(c.k), dev(c.ks), dev(c.ctx), off, dev(c.table), c.max_ctx, scale=c.scale)
    sums = mq.paged_attention_weights("mxfp4", q, lse, *pools[:2], dev(c.ctx), off, dev(table), c.max_ctx, scale=c.scale)
    assert torch.equal(sums, ref)
    free = np.array([nb - 5, nb - 6, 7], np.int32)
    e = mq.paged_kv_evict(sums, dev(c.ctx), dev(table), dev(free), pools, 100, 10, c.max_ctx)
    torch.cuda.synchronize()
    kept = e.kept[0].cpu().numpy()
    assert e.context_lens.tolist() == [100, 64] and (np.diff(kept) > 0).all()
    for p, small in zip(pools, (c.k, c.ks, c.v, c.vs)):
        rows = p[torch.from_numpy(free[np.arange(100) // bs]).long().cuda(), torch.arange(100).cuda() % bs].cpu().numpy()
        assert np.array_equal(rows, small[c.table[0, kept // bs], kept % bs])


def test_infinite_queries_stay_in_their_rows():
    for dtype in ("bf16", "fp16"):
        c = Case([300, 130], [40, 13], 10, 2, 128, 32, dtype, seed=4)
        clean, lse = c.run()
        c.q[7, 3, 5], c.q[45, 0, 0] = float("inf"), float("nan")
        out, lse_bad = c.run()
        same = torch.ones(53, 10, dtype=torch.bool, device="cuda")
        same[7, 3] = same[45, 0] = False
        assert torch.equal(out[same], clean[same]) and torch.equal(lse_bad[same], lse[same])


def test_fewer_candidates_than_stay_in_a_long_row():
    """NaNs of every kind are candidates, -inf is none."""
    import mqa_logits_amd as mq
    n, bs = 40000, 64
    w = np.full((2, n), -np.inf, np.float32)
    w.view(np.uint32)[0, [5, 17, 30000]] = 0xffffffff, 0xff800001, 0x7fffffff
    w[1, ::2] = -np.float32(3.0)
    args = dict(weights=w, context_lens=np.array([n, n], np.int32),
                block_table=np.arange(2 * 625, dtype=np.int32).reshape(2, 625), free_blocks=np.arange(1250, 2000, dtype=np.int32),
                pools=[np.random.default_rng(0).integers(0, 256, (2000, bs, 4), dtype=np.uint8)], keep=21000, recent=10,
                max_context_len=n)
    ref = cache.evict(**args)
    got = mq.paged_kv_evict(*(dev(args[x]) for x in ("weights", "context_lens", "block_table", "free_blocks")),
                            [dev(args["pools"][0])], 21000, 10, n)
    for name, g, r in zip(NAMES, got, ref):
        assert np.array_equal(g.cpu().numpy().view(np.int32), r.view(np.int32)), name
    assert got.context_lens.tolist() == [13, 19995 + 10]


def test_nothing_to_do():
    """No tokens, no context, or neither."""
    import mqa_logits_amd as mq
    c = Held([40, 7], [3, 2], 8, 2, 64, 16, "bf16", seed=1)
    free, zero = spare(c, 4), torch.zeros(3, dtype=torch.int32, device="cuda")
    q, sums = c.q.cuda(), torch.rand(2, c.max_ctx, device="cuda")
    pools = [c.dk, c.dks, c.dv, c.dvs]
    out, lse = mq.paged_chunk_attention("mxfp4", q[:0], *pools, c.dctx, zero, c.dtable, c.max_ctx, return_lse=True)
    assert out.shape == (0, 8, 64) and lse.shape == (0, 8)
    w = mq.paged_attention_weights("mxfp4", q[:0], lse, c.dk, c.dks, c.dctx, zero, c.dtable, c.max_ctx, weights=sums)
    seen = torch.arange(c.max_ctx, device="cuda") < c.dctx[:, None]
    assert torch.equal(w, torch.where(seen, sums, 0))
    # a bound of no keys
    out, lse = mq.paged_chunk_attention("mxfp4", q, *pools, c.dctx, c.doff, c.dtable[:, :0].contiguous(), 0, return_lse=True)
    assert not out.any() and bool((lse == -float("inf")).all())
    assert mq.paged_attention_weights("mxfp4", q, lse, c.dk, c.dks, c.dctx, c.doff, c.dtable, 0).shape == (2, 0)
    e = mq.paged_kv_evict(sums, c.dctx, c.dtable, free, pools, 20, 5, 0)
    assert e.context_lens.tolist() == [0, 0] and e.counts.tolist() == [0, 0] and bool((e.kept == -1).all())
    # an empty free list
    e = mq.paged_kv_evict(sums, c.dctx, c.dtable, free[:0], pools, 20, 5, c.max_ctx)
    assert e.context_lens.tolist() == [40, 7] and e.counts.tolist() == [2, 0] and torch.equal(e.weights, w)


def test_contexts_beyond_their_bound_and_of_negative_length():
    for hq, hkv, new in ((8, 2, 3), (64, 1, 6)):
        c = Held([300, 90, 500], [new] * 3, hq, hkv, 64, 16, "fp16", max_ctx=200, seed=3)
        c.ctx[1] = -4
        c.dctx = dev(c.ctx)
        out, lse = c.check("bounded")
        import mqa_logits_amd as mq
        w = mq.paged_attention_weights("mxfp4", c.q.cuda(), lse, c.dk, c.dks, c.dctx, c.doff, c.dtable, 200, scale=c.scale)
        assert not w[1].any() and bool((w[0] > 0).any()) and bool((w[2, -1:] > 0).all())
