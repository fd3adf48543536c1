"""GPU parity of attention's three kernels at their own edges.

Which kernel runs goes by the heads and by the steps of 128 keys that
max_context_len (or topk) allows for, so a large bound over short contexts
reaches each one with little work: 4, 8 .. KV heads of up to 16 rows a KV head
per wave, over 64 rows of a KV head the wide one, the others keys over waves.
"""

import numpy as np
import pytest
import torch

from oracle import cache
from tests.gpu_helpers import dev
from tests.test_gpu_attention import Case, assert_within

pytestmark = pytest.mark.gpu

# hq, hkv, next_n that make a kernel of a long bound
HEADS = [(8, 4, 1), (64, 8, 1), (8, 8, 3), (32, 4, 2), (12, 12, 16)]
WIDE = [(65, 1, 1), (128, 1, 1), (64, 1, 2), (64, 1, 4), (200, 2, 1), (40, 2, 16)]
TWO_GROUPS = [(33, 1, 1), (64, 1, 1), (16, 1, 4), (80, 2, 1), (4, 1, 12)]    # of 32 rows
LENGTHS = [0, 1, 15, 16, 17, 31, 33, 47, 48, 63, 64, 65, 95, 97, 127, 128, 129, 143, 160, 161, 255,
           256, 257, 300, 511, 513]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mqa_logits_amd  # noqa: F401


@pytest.mark.parametrize("d,dtype,bs", [(128, "bf16", 16), (64, "fp16", 32), (128, "fp16", 64),
                                        (64, "bf16", 16)])
@pytest.mark.parametrize("hq,hkv,next_n", HEADS)
def test_a_head_per_wave(hq, hkv, next_n, d, dtype, bs):
    Case(LENGTHS, next_n=next_n, hq=hq, hkv=hkv, d=d, bs=bs, dtype=dtype, max_ctx=65536,
         seed=hq + d).check("heads")


@pytest.mark.parametrize("d,dtype,bs", [(128, "bf16", 16), (64, "fp16", 32), (128, "fp16", 64),
                                        (64, "bf16", 16)])
@pytest.mark.parametrize("hq,hkv,next_n", WIDE + TWO_GROUPS)
def test_many_rows(hq, hkv, next_n, d, dtype, bs):
    Case(LENGTHS[::2], next_n=next_n, hq=hq, hkv=hkv, d=d, bs=bs, dtype=dtype, max_ctx=262144,
         seed=hq + d).check("wide")


@pytest.mark.parametrize("hq,hkv,next_n", [(8, 4, 2), (64, 1, 2), (20, 2, 3), (6, 2, 1), (64, 1, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_contexts_longer_than_a_stage(hq, hkv, next_n, dtype):
    # more keys than a workgroup holds places for at a time
    d = 64
    Case([40000, 16385, 16384, 33], next_n=next_n, hq=hq, hkv=hkv, d=d, bs=64, dtype=dtype,
         max_ctx=1 << 20, seed=hq).check("stages")


@pytest.mark.parametrize("batch", [63, 64, 65, 256, 257, 700])
@pytest.mark.parametrize("hq,hkv,next_n", [(2, 1, 1), (4, 4, 1), (33, 1, 2), (33, 1, 1)])
def test_batches(batch, hq, hkv, next_n):
    # the search for a worker's first sequence: up to 64 at once, or 256 by 256
    lens = np.random.default_rng(batch).integers(0, 200, batch)
    lens[::7] = 0
    for max_ctx in (200, 60000):
        Case(lens, next_n=next_n, hq=hq, hkv=hkv, d=64, bs=16, max_ctx=max_ctx, seed=batch).check("batch")


def wide_selection(c, topk, seed):
    """Few valid entries spread over a long list."""
    rng = np.random.default_rng(seed)
    rows = c.q.shape[0]
    c.topk = topk
    c.indices = np.full((rows, topk), -1, np.int32)
    for r in range(rows):
        n = int(rng.integers(0, 120))
        at = rng.permutation(topk)[:n]
        c.indices[r, at] = rng.integers(-3, 700, n)
    c.indices[0] = -1
    c.indices[1, :64] = np.arange(64)          # whole tiles of valid keys, nothing else
    c.indices[1, 64:] = -1
    return c


@pytest.mark.parametrize("hq,hkv,topk", [(64, 64, 3000), (8, 4, 8000), (130, 1, 70000), (50, 1, 70000)])
@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp16")])
def test_selected_keys_of_each_kernel(hq, hkv, topk, d, dtype):
    rng = np.random.default_rng(hq)
    c = Case(rng.integers(0, 700, 12), next_n=1, hq=hq, hkv=hkv, d=d, bs=16, dtype=dtype, max_ctx=700,
             seed=hq)
    wide_selection(c, topk, hq).check("selected")


@pytest.mark.parametrize("rows", [1, 2, 7, 256, 300, 512])
def test_selected_keys_whole_units(rows):
    # rows that divide evenly over the workers (nothing to join) and rows that do not
    Case([500] * rows, next_n=1, hq=40, hkv=1, d=64, bs=64, topk=200, seed=rows).check("units")


@pytest.mark.parametrize("hq,hkv,next_n,max_ctx", [(8, 4, 4, 65536), (64, 1, 4, 262144), (6, 2, 4, 600),
                                                    (14, 1, 4, 262144)])
@pytest.mark.parametrize("d", [64, 128])
def test_nan_in_each_kernel(hq, hkv, next_n, max_ctx, d):
    # NaN scales of K and of V in the middle of contexts, at tile and step
    # edges, and in keys that only the last query tokens see
    for side in ("k", "v"):
        c = Case([300, 131, 0, 520, 129], next_n=next_n, hq=hq, hkv=hkv, d=d, bs=16, max_ctx=max_ctx,
                 seed=d)
        at = c.kept()
        sf = c.ks if side == "k" else c.vs
        for b, j in ((0, 40), (0, 298), (1, 129), (1, 130), (3, 127), (3, 128), (4, 127)):
            sf[at(b, j)][(b + j) % hkv, j % (d // 32)] = 253 + j % 3
        out, _ = c.check("nan " + side)
        assert bool(torch.isnan(out).any()) and bool(torch.isfinite(out).any())


@pytest.mark.parametrize("hq,hkv,max_ctx", [(8, 4, 65536), (128, 1, 262144), (8, 2, 3000), (64, 1, 262144)])
def test_late_maxima_in_each_kernel(hq, hkv, max_ctx):
    # keys that grow along the context: the running maximum is left behind again
    # and again, by far
    c = Case([2900, 700], hq=hq, hkv=hkv, bs=64, max_ctx=max_ctx, q_size=20.0, seed=3)
    at = c.kept()
    for b, n in ((0, 2900), (1, 700)):
        for j in range(n):
            c.ks[at(b, j)] = 118 + 12 * j // n
    c.check("late maxima")


def test_every_tile_count_of_each_kernel():
    # one sequence of n tiles and a bit, n = 0 .. 17, joined with a neighbour
    for hq, hkv, max_ctx in ((4, 4, 65536), (70, 1, 262144), (3, 1, 700), (25, 1, 524288)):
        for n in range(18):
            Case([32 * n + 5, 70], next_n=2, hq=hq, hkv=hkv, d=64, bs=32, max_ctx=max_ctx,
                 seed=n).check("tiles")


@pytest.mark.parametrize("hq,hkv,next_n,max_ctx,topk", [
    (64, 8, 1, 65536, 0), (64, 1, 4, 262144, 0), (64, 1, 1, 524288, 0), (32, 4, 1, 4000, 0), (64, 1, 1, 4000, 600)])
def test_graph_replays_over_growing_contexts(hq, hkv, next_n, max_ctx, topk):
    # lengths, queries and indices change between the replays of one graph
    import mqa_logits_amd as mq
    c = Case([1500, 900, 2000], next_n=next_n, hq=hq, hkv=hkv, bs=64, max_ctx=max_ctx, topk=topk, seed=5)
    k, ks, v, vs = (dev(x) for x in (c.k, c.ks, c.v, c.vs))
    ctx, table, q = dev(c.ctx), dev(c.table), c.q.cuda()
    indices = dev(c.indices)

    def run():
        return mq.paged_attention("mxfp4", q, k, ks, v, vs, ctx, table, next_n, max_ctx,
                                  scale=c.scale, indices=indices, return_lse=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = run()
    rng = np.random.default_rng(0)
    for lens in ([1500, 900, 2000], [0, 1, 2000], [5, 900, 64], [1500, 0, 0], [1499, 17, 1999]):
        ctx.copy_(dev(np.array(lens, np.int32)))
        q.copy_(torch.from_numpy(rng.normal(size=c.q.shape)).to(q.dtype))
        if topk:
            indices.copy_(dev(rng.integers(-1, 2000, c.indices.shape).astype(np.int32)))
        ref = run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    c.ctx, c.q = np.array(lens, np.int32), q.cpu()
    if topk:
        c.indices = indices.cpu().numpy()
    want, want_lse, tol, tol_lse = c.reference()
    assert_within(out.double().cpu().numpy(), want, tol, "replayed out")
    assert_within(lse.double().cpu().numpy(), want_lse, tol_lse, "replayed lse")


def test_two_graphs_with_their_own_workspaces():
    import mqa_logits_amd as mq
    cases = [Case([3000, 100], hq=16, hkv=2, seed=s) for s in (1, 2)]
    state = []
    for c in cases:
        args = [c.q.cuda()] + [dev(x) for x in (c.k, c.ks, c.v, c.vs, c.ctx, c.table)]
        size = mq.paged_attention_workspace_size(2, 1, 16, 2, 128, c.max_ctx)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        ref = mq.paged_attention("mxfp4", *args, 1, c.max_ctx, workspace=ws).clone()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = mq.paged_attention("mxfp4", *args, 1, c.max_ctx, workspace=ws)
        state.append((g, out, ref, args, ws))
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        for s, (g, *_rest) in zip(streams, state):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for _, out, ref, *_rest in state:
            assert torch.equal(out, ref)


def test_outputs_hold_nothing_but_their_rows():
    # guard rows behind the output, lse and indices; a q view inside wider rows
    import mqa_logits_amd as mq
    for hq, hkv, max_ctx in ((8, 4, 65536), (128, 1, 262144), (10, 2, 300), (60, 1, 524288)):
        c = Case([300, 17], hq=hq, hkv=hkv, bs=16, max_ctx=max_ctx, seed=4)
        out = torch.full((4, hq, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((4, hq), 3.0, device="cuda")
        wide = torch.full((2, hq + 5, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, 3:hq + 3] = c.q.cuda()
        c.run(q=wide[:, 3:hq + 3], out=out[1:3], lse=lse[1:3])
        ref = c.run()
        assert torch.equal(out[1:3], ref[0]) and torch.equal(lse[1:3], ref[1])
        assert bool((out[[0, 3]] == 3).all()) and bool((lse[[0, 3]] == 3).all())


def test_slots_write_attend_and_select_together():
    """Prompts through slots, writes and attention, then three decoding steps whose indexer logits
    (FP8 pool, same table) choose the keys, against the oracle on the host."""
    import oracle
    import synth
    import mqa_logits_amd as mq
    rng = np.random.default_rng(9)
    batch, next_n, hkv, group, d, bs, max_ctx, topk = 4, 2, 2, 4, 64, 16, 160, 24
    nb, ih, idim = 60, 32, 128
    i32 = dict(dtype=torch.int32, device="cuda")
    ctx = np.array([37, 5, 100, 16], np.int32)
    table = torch.full((batch, max_ctx // bs), -1, **i32)
    free = rng.permutation(nb).astype(np.int32)
    host_table, taken_so_far = np.full((batch, max_ctx // bs), -1, np.int32), 0
    pools = [torch.full((nb, bs, hkv, d // 2), 0x77, dtype=torch.uint8, device="cuda") for _ in range(2)]
    sfs = [torch.full((nb, bs, hkv, d // 32), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    ipool = torch.full((nb, bs, idim), 0x7f, dtype=torch.uint8, device="cuda")
    iscale = torch.full((nb, bs), float("nan"), device="cuda")
    new = ctx.copy()
    for step in range(4):
        if step:
            ctx, new = ctx + next_n, np.full(batch, next_n, np.int32)
        total = int(new.sum())
        slots, _, taken = mq.paged_kv_slots(dev(ctx), dev(new), dev(free[taken_so_far:]), table, nb, bs,
                                            max_ctx, total + 3)
        ref_slots, _, ref_taken, host_table = cache.kv_slots(ctx, new, free[taken_so_far:], host_table,
                                                             nb, bs, max_ctx, total + 3)
        assert np.array_equal(slots.cpu().numpy(), ref_slots)
        assert np.array_equal(table.cpu().numpy(), host_table) and int(taken) == ref_taken[0]
        taken_so_far += int(taken)
        x = torch.from_numpy(rng.normal(size=(2, total + 3, hkv, d))).to(torch.bfloat16)
        key = torch.from_numpy(rng.normal(size=(total + 3, idim))).to(torch.bfloat16)
        for side in range(2):
            mq.paged_kv_write("mxfp4", x[side].cuda(), slots, pools[side], sfs[side])
        mq.paged_kv_write("fp8", key.cuda(), slots, ipool, None, iscale)
        if not step:
            continue
        iq = synth.encode_e4m3(rng.normal(size=(batch * next_n, ih, idim)))
        w = rng.normal(size=(batch * next_n, ih)).astype(np.float32)
        sched = mq.paged_mqa_logits_metadata(dev(ctx), next_n, bs, max_ctx, 16)
        logits = mq.paged_mqa_logits("fp8", dev(iq), None, ipool, None, iscale, dev(w), dev(ctx), table,
                                     sched, next_n, max_ctx)
        picked = mq.mqa_logits_topk(logits, topk)
        assert np.array_equal(picked.cpu().numpy(),
                              oracle.topk_indices(logits.cpu().numpy().astype(np.float32), topk))
        q = torch.from_numpy(rng.normal(size=(batch * next_n, hkv * group, d))).to(torch.bfloat16)
        for indices in (None, picked):
            out, lse = mq.paged_attention("mxfp4", q.cuda(), pools[0], sfs[0], pools[1], sfs[1],
                                          dev(ctx), table, next_n, max_ctx, indices=indices,
                                          return_lse=True)
            want, want_lse, tol, tol_lse = cache.attention(
                q.double().numpy(), *(t.cpu().numpy() for t in (pools[0], sfs[0], pools[1], sfs[1])), ctx,
                host_table, next_n, max_ctx, d ** -0.5, 2.0 ** -8, 2.0 ** -8,
                indices=None if indices is None else indices.cpu().numpy())
            assert_within(out.double().cpu().numpy(), want, tol, "together out")
            assert_within(lse.double().cpu().numpy(), want_lse, tol_lse, "together lse")


@pytest.mark.parametrize("batch,hq,hkv", [(1, 8, 1), (5, 70, 1), (300, 8, 4), (1200, 16, 2)])
@pytest.mark.parametrize("topk", [0, 100, 128])
def test_units_of_one_step(batch, hq, hkv, topk):
    # no unit is ever cut, so there is no workspace, however many workgroups there are
    import mqa_logits_amd as mq
    lens = np.random.default_rng(batch).integers(0, 129, batch)
    assert mq.paged_attention_workspace_size(batch, 1, hq, hkv, 64, 128, topk) == 0
    Case(lens, hq=hq, hkv=hkv, d=64, bs=16, max_ctx=128, topk=topk, seed=batch).check("one step")


@pytest.mark.parametrize("hq,hkv,max_ctx", [(8, 4, 65536), (128, 1, 262144), (8, 2, 300), (64, 1, 524288)])
def test_largest_scales(hq, hkv, max_ctx):
    # a factor whose product with log2(e) is beyond fp32: scores of 0 weigh the same
    c = Case([300, 0, 40], hq=hq, hkv=hkv, bs=16, max_ctx=max_ctx, seed=6)
    c.q.zero_()
    for c.scale in (3.4e38, -3.4e38):
        out, lse = c.check("largest scale")
        assert bool(torch.isfinite(out).all())
