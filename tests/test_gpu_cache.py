"""GPU parity of the cache's upkeep: slot maps and quantising writes.

Everything here is whole numbers or exactly defined codes, so every comparison
is bit for bit.
"""

import numpy as np
import pytest
import torch

import oracle
from oracle import cache
from tests.gpu_helpers import dev, log

pytestmark = pytest.mark.gpu

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mqa_logits_amd  # noqa: F401


# ---------------------------------------------------------------------------
# slots
# ---------------------------------------------------------------------------

def slots_case(ctx, new, block_size, max_context_len, max_tokens, seed=0, short=0, extra=3):
    rng = np.random.default_rng(seed)
    ctx, new = np.asarray(ctx, np.int32), np.asarray(new, np.int32)
    c = np.clip(ctx.astype(np.int64), 0, max_context_len)
    old = c - np.clip(new, 0, c)
    held = -(-old // block_size)
    take = int((-(-c // block_size) - held).sum())
    num_blocks = int(held.sum()) + take + 5
    ids = rng.permutation(num_blocks).astype(np.int32)
    width = -(-max_context_len // block_size) + extra
    table = np.full((len(ctx), width), -7, np.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = ids[at:at + n]
        at += n
    return (ctx, new, ids[at:at + max(take - short, 0)], table, num_blocks, block_size,
            max_context_len, max_tokens)


def check_slots(case, what):
    import mqa_logits_amd as mq
    ctx, new, free, table, num_blocks, bs, max_ctx, max_tokens = case
    log(f"[slots] {what} batch={len(ctx)} bs={bs} max_tokens={max_tokens}")
    ref = cache.kv_slots(ctx, new, free, table, num_blocks, bs, max_ctx, max_tokens)
    wide = torch.full((table.shape[0], table.shape[1] + 2), -9, dtype=torch.int32, device="cuda")
    view = wide[:, :table.shape[1]]
    view.copy_(dev(table))
    for _ in range(2):                            # the same call again changes nothing
        slots, offsets, taken = mq.paged_kv_slots(dev(ctx), dev(new), dev(free), view, num_blocks,
                                                  bs, max_ctx, max_tokens)
        for got, want, name in zip((slots, offsets, taken, view), ref,
                                   ("slots", "offsets", "taken", "table")):
            assert np.array_equal(got.cpu().numpy(), want), f"{what}: {name} differ"
        assert bool((wide[:, table.shape[1]:] == -9).all()), "columns behind the table"


@pytest.mark.parametrize("bs", [16, 32, 64])
def test_slots_edges(bs):
    ctx = [0, 1, bs - 1, bs, bs + 1, 5 * bs, 200, 7, -3, 10 ** 6]
    new = [0, 1, 1, bs, 1, 2 * bs + 3, 0, 99, 4, 5]
    check_slots(slots_case(ctx, new, bs, 400, 600, seed=bs), "edges")


def test_slots_block_boundaries():
    for old in range(0, 34):
        for n in (1, 15, 16, 17):
            check_slots(slots_case([old + n, old], [n, old], 16, 64, 60, seed=old), f"{old}+{n}")


@pytest.mark.parametrize("batch", [1, 63, 64, 65, 511, 512, 513, 1500, 8192])
def test_slots_batches(batch):
    rng = np.random.default_rng(batch)
    ctx = rng.integers(0, 300, batch)
    new = np.where(rng.random(batch) < 0.3, 0, rng.integers(0, 40, batch))
    total = int(np.minimum(new, ctx).sum())
    check_slots(slots_case(ctx, new, 16, 300, total + 17, seed=batch), "batches")


def test_slots_fresh_prompts():
    ctx = np.random.default_rng(8).integers(1, 4000, 90)
    check_slots(slots_case(ctx, ctx, 64, 4000, int(ctx.sum())), "prompts")


def test_slots_free_list_runs_out():
    check_slots(slots_case([100, 50, 70], [100, 20, 70], 16, 128, 200, short=6), "short list")
    check_slots(slots_case([100, 50, 70], [100, 20, 70], 16, 128, 200, short=100), "no list")


def test_slots_more_tokens_than_asked_for():
    check_slots(slots_case([100, 50, 70], [100, 20, 70], 16, 128, 131), "cut")
    check_slots(slots_case([100, 50, 70], [100, 20, 70], 16, 128, 0), "none")


def test_slots_missing_older_block():
    case = list(slots_case([40, 40, 40], [3, 3, 3], 16, 64, 9))
    case[3][0, 2], case[3][1, 2] = -1, case[4]        # new tokens 37..39 lie in these blocks
    check_slots(tuple(case), "bad ids")


def test_slots_no_context():
    check_slots(slots_case([0, 5], [0, 5], 16, 0, 4, extra=0), "max_context_len 0")


# ---------------------------------------------------------------------------
# writes
# ---------------------------------------------------------------------------

def rows_of(kind, n, heads, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, heads, d, generator=g)
    if kind == "normal":
        x = x * torch.exp2(torch.randint(-12, 12, (n, heads, 1), generator=g).float())
    elif kind == "ties":
        # multiples of 1/8 under a maximum of 6 (e2m1's ties) or 1/1024 under 448
        x = torch.randint(-48, 49, (n, heads, d), generator=g) / 8.0
        x[..., ::32] = 6.0
        x[: n // 2] = torch.randint(-448, 449, (n // 2, heads, d), generator=g).float()
        x[: n // 2, :, 0] = 448.0
    elif kind == "edges":
        x[::5] = 0.0
        x[1::5, :, 3] = float("inf")
        x[2::5, :, d - 1] = float("nan")
        x[3::5, :, 5] = -float("inf")
        x[4::5] *= 1e-30 if dtype == torch.float32 else 1e-7
        x[:, :, 7] = -0.0
    elif kind == "tiny":
        x = x * torch.exp2(torch.randint(-149, -118, (n, heads, 1), generator=g).double()).float()
    elif kind == "huge":
        x = (x.double() * torch.exp2(torch.randint(120, 127, (n, heads, 1), generator=g).double()))
        x = x.clamp(-3.3e38, 3.3e38).float()
    return x.to(dtype)


def check_write(fmt, x, bs, seed=0, drop=True, values=True, one_head_pool=False):
    import mqa_logits_amd as mq
    n, heads, d = x.shape
    rng = np.random.default_rng(seed)
    nb = -(-n // bs) + 2
    slots = rng.permutation(nb * bs)[:n].astype(np.int64)
    if drop and n > 3:
        slots[n // 2], slots[0], slots[n - 1] = -1, nb * bs, 2 ** 40
    width = d // 2 if fmt == "mxfp4" else d
    pool = rng.integers(0, 256, (nb, bs, heads, width), dtype=np.uint8)
    sf = None if fmt == "fp8" else rng.integers(0, 256, (nb, bs, heads, d // 32), dtype=np.uint8)
    scale = rng.random((nb, bs, heads)).astype(np.float32) if fmt == "fp8" else None
    X = x.cuda()
    P, S, C = dev(pool), dev(sf), dev(scale)
    args = X, P, S, C
    if one_head_pool:
        args = X[:, 0], P[:, :, 0], None if S is None else S[:, :, 0], None if C is None else C[:, :, 0]
    V = torch.full(args[0].shape, 7.0, dtype=x.dtype, device="cuda") if values else None
    log(f"[write] {fmt} n={n} heads={heads} D={d} {x.dtype}")
    mq.paged_kv_write(fmt, args[0], dev(slots), *args[1:], values=V)
    with np.errstate(all="ignore"):
        codes, scales, held = cache.quantise(fmt, x.double().numpy())
    kept = (slots >= 0) & (slots < nb * bs)
    pool.reshape(nb * bs, heads, width)[slots[kept]] = codes[kept]
    assert np.array_equal(P.cpu().numpy(), pool), "codes differ"
    if fmt == "fp8":
        scale.reshape(nb * bs, heads)[slots[kept]] = scales[kept]
        assert np.array_equal(C.cpu().numpy(), scale, equal_nan=True), "scales differ"
    else:
        sf.reshape(nb * bs, heads, d // 32)[slots[kept]] = scales[kept]
        assert np.array_equal(S.cpu().numpy(), sf), "block scales differ"
    if values:
        want = torch.from_numpy(held).to(x.dtype).numpy(force=True) if x.dtype != torch.bfloat16 \
            else torch.from_numpy(held).to(x.dtype).float().numpy()
        got = V.reshape(n, heads, d).float().cpu() if x.dtype == torch.bfloat16 else V.reshape(n, heads, d).cpu()
        assert np.array_equal(got.numpy(), want, equal_nan=True), "values differ"


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fmt", ["fp8", "mxfp8", "mxfp4"])
def test_write_formats(fmt, d, dtype):
    for kind in ("normal", "ties", "edges"):
        for n, heads in ((1, 1), (37, 1), (130, 3), (16, 8)):
            check_write(fmt, rows_of(kind, n, heads, d, DTYPES[dtype], n + d), 16, seed=n)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp8", "mxfp4"])
def test_write_extremes(fmt):
    for kind in ("tiny", "huge"):
        for dtype in ("fp32", "bf16"):
            check_write(fmt, rows_of(kind, 300, 2, 128, DTYPES[dtype], 5), 32)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp8", "mxfp4"])
def test_write_every_bf16(fmt):
    # every bf16 value once, each group with values of like magnitude
    bits = torch.arange(65536, dtype=torch.int32).to(torch.uint16).view(torch.bfloat16)
    check_write(fmt, bits.view(-1, 2, 64), 64, drop=False)
    mixed = bits.view(-1, 128, 2).transpose(1, 2).reshape(-1, 2, 128)
    check_write(fmt, mixed.contiguous(), 64, drop=False)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp8", "mxfp4"])
def test_write_one_head_pool(fmt):
    check_write(fmt, rows_of("normal", 50, 1, 128, torch.bfloat16, 2), 64, one_head_pool=True)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
def test_write_strided_rows(fmt):
    # K heads inside a fused projection: rows and heads apart, in either order
    import mqa_logits_amd as mq
    wide = torch.randn(70, 3, 4, 128, device="cuda").to(torch.bfloat16)
    for x in (wide[:, 1], wide[::2, 0], wide[:, :, 2], wide.transpose(0, 1)[1]):
        n, heads = x.shape[:2]
        slots = torch.randperm(128, device="cuda")[:n]
        outs = []
        for src in (x, x.contiguous()):
            pool = torch.zeros(4, 32, heads, 64 if fmt == "mxfp4" else 128, dtype=torch.uint8, device="cuda")
            sf = torch.zeros(4, 32, heads, 4, dtype=torch.uint8, device="cuda") if fmt == "mxfp4" else None
            sc = torch.zeros(4, 32, heads, device="cuda") if fmt == "fp8" else None
            mq.paged_kv_write(fmt, src, slots, pool, sf, sc)
            outs.append((pool, sf if sc is None else sc))
        for a, b in zip(*outs):
            assert torch.equal(a, b)


def test_write_values_in_place():
    import mqa_logits_amd as mq
    x = torch.randn(100, 2, 128, device="cuda").to(torch.bfloat16)
    y = x.clone()
    slots = torch.full((100,), -1, device="cuda")
    pool = torch.zeros(1, 16, 2, 64, dtype=torch.uint8, device="cuda")
    sf = torch.zeros(1, 16, 2, 4, dtype=torch.uint8, device="cuda")
    v = mq.paged_kv_write("mxfp4", x, slots, pool, sf, values=torch.empty_like(x))
    mq.paged_kv_write("mxfp4", y, slots, pool, sf, values=y)
    assert torch.equal(v, y) and not pool.any() and not sf.any()


def test_written_pool_feeds_the_paged_logits():
    # FP8 keys through the slot map into the pool that paged_mqa_logits reads: the
    # logits are those of a pool assembled on the host from the oracle's codes
    import mqa_logits_amd as mq
    rng = np.random.default_rng(11)
    batch, next_n, bs, h, d, max_ctx = 5, 2, 16, 64, 128, 200
    ctx = np.array([1, 200, 33, 64, 150], np.int32)
    table = torch.full((batch, 13), -1, dtype=torch.int32, device="cuda")
    nb = int((-(-ctx // bs)).sum()) + 4
    free = rng.permutation(nb).astype(np.int32)
    total = int(ctx.sum())
    slots, offsets, taken = mq.paged_kv_slots(dev(ctx), dev(ctx), dev(free), table, nb, bs, max_ctx,
                                              total)
    x = torch.from_numpy(rng.normal(size=(total, d))).to(torch.bfloat16)
    pool = torch.full((nb, bs, d), 0x7f, dtype=torch.uint8, device="cuda")
    scale = torch.full((nb, bs), float("nan"), device="cuda")
    mq.paged_kv_write("fp8", x.cuda(), slots, pool, None, scale)
    q = synth_codes(rng, (batch * next_n, h, d))
    w = rng.normal(size=(batch * next_n, h)).astype(np.float32)
    sched = mq.paged_mqa_logits_metadata(dev(ctx), next_n, bs, max_ctx, 64)
    got = mq.paged_mqa_logits("fp8", dev(q), None, pool, None, scale, dev(w), dev(ctx), table, sched,
                              next_n, max_ctx)
    codes, scales, _ = cache.quantise("fp8", x.double().numpy())
    rs, _, _, rt = cache.kv_slots(ctx, ctx, free, np.full((batch, 13), -1), nb, bs, max_ctx, total)
    rp, rsc = np.full((nb * bs, d), 0x7f, np.uint8), np.full(nb * bs, np.nan, np.float32)
    rp[rs], rsc[rs] = codes, scales
    ref, bound = oracle.paged_logits("fp8", q, None, rp.reshape(nb, bs, d), None, rsc.reshape(nb, bs),
                                     w, ctx, rt, next_n, bs, max_ctx)
    from tests.gpu_helpers import assert_close
    assert_close(got.cpu().numpy(), ref, bound, "written pool")


def synth_codes(rng, shape):
    import synth
    return synth.encode_e4m3(rng.normal(size=shape))
