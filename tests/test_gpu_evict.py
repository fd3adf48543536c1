"""GPU parity of eviction from the paged cache: every output and every pool byte."""

import numpy as np
import pytest
import torch

from oracle import cache
from tests.gpu_helpers import dev, log

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mqa_logits_amd  # noqa: F401


# bytes of a token in each pool (and shapes), every width of piece among them
POOLS = {"mqa": [(64,), (4,), (64,), (4,), (128,), ()], "odd": [(3, 32), (3, 2), (5,), (1,), (2, 3), (16,)],
         "one": [(8, 64)]}


def case(ctx, keep, recent, bs=16, pools="mqa", free=None, max_ctx=None, seed=0, extra=1):
    rng = np.random.default_rng(seed)
    ctx = np.asarray(ctx, np.int32)
    max_ctx = int(max(ctx.max(), 1)) if max_ctx is None else max_ctx
    n = np.clip(ctx, 0, max_ctx)
    need = -(-n // bs)
    enough = int(np.sum(-(-np.minimum(n, keep)[n > keep] // bs)))
    free = enough + 2 if free is None else free
    nb = int(need.sum()) + free + 3
    ids = rng.permutation(nb).astype(np.int32)
    table = rng.integers(-5, nb + 5, (len(ctx), -(-max_ctx // bs) + extra)).astype(np.int32)
    at = 0
    for b in range(len(ctx)):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
    data = []
    for i, shape in enumerate(POOLS[pools]):
        if shape == ():
            data.append(rng.random((nb, bs)).astype(np.float32))
        else:
            data.append(rng.integers(0, 256, (nb, bs, *shape), dtype=np.uint8))
    w = rng.gamma(0.2, size=(len(ctx), max_ctx + extra)).astype(np.float32)
    w[rng.random(w.shape) < 0.2] = 0.0
    w[rng.random(w.shape) < 0.1] = 0.5
    return dict(weights=w, context_lens=ctx, block_table=table, free_blocks=ids[at:at + free], pools=data,
                keep=keep, recent=recent, max_context_len=max_ctx)


NAMES = "context_lens block_table weights kept freed counts".split()


def check(c, **kw):
    import mqa_logits_amd as mq
    log(f"[evict] ctx={c['context_lens'][:5]}.. keep={c['keep']} recent={c['recent']} "
        f"pools={[p.shape for p in c['pools']]} free={len(c['free_blocks'])}")
    args = dict(c, pools=[dev(p) for p in c["pools"]])
    for name in ("weights", "context_lens", "block_table", "free_blocks"):
        args[name] = dev(c[name])
    got = mq.paged_kv_evict(**args, **kw)
    torch.cuda.synchronize()
    ref = cache.evict(**c)
    for name, g, r in zip(NAMES, got, ref):
        g = g.cpu().numpy()
        if name in ("block_table", "weights", "kept"):
            g = g[:, :r.shape[1]]
        assert np.array_equal(g.view(np.int32), r.view(np.int32)), name
    for i, (g, r) in enumerate(zip(args["pools"], ref[-1])):
        assert np.array_equal(g.cpu().numpy().view(np.uint8), r.view(np.uint8)), f"pool {i}"
    return got, args


@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("pools", list(POOLS))
@pytest.mark.parametrize("ctx,keep,recent", [
    ([0, 1, 50, 129, 200], 48, 16), ([100], 99, 0), ([100], 99, 99), ([100], 100, 5), ([300, 7], 1, 0),
    ([300, 7], 1, 1), ([700, 700, 700], 130, 65), ([1, 2, 3], 2, 1),
])
def test_lengths(ctx, keep, recent, pools, bs):
    check(case(ctx, keep, recent, bs, pools, seed=sum(ctx) + keep))


def test_many_sequences():
    rng = np.random.default_rng(1)
    check(case(rng.integers(0, 90, 1500), 33, 5, 16, "odd", seed=2))


def test_long():
    check(case([9000, 20, 5000], 1030, 100, 64, "mqa", seed=2))


@pytest.mark.parametrize("keep,recent", [(16000, 1000), (1, 0), (40000, 39999), (300, 300), (30000, 5)])
def test_long_rows(keep, recent):
    """Rows beyond what one workgroup selects from."""
    check(case([40960, 33000, 9000, 40000], keep, recent, 64, "one", seed=keep))


def test_long_rows_of_equal_and_unusual_weights():
    c = case([50000] * 7 + [100], 20000, 50, 64, "one", seed=6)
    w, n = c["weights"], 50000
    w[0] = 1.0
    w[1, ::2], w[1, 1::2] = np.inf, -0.0
    w[2, :40000] = -np.inf                   # fewer than keep can stay
    w[3] = -np.inf                           # the recent ones alone
    w[4, 5::3000] = np.nan
    w[5] = np.random.default_rng(1).integers(0, 2 ** 32, w.shape[1], dtype=np.uint32).view(np.float32)
    w[6] = np.float32(1.0) + np.arange(w.shape[1], dtype=np.float32) % 3 * np.float32(2.0 ** -23)
    check(c)


def test_limits_of_lengths():
    check(case([900, -4, 40], 64, 20, 16, max_ctx=600, seed=3))
    check(case([10, 20], 300, 20, 16, seed=3))                  # keep beyond every sequence
    check(case([0, 0], 5, 1, 16, max_ctx=0, seed=3, extra=1))


@pytest.mark.parametrize("free", [0, 1, 3, 4, 6, 7])
def test_free_list_runs_out(free):
    got, _ = check(case([100, 30, 200, 90, 64], 48, 16, 16, free=free, seed=5))
    assert got.counts[0] == 12


def test_equal_and_unusual_weights():
    c = case([200, 150, 90, 80, 70], 40, 8, 16, seed=6)
    w = c["weights"]
    w[0] = 1.0
    w[1, ::2], w[1, 1::2] = np.inf, -0.0
    w[2, :60] = -np.inf                      # fewer than keep can stay
    w[3] = -np.inf                           # the recent ones alone
    w[4, 5] = np.nan
    got, _ = check(c)
    assert got.context_lens.tolist() == [40, 40, 30, 8, 40]
    assert got.kept[0, :32].tolist() == list(range(32)) and 5 in got.kept[4].tolist()


def test_nothing_stays():
    c = case([50], 8, 0, 16, seed=6)
    c["weights"][:] = -np.inf
    got, _ = check(c)
    assert got.context_lens.tolist() == [0] and got.counts.tolist() == [0, 4]


def test_bad_blocks_are_passed_over():
    c = case([100, 120], 48, 16, 16, seed=7)
    c["block_table"][0, 2], c["block_table"][1, 0] = -1, 10 ** 6
    c["free_blocks"][1] = -7
    check(c)


def test_again_and_given_outputs():
    import mqa_logits_amd as mq
    c = case([100, 30, 200], 48, 16, 16, seed=8)
    got, args = check(c)
    i32 = dict(dtype=torch.int32, device="cuda")
    out = (torch.empty(3, **i32), torch.full((3, 20), 9, **i32), torch.full((3, 210), 9.0, device="cuda"),
           torch.full((3, 50), 9, **i32), torch.empty(3 * 13, **i32), torch.empty(2, **i32))
    ws = torch.empty(mq.paged_kv_evict_workspace_size(3, c["max_context_len"]), dtype=torch.uint8, device="cuda")
    again = mq.paged_kv_evict(**args, out=out, workspace=ws)
    for name, a, b in zip(NAMES, got, again):
        b = b[:, :a.shape[1]] if a.dim() == 2 else b
        assert torch.equal(a, b), name
    assert (out[1][:, 13:] == 9).all() and (out[2][:, 200:] == 9).all() and (out[3][:, 48:] == 9).all()


def test_shared_blocks_stay():
    c = case([100, 100], 48, 16, 16, seed=9)
    c["block_table"][1] = c["block_table"][0]                 # one prefix, two sequences
    check(c)
