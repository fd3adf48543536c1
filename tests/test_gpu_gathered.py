"""GPU parity of the attention weight that cached tokens gather, against float64.

Tolerances are the oracle's per-entry bounds (oracle.cache.gathered).  Unread pool
slots hold random codes under NaN scales, so a key that a row does not see, or a
wrong block, cannot pass.
"""

import numpy as np
import pytest
import torch

from oracle import cache
from tests.gpu_helpers import dev, log
from tests.test_gpu_attention import assert_within
from tests.test_gpu_chunk import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mqa_logits_amd  # noqa: F401


def lengths(c):
    return np.clip(c.ctx, 0, c.max_ctx)


def true_lse(c):
    """fp32 lse of every row, -inf without keys and for rows of nobody."""
    with np.errstate(all="ignore"):
        _, lse, _, _ = c.reference()
    return torch.from_numpy(lse.astype(np.float32))


def gather(c, lse, **kw):
    import mqa_logits_amd as mq
    args = dict(q=c.q.cuda(), token_offsets=dev(c.offsets))
    args.update(kw)
    return mq.paged_attention_weights("mxfp4", args.pop("q"), lse, dev(c.k), dev(c.ks), dev(c.ctx),
                                      args.pop("token_offsets"), dev(c.table), c.max_ctx, scale=c.scale, **args)


def check(c, what, before=True, lse=None):
    log(f"[gathered] {what} ctx={c.ctx[:4]}.. offsets={c.offsets[:5]}.. heads={c.q.shape[1]}/{c.k.shape[2]} "
        f"D={c.q.shape[2]} bs={c.bs} {c.dtype} max_ctx={c.max_ctx}")
    lse = true_lse(c) if lse is None else lse
    old = torch.rand(len(c.ctx), c.max_ctx + 3) if before else None
    out = torch.full((len(c.ctx), c.max_ctx + 5), 7.0, device="cuda")
    gather(c, lse.cuda(), weights=None if old is None else old.cuda(), out=out)
    torch.cuda.synchronize()
    got = out.double().cpu().numpy()
    assert np.all(got[:, c.max_ctx:] == 7.0)
    with np.errstate(all="ignore"):
        ref, tol = cache.gathered(c.q.double().numpy(), lse.numpy(), c.k, c.ks, c.table, *c.rows(), c.scale, lengths(c),
                                  None if old is None else old.numpy())
    ref, tol = [np.pad(x[:, :c.max_ctx], ((0, 0), (0, max(0, c.max_ctx - x.shape[1])))) for x in (ref, tol)]
    ref, tol = [x * (np.arange(c.max_ctx) < lengths(c)[:, None]) for x in (ref, tol)]
    assert_within(got[:, :c.max_ctx], ref, tol, what)
    return out, old, lse


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(8, 1), (15, 3), (33, 1), (64, 1), (8, 8)])
def test_heads(hq, hkv, d, dtype):
    check(Case([70, 1, 0, 300, 129], [3, 1, 0, 4, 33], hq, hkv, d, 32, dtype, seed=hq + d), "heads")


@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("ctx,new", [
    ([1], [1]), ([31], [1]), ([32], [2]), ([33], [33]), ([127, 128, 129], [1, 1, 1]), ([700], [70]),
    ([0, 5, 0, 64], [0, 5, 0, 1]), ([2100, 3], [2, 3]),
])
def test_lengths(ctx, new, bs):
    check(Case(ctx, new, 12, 2, 64, bs, "fp16", seed=sum(ctx) + bs, pad=3), "lengths", before=False)
    check(Case(ctx, new, 8, 2, 128, bs, "bf16", seed=sum(ctx) + bs), "lengths")


def test_limits_of_lengths():
    check(Case([900, 3, -4, 40], [20, 7, 2, 40], 8, 2, 128, 16, "bf16", max_ctx=600, seed=8), "limits")


@pytest.mark.parametrize("d", [64, 128])
def test_key_scales_outside_fp16(d):
    c = Case([300, 130], [7, 13], 10, 2, d, 32, "fp16", seed=d)
    rng = np.random.default_rng(2)
    held = (c.ks <= 252) & (rng.random(c.ks.shape) < 0.02)
    c.ks[held] = rng.integers(60, 104, held.sum())
    check(c, "K's scales")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_nan_keys_and_rows_without_lse(dtype):
    c = Case([300, 130], [7, 13], 10, 2, 128, 32, dtype, seed=4)
    lse = true_lse(c)
    for b, j in [(0, 250), (1, 129), (1, 120)]:
        page, at = c.slot(b, j)
        c.ks[page, at, 1, j % 4] = 253 + j % 3
    lse[3], lse[9, 2] = -np.inf, -np.inf
    out, old, _ = check(c, "NaN keys", lse=lse)
    assert torch.isnan(out).sum() == 3
    lse[15, 1] = np.nan                      # the eighth of 13 rows: its own keys, and no others
    out, _, _ = check(c, "NaN lse", lse=lse)
    assert torch.isnan(out[1]).sum() == 130 - 13 + 1 + 8 + 1


def test_in_place_and_uniform_rows():
    c = Case([300, 130], [4, 4], 8, 2, 128, 32, "bf16", seed=4)
    lse = true_lse(c).cuda()
    once = gather(c, lse)
    sums = torch.zeros_like(once)
    for _ in range(2):
        assert gather(c, lse, weights=sums, out=sums, token_offsets=None) is sums
    assert torch.equal(sums, once + once)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_after_attention(dtype):
    """The sums of a chunk's weights are its rows: each row gives 1 a head."""
    c = Case([400, 130, 64], [70, 13, 64], 8, 2, 128, 32, dtype, seed=4)
    out, lse = c.run()
    sums = gather(c, lse)
    got = sums.double().sum(1).cpu().numpy()
    assert np.allclose(got, 8 * np.array([70, 13, 64]), rtol=1e-5)
