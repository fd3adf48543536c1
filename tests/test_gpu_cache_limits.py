"""GPU tests of the cache calls at the ends of their ranges; whole numbers and
exactly defined codes, compared bit for bit."""

import numpy as np
import pytest
import torch

from oracle import cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mqa_logits_amd  # noqa: F401


@pytest.mark.parametrize("bs", [32, 64])
@pytest.mark.parametrize("length,new", [(2 ** 31 - 2, 70), (2 ** 31 - 2, 1), (2 ** 31 - 30, 50), (2 ** 31 - 66, 3)])
def test_slots_of_lengths_near_2_to_the_31(length, new, bs):
    # a length rounded up to whole blocks passes int32
    import mqa_logits_amd as mq
    print(f"[slots] length {length} new {new} block {bs}", flush=True)
    max_ctx, nb = 2 ** 31 - 2, 9
    first, last = -(-(length - new) // bs), -(-length // bs)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.full((1, -(-max_ctx // bs)), -1, **i32)
    table[0, first - 1] = 7
    free = [3, 8, 5, 0, 1]
    slots, offsets, taken = mq.paged_kv_slots(
        torch.tensor([length], **i32), torch.tensor([new], **i32), torch.tensor(free, **i32), table,
        nb, bs, max_ctx, new + 2)
    torch.cuda.synchronize()
    block = {first - 1: 7, **{first + i: free[i] for i in range(last - first)}}
    want = [block[j // bs] * bs + j % bs for j in range(length - new, length)] + [-1, -1]
    assert slots.tolist() == want
    assert offsets.tolist() == [0, new] and taken.tolist() == [last - first]
    assert table[0, first:last].tolist() == free[:last - first]
    assert int((table != -1).sum()) == 1 + last - first


TOP = 1.5 * 2.0 ** 127


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_near_the_end_of_fp32(dtype):
    # Up to 1.5 * 2^127 a group's scale is 2^125 at most (byte 252), which attention
    # reads; the next magnitude takes byte 253, which it counts as NaN.
    import mqa_logits_amd as mq
    x = torch.ones(2, 1, 64, dtype=dtype, device="cuda")
    x[0, 0, 5], x[0, 0, 40] = TOP, -TOP / 4
    x[1, 0, 5] = torch.nextafter(torch.tensor(TOP, dtype=dtype), torch.tensor(float("inf"), dtype=dtype))
    codes, sf, values = cache.quantise("mxfp4", x.double().cpu().numpy())
    assert sf[:, 0].tolist() == [[252, 250], [253, 127 - 2]] and np.isfinite(values).all()
    pool = torch.zeros(1, 16, 1, 32, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(1, 16, 1, 2, dtype=torch.uint8, device="cuda")
    got = torch.empty_like(x)
    mq.paged_kv_write("mxfp4", x, torch.tensor([0, 1], device="cuda"), pool, scales, values=got)
    torch.cuda.synchronize()
    assert np.array_equal(pool[0, :2].cpu().numpy(), codes) and np.array_equal(scales[0, :2].cpu().numpy(), sf)
    assert np.array_equal(got.double().cpu().numpy(), values)
    # keys of 0 and these values: of the first row alone, then of both
    zero = torch.zeros_like(pool), torch.full_like(scales, 127)
    q = torch.ones(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    for n in (1, 2):
        out = mq.paged_attention("mxfp4", q, *zero, pool, scales, torch.tensor([n], **i32),
                                 torch.zeros(1, 1, **i32), 1, 16)
        torch.cuda.synchronize()
        if n == 1:
            assert np.array_equal(out[0].double().cpu().numpy(), np.broadcast_to(values[0], (4, 64)))
        else:
            assert bool(torch.isnan(out[..., :32]).all()) and bool(torch.isfinite(out[..., 32:]).all())
