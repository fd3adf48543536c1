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
