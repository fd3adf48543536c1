"""Refusals of chunk attention, gathered weights and eviction (CPU only).

The C ABI is called with fake pointers that fail validation before any HIP call; the
binding with CPU tensors, which it refuses before the library.
"""

import ctypes

import pytest
import torch

mq = pytest.importorskip("mqa_logits_amd")
lib = mq.lib

INVALID, UNSUPPORTED = 1, 2
FAKE, OTHER = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x200000)
ODD = ctypes.c_void_p(0x100002)
NAN, INF = float("nan"), float("inf")


def call(fn, base, change):
    args = dict(base)
    assert set(change) <= set(args)
    args.update(change)
    return fn(*args.values())


def pools(*entries):
    words = [x for e in entries for x in e]
    return (ctypes.c_int64 * len(words))(*words)


CHUNK = dict(dt=2, q=FAKE, q_type=1, q_stride=1024, k=FAKE, ks=FAKE, v=FAKE, vs=FAKE, ctx=FAKE, offsets=FAKE,
             table=FAKE, table_stride=8, scale=0.1, out=FAKE, lse=None, ws=None, ws_bytes=0, batch=2, tokens=6,
             hq=8, hkv=2, d=128, bs=16, nb=10, max_ctx=128, stream=None)
WEIGHTS = dict(dt=2, q=FAKE, q_type=1, q_stride=1024, lse=FAKE, k=FAKE, ks=FAKE, ctx=FAKE, offsets=FAKE, table=FAKE,
               table_stride=8, scale=0.1, before=None, before_stride=0, out=FAKE, out_stride=128, ws=None,
               ws_bytes=0, batch=2, tokens=6, hq=8, hkv=2, d=128, bs=16, nb=10, max_ctx=128, stream=None)
EVICT = dict(weights=FAKE, stride=128, ctx=FAKE, table=FAKE, table_stride=8, free=FAKE, num_free=4,
             pools=pools((0x100000, 64)), num_pools=1, new_ctx=OTHER, new_table=OTHER, new_stride=8, new_weights=OTHER,
             new_weights_stride=128, kept=OTHER, kept_stride=32, freed=OTHER, counts=OTHER, ws=OTHER, ws_bytes=1 << 20,
             batch=2, bs=16, nb=10, max_ctx=128, keep=32, recent=8, stream=None)

SHARED = [
    (dict(dt=0), UNSUPPORTED), (dict(dt=1), UNSUPPORTED), (dict(dt=9), INVALID), (dict(q_type=0), UNSUPPORTED),
    (dict(q_type=5), INVALID), (dict(batch=0), UNSUPPORTED), (dict(batch=8193), UNSUPPORTED), (dict(tokens=-1), INVALID),
    (dict(hq=9), UNSUPPORTED), (dict(hkv=0), UNSUPPORTED), (dict(hkv=16), UNSUPPORTED), (dict(hq=2048, hkv=1), UNSUPPORTED),
    (dict(hq=512, hkv=512), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(bs=48), UNSUPPORTED),
    (dict(nb=0), INVALID), (dict(nb=1 << 28), UNSUPPORTED), (dict(max_ctx=-1), INVALID),
    (dict(max_ctx=(1 << 30) + 1), UNSUPPORTED), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(ks=None), INVALID),
    (dict(ctx=None), INVALID), (dict(table=None), INVALID), (dict(out=None), INVALID), (dict(q=ODD), INVALID),
    (dict(out=ODD), INVALID), (dict(lse=ODD), INVALID), (dict(offsets=ODD), INVALID), (dict(q_stride=1000), INVALID),
    (dict(q_stride=1028), INVALID), (dict(table_stride=7), INVALID), (dict(offsets=None, tokens=7), INVALID),
    (dict(scale=INF), INVALID), (dict(scale=NAN), INVALID),
]


@pytest.mark.parametrize("change,expect", SHARED + [
    (dict(v=None), INVALID), (dict(vs=None), INVALID), (dict(v=ODD), INVALID),
    (dict(max_ctx=1 << 16, table_stride=1 << 12), INVALID),           # needs a workspace
    (dict(max_ctx=1 << 16, table_stride=1 << 12, ws=FAKE, ws_bytes=100), INVALID),
    (dict(max_ctx=1 << 16, table_stride=1 << 12, ws=ODD, ws_bytes=1 << 40), INVALID),
])
def test_chunk_refusals(change, expect):
    assert call(lib.paged_chunk_attention, CHUNK, change) == expect
    assert lib.mqa_last_error()


@pytest.mark.parametrize("change,expect", SHARED + [
    (dict(lse=None), INVALID), (dict(before=ODD, before_stride=128), INVALID), (dict(before=FAKE, before_stride=127), INVALID),
    (dict(out_stride=127), INVALID),
    (dict(tokens=200, hq=64, max_ctx=1 << 12, table_stride=1 << 8, out_stride=1 << 12), INVALID),   # needs a workspace
    (dict(tokens=200, hq=64, max_ctx=1 << 12, table_stride=1 << 8, out_stride=1 << 12, ws=FAKE, ws_bytes=64), INVALID),
])
def test_weights_refusals(change, expect):
    if "hq" in change and change["hq"] == 64:
        change = dict(change, q_stride=64 * 128)
    assert call(lib.paged_attention_weights, WEIGHTS, change) == expect
    assert lib.mqa_last_error()


@pytest.mark.parametrize("change,expect", [
    (dict(batch=0), UNSUPPORTED), (dict(batch=8193), UNSUPPORTED), (dict(bs=48), UNSUPPORTED), (dict(nb=0), INVALID),
    (dict(nb=1 << 28), UNSUPPORTED), (dict(num_free=-1), INVALID), (dict(max_ctx=-1), INVALID), (dict(keep=0), INVALID),
    (dict(recent=-1), INVALID), (dict(recent=33), INVALID), (dict(num_pools=17), UNSUPPORTED), (dict(num_pools=-1), UNSUPPORTED),
    (dict(weights=None), INVALID), (dict(ctx=None), INVALID), (dict(table=None), INVALID), (dict(free=None), INVALID),
    (dict(pools=None), INVALID), (dict(new_ctx=None), INVALID), (dict(new_table=None), INVALID),
    (dict(new_weights=None), INVALID), (dict(kept=None), INVALID), (dict(freed=None), INVALID), (dict(counts=None), INVALID),
    (dict(ws=None), INVALID), (dict(weights=ODD), INVALID), (dict(kept=ODD), INVALID), (dict(ws=ODD), INVALID),
    (dict(stride=127), INVALID), (dict(new_weights_stride=127), INVALID), (dict(kept_stride=31), INVALID),
    (dict(table_stride=7), INVALID), (dict(new_stride=7), INVALID), (dict(ws_bytes=8), INVALID),
    (dict(pools=pools((0, 64))), INVALID), (dict(pools=pools((0x100000, 0))), INVALID),
    (dict(pools=pools((0x100000, (1 << 24) + 16))), UNSUPPORTED),
    (dict(new_ctx=FAKE), INVALID), (dict(new_table=FAKE), INVALID), (dict(new_weights=FAKE), INVALID), (dict(freed=FAKE), INVALID),
    (dict(batch=4096, max_ctx=1 << 19, stride=1 << 19, new_weights_stride=1 << 19, table_stride=1 << 15, new_stride=1 << 15),
     UNSUPPORTED),
    (dict(batch=4096, keep=1 << 19, kept_stride=1 << 19), UNSUPPORTED),
    (dict(batch=1, keep=(1 << 30) + 1, kept_stride=1 << 31), UNSUPPORTED),
])
def test_evict_refusals(change, expect):
    assert call(lib.paged_kv_evict, EVICT, change) == expect
    assert lib.mqa_last_error()


def test_workspace_sizes():
    chunk, weights, evict = (mq.paged_chunk_attention_workspace_size, mq.paged_attention_weights_workspace_size,
                             mq.paged_kv_evict_workspace_size)
    assert chunk(2, 0, 8, 2, 128, 100000) == 0 and chunk(1, 17, 16, 2, 128, 113) == 0
    assert chunk(1, 4096, 64, 8, 128, 65536) > 0
    assert weights(64, 256, 64, 1, 128, 32768) == 0 and weights(1, 256, 64, 8, 128, 32768) % (4 * 32768) == 0
    # (64 parts of 256 rows, three padding rows behind them: as many splits; then 16)
    assert weights(1, 259, 64, 8, 128, 32768) == 4 * 32768 * 64 and weights(1, 67, 64, 8, 128, 32768) == 4 * 32768 * 16
    assert weights(3, 0, 8, 2, 128, 1000) == 0 and weights(1, 4, 8, 2, 128, 0) >= 0
    assert evict(3, 600) < evict(64, 600) < 1 << 20 and evict(1, 131072) > 3 * 2048 * 4
    for fn, bad in ((chunk, (0, 1, 8, 1, 128, 1)), (chunk, (1, 1, 8, 3, 128, 1)), (chunk, (1, 1, 8, 1, 96, 1)),
                    (chunk, (1, -1, 8, 1, 128, 1)), (chunk, (1, 1, 8, 1, 128, -1)), (weights, (0, 1, 8, 1, 128, 1)),
                    (weights, (1, 1, 8, 1, 128, -1)), (weights, (1, 1, 0, 1, 128, 1)), (evict, (0, 1)), (evict, (1, -1))):
        with pytest.raises(mq.MqaError):
            fn(*bad)


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


Q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
CALLS = {
    mq.paged_chunk_attention: dict(fmt="mxfp4", q=Q, k_pool=u8(3, 16, 2, 32), k_sf_pool=u8(3, 16, 2, 2),
                                   v_pool=u8(3, 16, 2, 32), v_sf_pool=u8(3, 16, 2, 2), context_lens=i32(2),
                                   token_offsets=i32(3), block_table=i32(2, 4), max_context_len=16),
    mq.paged_attention_weights: dict(fmt="mxfp4", q=Q, lse=torch.zeros(3, 4), k_pool=u8(3, 16, 2, 32),
                                     k_sf_pool=u8(3, 16, 2, 2), context_lens=i32(2), token_offsets=i32(3),
                                     block_table=i32(2, 4), max_context_len=16),
    mq.paged_kv_evict: dict(weights=torch.zeros(2, 16), context_lens=i32(2), block_table=i32(2, 4), free_blocks=i32(3),
                            pools=[u8(3, 16, 2, 32)], keep=8, recent=2, max_context_len=16),
}
TENSORS = [(fn, name) for fn, args in CALLS.items() for name, x in args.items()
           if isinstance(x, torch.Tensor) and name != "token_offsets"]


@pytest.mark.parametrize("fn,name", TENSORS, ids=lambda x: x if isinstance(x, str) else x.__name__)
def test_what_is_missing_is_named(fn, name):
    with pytest.raises(ValueError, match=name + " is required"):
        fn(**{**CALLS[fn], name: None})
    with pytest.raises(ValueError):
        fn(**{**CALLS[fn], name: CALLS[fn][name].new_zeros(())})


@pytest.mark.parametrize("fn", CALLS, ids=lambda x: x.__name__)
def test_cpu_tensors_and_sizes_are_refused(fn):
    with pytest.raises(ValueError):
        fn(**CALLS[fn])
    for n in (-1, 2 ** 31, 2 ** 32 + 16):
        with pytest.raises(ValueError):
            fn(**{**CALLS[fn], "max_context_len": n})


@pytest.mark.parametrize("fn,change", [(fn, c) for fn in list(CALLS)[:2] for c in (
    dict(fmt="fp8"), dict(fmt="nope"), dict(q=Q.float()), dict(q=Q[0]), dict(q=torch.zeros(3, 4, 32, dtype=torch.bfloat16)),
    dict(q=torch.zeros(3, 64, 4, dtype=torch.bfloat16).transpose(1, 2)), dict(token_offsets=i32(2)),
    dict(token_offsets=i32(3).long()), dict(token_offsets=None), dict(k_pool=u8(3, 16, 2, 64)), dict(k_pool=u8(3, 8, 2, 32)),
    dict(k_sf_pool=u8(3, 16, 2, 1)), dict(k_pool=u8(3, 16, 4, 32)[:, :, ::2]), dict(context_lens=i32(2).long()),
    dict(block_table=i32(2, 0)), dict(block_table=i32(1, 4)), dict(out=torch.zeros(3, 4, 64)), dict(lse=torch.zeros(3, 5)),
    dict(workspace=torch.zeros(64)))] + [(mq.paged_kv_evict, c) for c in (
        dict(weights=torch.zeros(2, 15)), dict(weights=torch.zeros(2, 16).double()), dict(weights=torch.zeros(16, 2).t()),
        dict(context_lens=i32(3)), dict(block_table=i32(2, 0)), dict(free_blocks=i32(3, 1)), dict(free_blocks=i32(3).long()),
        dict(pools=[]), dict(pools=[None]), dict(pools=[u8(3, 16, 2), None]), dict(pools=[u8(3)]), dict(pools=[u8(3, 8, 2)]), dict(pools=[u8(3, 16, 2), u8(4, 16, 2)]),
        dict(pools=[u8(3, 16, 4)[:, :, ::2]]), dict(keep=0), dict(recent=9), dict(recent=-1), dict(workspace=torch.zeros(64)),
        dict(out=(i32(2), i32(2, 1), torch.zeros(2, 16), i32(2, 8), i32(2), i32(3))),
        dict(out=(i32(2), i32(2, 0), torch.zeros(2, 16), i32(2, 8), i32(2), i32(2))))],
    ids=lambda x: x.__name__ if callable(x) else "-".join(x))
def test_binding_refuses_what_does_not_fit(fn, change):
    with pytest.raises((ValueError, mq.MqaError)):   # (unsupported sizes: by the library)
        fn(**{**CALLS[fn], **change})
