"""Refusals of the cache and attention entry points (CPU only).

The C ABI is called with fake pointers that fail validation before any HIP
call; the binding with CPU tensors, which it refuses before the library.
"""

import ctypes

import pytest
import torch

mq = pytest.importorskip("mqa_logits_amd")
lib = mq.lib

OK, INVALID, UNSUPPORTED = 0, 1, 2
FAKE = ctypes.c_void_p(0x100000)
ODD = ctypes.c_void_p(0x100002)


def call(fn, base, change):
    args = dict(base)
    assert set(change) <= set(args)
    args.update(change)
    return fn(*args.values())


SLOTS = dict(ctx=FAKE, new=FAKE, free=FAKE, num_free=4, table=FAKE, stride=8, slots=FAKE,
             offsets=FAKE, taken=FAKE, batch=4, bs=16, nb=100, max_ctx=128, max_tokens=8, stream=None)
WRITE = dict(dt=2, x=FAKE, x_type=1, x_stride=256, x_head=128, slots=FAKE, pool=FAKE, sf=FAKE,
             scale=None, values=None, num_slots=64, rows=4, heads=2, d=128, stream=None)
ATTEND = dict(dt=2, q=FAKE, q_type=1, q_stride=1024, k=FAKE, ks=FAKE, v=FAKE, vs=FAKE, ctx=FAKE,
              table=FAKE, table_stride=8, idx=None, idx_stride=0, topk=0, scale=0.1, out=FAKE,
              lse=None, ws=None, ws_bytes=0, batch=2, next_n=1, hq=8, hkv=2, d=128, bs=16, nb=10,
              max_ctx=128, stream=None)


@pytest.mark.parametrize("change,expect", [
    (dict(batch=0), UNSUPPORTED), (dict(batch=8193), UNSUPPORTED), (dict(bs=8), UNSUPPORTED),
    (dict(bs=128), UNSUPPORTED), (dict(nb=0), INVALID), (dict(num_free=-1), INVALID),
    (dict(max_ctx=-1), INVALID), (dict(max_tokens=-1), INVALID), (dict(ctx=None), INVALID),
    (dict(new=None), INVALID), (dict(free=None), INVALID), (dict(table=None), INVALID),
    (dict(slots=None), INVALID), (dict(offsets=None), INVALID), (dict(taken=None), INVALID),
    (dict(slots=ctypes.c_void_p(0x100004)), INVALID), (dict(ctx=ODD), INVALID),
    (dict(stride=7), INVALID), (dict(batch=8192, max_ctx=1 << 18, stride=1 << 20), UNSUPPORTED),
])
def test_slots_refusals(change, expect):
    assert call(lib.paged_kv_slots, SLOTS, change) == expect
    assert mq.lib.mqa_last_error()


@pytest.mark.parametrize("change,expect", [
    (dict(dt=3), INVALID), (dict(dt=-1), INVALID), (dict(x_type=3), INVALID),
    (dict(d=32), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(heads=0), UNSUPPORTED),
    (dict(heads=2000), UNSUPPORTED), (dict(rows=-1), INVALID), (dict(num_slots=-1), INVALID),
    (dict(rows=1 << 30, heads=4), UNSUPPORTED), (dict(x_stride=260), INVALID),
    (dict(x_head=132), INVALID), (dict(x_stride=64), INVALID), (dict(x_head=64), INVALID),
    (dict(x_head=0), INVALID), (dict(x_stride=-256), INVALID),
    (dict(x_type=0, x_stride=258), INVALID), (dict(x=None), INVALID), (dict(slots=None), INVALID),
    (dict(pool=None), INVALID), (dict(sf=None), INVALID), (dict(scale=FAKE), INVALID),
    (dict(dt=0), INVALID), (dict(dt=0, sf=None), INVALID), (dict(x=ODD), INVALID),
    (dict(pool=ODD), INVALID), (dict(values=ODD), INVALID),
])
def test_write_refusals(change, expect):
    assert call(lib.paged_kv_write, WRITE, change) == expect


@pytest.mark.parametrize("change,expect", [
    (dict(dt=0), UNSUPPORTED), (dict(dt=1), UNSUPPORTED), (dict(dt=9), INVALID),
    (dict(q_type=0), UNSUPPORTED), (dict(q_type=5), INVALID), (dict(batch=0), UNSUPPORTED),
    (dict(next_n=17), UNSUPPORTED), (dict(next_n=0), UNSUPPORTED), (dict(hq=9), UNSUPPORTED),
    (dict(hkv=0), UNSUPPORTED), (dict(hkv=16), UNSUPPORTED), (dict(hq=2048, hkv=1), UNSUPPORTED),
    (dict(d=256), UNSUPPORTED), (dict(bs=48), UNSUPPORTED), (dict(nb=0), INVALID),
    (dict(nb=1 << 28), UNSUPPORTED), (dict(max_ctx=-1), INVALID), (dict(q=None), INVALID),
    (dict(k=None), INVALID), (dict(ks=None), INVALID), (dict(v=None), INVALID),
    (dict(vs=None), INVALID), (dict(ctx=None), INVALID), (dict(table=None), INVALID),
    (dict(out=None), INVALID), (dict(q=ODD), INVALID), (dict(out=ODD), INVALID),
    (dict(lse=ODD), INVALID), (dict(q_stride=1000), INVALID), (dict(q_stride=1028), INVALID),
    (dict(table_stride=7), INVALID), (dict(idx=FAKE), INVALID), (dict(topk=8), INVALID),
    (dict(idx=FAKE, topk=8, idx_stride=7), INVALID), (dict(topk=-1, idx=FAKE), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(max_ctx=1 << 14, table_stride=1 << 10), INVALID),           # needs a workspace
    (dict(max_ctx=1 << 14, table_stride=1 << 10, ws=FAKE, ws_bytes=100), INVALID),
])
def test_attention_refusals(change, expect):
    assert call(lib.paged_attention, ATTEND, change) == expect


def test_workspace_size():
    size = mq.paged_attention_workspace_size
    assert size(2, 1, 8, 2, 128, 0) == 0 and size(2, 1, 8, 2, 128, 128) == 0
    assert size(1, 1, 8, 1, 128, 100000) > 0
    assert size(1, 1, 8, 1, 128, 100000) % 4 == 0
    for bad in ((0, 1, 8, 1, 128, 1), (1, 1, 8, 3, 128, 1), (1, 1, 8, 1, 96, 1), (1, 1, 8, 1, 128, -1)):
        with pytest.raises(mq.MqaError):
            size(*bad)


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def test_binding_refuses_what_does_not_fit():
    x, slots = torch.zeros(4, 2, 128, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64)
    pool, sf = u8(3, 16, 2, 64), u8(3, 16, 2, 4)
    bad = [
        lambda: mq.paged_kv_write("fp4", x, slots, pool, sf),
        lambda: mq.paged_kv_write("mxfp4", x.double(), slots, pool, sf),
        lambda: mq.paged_kv_write("mxfp4", x, slots.int(), pool, sf),
        lambda: mq.paged_kv_write("mxfp4", x, slots[:3], pool, sf),
        lambda: mq.paged_kv_write("mxfp4", x, slots, u8(3, 16, 2, 128), sf),
        lambda: mq.paged_kv_write("mxfp4", x, slots, pool[:, :, :1], sf),
        lambda: mq.paged_kv_write("mxfp4", x, slots, pool, u8(3, 16, 2, 2)),
        lambda: mq.paged_kv_write("mxfp4", x, slots, pool),
        lambda: mq.paged_kv_write("mxfp4", x, slots, pool, sf, torch.zeros(3, 16, 2)),
        lambda: mq.paged_kv_write("fp8", x, slots, u8(3, 16, 2, 128), None, torch.zeros(3, 16)),
        lambda: mq.paged_kv_write("mxfp4", x.transpose(1, 2), slots, pool, sf),
        lambda: mq.paged_kv_write("mxfp4", x, slots, pool, sf, values=x.float()),
        lambda: mq.paged_kv_write("mxfp4", x, slots, pool, sf),                 # CPU tensors
    ]
    ctx, table = i32(2), i32(2, 8)
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)

    def attend(fmt="mxfp4", q=q, k=pool, ks=sf, v=pool, vs=sf, ctx=ctx, table=table, n=1, m=128, **kw):
        return lambda: mq.paged_attention(fmt, q, k, ks, v, vs, ctx, table, n, m, **kw)
    bad += [
        attend("fp8"), attend("nope"), attend(q=q.float()), attend(q=q[0]), attend(n=2),
        attend(k=pool[:, :, 0]), attend(v=u8(3, 16, 1, 64)), attend(vs=u8(3, 16, 2, 2)),
        attend(k=u8(3, 8, 2, 64)), attend(ctx=ctx.long()), attend(table=i32(2, 7)),
        attend(table=i32(1, 8)), attend(m=-1), attend(indices=i32(3, 4)), attend(indices=i32(2, 0)),
        attend(indices=i32(2, 4).long()), attend(out=q.half()), attend(out=q[:1]),
        attend(lse=torch.zeros(2, 7)), attend(workspace=torch.zeros(8)),
        attend(q=torch.zeros(2, 128, 8, dtype=torch.bfloat16).transpose(1, 2)), attend(),
    ]

    def step(ctx=ctx, new=ctx, free=i32(3), table=table, nb=10, bs=16, m=128, t=4, **kw):
        return lambda: mq.paged_kv_slots(ctx, new, free, table, nb, bs, m, t, **kw)
    bad += [
        step(new=i32(3)), step(ctx=ctx.long()), step(free=i32(3, 2)), step(table=i32(2, 7)),
        step(bs=8), step(m=-1), step(t=-1), step(table=i32(8, 2).t()),
        step(out=(torch.zeros(3, dtype=torch.int64), i32(3), i32(1))), step(),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()


@pytest.mark.parametrize("change", [dict(max_tokens=2 ** 32), dict(max_context_len=2 ** 32 + 16),
                                    dict(num_blocks=2 ** 32 + 5), dict(num_blocks=0),
                                    dict(max_tokens=-1), dict(max_context_len=-1)])
def test_binding_refuses_sizes_beyond_int32(change):
    # (they would reach the library cut to their low 32 bits)
    sizes = dict(num_blocks=9, block_size=16, max_context_len=16, max_tokens=4)
    sizes.update(change)
    with pytest.raises(ValueError, match="int32"):
        mq.paged_kv_slots(i32(2), i32(2), i32(3), i32(2, 4), **sizes)
    if "max_context_len" in change:
        q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
        with pytest.raises(ValueError, match="int32"):
            mq.paged_attention("mxfp4", q, u8(3, 16, 2, 32), u8(3, 16, 2, 2), u8(3, 16, 2, 32),
                               u8(3, 16, 2, 2), i32(2), i32(2, 4), 1, change["max_context_len"])


@pytest.mark.parametrize("at,name", [(3, "k_sf_pool"), (4, "v_pool"), (5, "v_sf_pool"), (7, "block_table")])
def test_binding_names_what_is_missing(at, name):
    args = ["mxfp4", torch.zeros(2, 4, 64, dtype=torch.bfloat16), u8(3, 16, 2, 32), u8(3, 16, 2, 2),
            u8(3, 16, 2, 32), u8(3, 16, 2, 2), i32(2), i32(2, 4), 1, 16]
    args[at] = None
    with pytest.raises(ValueError, match=name + " is required"):
        mq.paged_attention(*args)
    with pytest.raises(ValueError, match="slots is required"):
        mq.paged_kv_write("mxfp4", torch.zeros(2, 2, 64), None, u8(3, 16, 2, 32), u8(3, 16, 2, 2))
