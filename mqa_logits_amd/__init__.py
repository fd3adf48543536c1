"""Python binding of libmqa_logits (weighted MQA logits on MI355X / gfx950).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI declared in include/mqa_logits.h.  PyTorch supplies
device memory and the current stream; nothing here computes logits, and there
is no CPU fallback -- if the shared library is missing, importing the package
raises.

Entry points (same names as the C ABI):
  mqa_logits                      dense clean (or keep) logits
  mqa_logits_metadata             work schedule for the dense / compressed calls
  mqa_logits_topk                 top-k column indices of logits rows
  mqa_logits_compressed_offsets   row offsets of the packed layout
  mqa_logits_compressed           packed logits
  paged_mqa_logits_metadata       paged work split
  paged_mqa_logits                paged decode logits
  paged_kv_slots                  block-table entries and slot map of a step's new tokens
  paged_kv_write                  quantise rows and store them at their slots
  paged_attention                 attention over a paged MXFP4 cache, whole or selected keys
  paged_chunk_attention           the same for chunks of new tokens, a different number a sequence
  paged_attention_weights         the attention weight that every cached token has gathered
  paged_kv_evict                  cut long sequences to their heaviest and their last tokens
  mqa_num_cus, paged_mqa_logits_default_splits
"""

import collections
import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmqa_logits.so")

FORMATS = {"fp8": 0, "mxfp8": 1, "mxfp4": 2}
# mqa_precision of the C ABI: the matrix core's grouped summation, or every
# product exact (eight KV operand copies for fp8 elements)
PRECISIONS = {"default": 0, "exact": 1}
# mqa_float of the C ABI: element type of the weights and of the logits
FLOAT_TYPES = {torch.float32: 0, torch.bfloat16: 1}
ROW_TYPES = {**FLOAT_TYPES, torch.float16: 2}      # paged_kv_write's rows
QUERY_TYPES = {torch.bfloat16: 1, torch.float16: 2}    # paged_attention's q and output
BLOCK_SIZES = (16, 32, 64)


class MqaError(RuntimeError):
    """A non-OK status from the C ABI, with mqa_last_error()'s message."""

    def __init__(self, status, message):
        super().__init__(f"status {status}: {message}")
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python mqa_logits_amd/build.py` "
            "(there is no fallback implementation)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    sigs = {
        "mqa_logits": [I32, P, P, P, P, P, P, P, P, P, I64, I32, I32, I32, I32, I32, I32, I32,
                       P, I32, I32, P],
        "mqa_logits_metadata": [P, P, I32, I32, I32, P, P],
        "mqa_logits_topk": [P, I32, I64, P, P, I32, I32, I32, P, I64, P],
        "mqa_logits_compressed_offsets": [P, P, I32, I32, P, P],
        "mqa_logits_compressed": [I32, P, P, P, P, P, P, P, P, P, P, I32, I32, I32, I32, I32, I32,
                                  P, I32, I32, P],
        "paged_mqa_logits_metadata": [P, I32, I32, I32, I32, I32, P, P],
        "paged_mqa_logits": [I32, P, P, P, P, P, P, P, P, I64, P, P, I64,
                             I32, I32, I32, I32, I32, I32, I32, I32, I32, I32, I32, I32, P],
        "paged_kv_slots": [P, P, P, I32, P, I64, P, P, P, I32, I32, I32, I32, I32, P],
        "paged_kv_write": [I32, P, I32, I64, I64, P, P, P, P, P, I64, I32, I32, I32, P],
        "paged_attention": [I32, P, I32, I64, P, P, P, P, P, P, I64, P, I64, I32, ctypes.c_float,
                            P, P, P, I64, I32, I32, I32, I32, I32, I32, I32, I32, P],
        "paged_chunk_attention": [I32, P, I32, I64, P, P, P, P, P, P, P, I64, ctypes.c_float, P, P, P,
                                  I64, I32, I32, I32, I32, I32, I32, I32, I32, P],
        "paged_attention_weights": [I32, P, I32, I64, P, P, P, P, P, P, I64, ctypes.c_float, P, I64, P, I64,
                                    P, I64, I32, I32, I32, I32, I32, I32, I32, I32, P],
        "paged_kv_evict": [P, I64, P, P, I64, P, I32, P, I32, P, P, I64, P, I64, P, I64, P, P, P, I64,
                           I32, I32, I32, I32, I32, I32, P],
    }
    for name, argtypes in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = argtypes
        fn.restype = ctypes.c_int
    for name in ("paged_mqa_logits_metadata_size", "mqa_logits_metadata_size"):
        getattr(lib, name).argtypes = [I32]
        getattr(lib, name).restype = I64
    lib.paged_attention_workspace_size.argtypes = [I32] * 7
    lib.paged_attention_workspace_size.restype = I64
    lib.paged_chunk_attention_workspace_size.argtypes = [I32] * 6
    lib.paged_chunk_attention_workspace_size.restype = I64
    lib.paged_attention_weights_workspace_size.argtypes = [I32] * 6
    lib.paged_attention_weights_workspace_size.restype = I64
    lib.paged_kv_evict_workspace_size.argtypes = [I32, I32]
    lib.paged_kv_evict_workspace_size.restype = I64
    lib.mqa_num_cus.argtypes = [I32]
    lib.mqa_num_cus.restype = I32
    lib.paged_mqa_logits_default_splits.argtypes = [I32]
    lib.paged_mqa_logits_default_splits.restype = I32
    lib.mqa_last_error.argtypes = []
    lib.mqa_last_error.restype = ctypes.c_char_p
    return lib


lib = _load()

EXPORTED = ("mqa_logits", "mqa_logits_metadata_size", "mqa_logits_metadata", "mqa_logits_topk",
            "mqa_logits_compressed_offsets", "mqa_logits_compressed",
            "paged_mqa_logits_metadata_size", "paged_mqa_logits_metadata",
            "paged_mqa_logits", "paged_kv_slots", "paged_kv_write",
            "paged_attention_workspace_size", "paged_attention",
            "paged_chunk_attention_workspace_size", "paged_chunk_attention",
            "paged_attention_weights_workspace_size", "paged_attention_weights",
            "paged_kv_evict_workspace_size", "paged_kv_evict",
            "mqa_num_cus", "paged_mqa_logits_default_splits",
            "mqa_last_error")


def _check(status):
    if status != 0:
        raise MqaError(status, lib.mqa_last_error().decode())


def _ptr(t):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libmqa_logits must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


I32_T, I64_T = (torch.int32,), (torch.int64,)


class _Args:
    """The tensor arguments of one call, checked against what the C ABI will
    read or write through their pointers: shape (None entries are free),
    element type or size, layout (contiguous, or rows contiguous when
    `rows`), then one GPU for all of them.  The library sees only pointers
    and sizes, so a mismatch would read or write outside a tensor."""

    def __init__(self):
        self.seen = []

    def want(self, t, name, shape, dtypes=None, itemsize=None, rows=False):
        if t is None:
            raise ValueError(f"{name} is required")
        got = t.shape                           # a tuple: compared whole when no entry is free
        if (got != shape) if None not in shape else (
                len(got) != len(shape) or not all(w is None or g == w for g, w in zip(got, shape))):
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(got)}")
        dt = t.dtype
        if dtypes is not None and dt not in dtypes:
            raise ValueError(f"{name} must be {' or '.join(map(str, dtypes))}, got {dt}")
        if itemsize is not None and dt.itemsize != itemsize:
            raise ValueError(f"{name} must have {itemsize}-byte elements, got {dt}")
        if rows:
            if len(got) and t.stride(-1) != 1 and got[-1] > 1:
                raise ValueError(f"{name} rows must be contiguous")
        elif not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        self.seen.append((name, t))

    def on_gpu(self):
        # device indices compared as integers (-1 for a CPU tensor); returns theirs
        first = self.seen[0][1].get_device()
        for name, t in self.seen:
            dev = t.get_device()
            if dev < 0:
                raise ValueError(f"{name} must be a GPU tensor (the library reads device memory)")
            if dev != first:
                raise ValueError(f"{name} must be on cuda:{first}, got {t.device}")
        return first


def _codes(a, fmt, q, kv, q_sf, kv_sf, kv_scale, rows_shape, kv_shape):
    """The Q and KV operands of a call: byte codes (two e2m1 per byte for
    mxfp4), e8m0 block scales for the MX formats, fp32 token scales for fp8.
    rows_shape: Q's leading dims; kv_shape: KV's leading dims.  Returns D."""
    _fmt(fmt)
    d = _head_dim(fmt, q)
    a.want(q, "q", (*rows_shape, q.shape[-1] if q.dim() else None), itemsize=1)
    a.want(kv, "kv", (*kv_shape, q.shape[-1]), itemsize=1)
    if fmt == "fp8":
        if q_sf is not None or kv_sf is not None:
            raise ValueError("fp8 takes no block scales (q_sf, kv_sf)")
        a.want(kv_scale, "kv_scale", tuple(kv_shape), (torch.float32,))
    else:
        if kv_scale is not None:
            raise ValueError(f"{fmt} takes no kv_scale")
        a.want(q_sf, "q_sf", (*rows_shape, d // 32), itemsize=1)
        a.want(kv_sf, "kv_sf", (*kv_shape, d // 32), itemsize=1)
    return d


def _rows_ptr(t, what):
    """A 2-D tensor whose rows are contiguous (its row stride is passed apart)."""
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{what} rows must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(t):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _fmt(fmt):
    if fmt not in FORMATS:
        raise ValueError(f"format must be one of {sorted(FORMATS)}, got {fmt!r}")
    return FORMATS[fmt]


def _precision(precision):
    if precision not in PRECISIONS:
        raise ValueError(f"precision must be one of {sorted(PRECISIONS)}, got {precision!r}")
    return PRECISIONS[precision]


def _head_dim(fmt, q):
    return q.shape[-1] * (2 if fmt == "mxfp4" else 1)


def _float_type(dtype, what):
    if dtype not in FLOAT_TYPES:
        raise ValueError(f"{what} must be float32 or bfloat16, got {dtype}")
    return FLOAT_TYPES[dtype]


def _logits_rows(rows, cols, dtype, device):
    """[rows, cols] logits; bf16 rows get an even stride (the C ABI needs one)."""
    width = cols + (cols & 1) if dtype == torch.bfloat16 else cols
    out = torch.empty(rows, width, dtype=dtype, device=device)
    return out[:, :cols] if width != cols else out


def mqa_num_cus(device=0):
    n = lib.mqa_num_cus(int(device))
    if n < 0:
        raise MqaError(3, lib.mqa_last_error().decode())
    return n


def paged_mqa_logits_default_splits(device=0):
    n = lib.paged_mqa_logits_default_splits(int(device))
    if n < 0:
        raise MqaError(3, lib.mqa_last_error().decode())
    return n


def _schedule(schedule):
    if schedule is None:
        return None, 0
    return _ptr(schedule), schedule.shape[0] - 1


def _dense_args(a, fmt, q, q_sf, kv, kv_sf, kv_scale, weights, k_start, k_end, schedule):
    sq, h = weights.shape
    _codes(a, fmt, q, kv, q_sf, kv_sf, kv_scale, (sq, h), (kv.shape[0],))
    a.want(weights, "weights", (sq, h), tuple(FLOAT_TYPES))
    a.want(k_start, "k_start", (sq,), I32_T)
    a.want(k_end, "k_end", (sq,), I32_T)
    if schedule is not None:
        a.want(schedule, "schedule", (None, 2), I32_T)


def mqa_logits_metadata(k_start, k_end, skv, num_splits=None, out=None):
    """int32 [num_splits + 1, 2] work schedule for mqa_logits /
    mqa_logits_compressed with these ranges."""
    a = _Args()
    if num_splits is None:
        num_splits = paged_mqa_logits_default_splits(k_start.device.index or 0)
    sq = k_start.shape[0]
    a.want(k_start, "k_start", (sq,), I32_T)
    a.want(k_end, "k_end", (sq,), I32_T)
    if out is None:
        out = torch.empty(num_splits + 1, 2, dtype=torch.int32, device=k_start.device)
    a.want(out, "out", (num_splits + 1, 2), I32_T)
    a.on_gpu()
    _check(lib.mqa_logits_metadata(_ptr(k_start), _ptr(k_end), k_start.shape[0], skv,
                                   num_splits, _ptr(out), _stream(k_start)))
    return out


def mqa_logits(fmt, q, q_sf, kv, kv_sf, kv_scale, weights, k_start, k_end,
               clean_logits=True, out=None, logits_dtype=torch.float32, schedule=None,
               precision="default"):
    """Dense logits [Sq, Skv] of logits_dtype (out may be a wider-strided row
    view; its dtype then decides).  weights: float32 or bfloat16.  schedule:
    None or mqa_logits_metadata's result for the same ranges.  precision:
    "default" or "exact" (mqa_precision)."""
    sq, h = weights.shape
    skv = kv.shape[0]
    a = _Args()
    _dense_args(a, fmt, q, q_sf, kv, kv_sf, kv_scale, weights, k_start, k_end, schedule)
    if out is None:
        out = _logits_rows(sq, skv, logits_dtype, q.device)
    a.want(out, "out", (sq, skv), tuple(FLOAT_TYPES), rows=True)
    a.on_gpu()
    _check(lib.mqa_logits(
        _fmt(fmt), _ptr(q), _ptr(q_sf), _ptr(kv), _ptr(kv_sf), _ptr(kv_scale),
        _ptr(weights), _ptr(k_start), _ptr(k_end), ctypes.c_void_p(out.data_ptr()),
        out.stride(0) if sq > 0 else skv, sq, skv, h, _head_dim(fmt, q),
        1 if clean_logits else 0, _float_type(weights.dtype, "weights"),
        _float_type(out.dtype, "logits"), *_schedule(schedule), _precision(precision),
        _stream(q)))
    return out


def mqa_logits_topk(logits, topk, k_start=None, k_end=None, out=None):
    """int32 [Sq, topk] columns of each row's topk largest non--inf logits in
    [k_start, k_end) (the whole row without ranges), ascending, -1 padded."""
    a = _Args()
    sq, skv = logits.shape
    a.want(logits, "logits", (sq, skv), tuple(FLOAT_TYPES), rows=True)
    if (k_start is None) != (k_end is None):
        raise ValueError("k_start and k_end go together")
    if k_start is not None:
        a.want(k_start, "k_start", (sq,), I32_T)
        a.want(k_end, "k_end", (sq,), I32_T)
    if out is None:
        out = torch.empty(sq, topk, dtype=torch.int32, device=logits.device)
    a.want(out, "out", (sq, topk), I32_T, rows=True)
    a.on_gpu()
    _check(lib.mqa_logits_topk(
        ctypes.c_void_p(logits.data_ptr()), _float_type(logits.dtype, "logits"),
        logits.stride(0) if sq > 0 else skv, _ptr(k_start), _ptr(k_end), sq, skv, topk,
        ctypes.c_void_p(out.data_ptr()), out.stride(0) if sq > 0 else topk,
        _stream(logits)))
    return out


def mqa_logits_compressed_offsets(k_start, k_end, skv, out=None):
    """int64 [Sq + 1] exclusive prefix sum of the clamped row lengths."""
    a = _Args()
    sq = k_start.shape[0]
    a.want(k_start, "k_start", (sq,), I32_T)
    a.want(k_end, "k_end", (sq,), I32_T)
    if out is None:
        out = torch.empty(sq + 1, dtype=torch.int64, device=k_start.device)
    a.want(out, "out", (sq + 1,), I64_T)
    a.on_gpu()
    _check(lib.mqa_logits_compressed_offsets(_ptr(k_start), _ptr(k_end), sq, skv,
                                             _ptr(out), _stream(k_start)))
    return out


def mqa_logits_compressed(fmt, q, q_sf, kv, kv_sf, kv_scale, weights, k_start, k_end,
                          row_offsets=None, out=None, logits_dtype=torch.float32,
                          schedule=None, precision="default"):
    """Packed logits; returns (packed [total] of logits_dtype, row_offsets int64
    [Sq+1]).

    Without `out`, the total length is read back from the device (a sync)."""
    sq, h = weights.shape
    skv = kv.shape[0]
    a = _Args()
    _dense_args(a, fmt, q, q_sf, kv, kv_sf, kv_scale, weights, k_start, k_end, schedule)
    if row_offsets is None:
        row_offsets = mqa_logits_compressed_offsets(k_start, k_end, skv)
    a.want(row_offsets, "row_offsets", (sq + 1,), I64_T)
    if out is None:
        out = torch.empty(int(row_offsets[-1].item()), dtype=logits_dtype, device=q.device)
    # out must hold row_offsets[-1] values (not checked here: that would read
    # the offsets back from the device)
    a.want(out, "out", (None,), tuple(FLOAT_TYPES))
    a.on_gpu()
    _check(lib.mqa_logits_compressed(
        _fmt(fmt), _ptr(q), _ptr(q_sf), _ptr(kv), _ptr(kv_sf), _ptr(kv_scale),
        _ptr(weights), _ptr(k_start), _ptr(k_end), _ptr(row_offsets), _ptr(out),
        sq, skv, h, _head_dim(fmt, q), _float_type(weights.dtype, "weights"),
        _float_type(out.dtype, "logits"), *_schedule(schedule), _precision(precision),
        _stream(q)))
    return out, row_offsets


def paged_mqa_logits_metadata(context_lens, next_n, block_size, max_context_len,
                              num_splits=None, out=None):
    """int32 [num_splits + 1, 2] schedule for paged_mqa_logits."""
    a = _Args()
    if num_splits is None:
        num_splits = paged_mqa_logits_default_splits(context_lens.device.index or 0)
    a.want(context_lens, "context_lens", (context_lens.shape[0],), I32_T)
    if out is None:
        out = torch.empty(num_splits + 1, 2, dtype=torch.int32, device=context_lens.device)
    a.want(out, "out", (num_splits + 1, 2), I32_T)
    a.on_gpu()
    _check(lib.paged_mqa_logits_metadata(_ptr(context_lens), context_lens.shape[0], next_n,
                                         block_size, max_context_len, num_splits, _ptr(out),
                                         _stream(context_lens)))
    return out


def paged_mqa_logits(fmt, q, q_sf, kv_pool, kv_sf_pool, kv_scale_pool, weights,
                     context_lens, block_table, schedule, next_n, max_context_len,
                     clean_logits=True, out=None, logits_dtype=torch.float32,
                     precision="default"):
    """Paged decode logits [batch * next_n, max_context_len] of logits_dtype."""
    a = _Args()
    batch = context_lens.shape[0]
    rows, h = weights.shape
    num_blocks, block_size = kv_pool.shape[0], kv_pool.shape[1]
    num_splits = schedule.shape[0] - 1
    if rows != batch * next_n:
        raise ValueError(f"weights must have batch * next_n = {batch * next_n} rows, got {rows}")
    _codes(a, fmt, q, kv_pool, q_sf, kv_sf_pool, kv_scale_pool, (rows, h), (num_blocks, block_size))
    a.want(weights, "weights", (rows, h), tuple(FLOAT_TYPES))
    a.want(context_lens, "context_lens", (batch,), I32_T)
    a.want(block_table, "block_table", (batch, None), I32_T, rows=True)
    need = -(-max_context_len // block_size) if block_size > 0 else 0
    if block_table.shape[1] < need:
        raise ValueError(f"block_table rows must hold ceil(max_context_len / block_size) = {need} "
                         f"blocks, got {block_table.shape[1]}")
    a.want(schedule, "schedule", (num_splits + 1, 2), I32_T)
    if out is None:
        out = _logits_rows(rows, max_context_len, logits_dtype, q.device)
    a.want(out, "out", (rows, max_context_len), tuple(FLOAT_TYPES), rows=True)
    a.on_gpu()
    _check(lib.paged_mqa_logits(
        _fmt(fmt), _ptr(q), _ptr(q_sf), _ptr(kv_pool), _ptr(kv_sf_pool), _ptr(kv_scale_pool),
        _ptr(weights), _ptr(context_lens), _rows_ptr(block_table, "block_table"),
        block_table.stride(0),
        _ptr(schedule), ctypes.c_void_p(out.data_ptr()), out.stride(0), batch, next_n, h,
        _head_dim(fmt, q), block_size, num_blocks, max_context_len, num_splits,
        1 if clean_logits else 0, _float_type(weights.dtype, "weights"),
        _float_type(out.dtype, "logits"), _precision(precision), _stream(q)))
    return out


# The calls below run once per layer and step, so their checks are made twice:
# first one expression over everything a call takes; only where that fails, the
# checks one by one, which name what does not fit.


def _call(fn, device, *args):
    """fn(*args, stream) on GPU `device` (kernels go to the current device)."""
    # the bindings under torch.cuda's current_device and current_stream, a
    # microsecond sooner; a build of torch without GPU support lacks them
    current = torch._C._cuda_getDevice
    stream = torch._C._cuda_getCurrentRawStream
    if current() == device:
        status = fn(*args, stream(device))
    else:
        with torch.cuda.device(device):
            status = fn(*args, stream(device))
    if status != 0:
        _check(status)


def _data(t):
    return None if t is None else t.data_ptr()


def _row_stride(t, width):
    """Elements from row to row of a tensor whose rows of `width` are contiguous."""
    return t.stride(0) if t.shape[0] > 1 else max(width, 1)


def _block_size(block_size):
    if block_size not in BLOCK_SIZES:
        raise ValueError(f"block_size must be one of {BLOCK_SIZES}, got {block_size}")


def _required(**tensors):
    for name, t in tensors.items():
        if t is None:
            raise ValueError(f"{name} is required")


def _fits(t, shape, dtype, device):
    return (t is not None and t.shape == shape and t.dtype is dtype and t.get_device() == device
            and t.is_contiguous())


def _table_fits(t, batch, blocks, device):
    if t is None:
        return False
    shape = t.shape
    return (len(shape) == 2 and shape[0] == batch and shape[1] >= blocks
            and t.dtype is torch.int32 and t.get_device() == device
            and (t.stride(1) == 1 or shape[1] <= 1))


def _want_table(a, block_table, batch, block_size, max_context_len):
    a.want(block_table, "block_table", (batch, None), I32_T, rows=True)
    need = -(-max_context_len // block_size)
    if block_table.shape[1] < need:
        raise ValueError(f"block_table rows must hold ceil(max_context_len / block_size) = {need} "
                         f"blocks, got {block_table.shape[1]}")


def paged_kv_slots(context_lens, new_lens, free_blocks, block_table, num_blocks, block_size,
                   max_context_len, max_tokens, out=None):
    """Block-table entries and slot map of a step's new tokens.

    context_lens counts the new_lens new tokens; block_table (int32, updated in
    place) gets the blocks they need from free_blocks in order.  Returns (slots
    int64 [max_tokens], -1 padded; token_offsets int32 [batch + 1];
    blocks_taken int32 [1], which exceeds len(free_blocks) when the list ran
    out); `out` may hold these three."""
    _block_size(block_size)
    if not (0 <= max_tokens < 2 ** 31 and 0 <= max_context_len < 2 ** 31 and 0 < num_blocks < 2 ** 31):
        raise ValueError("max_tokens, max_context_len and num_blocks must be int32 and not negative")
    if context_lens is None or free_blocks is None:
        _required(context_lens=context_lens, free_blocks=free_blocks)
    batch, dev = context_lens.numel(), context_lens.get_device()
    i32, given = torch.int32, out is not None
    if not given:
        out = (context_lens.new_empty(max_tokens, dtype=torch.int64),
               context_lens.new_empty(batch + 1, dtype=i32), context_lens.new_empty(1, dtype=i32))
    slots, offsets, taken = out
    if not (dev >= 0 and _fits(context_lens, (batch,), i32, dev)
            and _fits(new_lens, (batch,), i32, dev)
            and _fits(free_blocks, (free_blocks.numel(),), i32, dev)
            and _table_fits(block_table, batch, -(-max_context_len // block_size), dev)
            and (not given or (_fits(slots, (max_tokens,), torch.int64, dev)
                               and _fits(offsets, (batch + 1,), i32, dev)
                               and _fits(taken, (1,), i32, dev)))):
        a = _Args()
        a.want(context_lens, "context_lens", (batch,), I32_T)
        a.want(new_lens, "new_lens", (batch,), I32_T)
        a.want(free_blocks, "free_blocks", (None,), I32_T)
        _want_table(a, block_table, batch, block_size, max_context_len)
        a.want(slots, "slots", (max_tokens,), I64_T)
        a.want(offsets, "token_offsets", (batch + 1,), I32_T)
        a.want(taken, "blocks_taken", (1,), I32_T)
        a.on_gpu()
    _call(lib.paged_kv_slots, dev, context_lens.data_ptr(), new_lens.data_ptr(),
          free_blocks.data_ptr(), free_blocks.shape[0], block_table.data_ptr(),
          _row_stride(block_table, block_table.shape[1]), slots.data_ptr(), offsets.data_ptr(),
          taken.data_ptr(), batch, block_size, num_blocks, max_context_len, max_tokens)
    return out


def paged_kv_write(fmt, x, slots, kv_pool, kv_sf_pool=None, kv_scale_pool=None, values=None):
    """Quantise rows x [n, D] or [n, heads, D] (fp32, bf16 or fp16; rows and
    heads may be strided) and store them at `slots` (int64 [n]; outside the
    pool: not stored) of kv_pool [num_blocks, block_size(, heads), D or D/2]
    with kv_sf_pool [.., D/32] (MX formats) or kv_scale_pool (fp8).  Slots that
    are stored must differ.  (paged_attention counts mxfp4 groups with a magnitude
    over 1.5 * 2 ** 127 as NaN.)  values (x's shape and type, contiguous) receives
    what the codes stand for."""
    code = _fmt(fmt)
    if x is None or kv_pool is None:
        _required(x=x, kv_pool=kv_pool)
    shape = x.shape
    if len(shape) not in (2, 3) or x.dtype not in ROW_TYPES:
        raise ValueError(f"x must be [n, D] or [n, heads, D] of {sorted(map(str, ROW_TYPES))}, "
                         f"got {tuple(shape)} {x.dtype}")
    n, d, dev = shape[0], shape[-1], x.get_device()
    heads = shape[1] if len(shape) == 3 else 1
    lead = kv_pool.shape[:2] + shape[1:-1]
    pool_shape = (*lead, d // 2 if fmt == "mxfp4" else d)
    if fmt == "fp8":
        scales, scale_shape, scale_size = kv_scale_pool, lead, 4
    else:
        scales, scale_shape, scale_size = kv_sf_pool, (*lead, d // 32), 1
    if not (dev >= 0 and scales is not None and (kv_sf_pool is None or kv_scale_pool is None)
            and x.stride(-1) == 1 and _fits(slots, (n,), torch.int64, dev)
            and _fits(kv_pool, pool_shape, kv_pool.dtype, dev) and kv_pool.dtype.itemsize == 1
            and _fits(scales, scale_shape, scales.dtype, dev)
            and (scales.dtype.itemsize == 1 if scale_size == 1 else scales.dtype is torch.float32)
            and (values is None or _fits(values, shape, x.dtype, dev))):
        a = _Args()
        a.want(x, "x", tuple(shape), rows=True)
        a.want(slots, "slots", (n,), I64_T)
        a.want(kv_pool, "kv_pool", (None, None, *pool_shape[2:]), itemsize=1)
        if fmt == "fp8":
            if kv_sf_pool is not None:
                raise ValueError("fp8 takes no block scales (kv_sf_pool)")
            a.want(kv_scale_pool, "kv_scale_pool", tuple(lead), (torch.float32,))
        else:
            if kv_scale_pool is not None:
                raise ValueError(f"{fmt} takes no kv_scale_pool")
            a.want(kv_sf_pool, "kv_sf_pool", tuple(scale_shape), itemsize=1)
        if values is not None:
            a.want(values, "values", tuple(shape), (x.dtype,))
        a.on_gpu()
    _call(lib.paged_kv_write, dev, code, x.data_ptr(), ROW_TYPES[x.dtype], _row_stride(x, d),
          x.stride(1) if heads > 1 else d, slots.data_ptr(), kv_pool.data_ptr(), _data(kv_sf_pool),
          _data(kv_scale_pool), _data(values), lead[0] * lead[1], n, heads, d)
    return values


@functools.lru_cache(maxsize=1024)
def paged_attention_workspace_size(batch, next_n, q_heads, kv_heads, d, max_context_len, topk=0):
    """Bytes of workspace of a paged_attention call of these sizes."""
    n = lib.paged_attention_workspace_size(batch, next_n, q_heads, kv_heads, d, max_context_len,
                                           topk)
    if n < 0:
        raise MqaError(2, lib.mqa_last_error().decode())
    return n


def paged_attention(fmt, q, k_pool, k_sf_pool, v_pool, v_sf_pool, context_lens, block_table,
                    next_n, max_context_len, scale=None, indices=None, out=None, lse=None,
                    return_lse=False, workspace=None):
    """Attention of next_n query tokens a sequence over a paged 4-bit cache.

    fmt "mxfp4"; q [batch * next_n, Hq, D] bf16 or fp16 (rows may be strided),
    pools [num_blocks, block_size, Hkv, D/2] with e8m0 [.., D/32].  Row
    b * next_n + t sees the first context_lens[b] - next_n + 1 + t keys; with
    indices (int32 [rows, topk], as mqa_logits_topk gives them) it attends to
    the listed ones among them.  scale defaults to D ** -0.5; scores must stay
    within +-2 ** 24 octaves.  Returns out
    (q's shape and type; zeros for a row without keys), or (out, lse fp32
    [rows, Hq]) with return_lse or an lse to fill.  workspace: a uint8 tensor
    of paged_attention_workspace_size bytes to keep between calls on one
    stream, or None."""
    if fmt != "mxfp4":
        _fmt(fmt)
        raise ValueError(f"paged_attention reads an mxfp4 cache, got {fmt!r}")
    if q is None or k_pool is None or context_lens is None:
        _required(q=q, k_pool=k_pool, context_lens=context_lens)
    if q.dim() != 3 or q.dtype not in QUERY_TYPES:
        raise ValueError(f"q must be [rows, Hq, D] of bfloat16 or float16, got {tuple(q.shape)} {q.dtype}")
    if k_pool.dim() != 4:
        raise ValueError(f"k_pool must be [num_blocks, block_size, Hkv, D/2], got {tuple(k_pool.shape)}")
    q_shape, q_stride, dev = q.shape, q.stride(), q.get_device()
    rows, hq, d = q_shape
    batch = context_lens.numel()
    num_blocks, block_size, hkv, _ = k_pool.shape
    _block_size(block_size)
    if not 0 <= max_context_len < 2 ** 31:
        raise ValueError("max_context_len must be int32 and not negative")
    if rows != batch * next_n:
        raise ValueError(f"q must have batch * next_n = {batch * next_n} rows, got {rows}")
    if q_stride[2] != 1 or (hq > 1 and q_stride[1] != d):
        raise ValueError("q rows must be contiguous")
    topk = 0
    if indices is not None:
        topk = indices.shape[1] if indices.dim() == 2 else 0
        if topk < 1:
            raise ValueError("indices must be [rows, topk] with at least one column")
    # (what is made here needs no check)
    given_out, given_lse, given_workspace = out is not None, lse is not None, workspace is not None
    if not given_out:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if not given_lse and return_lse:
        lse = q.new_empty((rows, hq), dtype=torch.float32)
    need = paged_attention_workspace_size(batch, next_n, hq, hkv, d, max_context_len, topk)
    if not given_workspace:
        workspace, size = (q.new_empty(need, dtype=torch.uint8), need) if need else (None, 0)
    else:
        size = workspace.numel()
    codes, scales = (num_blocks, block_size, hkv, d // 2), (num_blocks, block_size, hkv, d // 32)
    byte, i32 = k_pool.dtype, torch.int32
    if not (dev >= 0 and byte.itemsize == 1 and _fits(k_pool, codes, byte, dev)
            and _fits(v_pool, codes, byte, dev)
            and k_sf_pool is not None and k_sf_pool.dtype.itemsize == 1 and _fits(k_sf_pool, scales, k_sf_pool.dtype, dev)
            and _fits(v_sf_pool, scales, k_sf_pool.dtype, dev)
            and _fits(context_lens, (batch,), i32, dev)
            and _table_fits(block_table, batch, -(-max_context_len // block_size), dev)
            and (topk == 0 or _table_fits(indices, rows, topk, dev))
            and (not given_out or _fits(out, q_shape, q.dtype, dev))
            and (not given_lse or _fits(lse, (rows, hq), torch.float32, dev))
            and (not given_workspace or _fits(workspace, (size,), torch.uint8, dev))):
        a = _Args()
        a.want(q[:0], "q", (0, hq, d))
        for name, pool, sf in (("k", k_pool, k_sf_pool), ("v", v_pool, v_sf_pool)):
            a.want(pool, name + "_pool", codes, itemsize=1)
            a.want(sf, name + "_sf_pool", scales, itemsize=1)
        a.want(context_lens, "context_lens", (batch,), I32_T)
        _want_table(a, block_table, batch, block_size, max_context_len)
        if topk:
            a.want(indices, "indices", (rows, topk), I32_T, rows=True)
        a.want(out, "out", (rows, hq, d), (q.dtype,))
        if lse is not None:
            a.want(lse, "lse", (rows, hq), (torch.float32,))
        if workspace is not None:
            a.want(workspace, "workspace", (None,), itemsize=1)
        a.on_gpu()
    _call(lib.paged_attention, dev, 2, q.data_ptr(), QUERY_TYPES[q.dtype],
          q_stride[0] if rows > 1 else hq * d, k_pool.data_ptr(), k_sf_pool.data_ptr(),
          v_pool.data_ptr(), v_sf_pool.data_ptr(), context_lens.data_ptr(), block_table.data_ptr(),
          _row_stride(block_table, block_table.shape[1]), _data(indices),
          _row_stride(indices, topk) if topk else 0, topk,
          d ** -0.5 if scale is None else float(scale), out.data_ptr(), _data(lse),
          _data(workspace), size, batch, next_n, hq, hkv, d, block_size, num_blocks, max_context_len)
    return out if lse is None else (out, lse)


@functools.lru_cache(maxsize=1024)
def paged_chunk_attention_workspace_size(batch, tokens, q_heads, kv_heads, d, max_context_len):
    """Bytes of workspace of a paged_chunk_attention call of these sizes."""
    n = lib.paged_chunk_attention_workspace_size(batch, tokens, q_heads, kv_heads, d, max_context_len)
    if n < 0:
        raise MqaError(2, lib.mqa_last_error().decode())
    return n


def _chunk_sizes(what, fmt, q, k_pool, context_lens, token_offsets, max_context_len):
    """Sizes of a call for ragged tokens, from its first arguments: (tokens, Hq, D, batch, pool
    shape, q's stride), once they make sense together."""
    if fmt != "mxfp4":
        _fmt(fmt)
        raise ValueError(f"{what} reads an mxfp4 cache, got {fmt!r}")
    if q is None or k_pool is None or context_lens is None:
        _required(q=q, k_pool=k_pool, context_lens=context_lens)
    if q.dim() != 3 or q.dtype not in QUERY_TYPES:
        raise ValueError(f"q must be [tokens, Hq, D] of bfloat16 or float16, got {tuple(q.shape)} {q.dtype}")
    if k_pool.dim() != 4:
        raise ValueError(f"k_pool must be [num_blocks, block_size, Hkv, D/2], got {tuple(k_pool.shape)}")
    tokens, hq, d = q.shape
    stride, batch = q.stride(), context_lens.numel()
    _block_size(k_pool.shape[1])
    if not (0 <= max_context_len < 2 ** 31 and tokens < 2 ** 31):
        raise ValueError("max_context_len and the number of tokens must be int32 and not negative")
    if stride[2] != 1 or (hq > 1 and stride[1] != d):
        raise ValueError("q rows must be contiguous")
    if token_offsets is None and (batch == 0 or tokens % batch):
        raise ValueError(f"{tokens} tokens of {batch} sequences need token_offsets")
    return tokens, hq, d, batch, k_pool.shape, stride[0] if tokens > 1 else hq * d


def paged_chunk_attention(fmt, q, k_pool, k_sf_pool, v_pool, v_sf_pool, context_lens, token_offsets,
                          block_table, max_context_len, scale=None, out=None, lse=None,
                          return_lse=False, workspace=None):
    """Attention of chunks of new tokens over a paged 4-bit cache that holds them already.

    fmt "mxfp4"; q [tokens, Hq, D] bf16 or fp16 (rows may be strided), pools [num_blocks,
    block_size, Hkv, D/2] with e8m0 [.., D/32].  The rows of sequence b are token_offsets[b] ..
    token_offsets[b + 1] - 1 (int32 [batch + 1], as paged_kv_slots gives them; None: as many for
    every sequence), its last tokens: row t of n sees the first context_lens[b] - n + 1 + t keys.
    scale defaults to D ** -0.5; scores must stay within +-2 ** 24 octaves.  Returns out (q's
    shape and type; zeros for a row without keys), or (out, lse fp32 [tokens, Hq]) with return_lse
    or an lse to fill; rows that no sequence has are left as they were.  workspace: a uint8 tensor of
    paged_chunk_attention_workspace_size bytes to keep between calls on one stream, or None."""
    tokens, hq, d, batch, (num_blocks, block_size, hkv, _), q_stride = _chunk_sizes(
        "paged_chunk_attention", fmt, q, k_pool, context_lens, token_offsets, max_context_len)
    dev = q.get_device()
    # (what is made here needs no check)
    given_out, given_lse, given_workspace = out is not None, lse is not None, workspace is not None
    if not given_out:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if not given_lse and return_lse:
        lse = q.new_empty((tokens, hq), dtype=torch.float32)
    need = paged_chunk_attention_workspace_size(batch, tokens, hq, hkv, d, max_context_len)
    if not given_workspace:
        workspace, size = (q.new_empty(need, dtype=torch.uint8), need) if need else (None, 0)
    else:
        size = workspace.numel()
    codes, scales = (num_blocks, block_size, hkv, d // 2), (num_blocks, block_size, hkv, d // 32)
    byte, i32 = k_pool.dtype, torch.int32
    if not (dev >= 0 and byte.itemsize == 1 and _fits(k_pool, codes, byte, dev)
            and _fits(v_pool, codes, byte, dev)
            and k_sf_pool is not None and k_sf_pool.dtype.itemsize == 1 and _fits(k_sf_pool, scales, k_sf_pool.dtype, dev)
            and _fits(v_sf_pool, scales, k_sf_pool.dtype, dev)
            and _fits(context_lens, (batch,), i32, dev)
            and (token_offsets is None or _fits(token_offsets, (batch + 1,), i32, dev))
            and _table_fits(block_table, batch, -(-max_context_len // block_size), dev)
            and (not given_out or _fits(out, q.shape, q.dtype, dev))
            and (not given_lse or _fits(lse, (tokens, hq), torch.float32, dev))
            and (not given_workspace or _fits(workspace, (size,), torch.uint8, dev))):
        a = _Args()
        a.want(q[:0], "q", (0, hq, d))
        for name, pool, sf in (("k", k_pool, k_sf_pool), ("v", v_pool, v_sf_pool)):
            a.want(pool, name + "_pool", codes, itemsize=1)
            a.want(sf, name + "_sf_pool", scales, itemsize=1)
        a.want(context_lens, "context_lens", (batch,), I32_T)
        if token_offsets is not None:
            a.want(token_offsets, "token_offsets", (batch + 1,), I32_T)
        _want_table(a, block_table, batch, block_size, max_context_len)
        a.want(out, "out", (tokens, hq, d), (q.dtype,))
        if lse is not None:
            a.want(lse, "lse", (tokens, hq), (torch.float32,))
        if workspace is not None:
            a.want(workspace, "workspace", (None,), itemsize=1)
        a.on_gpu()
    _call(lib.paged_chunk_attention, dev, 2, q.data_ptr(), QUERY_TYPES[q.dtype], q_stride,
          k_pool.data_ptr(), k_sf_pool.data_ptr(), v_pool.data_ptr(), v_sf_pool.data_ptr(),
          context_lens.data_ptr(), _data(token_offsets), block_table.data_ptr(),
          _row_stride(block_table, block_table.shape[1]), d ** -0.5 if scale is None else float(scale),
          out.data_ptr(), _data(lse), _data(workspace), size, batch, tokens, hq, hkv, d, block_size,
          num_blocks, max_context_len)
    return out if lse is None else (out, lse)


@functools.lru_cache(maxsize=1024)
def paged_attention_weights_workspace_size(batch, tokens, q_heads, kv_heads, d, max_context_len):
    """Bytes of workspace of a paged_attention_weights call of these sizes."""
    n = lib.paged_attention_weights_workspace_size(batch, tokens, q_heads, kv_heads, d, max_context_len)
    if n < 0:
        raise MqaError(2, lib.mqa_last_error().decode())
    return n


def paged_attention_weights(fmt, q, lse, k_pool, k_sf_pool, context_lens, token_offsets, block_table,
                            max_context_len, scale=None, weights=None, out=None, workspace=None):
    """The attention weight that every cached token has gathered, after one more step.

    out[b, j] = weights[b, j] (0 without weights) + the sum of exp(scale <q, k_j> - lse) over
    the rows of sequence b that see key j and over query heads, 0 behind the context: fp32
    [batch, max_context_len].  q, the pools, token_offsets and what a row sees are as in
    paged_chunk_attention, lse [tokens, Hq] is what that (or paged_attention) gave for q; rows of
    -inf give nothing.  weights and out may have wider rows, and be the same tensor.
    workspace: a uint8 tensor of paged_attention_weights_workspace_size bytes to keep between
    calls on one stream, or None."""
    tokens, hq, d, batch, (num_blocks, block_size, hkv, _), q_stride = _chunk_sizes(
        "paged_attention_weights", fmt, q, k_pool, context_lens, token_offsets, max_context_len)
    dev = q.get_device()
    given_out, given_workspace = out is not None, workspace is not None
    if not given_out:
        out = q.new_empty((batch, max_context_len), dtype=torch.float32)
    need = paged_attention_weights_workspace_size(batch, tokens, hq, hkv, d, max_context_len)
    if not given_workspace:
        workspace, size = (q.new_empty(need, dtype=torch.uint8), need) if need else (None, 0)
    else:
        size = workspace.numel()
    codes, scales = (num_blocks, block_size, hkv, d // 2), (num_blocks, block_size, hkv, d // 32)
    byte, i32 = k_pool.dtype, torch.int32
    if not (dev >= 0 and byte.itemsize == 1 and _fits(k_pool, codes, byte, dev)
            and k_sf_pool is not None and k_sf_pool.dtype.itemsize == 1 and _fits(k_sf_pool, scales, k_sf_pool.dtype, dev)
            and _fits(lse, (tokens, hq), torch.float32, dev)
            and _fits(context_lens, (batch,), i32, dev)
            and (token_offsets is None or _fits(token_offsets, (batch + 1,), i32, dev))
            and _table_fits(block_table, batch, -(-max_context_len // block_size), dev)
            and (weights is None or _rows_fit(weights, batch, max_context_len, dev))
            and (not given_out or _rows_fit(out, batch, max_context_len, dev))
            and (not given_workspace or _fits(workspace, (size,), torch.uint8, dev))):
        a = _Args()
        a.want(q[:0], "q", (0, hq, d))
        a.want(lse, "lse", (tokens, hq), (torch.float32,))
        a.want(k_pool, "k_pool", codes, itemsize=1)
        a.want(k_sf_pool, "k_sf_pool", scales, itemsize=1)
        a.want(context_lens, "context_lens", (batch,), I32_T)
        if token_offsets is not None:
            a.want(token_offsets, "token_offsets", (batch + 1,), I32_T)
        _want_table(a, block_table, batch, block_size, max_context_len)
        for name, t in (("weights", weights), ("out", out)):
            if t is not None:
                _want_rows(a, t, name, batch, max_context_len)
        if workspace is not None:
            a.want(workspace, "workspace", (None,), itemsize=1)
        a.on_gpu()
    _call(lib.paged_attention_weights, dev, 2, q.data_ptr(), QUERY_TYPES[q.dtype], q_stride, lse.data_ptr(),
          k_pool.data_ptr(), k_sf_pool.data_ptr(), context_lens.data_ptr(), _data(token_offsets),
          block_table.data_ptr(), _row_stride(block_table, block_table.shape[1]),
          d ** -0.5 if scale is None else float(scale), _data(weights),
          0 if weights is None else _row_stride(weights, weights.shape[1]), out.data_ptr(),
          _row_stride(out, out.shape[1]), _data(workspace), size, batch, tokens, hq, hkv, d, block_size,
          num_blocks, max_context_len)
    return out


def _rows_fit(t, batch, width, device):
    """fp32 rows of at least `width`, a row for each sequence, elements of a row adjacent."""
    shape = t.shape
    return (len(shape) == 2 and shape[0] == batch and shape[1] >= width and t.dtype is torch.float32
            and t.get_device() == device and (t.stride(1) == 1 or shape[1] <= 1))


def _want_rows(a, t, name, batch, width):
    a.want(t, name, (batch, None), (torch.float32,), rows=True)
    if t.shape[1] < width:
        raise ValueError(f"{name} rows must hold max_context_len = {width} values, got {t.shape[1]}")


Eviction = collections.namedtuple("Eviction", "context_lens block_table weights kept freed counts")


def paged_kv_evict(weights, context_lens, block_table, free_blocks, pools, keep, recent, max_context_len,
                   out=None, workspace=None):
    """Cut sequences longer than `keep` tokens to their last `recent` and the heaviest of the others.

    weights fp32 [batch, >= max_context_len] (paged_attention_weights); context_lens, block_table
    and free_blocks (int32, in the order to take them) are only read.  The tokens that stay
    are copied, in order, to free blocks of every pool in `pools` (contiguous
    [num_blocks, block_size, ...] tensors of any type: K, V, their scales, the indexer's keys),
    whose old blocks are not written.  Returns Eviction(context_lens int32 [batch], block_table
    int32 [batch, blocks] (-1 behind), weights fp32 [batch, max_context_len] (0 behind), kept
    int32 [batch, keep] (the old positions, -1 behind), freed int32 [batch * blocks] (the old
    blocks of cut sequences, -1 behind), counts int32 [2]: blocks asked of the free list
    and blocks in freed); `out` may hold these.  Where the first count exceeds
    len(free_blocks), the sequences that the list did not reach stay as they are.  Sequences of
    up to `keep` tokens stay as they are.  workspace: a uint8 tensor of
    paged_kv_evict_workspace_size bytes to keep between calls on one stream, or None."""
    if weights is None or context_lens is None or free_blocks is None or pools is None:
        _required(weights=weights, context_lens=context_lens, free_blocks=free_blocks, pools=pools)
    if not pools or any([p is None for p in pools]):
        raise ValueError("pools must hold tensors, at least one")
    if len(pools[0].shape) < 2:
        raise ValueError(f"pools must be [num_blocks, block_size, ...], got {tuple(pools[0].shape)}")
    lead = pools[0].shape[:2]
    num_blocks, block_size = lead
    _block_size(block_size)
    if not (1 <= keep < 2 ** 31 and 0 <= recent <= keep and 0 <= max_context_len < 2 ** 31
            and num_blocks < 2 ** 31):
        raise ValueError("keep must be at least 1, recent within [0, keep], sizes int32 and not negative")
    batch, dev = context_lens.numel(), context_lens.get_device()
    width = -(-max_context_len // block_size)
    i32, given = torch.int32, out is not None
    if not given:
        new = context_lens.new_empty
        out = Eviction(new(batch, dtype=i32), new((batch, width), dtype=i32),
                       new((batch, max_context_len), dtype=torch.float32), new((batch, keep), dtype=i32),
                       new(batch * width, dtype=i32), new(2, dtype=i32))
        strides = max(width, 1), max(max_context_len, 1), keep
    else:
        out = Eviction(*out)
    size = paged_kv_evict_workspace_size(batch, max_context_len)
    if workspace is None:
        workspace, given_workspace = context_lens.new_empty(size, dtype=torch.uint8), False
    else:
        size, given_workspace = workspace.numel(), True
    if not (dev >= 0 and _rows_fit(weights, batch, max_context_len, dev)
            and _fits(context_lens, (batch,), i32, dev) and _table_fits(block_table, batch, width, dev)
            and _fits(free_blocks, (free_blocks.numel(),), i32, dev)
            and all([p.get_device() == dev and p.shape[:2] == lead and p.is_contiguous() for p in pools])
            and (not given or (_fits(out.context_lens, (batch,), i32, dev)
                               and _table_fits(out.block_table, batch, width, dev)
                               and _rows_fit(out.weights, batch, max_context_len, dev)
                               and _table_fits(out.kept, batch, keep, dev)
                               and _fits(out.freed, (batch * width,), i32, dev)
                               and _fits(out.counts, (2,), i32, dev)))
            and (not given_workspace or _fits(workspace, (size,), torch.uint8, dev))):
        a = _Args()
        _want_rows(a, weights, "weights", batch, max_context_len)
        a.want(context_lens, "context_lens", (batch,), I32_T)
        _want_table(a, block_table, batch, block_size, max_context_len)
        a.want(free_blocks, "free_blocks", (None,), I32_T)
        for i, p in enumerate(pools):
            a.want(p, f"pools[{i}]", (num_blocks, block_size, *p.shape[2:]))
        a.want(out.context_lens, "out.context_lens", (batch,), I32_T)
        a.want(out.block_table, "out.block_table", (batch, None), I32_T, rows=True)
        if out.block_table.shape[1] < width:
            raise ValueError(f"out.block_table rows must hold {width} blocks, got {out.block_table.shape[1]}")
        _want_rows(a, out.weights, "out.weights", batch, max_context_len)
        a.want(out.kept, "out.kept", (batch, None), I32_T, rows=True)
        if out.kept.shape[1] < keep:
            raise ValueError(f"out.kept rows must hold keep = {keep} positions, got {out.kept.shape[1]}")
        a.want(out.freed, "out.freed", (batch * width,), I32_T)
        a.want(out.counts, "out.counts", (2,), I32_T)
        a.want(workspace, "workspace", (None,), itemsize=1)
        a.on_gpu()
    if given:
        strides = [_row_stride(t, t.shape[1]) for t in (out.block_table, out.weights, out.kept)]
    # the C structs {data, bytes of a token}, as words: of a contiguous tensor, the stride
    # of a token is its size
    words = []
    for p in pools:
        words += p.data_ptr(), p.stride(1) * p.itemsize
    described = (ctypes.c_int64 * len(words))(*words)
    _call(lib.paged_kv_evict, dev, weights.data_ptr(), _row_stride(weights, weights.shape[1]),
          context_lens.data_ptr(), block_table.data_ptr(), _row_stride(block_table, block_table.shape[1]),
          free_blocks.data_ptr(), free_blocks.shape[0], described, len(pools), out.context_lens.data_ptr(),
          out.block_table.data_ptr(), strides[0], out.weights.data_ptr(), strides[1], out.kept.data_ptr(),
          strides[2], out.freed.data_ptr(), out.counts.data_ptr(),
          workspace.data_ptr(), size, batch, block_size, num_blocks, max_context_len, keep, recent)
    return out


@functools.lru_cache(maxsize=1024)
def paged_kv_evict_workspace_size(batch, max_context_len):
    """Bytes of workspace of a paged_kv_evict call of these sizes."""
    n = lib.paged_kv_evict_workspace_size(batch, max_context_len)
    if n < 0:
        raise MqaError(2, lib.mqa_last_error().decode())
    return n
