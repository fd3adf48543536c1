"""Cases for the paged-cache operators: tables and slot maps, the quantising
cache write, and attention over the 4-bit cache (whole contexts, or the tokens
a top-k selected).

`run` computes a case either with elementary torch operations (`own` false) or
with the library's entry points (`own` true); `exact` is the same result in 64
bits, from the definition.

Shapes follow the library's own paged workload (64 sequences of 1024..32768
tokens, 4 query tokens each, 64 heads of 128, blocks of 64, top-k of 2048) and
generic grouped-head ones around it.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CODE_MAX = {"fp8": 448.0, "mxfp8": 448.0, "mxfp4": 6.0}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def slots_case(name, batch, lo, hi, new, block):
    """new = 0: fresh prompts (every token is new); otherwise tokens per step."""
    return {"name": name, "op": "slots", "batch": batch, "lo": lo, "hi": hi, "new": new,
            "block": block}


def write_case(name, fmt, rows, heads, d, dtype, block, values):
    return {"name": name, "op": "write", "fmt": fmt, "rows": rows, "heads": heads, "d": d,
            "dtype": dtype, "block": block, "values": values}


def attend_case(name, batch, next_n, kv_heads, group, d, lo, hi, block, dtype, topk=0):
    return {"name": name, "op": "attend", "batch": batch, "next_n": next_n,
            "kv_heads": kv_heads, "group": group, "d": d, "lo": lo, "hi": hi, "block": block,
            "dtype": dtype, "topk": topk}


def listed():
    return [
        # one decoding step of the paged workload: 4 new tokens a sequence
        slots_case("slots_step", 64, 1024, 32768, 4, 64),
        # a batch of fresh, ragged prompts in small blocks: half a million slots
        slots_case("slots_prompts", 513, 1, 1900, 0, 16),
        # the indexer keys of one decoding step, into the FP8 pool the paged logits read
        write_case("write_fp8_step", "fp8", 256, 1, 128, "bf16", 64, False),
        # keys (or values) of a prompt chunk into the 4-bit cache, 8 heads, and what
        # the cache now stands for, for the chunk's own attention
        write_case("write_mxfp4_prompt", "mxfp4", 32768, 8, 128, "bf16", 64, True),
        # an odd number of fp32 rows of odd head count, D = 64
        write_case("write_mxfp8_odd", "mxfp8", 2047, 3, 64, "fp32", 32, False),
        # a single short request: latency
        attend_case("attend_one", 1, 1, 2, 8, 128, 113, 113, 16, "bf16"),
        # the paged workload: 4 query tokens x 64 heads share one KV head
        attend_case("attend_mqa_step", 64, 4, 1, 64, 128, 1024, 32768, 64, "bf16"),
        # plain decoding with grouped heads, ragged contexts
        attend_case("attend_gqa_step", 32, 1, 8, 8, 128, 1024, 32768, 64, "fp16"),
        # one request with a long context and a draft token
        attend_case("attend_long", 1, 2, 4, 8, 128, 131072, 131072, 64, "bf16"),
        # D = 64, groups of 5, three query tokens, lengths from zero
        attend_case("attend_odd", 29, 3, 3, 5, 64, 0, 5000, 32, "fp16"),
        # sparse decoding: each query token attends to the 2048 tokens its indexer chose
        attend_case("topk_step", 64, 4, 1, 64, 128, 1024, 32768, 64, "bf16", 2048),
        # the same for a single request
        attend_case("topk_one", 1, 1, 1, 64, 128, 9001, 9001, 64, "bf16", 2048),
    ]


def draw(rng):
    def spread(lo, hi):                      # log-uniform integer
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["slots", "write", "attend", "attend", "topk"])
    if op == "slots":
        batch, hi = spread(1, 2048), spread(1, 32768)
        new = rng.choice([0, 1, 2, 4, 7])
        if new == 0:
            hi = max(1, min(hi, 500000 // batch))
        hi = min(hi, 2000000 // batch)
        return slots_case(None, batch, rng.randint(0, hi), hi, new, rng.choice([16, 32, 64]))
    if op == "write":
        heads, d = rng.choice([1, 1, 2, 3, 4, 8]), rng.choice([64, 128])
        rows = spread(1, 32768 * 1024 // (heads * d) if heads * d > 1024 else 32768)
        return write_case(None, rng.choice(["fp8", "mxfp8", "mxfp4"]), rows, heads, d,
                          rng.choice(["bf16", "fp16", "fp32"]) if rows < 9000 else "bf16",
                          rng.choice([16, 32, 64]), rng.random() < 0.5)
    kv_heads = rng.choice([1, 1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16] if kv_heads > 1 else [1, 4, 8, 16, 24, 33, 64])
    next_n = rng.choice([1, 1, 1, 2, 3, 4, 7, 16])
    d = rng.choice([64, 128, 128])
    batch = spread(1, 128)
    hi = spread(1, 131072)
    while batch * hi * kv_heads > 3000000 or batch * hi * next_n * kv_heads * group > 130000000:
        if hi > 64 * batch:
            hi = hi // 2 + 1
        else:
            batch = max(1, batch // 2)
            hi = hi * 3 // 4 + 1
    topk = 0
    if op == "topk":
        topk = spread(16, 2048)
        batch = max(1, min(batch, 256 // next_n))
    return attend_case(None, batch, next_n, kv_heads, group, d, rng.randint(0, hi), hi,
                       rng.choice([16, 32, 64]), rng.choice(["bf16", "fp16"]), topk)


def lengths(case):
    """Ragged lengths over [lo, hi], the same for every seed."""
    lo, hi = case["lo"], case["hi"]
    return [lo + int(((0.5 + b * 0.6180339887498949) % 1.0) * (hi - lo + 1))
            for b in range(case["batch"])]


def new_tokens(case):
    return [n if case["new"] == 0 else min(n, case["new"]) for n in lengths(case)]


def blocks(n, block):
    return -(-n // block)


def work(case):
    if case["op"] == "slots":
        size, lens, new = case["block"], lengths(case), new_tokens(case)
        taken = sum(blocks(n, size) - blocks(n - m, size) for n, m in zip(lens, new))
        # lengths, free ids and the blocks behind the new tokens in; table entries, slots and offsets out
        touched = sum(blocks(n, size) - (n - m) // size for n, m in zip(lens, new) if m)
        return {"bytes": 8 * len(lens) + 4 * touched + 4 * taken + 8 * sum(new)
                + 4 * (len(lens) + 1) + 4, "flops": 0}
    if case["op"] == "write":
        n = case["rows"] * case["heads"]
        d, size = case["d"], torch.finfo(DTYPES[case["dtype"]]).bits // 8
        stored = d / 2 + d / 32 if case["fmt"] == "mxfp4" else (
            d + d / 32 if case["fmt"] == "mxfp8" else d + 4)
        out = stored + (d * size if case["values"] else 0)
        return {"bytes": n * (d * size + out) + 8 * case["rows"], "flops": 0}
    rows = case["batch"] * case["next_n"]
    heads, d, lens = case["kv_heads"] * case["group"], case["d"], lengths(case)
    token = 2 * case["kv_heads"] * (d // 2 + d // 32)
    seen = [max(0, n - case["next_n"] + 1 + t) for n in lens for t in range(case["next_n"])]
    if case["topk"]:
        seen = [min(case["topk"], n) for n in seen]
        # a token is read once for a sequence, however many of its rows chose it
        # (the expected number of tokens that independent choices name)
        read = sum(round(n * (1 - math.prod(1 - s / n for s in seen[b * case["next_n"]:
                                                                    (b + 1) * case["next_n"]])))
                   for b, n in enumerate(lens) if n)
        extra = 4 * rows * case["topk"]
    else:
        read, extra = sum(lens), 0
    pages = 4 * sum(blocks(n, case["block"]) for n in lens)
    return {"bytes": read * token + extra + pages + 4 * len(lens)
            + rows * heads * (4 * d + 4), "flops": 4 * d * heads * sum(seen)}


# --------------------------------------------------------------------------
# formats, in elementary operations
# --------------------------------------------------------------------------

def e2m1_pairs(device):
    grid = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    grid = torch.tensor(grid + [-g for g in grid], device=device)
    byte = torch.arange(256, device=device)
    return torch.stack([grid[byte & 15], grid[byte >> 4]], -1)


def powers_of_two(device):
    """2^-127 .. 2^127 at 0 .. 254 (a table: pow on the device need not be exact)."""
    return torch.tensor([2.0 ** k for k in range(-127, 128)], dtype=torch.float64, device=device)


def e8m0_values(device):
    # bytes over 252 could overflow the product and count as NaN
    v = powers_of_two(device).float()
    return torch.cat([v[:253], v.new_full((3,), math.nan)])


def decode_mxfp4(codes, sf):
    v = e2m1_pairs(codes.device)[codes.long()].flatten(-2)
    s = e8m0_values(codes.device)[sf.long()]
    return (v.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def encode(fmt, x):
    """Codes and scales of rows [.., D], and the values they stand for: the scale of a group is the
    smallest power of two under which none of its elements exceeds the largest code."""
    top = CODE_MAX[fmt]
    x = x.float()
    group = x.shape[-1] if fmt == "fp8" else 32
    x = x.unflatten(-1, (-1, group))
    amax = x.abs().amax(-1)
    part, exponent = torch.frexp(amax)
    part_top, exponent_top = math.frexp(top)
    e = exponent.long() - exponent_top + (part > part_top).long()
    e = e.clamp(-126 if fmt == "fp8" else -127, 127)
    e = torch.where(amax == 0, torch.zeros_like(e), e)
    fine = torch.isfinite(amax)
    two = powers_of_two(x.device)[e + 127]
    y = torch.where(fine[..., None], x.double() / two[..., None], 0.0).float()
    if fmt == "mxfp4":
        a = y.abs()
        code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
                + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5.0).byte())
        code = code + 8 * torch.signbit(y).byte()
        low, high = code.flatten(-2)[..., 0::2], code.flatten(-2)[..., 1::2]
        codes = low + 16 * high
        held = e2m1_pairs(x.device)[codes.long()].flatten(-2).unflatten(-1, (-1, group))
    else:
        code = y.to(torch.float8_e4m3fn)
        codes = code.view(torch.uint8).flatten(-2)
        held = code.float()
    values = torch.where(fine[..., None], held.double() * two[..., None], math.nan)
    if fmt == "fp8":
        scales = torch.where(fine, two, math.nan).float()[..., 0]
    else:
        scales = torch.where(fine, e + 127, 255).to(torch.uint8)
    return codes, scales, values.flatten(-2)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    i32 = dict(dtype=torch.int32, device=dev)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def order(n):
        return torch.randperm(n, generator=g, device=dev).int()

    if case["op"] == "slots":
        size, lens, new = case["block"], lengths(case), new_tokens(case)
        width = max(1, blocks(max(lens), size))
        held = torch.tensor([blocks(n - m, size) for n, m in zip(lens, new)], device=dev)
        taken = sum(blocks(n, size) for n in lens) - int(held.sum())
        pool = int(held.sum()) + taken + 64
        ids = order(pool)
        table = torch.full((len(lens), width), -1, **i32)
        table[torch.arange(width, device=dev)[None] < held[:, None]] = ids[:int(held.sum())]
        return {"case": case, "context_lens": torch.tensor(lens, **i32),
                "new_lens": torch.tensor(new, **i32), "free": ids[int(held.sum()):].clone(),
                "table": table, "pool": pool,
                # a step's buffers are sized for its padded batch
                "max_tokens": max(1, sum(new) + 3), "max_context_len": max(1, max(lens))}

    if case["op"] == "write":
        n, heads, d, fmt = case["rows"], case["heads"], case["d"], case["fmt"]
        # a view of a wider projection; channels of unlike size, a few large rows
        size = torch.exp(normal(2, heads, d)) * torch.exp(normal(n, 1, 1, 1))
        wide = (normal(n, 2, heads, d) * size).to(DTYPES[case["dtype"]])
        num_blocks = blocks(n, case["block"]) + 3
        total = num_blocks * case["block"]
        slots = order(total)[:n].long()
        slots[n - 1 - n // 64:n - 1] = -1                     # padded rows write nothing
        shape = (num_blocks, case["block"]) + ((heads,) if heads > 1 else ())
        pool = torch.randint(0, 0x77, shape + (d // 2 if fmt == "mxfp4" else d,), generator=g,
                             device=dev, dtype=torch.uint8)
        x = wide[:, 1] if heads > 1 else wide[:, 1, 0]
        state = {"case": case, "x": x, "slots": slots, "pool": pool, "sf": None, "scale": None,
                 "values": torch.empty(x.shape, dtype=x.dtype, device=dev) if case["values"] else None}
        if fmt == "fp8":
            state["scale"] = torch.rand(shape, generator=g, device=dev)
        else:
            state["sf"] = torch.randint(120, 130, shape + (d // 32,), generator=g, device=dev,
                                        dtype=torch.uint8)
        return state

    lens, size, heads, d = lengths(case), case["block"], case["kv_heads"], case["d"]
    width = max(1, blocks(max(lens), size))
    need = torch.tensor([blocks(n, size) for n in lens], device=dev)
    used = int(need.sum())
    num_blocks = used + max(1, used // 10)
    ids = order(num_blocks)
    table = torch.full((len(lens), width), -1, **i32)
    table[torch.arange(width, device=dev)[None] < need[:, None]] = ids[:used]
    state = {"case": case, "context_lens": torch.tensor(lens, **i32), "table": table,
             "max_context_len": max(1, max(lens)), "scale": d ** -0.5, "indices": None}
    # what no sequence holds is never written: its scales are the NaN byte
    held = torch.zeros(num_blocks, size, dtype=torch.bool, device=dev)
    tokens = torch.arange(width * size, device=dev)
    inside = tokens[None] < state["context_lens"][:, None]
    slot = table.clamp_min(0).long().repeat_interleave(size, 1) * size + tokens % size
    held.view(-1)[slot[inside]] = True
    for side in ("k", "v"):
        codes = torch.empty(num_blocks, size, heads, d // 2, dtype=torch.uint8, device=dev)
        sf = torch.empty(num_blocks, size, heads, d // 32, dtype=torch.uint8, device=dev)
        spread = torch.exp(0.5 * normal(heads, d))
        step = max(1, (1 << 26) // (size * heads * d))
        for b in range(0, num_blocks, step):
            n = min(step, num_blocks - b)
            codes[b:b + n], sf[b:b + n] = encode("mxfp4", normal(n, size, heads, d) * spread)[:2]
        sf[~held] = 255
        state[side], state[side + "_sf"] = codes, sf
    rows = case["batch"] * case["next_n"]
    state["q"] = (2.0 * normal(rows, heads * case["group"], d)).to(DTYPES[case["dtype"]])
    if case["topk"]:
        k, seen = case["topk"], visible(state)
        picked = torch.full((rows, k), -1, **i32)
        for r in range(0, rows, 64):
            n = min(k, state["max_context_len"])
            score = torch.rand(min(64, rows - r), state["max_context_len"], generator=g, device=dev)
            score.masked_fill_(torch.arange(state["max_context_len"], device=dev)[None]
                               >= seen[r:r + 64, None], -1.0)
            best, at = score.topk(n, dim=1)
            at = torch.where(best < 0, torch.iinfo(torch.int32).max, at).sort(1).values
            at = torch.where(at == torch.iinfo(torch.int32).max, -1, at)
            picked[r:r + 64, :n] = at.int()
        state["indices"] = picked
    return state


def visible(state):
    """Keys that each query row may see."""
    n = state["case"]["next_n"]
    lens = state["context_lens"].long()
    t = torch.arange(n, device=lens.device)
    return (lens[:, None] - n + 1 + t[None]).clamp_min(0).flatten()


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return run_own(op, state)
    if op == "slots":
        return slots_plain(state)
    if op == "write":
        return write_plain(state)
    return attend_topk_plain(state) if state["indices"] is not None else attend_plain(state)


def run_own(op, state):
    import mqa_logits_amd as mq
    case = state["case"]
    if op == "slots":
        slots, offsets, taken = mq.paged_kv_slots(
            state["context_lens"], state["new_lens"], state["free"], state["table"], state["pool"],
            case["block"], state["max_context_len"], state["max_tokens"])
        return {"slots": slots, "offsets": offsets, "taken": taken, "table": state["table"]}
    if op == "write":
        mq.paged_kv_write(case["fmt"], state["x"], state["slots"], state["pool"], state["sf"],
                          state["scale"], values=state["values"])
        return written(state)
    out, lse = mq.paged_attention("mxfp4", state["q"], state["k"], state["k_sf"], state["v"],
                                  state["v_sf"], state["context_lens"], state["table"],
                                  case["next_n"], state["max_context_len"], scale=state["scale"],
                                  indices=state["indices"], return_lse=True)
    return {"out": out, "lse": lse}


def written(state):
    pool = state["pool"]
    if state["case"]["fmt"] != "mxfp4":
        pool = pool.view(torch.float8_e4m3fn)
    out = {"pool": pool, "scales": state["scale"] if state["sf"] is None else state["sf"]}
    if state["values"] is not None:
        out["values"] = state["values"]
    return out


def slots_plain(state):
    case, table, free = state["case"], state["table"], state["free"]
    size, dev = case["block"], table.device
    lens = state["context_lens"].clamp(0, state["max_context_len"])
    new = torch.minimum(state["new_lens"].clamp_min(0), lens)
    old = lens - new
    first, last = (old + size - 1) // size, (lens + size - 1) // size
    ends = torch.cumsum(last - first, 0)
    base = ends - (last - first)
    column = torch.arange(table.shape[1], device=dev)[None]
    at = base[:, None] + column - first[:, None]
    ids = torch.where(at < free.numel(), free[at.clamp(0, free.numel() - 1)], -1)
    table.copy_(torch.where((column >= first[:, None]) & (column < last[:, None]), ids, table))
    offsets = torch.cat([torch.zeros_like(ends[:1]), torch.cumsum(new, 0)])
    token = torch.arange(state["max_tokens"], device=dev)
    row = torch.searchsorted(offsets[1:], token, right=True)
    inside = row < lens.numel()
    row = row.clamp_max(lens.numel() - 1)
    position = old[row].long() + token - offsets[row]
    position = torch.where(inside, position, 0)
    block = table[row, position // size].long()
    slots = torch.where(inside & (block >= 0) & (block < state["pool"]),
                        block * size + position % size, -1)
    return {"slots": slots, "offsets": offsets.int(), "taken": ends[-1:].int(), "table": table}


def write_plain(state):
    case, x, slots = state["case"], state["x"], state["slots"]
    codes, scales, values = encode(case["fmt"], x)
    kept = (slots >= 0) & (slots < state["pool"].shape[0] * state["pool"].shape[1])
    at = slots[kept]
    state["pool"].flatten(0, 1)[at] = codes[kept]
    into = state["scale"] if state["sf"] is None else state["sf"]
    into.flatten(0, 1)[at] = scales[kept]
    if state["values"] is not None:
        state["values"].copy_(values)
    return written(state)


def softmax_parts(scores, mask):
    """exp(score - max) under a mask that may leave a row empty, their sum, and log of the sum of exponentials."""
    scores = scores.masked_fill(~mask, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isneginf(top), 0.0, top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    return p, total, (top + torch.log(total)).squeeze(-1)


def attend_plain(state):
    case, q, table = state["case"], state["q"], state["table"]
    batch, n, heads, group, d = (case["batch"], case["next_n"], case["kv_heads"], case["group"],
                                 case["d"])
    page = table.clamp_min(0).long()
    span = page.shape[1] * case["block"]
    token = torch.arange(span, device=q.device)
    inside = token[None] < state["context_lens"][:, None]

    def gather(codes, sf):                                   # [batch, heads, span, d]
        v = decode_mxfp4(codes[page], sf[page]).reshape(batch, span, heads, d)
        return torch.where(inside[:, :, None, None], v, 0.0).transpose(1, 2).contiguous()

    rows = q.float().view(batch, n, heads, group, d).transpose(1, 2).reshape(batch, heads, n * group, d)
    keys = gather(state["k"], state["k_sf"]).transpose(2, 3).contiguous()
    scores = (rows @ keys) * state["scale"]
    seen = visible(state).view(batch, 1, n, 1, 1)
    mask = (token < seen).expand(batch, heads, n, group, span).reshape(batch, heads, n * group, span)
    p, total, lse = softmax_parts(scores, mask)
    out = (p @ gather(state["v"], state["v_sf"])) / torch.where(total == 0, 1.0, total)
    out = out.view(batch, heads, n, group, d).transpose(1, 2).reshape(q.shape)
    lse = lse.view(batch, heads, n, group).transpose(1, 2).reshape(q.shape[:2])
    return {"out": out.to(q.dtype), "lse": lse}


def attend_topk_plain(state):
    case, q, at = state["case"], state["q"], state["indices"].long()
    heads, group, d = case["kv_heads"], case["group"], case["d"]
    mask = (at >= 0) & (at < visible(state)[:, None])
    at = torch.where(mask, at, 0)
    row = torch.arange(q.shape[0], device=q.device)[:, None] // case["next_n"]
    block = state["table"][row, at // case["block"]].clamp_min(0).long()

    def gather(codes, sf):                                   # [rows, heads, topk, d]
        v = decode_mxfp4(codes[block, at % case["block"]], sf[block, at % case["block"]])
        return torch.where(mask[:, :, None, None], v, 0.0).transpose(1, 2).contiguous()

    keys = gather(state["k"], state["k_sf"]).transpose(2, 3).contiguous()
    scores = (q.float().view(-1, heads, group, d) @ keys) * state["scale"]
    p, total, lse = softmax_parts(scores, mask[:, None, None, :])
    out = (p @ gather(state["v"], state["v_sf"])) / torch.where(total == 0, 1.0, total)
    return {"out": out.reshape(q.shape).to(q.dtype), "lse": lse.reshape(q.shape[:2])}


# --------------------------------------------------------------------------
# 64 bits, from the definitions
# --------------------------------------------------------------------------

def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "slots":
        return slots_exact(state)
    if case["op"] == "write":
        return write_exact(state)
    return attend_exact(state)


def slots_exact(state):
    """Sequence by sequence, on the host."""
    size = state["case"]["block"]
    table = state["table"].cpu().numpy().copy()
    free = state["free"].cpu().numpy()
    slots = np.full(state["max_tokens"], -1, np.int64)
    offsets, taken = [0], 0
    for b, (n, m) in enumerate(zip(state["context_lens"].tolist(), state["new_lens"].tolist())):
        for j in range(-(-(n - m) // size), -(-n // size)):
            table[b, j] = free[taken] if taken < len(free) else -1
            taken += 1
        position = np.arange(n - m, n)
        block = table[b, position // size].astype(np.int64)
        slots[offsets[-1]:offsets[-1] + m] = np.where(block >= 0, block * size + position % size, -1)
        offsets.append(offsets[-1] + m)
    dev = state["table"].device
    return {"slots": torch.from_numpy(slots).to(dev),
            "offsets": torch.tensor(offsets, dtype=torch.int32, device=dev),
            "taken": torch.tensor([taken], dtype=torch.int32, device=dev),
            "table": torch.from_numpy(table).to(dev)}


def code_values(fmt, device):
    """The value of every non-negative code, by its fields."""
    bits, mantissa, bias = (3, 1, 1) if fmt == "mxfp4" else (7, 3, 7)
    values = []
    for code in range(2 ** bits - (0 if fmt == "mxfp4" else 1)):
        exponent, fraction = code >> mantissa, (code & (2 ** mantissa - 1)) / 2 ** mantissa
        values.append(fraction * 2.0 ** (1 - bias) if exponent == 0
                      else (1 + fraction) * 2.0 ** (exponent - bias))
    return torch.tensor(values, dtype=torch.float64, device=device)


def write_exact(state):
    case, fmt = state["case"], state["case"]["fmt"]
    x = state["x"].double()
    group = case["d"] if fmt == "fp8" else 32
    x = x.reshape(*x.shape[:-1], -1, group)
    amax = x.abs().amax(-1, keepdim=True)
    low = -126 if fmt == "fp8" else -127
    e = torch.full_like(amax, low)
    for k in range(low, 127):                                # smallest power of two that is enough
        e = torch.where(amax > CODE_MAX[fmt] * 2.0 ** k, k + 1, e)
    two = torch.where(amax == 0, 1.0, powers_of_two(x.device)[e.long() + 127])
    y = x / two
    grid = code_values(fmt, x.device)
    above = torch.searchsorted(grid, y.abs().contiguous()).clamp(1, grid.numel() - 1)
    below = above - 1
    up, down = grid[above] - y.abs(), y.abs() - grid[below]
    code = torch.where((up < down) | ((up == down) & (above % 2 == 0)), above, below)
    held = torch.copysign(grid[code], y)
    byte = code + torch.signbit(y) * (8 if fmt == "mxfp4" else 128)
    kept = (state["slots"] >= 0) & (state["slots"] < state["pool"].shape[0] * state["pool"].shape[1])
    at = state["slots"][kept]
    if fmt == "mxfp4":
        byte = byte.flatten(-2)
        pool = state["pool"].clone()
        pool.flatten(0, 1)[at] = (byte[..., 0::2] | (byte[..., 1::2] << 4)).to(torch.uint8)[kept]
    else:
        pool = state["pool"].view(torch.float8_e4m3fn).float().double()
        pool.flatten(0, 1)[at] = held.flatten(-2)[kept]
    if fmt == "fp8":
        scales = state["scale"].double()
        scales.flatten(0, 1)[at] = two[..., 0, 0][kept]
    else:
        scales = state["sf"].clone()
        scales.flatten(0, 1)[at] = (torch.log2(two[..., 0]).round() + 127).to(torch.uint8)[kept]
    out = {"pool": pool, "scales": scales}
    if state["values"] is not None:
        out["values"] = (held * two).flatten(-2)
    return out


def attend_exact(state):
    """Row by row, gathering only the tokens that the row attends to."""
    case, q = state["case"], state["q"].double()
    heads, group, size, n = case["kv_heads"], case["group"], case["block"], case["next_n"]
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    grid = code_values("mxfp4", q.device)

    def values(codes, sf):
        nibble = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
        v = grid[nibble & 7] * (1 - 2 * (nibble >> 3)).double()
        return v * powers_of_two(sf.device)[sf.long()].repeat_interleave(32, -1)

    lens = state["context_lens"].tolist()
    for b, length in enumerate(lens):
        if length == 0:
            continue
        token = torch.arange(length, device=q.device)
        slot = state["table"][b, token // size].long() * size + token % size
        k = values(state["k"].flatten(0, 1)[slot], state["k_sf"].flatten(0, 1)[slot])
        v = values(state["v"].flatten(0, 1)[slot], state["v_sf"].flatten(0, 1)[slot])
        for t in range(n):
            r, seen = b * n + t, max(0, length - n + 1 + t)
            at = token[:seen]
            if state["indices"] is not None:
                at = state["indices"][r].long()
                at = at[(at >= 0) & (at < seen)]
            if at.numel() == 0:
                continue
            for h in range(heads):
                own_rows = slice(h * group, (h + 1) * group)
                s = (q[r, own_rows] @ k[at, h].T.contiguous()) * state["scale"]
                lse[r, own_rows] = torch.logsumexp(s, -1)
                out[r, own_rows] = torch.softmax(s, -1) @ v[at, h]
    return {"out": out, "lse": lse}
