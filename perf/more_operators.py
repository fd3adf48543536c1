"""Cases for attention of chunks of new tokens over the paged 4-bit cache, the
attention weight that every cached token has gathered, and the eviction of the
tokens that gathered least.

`run` computes a case either with elementary torch operations (`own` false) or
with the library's entry points (`own` true); `exact` is the same result in 64
bits, from the definition.

Shapes follow the library's own paged workload (64 sequences of 1024..32768
tokens, 4 query tokens each, 64 heads of 128, blocks of 64) and generic
grouped-head ones around it.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def attend_case(name, op, batch, new, kv_heads, group, d, lo, hi, block, dtype):
    """op "chunk" or "weights"; new = 0: fresh prompts (every token is new); otherwise new
    tokens a sequence, as far as it has them."""
    return {"name": name, "op": op, "batch": batch, "new": new, "kv_heads": kv_heads,
            "group": group, "d": d, "lo": lo, "hi": hi, "block": block, "dtype": dtype}


def evict_case(name, batch, lo, hi, keep, recent, kv_heads, d, block, index):
    """index: the indexer's fp8 keys lie in a pool of their own beside K and V."""
    return {"name": name, "op": "evict", "batch": batch, "lo": lo, "hi": hi, "keep": keep,
            "recent": recent, "kv_heads": kv_heads, "d": d, "block": block, "index": index}


def listed():
    return [
        # the last few tokens of a short prompt: latency
        attend_case("chunk_one", "chunk", 1, 17, 2, 8, 128, 113, 113, 16, "bf16"),
        # the paged workload's sequences, each with a chunk of 32 tokens (drafts to verify, or
        # prompts that go on beside decoding); 64 heads share one KV head
        attend_case("chunk_mqa", "chunk", 64, 32, 1, 64, 128, 1024, 32768, 64, "bf16"),
        # a batch of fresh, ragged prompts
        attend_case("chunk_prompts", "chunk", 33, 0, 8, 4, 128, 1, 1900, 16, "bf16"),
        # one chunk of a long document
        attend_case("chunk_long", "chunk", 1, 4096, 8, 8, 128, 65536, 65536, 64, "bf16"),
        # D = 64, groups of 5, lengths from zero
        attend_case("chunk_odd", "chunk", 29, 201, 3, 5, 64, 0, 5000, 32, "fp16"),
        # the weight that one decoding step of the paged workload gives to every cached token
        attend_case("weights_step", "weights", 64, 4, 1, 64, 128, 1024, 32768, 64, "bf16"),
        # plain decoding with grouped heads, ragged contexts
        attend_case("weights_gqa", "weights", 32, 1, 8, 8, 128, 1024, 32768, 64, "fp16"),
        # the last 256 tokens of a long prompt judge all of it
        attend_case("weights_window", "weights", 1, 256, 8, 8, 128, 32768, 32768, 64, "bf16"),
        # D = 64, groups of 5, lengths from zero
        attend_case("weights_odd", "weights", 29, 3, 3, 5, 64, 0, 5000, 32, "fp16"),
        # short requests of a small cache: latency
        evict_case("evict_small", 3, 0, 600, 128, 32, 2, 64, 16, False),
        # the paged workload's sequences, cut to 4096 tokens, indexer keys and all
        evict_case("evict_mqa", 64, 1024, 32768, 4096, 256, 1, 128, 64, True),
        # one long request with eight KV heads, cut to an eighth
        evict_case("evict_long", 1, 131072, 131072, 16384, 1024, 8, 128, 64, False),
    ]


def draw(rng):
    def spread(lo, hi):                      # log-uniform integer
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["chunk", "chunk", "weights", "evict"])
    block = rng.choice([16, 32, 64])
    d = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 1, 2, 3, 4, 8])
    if op == "evict":
        batch, hi = spread(1, 128), spread(1, 131072)
        hi = max(1, min(hi, 1500000 // (batch * kv_heads)))
        keep = spread(1, hi)
        return evict_case(None, batch, rng.randint(0, hi), hi, keep, rng.randint(0, keep // 2),
                          kv_heads, d, block, rng.random() < 0.5)
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16] if kv_heads > 1 else [1, 4, 8, 16, 24, 33, 64])
    batch, hi = spread(1, 128), spread(1, 65536)
    if op == "weights":
        new = rng.choice([1, 1, 1, 2, 3, 4, 7, 16, 64, 200])
        most = 3e8                           # (row, head, key) triples
    else:
        new = rng.choice([0, 0, spread(1, 64), spread(1, 4096)])
        most = 2e9
    while True:
        n = hi if new == 0 else min(new, hi)
        if (batch * hi * kv_heads <= 3000000
                and batch * n * hi * kv_heads * group * (0.5 if new == 0 else 1.0) <= most
                and batch * n * kv_heads * group * d <= 1 << 28):
            break
        if batch > 1:
            batch = batch // 2
        else:
            hi = hi * 3 // 4 + 1
    return attend_case(None, op, batch, new, kv_heads, group, d, rng.randint(0, hi), hi, block,
                       rng.choice(["bf16", "fp16"]))


def lengths(case):
    """Ragged lengths over [lo, hi], the same for every seed."""
    lo, hi = case["lo"], case["hi"]
    return [lo + int(((0.5 + b * 0.6180339887498949) % 1.0) * (hi - lo + 1))
            for b in range(case["batch"])]


def new_tokens(case):
    return [n if case["new"] == 0 else min(n, case["new"]) for n in lengths(case)]


def blocks(n, block):
    return -(-n // block)


def row_bytes(case):
    """Bytes of a token in each pool."""
    heads, d = case["kv_heads"], case["d"]
    return [heads * d // 2, heads * d // 32] * 2 + ([d, 4] if case["index"] else [])


def work(case):
    lens, size = lengths(case), case["block"]
    if case["op"] == "evict":
        cut = [n for n in lens if n > case["keep"]]
        width = max(1, blocks(max(lens), size))
        judged = sum(n - case["recent"] for n in cut)
        moved = case["keep"] * len(cut)
        left = sum(min(n, case["keep"]) for n in lens)
        # weights and kept rows in, rows, weights and positions out, both tables
        return {"bytes": 4 * judged + 2 * moved * sum(row_bytes(case)) + 4 * left
                + 4 * case["batch"] * (case["keep"] + max(1, max(lens)) + 3 * width + 2),
                "flops": 0}
    heads, d = case["kv_heads"] * case["group"], case["d"]
    pairs = sum(m * (n - m) + m * (m + 1) // 2 for n, m in zip(lens, new_tokens(case)))
    rows = sum(new_tokens(case))
    pages = 4 * sum(blocks(n, size) for n in lens) + 8 * len(lens)
    key = case["kv_heads"] * (d // 2 + d // 32)
    if case["op"] == "chunk":
        return {"bytes": 2 * key * sum(lens) + pages + rows * heads * (4 * d + 4),
                "flops": 4 * d * heads * pairs}
    return {"bytes": (key + 4) * sum(lens) + 4 * case["batch"] * max(1, max(lens)) + pages
            + rows * heads * (2 * d + 4), "flops": 2 * d * heads * pairs}


# --------------------------------------------------------------------------
# the cache's format, in elementary operations
# --------------------------------------------------------------------------

def e2m1_pairs(device):
    grid = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    grid = torch.tensor(grid + [-g for g in grid], device=device)
    byte = torch.arange(256, device=device)
    return torch.stack([grid[byte & 15], grid[byte >> 4]], -1)


def powers_of_two(device):
    """2^-127 .. 2^127 at 0 .. 254 (a table: pow on the device need not be exact)."""
    return torch.tensor([2.0 ** k for k in range(-127, 128)], dtype=torch.float64, device=device)


def decode(codes, sf):
    """[.., D] fp32 values of packed e2m1 codes under e8m0 scales (of at most 252)."""
    v = e2m1_pairs(codes.device)[codes.long()].flatten(-2)
    s = powers_of_two(codes.device).float()[sf.long()]
    return (v.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def encode(x):
    """Codes and scales of fp32 rows [.., D]: every 32 elements share the smallest power of two
    under which none of them exceeds 6."""
    x = x.unflatten(-1, (-1, 32))
    part, exponent = torch.frexp(x.abs().amax(-1))
    e = (exponent.long() - 3 + (part > 0.75).long()).clamp(-127, 125)
    a = (x.double() / powers_of_two(x.device)[e + 127][..., None]).float()
    code = torch.zeros_like(a, dtype=torch.uint8)
    for border in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
        code += a.abs() > border
    code = (code + 8 * torch.signbit(a).byte()).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], (e + 127).to(torch.uint8)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    i32 = dict(dtype=torch.int32, device=dev)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    lens, size, heads, d = lengths(case), case["block"], case["kv_heads"], case["d"]
    width = max(1, blocks(max(lens), size))
    need = torch.tensor([blocks(n, size) for n in lens], device=dev)
    used = int(need.sum())
    # an eviction repacks into free blocks
    free = blocks(case["keep"], size) * len(lens) + 5 if case["op"] == "evict" else 0
    num_blocks = used + max(1, used // 10) + free
    ids = torch.randperm(num_blocks, generator=g, device=dev).int()
    table = torch.full((len(lens), width), -1, **i32)
    table[torch.arange(width, device=dev)[None] < need[:, None]] = ids[:used]
    state = {"case": case, "context_lens": torch.tensor(lens, **i32), "table": table,
             "max_context_len": max(1, max(lens)), "scale": d ** -0.5}

    def pool(spread):
        codes = torch.empty(num_blocks, size, heads, d // 2, dtype=torch.uint8, device=dev)
        sf = torch.empty(num_blocks, size, heads, d // 32, dtype=torch.uint8, device=dev)
        step = max(1, (1 << 26) // (size * heads * d))
        for b in range(0, num_blocks, step):
            n = min(step, num_blocks - b)
            codes[b:b + n], sf[b:b + n] = encode(normal(n, size, heads, d) * spread)
        return codes, sf

    (state["k"], state["k_sf"]), (state["v"], state["v_sf"]) = [
        pool(torch.exp(0.5 * normal(heads, d))) for _ in range(2)]

    if case["op"] == "evict":
        # sums of many steps: a few tokens gather most, some exactly nothing
        w = torch.exp(2.5 * normal(len(lens), state["max_context_len"]))
        w[torch.rand(w.shape, generator=g, device=dev) < 0.05] = 0.0
        w[torch.arange(w.shape[1], device=dev)[None] >= state["context_lens"][:, None]] = 0.0
        state["weights"], state["free"] = w, ids[used:used + free].clone()
        state["pools"] = [state["k"], state["k_sf"], state["v"], state["v_sf"]]
        if case["index"]:
            state["pools"] += [torch.randint(0, 0x77, (num_blocks, size, d), generator=g,
                                             device=dev, dtype=torch.uint8),
                               torch.rand(num_blocks, size, generator=g, device=dev)]
        return state

    new = new_tokens(case)
    state["offsets"] = torch.tensor([0] + np.cumsum(new).tolist(), **i32)
    state["new"] = new
    # a step's buffers are sized for its padded batch
    rows, q_heads = sum(new) + 3, heads * case["group"]
    state["q"] = (2.0 * normal(rows, q_heads, d)).to(DTYPES[case["dtype"]])
    state["lse"] = torch.zeros(rows, q_heads, device=dev)
    if case["op"] == "chunk":
        state["out"] = torch.zeros_like(state["q"])
        return state
    # what attention gave for these queries, and the sums so far
    for b, h, r, scores in score_tiles(state):
        top = scores.amax(-1, keepdim=True)
        lse = top + torch.log(torch.exp(scores - top).sum(-1, keepdim=True))
        by_head(state, state["lse"], b, h)[r] = torch.where(torch.isneginf(top), top, lse)[:, :, 0]
    state["weights"] = torch.exp(2.0 * normal(len(lens), state["max_context_len"]))
    state["sums"] = torch.zeros_like(state["weights"])
    return state


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return run_own(op, state)
    return {"chunk": chunk_plain, "weights": weights_plain, "evict": evict_plain}[op](state)


def run_own(op, state):
    import mqa_logits_amd as mq
    if op == "chunk":
        out, lse = mq.paged_chunk_attention(
            "mxfp4", state["q"], state["k"], state["k_sf"], state["v"], state["v_sf"],
            state["context_lens"], state["offsets"], state["table"], state["max_context_len"],
            scale=state["scale"], out=state["out"], lse=state["lse"])
        return {"out": out, "lse": lse}
    if op == "weights":
        return {"sums": mq.paged_attention_weights(
            "mxfp4", state["q"], state["lse"], state["k"], state["k_sf"], state["context_lens"],
            state["offsets"], state["table"], state["max_context_len"], scale=state["scale"],
            weights=state["weights"], out=state["sums"])}
    case = state["case"]
    got = mq.paged_kv_evict(state["weights"], state["context_lens"], state["table"], state["free"],
                            state["pools"], case["keep"], case["recent"], state["max_context_len"])
    return {"lens": got.context_lens, "table": got.block_table, "weights": got.weights,
            "kept": got.kept, "freed": got.freed, "counts": got.counts, **pools_of(state)}


def pools_of(state):
    # (the indexer's fp8 keys come back as the values they stand for)
    return {"pool%d" % i: p.view(torch.float8_e4m3fn) if i == 4 else p
            for i, p in enumerate(state["pools"])}


def by_head(state, x, b, h):
    """Rows of sequence b and the query heads of KV head h: a view of x [rows, Hq, ..]."""
    first = sum(state["new"][:b])
    group = state["case"]["group"]
    return x[first:first + state["new"][b], h * group:(h + 1) * group]


def cached(state, b, side):
    """[length, kv_heads, d] keys or values of sequence b."""
    n, size = int(lengths(state["case"])[b]), state["case"]["block"]
    at = torch.arange(n, device=state["table"].device)
    slot = state["table"][b].long()[at // size] * size + at % size
    return decode(state[side].flatten(0, 1)[slot], state[side + "_sf"].flatten(0, 1)[slot])


def score_tiles(state, values=False):
    """Masked fp32 scores [rows, group, length] of a sequence, KV head and slice of its rows."""
    for b, m in enumerate(state["new"]):
        if m == 0:
            continue
        keys = cached(state, b, "k")
        n = keys.shape[0]
        v = cached(state, b, "v") if values else None
        position = torch.arange(n, device=keys.device)
        step = max(1, (1 << 28) // (n * state["case"]["group"]))
        for h in range(state["case"]["kv_heads"]):
            q, k = by_head(state, state["q"], b, h), keys[:, h].T.contiguous()
            for t in range(0, m, step):
                rows = q[t:t + step].float()
                scores = (rows.flatten(0, 1) @ k).unflatten(0, rows.shape[:2]) * state["scale"]
                seen = n - m + 1 + t + torch.arange(rows.shape[0], device=keys.device)
                scores.masked_fill_((position >= seen[:, None])[:, None], -math.inf)
                item = (b, h, slice(t, t + step), scores)
                yield item + (v[:, h].contiguous(),) if values else item


def chunk_plain(state):
    for b, h, r, scores, v in score_tiles(state, True):
        top = scores.amax(-1, keepdim=True)
        p = torch.exp(scores - top)
        total = p.sum(-1, keepdim=True)
        o = (p.flatten(0, 1) @ v).unflatten(0, p.shape[:2]) / total
        by_head(state, state["out"], b, h)[r] = o.to(state["out"].dtype)
        by_head(state, state["lse"], b, h)[r] = (top + torch.log(total))[:, :, 0]
    return {"out": state["out"], "lse": state["lse"]}


def weights_plain(state):
    sums = state["sums"]
    position = torch.arange(sums.shape[1], device=sums.device)
    inside = position < state["context_lens"][:, None]
    sums.copy_(torch.where(inside, state["weights"], 0.0))
    for b, h, r, scores in score_tiles(state):
        p = torch.exp(scores - by_head(state, state["lse"], b, h)[r][:, :, None])
        sums[b, :p.shape[2]] += p.sum((0, 1))
    return {"sums": sums}


def evict_plain(state):
    case, table, weights = state["case"], state["table"], state["weights"]
    size, keep, recent, width = case["block"], case["keep"], case["recent"], table.shape[1]
    dev, lens = table.device, state["context_lens"].long()
    batch = lens.numel()
    cut = lens > keep
    # the largest weights before the recent tokens; a stable sort puts ties in order
    position = torch.arange(weights.shape[1], device=dev)
    old = position < (lens - recent)[:, None]
    order = torch.sort(torch.where(old, weights, -math.inf), dim=1, descending=True,
                       stable=True).indices[:, :keep - recent]
    chosen = torch.zeros(weights.shape, dtype=torch.bool, device=dev)
    chosen.scatter_(1, order, True)
    chosen &= old
    chosen |= ~old & (position < lens[:, None])
    chosen = torch.where(cut[:, None], chosen, position < lens[:, None])
    new_lens = chosen.sum(1)
    kept = torch.full((batch, keep), -1, dtype=torch.long, device=dev)
    row, at = chosen.nonzero(as_tuple=True)
    start = torch.cumsum(new_lens, 0) - new_lens
    place = torch.arange(row.numel(), device=dev) - start[row]
    kept[row, place] = at
    new_weights = torch.zeros_like(weights)
    new_weights[row, place] = weights[row, at]
    # tables: blocks of cut sequences come from the free list, their old ones go back
    entry = torch.arange(width, device=dev)
    want = torch.where(cut, (new_lens + size - 1) // size, 0)
    first = torch.cumsum(want, 0) - want
    fresh = state["free"][(first[:, None] + entry).clamp_max(state["free"].numel() - 1)]
    held = entry < ((lens + size - 1) // size)[:, None]
    new_table = torch.where(cut[:, None], torch.where(entry < want[:, None], fresh, -1),
                            torch.where(held, table, -1))
    back = table[held & cut[:, None]]
    freed = torch.full((batch * width,), -1, dtype=torch.int32, device=dev)
    freed[:back.numel()] = back
    counts = torch.stack([want.sum(), torch.tensor(back.numel(), device=dev)])
    moved = cut[row]
    row, at, place = row[moved], at[moved], place[moved]
    source = table[row, at // size].long() * size + at % size
    target = new_table[row, place // size].long() * size + place % size
    for p in state["pools"]:
        flat = p.flatten(0, 1)
        flat[target] = flat[source]
    return {"lens": new_lens.int(), "table": new_table, "weights": new_weights,
            "kept": kept.int(), "freed": freed, "counts": counts.int(), **pools_of(state)}


# --------------------------------------------------------------------------
# 64 bits, from the definitions
# --------------------------------------------------------------------------

def exact(case, seed):
    state = prepare(case, seed)
    return evict_exact(state) if case["op"] == "evict" else attend_exact(state)


def values_of(codes, sf):
    """fp64 values from the fields of the codes."""
    nibble = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    exponent, fraction = (nibble >> 1) & 3, (nibble & 1).double()
    v = torch.where(exponent == 0, 0.5 * fraction,
                    (1 + 0.5 * fraction) * (2 ** (exponent - 1).clamp_min(0)).double())
    v = torch.where(nibble >= 8, -v, v)
    return v * powers_of_two(sf.device)[sf.long()].repeat_interleave(32, -1)


def attend_exact(state):
    """Sequence by sequence, gathering its tokens; rows in slices."""
    case = state["case"]
    group, size = case["group"], case["block"]
    q = state["q"]
    if case["op"] == "chunk":
        out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
        lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    else:
        sums = torch.zeros(state["weights"].shape, dtype=torch.float64, device=q.device)
    offsets = state["offsets"].tolist()
    for b, n in enumerate(state["context_lens"].tolist()):
        first, m = offsets[b], offsets[b + 1] - offsets[b]
        if case["op"] == "weights":
            sums[b, :n] = state["weights"][b, :n].double()
        if m == 0:
            continue
        token = torch.arange(n, device=q.device)
        slot = state["table"][b, token // size].long() * size + token % size
        k = values_of(state["k"].flatten(0, 1)[slot], state["k_sf"].flatten(0, 1)[slot])
        v = values_of(state["v"].flatten(0, 1)[slot], state["v_sf"].flatten(0, 1)[slot])
        step = max(1, (1 << 27) // (n * group))
        for t in range(0, m, step):
            r = slice(first + t, first + min(m, t + step))
            seen = n - m + torch.arange(t, min(m, t + step), device=q.device) + 1
            hidden = (token[None] >= seen[:, None])[:, None]
            for h in range(case["kv_heads"]):
                g = slice(h * group, (h + 1) * group)
                rows = q[r, g].double()
                s = (rows.reshape(-1, case["d"]) @ k[:, h].T.contiguous()) * state["scale"]
                s = s.view(rows.shape[0], group, n).masked_fill(hidden, -math.inf)
                if case["op"] == "weights":
                    sums[b, :n] += torch.exp(s - state["lse"][r, g].double()[..., None]).sum((0, 1))
                    continue
                lse[r, g] = torch.logsumexp(s, -1)
                p = torch.exp(s - lse[r, g][..., None])
                out[r, g] = (p.view(-1, n) @ v[:, h].contiguous()).view(rows.shape)
    return {"out": out, "lse": lse} if case["op"] == "chunk" else {"sums": sums}


def evict_exact(state):
    """Sequence by sequence, on the host."""
    case = state["case"]
    size, keep, recent = case["block"], case["keep"], case["recent"]
    table, weights = state["table"].cpu().numpy(), state["weights"].cpu().numpy()
    free = state["free"].tolist()
    new_table, new_weights = np.full_like(table, -1), np.zeros_like(weights)
    kept = np.full((len(table), keep), -1, np.int32)
    lens, freed, taken, moves = [], [], 0, []
    for b, n in enumerate(state["context_lens"].tolist()):
        old, at = table[b, :-(-n // size)], np.arange(n)
        if n > keep:
            best = np.lexsort((at[:n - recent], -weights[b, :n - recent]))[:keep - recent]
            at = np.concatenate([np.sort(best), at[n - recent:]])
            m = -(-len(at) // size)
            mine = np.array(free[taken:taken + m], np.int32)
            taken, freed = taken + m, freed + old.tolist()
            place = np.arange(len(at))
            moves.append((old[at // size].astype(np.int64) * size + at % size,
                          mine[place // size].astype(np.int64) * size + place % size))
            old = mine
        new_table[b, :len(old)] = old
        kept[b, :len(at)] = at
        new_weights[b, :len(at)] = weights[b, at]
        lens.append(len(at))
    dev = state["table"].device
    out = {}
    for i, p in enumerate(state["pools"]):
        flat = p.flatten(0, 1)
        for source, target in moves:
            flat[torch.from_numpy(target).to(dev)] = flat[torch.from_numpy(source).to(dev)]
        out["pool%d" % i] = p.view(torch.float8_e4m3fn).double() if i == 4 else p
    freed = np.array(freed + [-1] * (table.size - len(freed)), np.int32)
    return {"lens": torch.tensor(lens, dtype=torch.int32, device=dev),
            "table": torch.from_numpy(new_table).to(dev),
            "weights": torch.from_numpy(new_weights).to(dev).double(),
            "kept": torch.from_numpy(kept).to(dev), "freed": torch.from_numpy(freed).to(dev),
            "counts": torch.tensor([taken, len(freed[freed >= 0])], dtype=torch.int32, device=dev),
            **out}
