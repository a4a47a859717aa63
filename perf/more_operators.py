"""The operators of a paged KV cache whose contexts are kept short by evicting tokens that attract little attention.

Beside a sequence's block table the cache keeps, for every cached token and kv head, the attention weight that the
token has drawn so far (float32 [num_seqs][num_kv_heads][width]) and the token's place in the sequence (int32 of the
same shape), since after an eviction that is no longer its place in the cache.  Keys are stored rotated, each by its own
position on several axes (time, height, width; one axis for text).

rope     rotary positions with several axes on q and k: pair i of a head turns by pos[axis[i]] * inv_freq[i].
write    the same on a step's new tokens, q returned, k and v stored at their slots of the pools, the tokens' weights
         set to 0 and their places noted.
decode   softmax(scale q K^T) V for one query token per sequence, and each key's softmax weight, summed over the query
         heads of its kv head, added to its accumulated weight.
prefill  the same for chunks of query tokens, each of which sees the keys up to its own position.
evict    of every (sequence, kv head) with more than `budget` tokens the `budget` best stay: the sequence's first and
         most recent tokens before all others, the others by accumulated weight (ties: the lowest index).  Kept tokens
         beyond the budget move, in order, into the places that are free below it.

With ``own`` false, `run` computes these with elementary torch operations in 32 bits; with it true, it makes the
framework's calls.
"""
import math
import random

import torch

own = False


def listed():
    return [
        # one decode step's queries and keys, turned before a write of the caller's own
        {"name": "rope_step", "op": "rope", "decode": 64, "chunks": 0, "chunk": 0, "lo": 128, "hi": 4096, "hq": 32,
         "hkv": 8, "dim": 128, "rot": 128, "axes": 1, "theta": 10000.0, "inter": False, "type": "bf16", "lens": 1},
        # four prompts of text and images, pairs interleaved, half of a head turned
        {"name": "rope_prompts", "op": "rope", "decode": 0, "chunks": 4, "chunk": 2047, "lo": 0, "hi": 4096, "hq": 32,
         "hkv": 8, "dim": 128, "rot": 64, "axes": 3, "theta": 10000.0, "inter": True, "type": "bf16", "lens": 2},
        # the new tokens of one decode step
        {"name": "write_step", "op": "write", "decode": 64, "chunks": 0, "chunk": 0, "lo": 128, "hi": 4096, "hq": 32,
         "hkv": 8, "dim": 128, "rot": 128, "axes": 3, "theta": 1000000.0, "inter": False, "block": 16, "type": "bf16",
         "lens": 3},
        # a continuous-batching step's decode tokens and four prompts' chunks
        {"name": "write_prompts", "op": "write", "decode": 256, "chunks": 4, "chunk": 2048, "lo": 16, "hi": 4096,
         "hq": 32, "hkv": 8, "dim": 128, "rot": 128, "axes": 3, "theta": 1000000.0, "inter": False, "block": 32,
         "type": "bf16", "lens": 4},
        # the smallest decode call: four sequences of a few tokens, 32-bit pools
        {"name": "decode_tiny", "op": "decode", "seqs": 4, "lo": 1, "hi": 40, "hq": 32, "hkv": 8, "dim": 128,
         "block": 16, "type": "f32", "lens": 5},
        # a serving batch's decode step
        {"name": "decode_batch", "op": "decode", "seqs": 64, "lo": 128, "hi": 4096, "hq": 32, "hkv": 8, "dim": 128,
         "block": 16, "type": "bf16", "lens": 6},
        # few long contexts, many query heads
        {"name": "decode_long", "op": "decode", "seqs": 16, "lo": 1024, "hi": 32768, "hq": 64, "hkv": 8, "dim": 128,
         "block": 16, "type": "bf16", "lens": 7},
        # the last, ragged piece of one prompt
        {"name": "prefill_tail", "op": "prefill", "chunks": 1, "chunk": 37, "lo": 2900, "hi": 3050, "hq": 32, "hkv": 8,
         "dim": 128, "block": 16, "type": "bf16", "lens": 8},
        # the prompt chunks of a continuous-batching step
        {"name": "prefill_mixed", "op": "prefill", "chunks": 4, "chunk": 512, "lo": 1, "hi": 4096, "hq": 32, "hkv": 8,
         "dim": 128, "block": 32, "type": "bf16", "lens": 9},
        # one large chunk deep in a long prompt
        {"name": "prefill_long", "op": "prefill", "chunks": 1, "chunk": 2048, "lo": 5900, "hi": 6100, "hq": 64,
         "hkv": 8, "dim": 128, "block": 64, "type": "bf16", "lens": 10},
        # a serving batch back to its budget after 16 decode steps
        {"name": "evict_step", "op": "evict", "seqs": 64, "lo": 2064, "hi": 2064, "budget": 2048, "first": 4,
         "recent": 128, "hkv": 8, "dim": 128, "block": 16, "type": "bf16", "lens": 11},
        # long prompts cut down before their first decode step
        {"name": "evict_prompts", "op": "evict", "seqs": 16, "lo": 1024, "hi": 32768, "budget": 4096, "first": 4,
         "recent": 512, "hkv": 8, "dim": 128, "block": 16, "type": "bf16", "lens": 12},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "write", "decode", "prefill", "evict"])
    case = {"op": op, "hkv": rng.choice([1, 2, 4, 8]), "dim": rng.choice([64, 128, 128, 128]),
            "block": rng.choice([16, 32, 64]), "type": rng.choice(["bf16", "bf16", "bf16", "f32"]),
            "lens": rng.randrange(1 << 30)}
    if op != "evict":
        case["hq"] = case["hkv"] * rng.choice([1, 2, 3, 4, 8])
    if op in ("rope", "write"):
        case |= {"decode": _log_int(rng, 1, 256), "chunks": rng.randrange(4), "chunk": _log_int(rng, 1, 1500),
                 "lo": 1, "hi": _log_int(rng, 16, 4096), "rot": rng.choice([case["dim"], case["dim"], case["dim"] // 2]),
                 "axes": rng.choice([1, 2, 3]), "theta": rng.choice([1e4, 5e5, 1e6]), "inter": rng.random() < 0.3}
        case["hq"] = min(case["hq"], 4 * case["hkv"])
    elif op == "decode":
        seqs = _log_int(rng, 1, 96)
        case |= {"seqs": seqs, "lo": 1, "hi": _log_int(rng, 2, min(32768, 160000 // seqs))}
    elif op == "prefill":
        case |= {"chunks": rng.randrange(1, 5), "chunk": _log_int(rng, 1, 512), "lo": 1, "hi": _log_int(rng, 8, 4096)}
    else:
        seqs = _log_int(rng, 1, 64)
        hi = _log_int(rng, 64, min(32768, 150000 // seqs))
        budget = _log_int(rng, 16, hi)
        case |= {"seqs": seqs, "lo": max(1, hi // 8), "hi": hi, "budget": budget, "first": rng.randrange(5),
                 "recent": rng.randrange(budget // 4 + 1)}
    return case


# ---------------------------------------------------------------- a case's lengths, from the case alone
def _lengths(case, n, salt):
    """n whole numbers spread over [lo, hi], over their logarithm."""
    rng = random.Random(case["lens"] * 8 + salt)
    return [min(case["hi"], max(case["lo"], _log_int(rng, max(case["lo"], 1), max(case["hi"], 1)))) for _ in range(n)]


def _layout(case):
    """(context length of every sequence, first new position of every sequence or None)."""
    if case["op"] in ("decode", "evict"):
        return _lengths(case, case["seqs"], 0), None
    chunks = _lengths(case, case["chunks"], 1)
    if case["op"] == "prefill":
        return [o + case["chunk"] for o in chunks], chunks
    steps = _lengths(case, case["decode"], 0)
    return [o + 1 for o in steps] + [o + case["chunk"] for o in chunks], steps + chunks


def _pairs(first, lens):
    seq = [s for s in range(len(lens)) for _ in range(lens[s] - first[s])]
    pos = [p for s in range(len(lens)) for p in range(first[s], lens[s])]
    return seq, pos


# ---------------------------------------------------------------- inputs
def _type(case):
    return torch.float32 if case["type"] == "f32" else torch.bfloat16


def _rows(gen, n, heads, case):
    """Rows as a model's projections make them: heads, and some columns, of different size."""
    dev, d = torch.device("cuda"), case["dim"]
    gain = torch.exp(0.3 * torch.randn(heads, 1, generator=gen, device=dev))
    col = 1 + 3 * (torch.rand(heads, d, generator=gen, device=dev) < 0.03)
    return (torch.randn(n, heads, d, generator=gen, device=dev) * gain * col).to(_type(case))


def _tables(gen, lens, block):
    dev = torch.device("cuda")
    count = [-(-n // block) for n in lens]
    blocks = sum(count) + max(4, sum(count) // 10)
    order = torch.randperm(blocks, generator=gen, device=dev).to(torch.int32)
    col = torch.arange(max(count), device=dev)
    start = torch.tensor([sum(count[:s]) for s in range(len(count))], device=dev)
    have = col[None] < torch.tensor(count, device=dev)[:, None]
    return torch.where(have, order[(start[:, None] + col[None]).clamp_max(blocks - 1)], -1).to(torch.int32), blocks


def _rope_inputs(st, case, gen, lens, first):
    """q, k and v as views of one projection, positions of text with images in it, and the pairs' frequencies."""
    dev, hq, hkv, d = torch.device("cuda"), case["hq"], case["hkv"], case["dim"]
    seq, pos = _pairs(first, lens)
    t = len(seq)
    st["seq"] = torch.tensor(seq, dtype=torch.int32, device=dev)
    st["pos"] = torch.tensor(pos, dtype=torch.int32, device=dev)
    st["qkv"] = _rows(gen, t, hq + 2 * hkv, case)
    st["q"], st["k_new"], st["v_new"] = st["qkv"][:, :hq], st["qkv"][:, hq:hq + hkv], st["qkv"][:, hq + hkv:]
    half = case["rot"] // 2
    st["inv_freq"] = (case["theta"] ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)).float()
    # the time axis takes the highest frequencies, as far as they go, height and width three eighths each
    side = half * 3 // 8 if case["axes"] == 3 else half // 2
    axis = torch.zeros(half, dtype=torch.int32, device=dev)
    for a in range(1, case["axes"]):
        axis[half - (case["axes"] - a) * side: half - (case["axes"] - a - 1) * side] = a
    st["axis"] = axis
    # a stretch of 256 tokens in every 1024 is an image 16 wide: one time, a row and a column for each
    p = st["pos"].long()
    far = torch.randint(0, 100000, (len(lens),), generator=gen, device=dev)[st["seq"].long()]
    image, i = (p % 1024) >= 768, p % 1024 - 768
    grid = [torch.where(image, p - i, p), torch.where(image, p - i + i // 16, p), torch.where(image, p - i + i % 16, p)]
    st["rope_pos"] = torch.stack([g + far for g in grid[:case["axes"]]]).to(torch.int32).contiguous()
    st["token_pos"] = (p + far).to(torch.int32)
    st["inter"] = case["inter"]


def prepare(case, seed):
    dev, hkv, d = torch.device("cuda"), case["hkv"], case["dim"]
    gen = torch.Generator(dev).manual_seed(seed)
    lens, first = _layout(case)
    st = {"op": case["op"], "scale": d ** -0.5}
    if case["op"] == "rope":
        _rope_inputs(st, case, gen, lens, first)
        return st
    block = st["block"] = case["block"]
    st["table"], blocks = _tables(gen, lens, block)
    st["max_len"] = max(lens)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    st["k"] = _rows(gen, blocks * block, hkv, case).view(blocks, block, hkv, d)
    st["v"] = _rows(gen, blocks * block, hkv, case).view(blocks, block, hkv, d)
    width = max(lens) + 24  # room for the next steps' tokens
    weights = torch.exp(2 * torch.randn(len(lens), hkv, width, generator=gen, device=dev) - 2)
    # some tokens have drawn nothing yet, and are equal
    weights *= torch.rand(len(lens), hkv, width, generator=gen, device=dev) > 0.05
    if case["op"] == "evict":
        budget = case["budget"]
        place = torch.arange(width, dtype=torch.int32, device=dev)[None, None].repeat(len(lens), hkv, 1)
        if max(lens) <= budget + 64:
            # after earlier evictions: the older tokens in any order, with gaps where others have gone
            order = torch.rand(len(lens), hkv, min(lens), generator=gen, device=dev).argsort(dim=-1)
            place[:, :, :min(lens)] = torch.where(order < min(lens) - case["recent"], 2 * order, order + min(lens)).int()
            place[:, :, min(lens):] += min(lens)
        st["next"] = place.gather(2, (st["lens"].long() - 1)[:, None, None].expand(-1, hkv, 1)).amax(dim=(1, 2)) + 1
        if max(lens) <= budget + 64:
            st["next"] = torch.maximum(st["next"], torch.full_like(st["next"], 2 * min(lens)))
        st["next"] = st["next"].to(torch.int32).contiguous()
        # a pass begins with the weights and places that the step's attention has left
        st["begin"] = torch.stack([weights, place.view(torch.float32)])
        st["pair"] = st["begin"].clone()
        st["weights"], st["place"] = st["pair"][0], st["pair"][1].view(torch.int32)
        st["budget"], st["first"], st["recent"] = budget, case["first"], case["recent"]
    else:
        st["weights"] = weights
    if case["op"] == "write":
        _rope_inputs(st, case, gen, lens, first)
        st["place"] = torch.full((len(lens), hkv, width), -1, dtype=torch.int32, device=dev)
    elif case["op"] == "decode":
        st["q"] = _rows(gen, len(lens), case["hq"], case)
    elif case["op"] == "prefill":
        chunk, n = case["chunk"], case["chunks"]
        st["q"] = _rows(gen, n * chunk, case["hq"], case)
        st["cu"] = torch.arange(n + 1, dtype=torch.int32, device=dev) * chunk
        st["start"] = torch.tensor(first, dtype=torch.int32, device=dev)
        st["seq_of"] = torch.arange(n, dtype=torch.int32, device=dev)
        st["max_q"] = chunk
    if own:
        from paged_kv_cache_313_gb300 import pa
        if case["op"] == "decode":
            st["ws"] = pa.new_decode_weights_workspace(len(lens), case["hq"], hkv, d, block, max(lens))
        elif case["op"] == "prefill":
            st["ws"] = pa.new_prefill_weights_workspace(case["chunks"], st["q"].shape[0], case["chunk"], case["hq"], hkv,
                                                        d, block, max(lens))
        elif case["op"] == "evict":
            st["ws"] = pa.new_evict_workspace(len(lens), hkv, max(lens), case["budget"])
    return st


# ---------------------------------------------------------------- the plain forms
def _turn(x, rope_pos, inv_freq, axis, inter):
    """Rotary positions, in 32 bits; the angles, which pass 10^5 turns, in 64."""
    angle = rope_pos.double()[axis.long()].T * inv_freq.double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    half = inv_freq.numel()
    y = x.float()
    a, b = (y[..., 0:2 * half:2], y[..., 1:2 * half:2]) if inter else (y[..., :half], y[..., half:2 * half])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], dim=-1).flatten(-2) if inter else torch.cat([ra, rb], dim=-1)
    return torch.cat([turned, y[..., 2 * half:]], dim=-1).to(x.dtype)


def _plain_rope(st):
    return tuple(_turn(st[n], st["rope_pos"], st["inv_freq"], st["axis"], st["inter"]) for n in ("q", "k_new"))


def _plain_write(st):
    q, k = _plain_rope(st)
    seq, pos = st["seq"].long(), st["pos"].long()
    phys, off = st["table"][seq, pos // st["block"]].long(), pos % st["block"]
    st["k"][phys, off] = k
    st["v"][phys, off] = st["v_new"]
    st["weights"][seq, :, pos] = 0.0
    st["place"][seq, :, pos] = st["token_pos"][:, None].expand(-1, st["k"].shape[2])
    return {"q": q, "k": st["k"], "v": st["v"], "weights": st["weights"], "place": st["place"]}


def _contexts(st, pool, table):
    n, width = table.shape
    x = pool[table.clamp_min(0).long().view(-1)].float()
    return x.view(n, width * st["block"], x.shape[2], x.shape[3])


def _attend(q, k, v, see, scale):
    """q [n, m, hkv, g, d], k and v [n, l, hkv, d], see [n, m, l]: softmax over the keys that are seen, and its sums over
    the queries and heads of a kv head."""
    s = torch.einsum("nmhgd,nlhd->nhgml", q, k) * scale
    s = s.masked_fill_(~see[:, None, None], -math.inf)
    p = torch.exp(s - s.amax(dim=-1, keepdim=True))
    p = p / p.sum(dim=-1, keepdim=True)
    return torch.einsum("nhgml,nlhd->nmhgd", p, v), p.sum(dim=(2, 3))


def _plain_decode(st):
    hkv = st["k"].shape[2]
    k, v = _contexts(st, st["k"], st["table"]), _contexts(st, st["v"], st["table"])
    n, hq, d = st["q"].shape
    see = torch.arange(k.shape[1], device=k.device)[None, None] < st["lens"][:, None, None]
    o, w = _attend(st["q"].float().view(n, 1, hkv, hq // hkv, d), k, v, see, st["scale"])
    l = st["max_len"]
    st["weights"][:, :, :l] += w[:, :, :l]
    return {"out": o.reshape(n, hq, d).to(st["q"].dtype), "weights": st["weights"]}


def _plain_prefill(st):
    hkv, m = st["k"].shape[2], st["max_q"]
    table = st["table"][st["seq_of"].long()]
    k, v = _contexts(st, st["k"], table), _contexts(st, st["v"], table)
    rows, hq, d = st["q"].shape
    n = rows // m
    last = st["start"][:, None] + torch.arange(m, device=k.device)[None]
    see = torch.arange(k.shape[1], device=k.device)[None, None] <= last[:, :, None]
    o, w = _attend(st["q"].float().view(n, m, hkv, hq // hkv, d), k, v, see, st["scale"])
    l = st["max_len"]
    st["weights"].index_add_(0, st["seq_of"], torch.nn.functional.pad(w[:, :, :l], (0, st["weights"].shape[2] - l)))
    return {"out": o.reshape(rows, hq, d).to(st["q"].dtype), "weights": st["weights"]}


def _plain_evict(st):
    budget, block, hkv = st["budget"], st["block"], st["k"].shape[2]
    st["pair"].copy_(st["begin"])
    w, place, n = st["weights"], st["place"], st["lens"].long()[:, None, None]
    l = st["max_len"]
    j = torch.arange(l, device=w.device)[None, None]
    safe = (place[:, :, :l] < st["first"]) | (place[:, :, :l] >= st["next"][:, None, None] - st["recent"])
    safe &= j < n
    score = torch.where(safe, 0.0, torch.nan_to_num(w[:, :, :l], nan=-math.inf, posinf=math.inf, neginf=-math.inf))
    score = torch.where(j < n, score, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices
    order = order.gather(2, torch.sort(safe.gather(2, order).int(), dim=-1, descending=True, stable=True).indices)
    rank = torch.empty_like(order).scatter_(2, order, torch.arange(l, device=w.device).expand_as(order))
    kept = (rank < budget) & (j < n)
    source, free = kept & (j >= budget), ~kept & (j < budget) & (j < n)
    m = max(0, min(budget, l - budget))
    if m:
        src = torch.sort(torch.where(source, j, l), dim=-1).values[:, :, :m]
        dst = torch.sort(torch.where(free, j, l), dim=-1).values[:, :, :m]
        # where there is nothing to move, a token that is no destination stays in its place
        stay = torch.where(n > budget, budget, 0)
        move = src < l
        src, dst = torch.where(move, src, stay), torch.where(move, dst, stay)
        seq = torch.arange(src.shape[0], device=w.device)[:, None, None]
        head = torch.arange(hkv, device=w.device)[None, :, None]
        at = [st["table"][seq, t // block].long() * block + t % block for t in (src, dst)]
        for pool in (st["k"], st["v"]):
            rows = pool.view(-1, hkv, pool.shape[3])
            rows[at[1], head] = rows[at[0], head]
        for state in (w, place):
            state.scatter_(2, dst, state.gather(2, src))
    new = st["lens"].clamp_max(budget)
    return {"k": st["k"], "v": st["v"], "weights": w, "place": place, "lens": new}


def run(state):
    st = state
    if own:
        return _own(st)
    return {"rope": _plain_rope, "write": _plain_write, "decode": _plain_decode, "prefill": _plain_prefill,
            "evict": _plain_evict}[st["op"]](st)


def _own(st):
    from paged_kv_cache_313_gb300 import pa
    if st["op"] == "rope":
        return pa.pa_rope(st["q"], st["k_new"], st["rope_pos"], st["inv_freq"], st["axis"], interleaved=st["inter"])
    if st["op"] == "write":
        q = pa.pa_rope_write_kv_paged(st["q"], st["k_new"], st["v_new"], st["rope_pos"], st["inv_freq"], st["axis"],
                                      st["k"], st["v"], st["table"], st["seq"], st["pos"], interleaved=st["inter"],
                                      key_weights=st["weights"], key_pos=st["place"], token_pos=st["token_pos"])
        return {"q": q, "k": st["k"], "v": st["v"], "weights": st["weights"], "place": st["place"]}
    if st["op"] == "decode":
        out = pa.pa_decode_weights(st["q"], st["k"], st["v"], st["table"], st["lens"], st["max_len"], st["scale"],
                                   st["weights"], st["ws"])
        return {"out": out, "weights": st["weights"]}
    if st["op"] == "prefill":
        out = pa.pa_prefill_chunk_weights(st["q"], st["cu"], st["start"], st["seq_of"], st["max_q"], st["k"], st["v"],
                                          st["table"], st["lens"], st["max_len"], st["scale"], st["weights"], st["ws"])
        return {"out": out, "weights": st["weights"]}
    st["pair"].copy_(st["begin"])
    new = pa.pa_evict_tokens(st["k"], st["v"], st["table"], st["lens"], st["max_len"], st["weights"], st["place"],
                             st["next"], st["budget"], st["first"], st["recent"], st["ws"])
    return {"k": st["k"], "v": st["v"], "weights": st["weights"], "place": st["place"], "lens": new}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    lens, first = _layout(case)
    hkv, d = case["hkv"], case["dim"]
    size = 4 if case["type"] == "f32" else 2
    if case["op"] in ("rope", "write"):
        new = sum(n - f for n, f in zip(lens, first))
        turned = new * (case["hq"] + hkv) * case["rot"]
        heads = case["hq"] + hkv + (hkv if case["op"] == "write" else 0)
        state = 4 * new * (4 + 2 * hkv) if case["op"] == "write" else 0  # indices, and a weight and a place for each head
        return {"bytes": 2 * size * new * heads * d + 4 * case["axes"] * new + state, "flops": 3 * turned}
    if case["op"] == "evict":
        rows = moves = 0
        for n in lens:
            tail = n - case["budget"]
            if tail > 0:
                kept = min(case["recent"], tail)
                free = case["first"] + case["recent"]
                rows += n
                moves += kept + (tail - kept) * (case["budget"] - free) / (n - free)
        return {"bytes": int(hkv * (8 * rows + 2 * moves * (2 * d * size + 8))) + 8 * len(lens), "flops": hkv * rows}
    cache = 2 * size * sum(lens) * hkv * d
    pages = 4 * sum(-(-n // case["block"]) for n in lens)
    weights = 8 * sum(lens) * hkv
    if case["op"] == "decode":
        return {"bytes": cache + pages + weights + 2 * size * len(lens) * case["hq"] * d,
                "flops": 4 * sum(lens) * case["hq"] * d}
    seen = sum((f + 1 + n) * (n - f) // 2 for n, f in zip(lens, first))
    queries = sum(n - f for n, f in zip(lens, first))
    return {"bytes": cache + pages + weights + 2 * size * queries * case["hq"] * d,
            "flops": 4 * seen * case["hq"] * d}


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_turn(x, st):
    """Each pair as a complex number, times e^(i angle)."""
    x, half = x.double(), st["inv_freq"].numel()
    pos = torch.stack([st["rope_pos"][int(a)].double() for a in st["axis"].tolist()], dim=1)
    by = torch.polar(torch.ones_like(pos), pos * st["inv_freq"].double()[None])[:, None]
    out = x.clone()
    if st["inter"]:
        pairs = torch.view_as_complex(x[..., :2 * half].unflatten(-1, (half, 2)).contiguous()) * by
        out[..., :2 * half] = torch.view_as_real(pairs).flatten(-2)
    else:
        pairs = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * by
        out[..., :half], out[..., half:2 * half] = pairs.real, pairs.imag
    return out


def _exact_write(st, case):
    lens, first = _layout(case)
    table = st["table"].cpu().tolist()
    k = _exact_turn(st["k_new"], st)
    pk, pv, w = st["k"].double(), st["v"].double(), st["weights"].double()
    t = 0
    for s in range(len(lens)):
        p = first[s]
        w[s, :, first[s]:lens[s]] = 0
        while p < lens[s]:
            n = min(case["block"] - p % case["block"], lens[s] - p)
            b, o = table[s][p // case["block"]], p % case["block"]
            pk[b, o:o + n], pv[b, o:o + n] = k[t:t + n], st["v_new"][t:t + n].double()
            t, p = t + n, p + n
    return {"q": _exact_turn(st["q"], st), "k": pk, "v": pv, "weights": w, "place": None}


def _exact_evict(st, case):
    lens, _ = _layout(case)
    budget, block, hkv = case["budget"], case["block"], case["hkv"]
    pk, pv, w = st["k"].clone(), st["v"].clone(), st["weights"].double()
    weights, place, table = st["weights"].cpu(), st["place"].cpu(), st["table"].cpu()
    for s, n in enumerate(lens):
        if n <= budget:
            continue
        for h in range(hkv):
            old = place[s, h, :n].tolist()
            late = int(st["next"][s]) - case["recent"] if h == 0 else late
            got = weights[s, h, :n].tolist()
            best = sorted(range(n), key=lambda i: (0, 0.0, i) if old[i] < case["first"] or old[i] >= late
                          else (1, -got[i], i))[:budget]
            keep = set(best)
            src = torch.tensor([i for i in range(budget, n) if i in keep], dtype=torch.long)
            dst = torch.tensor([i for i in range(budget) if i not in keep], dtype=torch.long)
            a, b = (table[s, t // block].long().cuda() * block + (t % block).cuda() for t in (src, dst))
            for pool in (pk, pv):
                rows = pool.view(-1, hkv, case["dim"])
                rows[b, h] = rows[a, h]
            w[s, h, dst.cuda()] = w[s, h, src.cuda()]
    return {"k": pk.double(), "v": pv.double(), "weights": w, "place": None, "lens": None}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_turn(st["q"], st), _exact_turn(st["k_new"], st)
    if case["op"] == "write":
        return _exact_write(st, case)
    if case["op"] == "evict":
        return _exact_evict(st, case)
    lens, first = _layout(case)
    hkv, d, g = case["hkv"], case["dim"], case["hq"] // case["hkv"]
    weights, outs = st["weights"].double(), []
    for s, n in enumerate(lens):
        blocks = st["table"][s, : -(-n // st["block"])].long()
        k, v = (st[x][blocks].double().flatten(0, 1)[:n].transpose(0, 1) for x in ("k", "v"))  # [hkv, n, d]
        q = st["q"][s: s + 1] if case["op"] == "decode" else st["q"][s * case["chunk"]: (s + 1) * case["chunk"]]
        start = n - 1 if case["op"] == "decode" else first[s]
        for i in range(0, q.shape[0], 256):
            part = q[i:i + 256].double().view(-1, hkv, g, d).permute(1, 2, 0, 3)  # [hkv, g, m, d]
            sc = part @ k[:, None].transpose(2, 3) * st["scale"]
            last = start + i + torch.arange(part.shape[2], device="cuda")
            sc = sc.masked_fill(torch.arange(n, device="cuda")[None] > last[:, None], -math.inf)
            p = torch.softmax(sc, dim=-1)
            outs.append((p @ v[:, None]).permute(2, 0, 1, 3).flatten(1, 2))
            weights[s, :, :n] += p.sum(dim=(1, 2))
    return {"out": torch.cat(outs), "weights": weights}
