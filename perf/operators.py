"""The prompt side of the paged cache: cases, plain forms and exact values.

Four operators, used one after another when a batch of requests is served:

* ``append``   block tables and slot maps grown on the GPU from request lengths
               and a device free list (``pa.pa_append_slots_device``);
* ``trim``     the reverse: blocks behind each request's new length go back on
               the free list (``pa.pa_trim_slots_device``);
* ``prefill``  causal attention of each sequence's newest tokens over its paged
               cache (``pa.pa_prefill``);
* ``cross``    attention of a decoder's tokens to an encoder's states of another
               length, held in a paged cache (``pa.pa_cross_attention``).

``run`` computes a case in elementary torch operations, in 32 bits, or (``own``)
by the library's calls; ``exact`` computes it again in 64 bits (attention) or in
Python integers (block bookkeeping).

A case's lengths come from its own ``mix`` number; the seed makes the values,
the block order and the free list.
"""
import math
import random

import torch

own = False

# One scratch buffer, as a serving program keeps for all its layers.
WORKSPACE_BYTES = 96 << 20


def attention(op, kv, heads, kv_heads, dim, block, seqs, new, ctx, mix):
    return {"op": op, "kv": kv, "heads": heads, "kv_heads": kv_heads, "dim": dim, "block": block, "seqs": seqs,
            "new_lo": new[0], "new_hi": new[1], "ctx_lo": ctx[0], "ctx_hi": ctx[1], "mix": mix}


def slots(op, block, seqs, new, ctx, mix):
    return {"op": op, "block": block, "seqs": seqs, "new_lo": new[0], "new_hi": new[1], "ctx_lo": ctx[0], "ctx_hi": ctx[1],
            "mix": mix}


def listed():
    return [
        # a decode step: every request of a batch grows by one token
        {"name": "append_step", **slots("append", 16, 256, (1, 1), (16, 4096), 1)},
        # a batch of new prompts is admitted: no blocks yet, long slot maps
        {"name": "append_prompts", **slots("append", 16, 48, (64, 4096), (0, 0), 2)},
        # a quarter of the batch has finished: all its blocks go back
        {"name": "trim_finished", **slots("trim", 16, 256, (0, 0), (16, 4096), 3)},
        # after a speculative step: each request gives back its rejected tokens (1 to 8)
        {"name": "trim_rejected", **slots("trim", 8, 1500, (1, 8), (16, 1024), 4)},
        # the smallest prompts: four requests of a small model, latency alone
        {"name": "prefill_tiny", **attention("prefill", "bf16", 4, 2, 64, 16, 4, (7, 50), (0, 0), 5)},
        # ragged prompts of one admission, 8B-shaped layer
        {"name": "prefill_ragged", **attention("prefill", "bf16", 32, 8, 128, 16, 8, (64, 2048), (0, 0), 6)},
        # one long prompt, 8B-shaped layer: tensor-core bound
        {"name": "prefill_long", **attention("prefill", "bf16", 32, 8, 128, 16, 1, (8192, 8192), (0, 0), 7)},
        # a prompt's next chunk over a long FP8 cache, 70B-shaped layer
        {"name": "prefill_chunk_fp8", **attention("prefill", "fp8", 64, 8, 128, 16, 2, (1021, 1021), (8000, 9000), 8)},
        # checking drafted tokens: a few queries a request over long contexts, bound by the cache's bytes
        {"name": "prefill_verify", **attention("prefill", "bf16", 32, 8, 128, 16, 48, (4, 8), (512, 4096), 9)},
        # decoder prompts against encoder states, 1B-shaped heads
        {"name": "cross_prompt", **attention("cross", "bf16", 32, 8, 64, 16, 24, (16, 256), (128, 2048), 10)},
        # one decoder token a request against encoder states
        {"name": "cross_step", **attention("cross", "bf16", 32, 8, 64, 16, 64, (1, 1), (128, 2048), 11)},
        # decoder prompts against a long FP8 encoder cache
        {"name": "cross_prompt_fp8", **attention("cross", "fp8", 64, 8, 128, 32, 4, (33, 300), (2000, 12000), 12)},
    ]


def _log_int(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(("append", "trim", "prefill", "prefill", "cross", "cross"))
    mix = rng.randrange(1 << 30)
    block = rng.choice((8, 16, 32, 64))
    if op in ("append", "trim"):
        seqs = _log_int(rng, 1, 2000)
        ctx_hi = _log_int(rng, 16, 4096)
        new_hi = min(_log_int(rng, 1, 4096), max(1, 200000 // seqs)) if op == "append" else rng.choice((0, 1, 8, 16))
        return slots(op, block, seqs, (min(1, new_hi), new_hi), (rng.choice((0, 1, 16)), ctx_hi), mix)
    kv = rng.choice(("bf16", "bf16", "fp8"))
    heads, kv_heads, dim = rng.choice(((4, 2, 64), (32, 8, 64), (32, 8, 128), (64, 8, 128), (12, 4, 128), (8, 8, 64),
                                       (16, 16, 128), (8, 1, 128)))
    new_hi = rng.choice((1, _log_int(rng, 2, 16), _log_int(rng, 16, 2048))) if op == "cross" else _log_int(rng, 2, 2048)
    ctx_hi = _log_int(rng, 16, 12000)
    widest = ctx_hi + (new_hi if op == "prefill" else 0)
    seqs = min(_log_int(rng, 1, 64), max(1, (1 << 30) // (heads * new_hi * widest)), max(1, 120000 // widest))
    new_lo = max(1, new_hi // rng.choice((1, 4, 16)))
    return attention(op, kv, heads, kv_heads, dim, block, seqs, (new_lo, new_hi), (rng.choice((0, ctx_hi // 4, ctx_hi)), ctx_hi),
                     mix)


def lengths(case):
    """(new, ctx) of each sequence: tokens of this call, and tokens cached before it (cross: encoder states)."""
    r = random.Random(case["mix"])
    pick = lambda lo, hi: lo if lo == hi else _log_int(r, lo + 1, hi + 1) - 1  # noqa: E731
    pairs = [(pick(case["new_lo"], case["new_hi"]), pick(case["ctx_lo"], case["ctx_hi"])) for _ in range(case["seqs"])]
    return [p[0] for p in pairs], [p[1] for p in pairs]


def _cdiv(a, b):
    return -(-a // b)


def trimmed(case):
    """(lens, new_lens) of a trim: a quarter finished where new_hi is 0, else the last few tokens rejected."""
    new, lens = lengths(case)
    if case["new_hi"] == 0:
        return lens, [0 if i % 4 == 1 else n for i, n in enumerate(lens)]
    return lens, [max(0, n - k) for n, k in zip(lens, new)]


def _tables(need, width, pool, g):
    """Scattered, private blocks for each sequence, and the free ones in the order of the stack."""
    order = torch.randperm(pool, generator=g).to(torch.int32)
    table = torch.full((len(need), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, order[at:]


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    bs, dev = case["block"], "cuda"
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    if case["op"] in ("append", "trim"):
        if case["op"] == "append":
            new, lens = lengths(case)
            after = [a + b for a, b in zip(lens, new)]
        else:
            lens, new = trimmed(case)
            after = lens
        need = [_cdiv(n, bs) for n in lens]
        total = sum(_cdiv(n, bs) for n in after)
        pool = math.ceil(1.3 * total) + 8
        width = max(1, max(_cdiv(n, bs) for n in after))
        table, free = _tables(need, width, pool, g)
        free_ids = torch.full((pool,), -1, dtype=torch.int32)
        free_ids[:len(free)] = free
        s = {"op": case["op"], "block": bs, "lens": ints(lens), "table": table.to(dev), "free_ids": free_ids.to(dev),
             "num_free": ints([len(free)]), "num_free_out": ints([0]), "seq_lens": ints(lens)}
        if case["op"] == "append":
            s |= {"new": ints(new), "slots": torch.empty(sum(new), dtype=torch.int64, device=dev),
                  "q_start": torch.empty(len(new) + 1, dtype=torch.int32, device=dev), "done": ints([0])}
        else:
            s["new_lens"] = ints(new)
        return s
    new, ctx = lengths(case)
    kv_lens = [c + (n if case["op"] == "prefill" else 0) for n, c in zip(new, ctx)]
    need = [_cdiv(n, bs) for n in kv_lens]
    pool, width = math.ceil(1.3 * sum(need)) + 1, max(1, max(need))
    table, _ = _tables(need, width, pool, g)
    gd = torch.Generator(device=dev).manual_seed(seed)
    shape = (pool, case["kv_heads"], bs, case["dim"])

    def cache():
        x = torch.randn(shape, generator=gd, device=dev, dtype=torch.float32)
        if case["kv"] == "bf16":
            return x.to(torch.bfloat16), None
        x = torch.where(torch.rand(shape, generator=gd, device=dev) < 0.01, x * 20, x)
        scale = x.abs().amax((2, 3)) / 448
        return (x / scale[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8), scale

    (k, ks), (v, vs) = cache(), cache()
    tokens = sum(new)
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    q = torch.randn((tokens, case["heads"], case["dim"]), generator=gd, device=dev).to(torch.bfloat16)
    return {"op": case["op"], "block": bs, "scale": case["dim"] ** -0.5, "k": k, "v": v, "k_scale": ks, "v_scale": vs, "q": q,
            "out": torch.empty_like(q), "table": table.to(dev), "q_start": ints(start), "kv_lens": ints(kv_lens),
            "single": max(new) == 1 and min(new) == 1, "most_new": max(new),
            "workspace": torch.empty(WORKSPACE_BYTES, dtype=torch.uint8, device=dev)}


# ------------------------------------------------------------ plain forms ---
def _append(s):
    bs, lens, new, table = s["block"], s["lens"].long(), s["new"].long(), s["table"]
    have, want = (lens + bs - 1) // bs, (lens + new + bs - 1) // bs
    taken = torch.cumsum(want - have, 0)
    start = torch.cat((torch.zeros_like(new[:1]), torch.cumsum(new, 0)))
    fits = (taken <= s["num_free"].long()) & (want <= table.shape[1])
    fits = torch.cumprod(fits.long(), 0)
    j = torch.arange(table.shape[1], device=table.device)[None, :]
    fresh = (j >= have[:, None]) & (j < want[:, None]) & (fits[:, None] > 0)
    top = s["num_free"].long() - 1 - ((taken - want + have)[:, None] + j - have[:, None])
    table.copy_(torch.where(fresh, s["free_ids"][top.clamp(0, s["free_ids"].shape[0] - 1)], table))
    t = torch.arange(s["slots"].shape[0], device=table.device)
    b = torch.searchsorted(start, t, right=True) - 1
    p = lens[b] + t - start[b]
    s["slots"].copy_(torch.where(fits[b] > 0, table[b, (p // bs).clamp(max=table.shape[1] - 1)].long() * bs + p % bs, -1))
    s["q_start"].copy_(start)
    s["seq_lens"].copy_(lens + new * fits)
    s["done"].copy_(fits.sum(0, keepdim=True))
    s["num_free_out"].copy_(s["num_free"] - ((want - have) * fits).sum(0, keepdim=True))


def _trim(s):
    bs, lens, keep, table = s["block"], s["lens"].long(), s["new_lens"].long(), s["table"]
    have, left = (lens + bs - 1) // bs, (keep + bs - 1) // bs
    before = torch.cumsum(have - left, 0) - (have - left)
    j = torch.arange(table.shape[1], device=table.device)[None, :]
    gone = (j >= left[:, None]) & (j < have[:, None])
    at = torch.where(gone, s["num_free"].long() + before[:, None] + j - left[:, None], s["free_ids"].shape[0])
    ids = torch.cat((s["free_ids"], s["free_ids"][:1]))
    ids[at.reshape(-1)] = table.reshape(-1)
    s["free_ids"].copy_(ids[:-1])
    s["seq_lens"].copy_(keep)
    s["num_free_out"].copy_(s["num_free"] + (have - left).sum(0, keepdim=True))


def _gathered(cache, scale, table, dtype):
    """[seqs, kv heads, tokens, dim] of a paged cache."""
    at = table.clamp(min=0).long()
    x = cache[at]
    x = x.to(dtype) if scale is None else x.view(torch.float8_e4m3fn).to(dtype) * scale[at][..., None, None].to(dtype)
    return x.transpose(1, 2).flatten(2, 3)


def _attend(s):
    q, start, n = s["q"], s["q_start"].long(), s["kv_lens"].long()
    k = _gathered(s["k"], s["k_scale"], s["table"], torch.float32)
    v = _gathered(s["v"], s["v_scale"], s["table"], torch.float32)
    i = torch.arange(s["most_new"], device=q.device)
    new = start[1:] - start[:-1]
    x = q[(start[:-1, None] + i).clamp(max=q.shape[0] - 1)].float()  # [seqs, new, heads, dim]
    seqs, most, heads, dim = x.shape
    kv_heads, group = k.shape[1], heads // k.shape[1]
    x = x.view(seqs, most, kv_heads, group, dim).permute(0, 2, 3, 1, 4).reshape(seqs, kv_heads, group * most, dim)
    a = (x @ k.transpose(2, 3)).mul_(s["scale"]).view(seqs, kv_heads, group, most, -1)
    t = torch.arange(a.shape[-1], device=q.device)
    seen = t < n[:, None, None]
    if s["op"] == "prefill":
        seen = seen & (t <= (n - new)[:, None, None] + i[None, :, None])
    a.masked_fill_(~seen[:, None, None], -math.inf)
    top = a.amax(-1, keepdim=True)
    a.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = a.sum(-1, keepdim=True)
    o = (a.view(seqs, kv_heads, group * most, -1) @ v).view(seqs, kv_heads, group, most, dim)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(seqs, most, heads, dim)
    r = torch.arange(q.shape[0], device=q.device)
    b = torch.searchsorted(start, r, right=True) - 1
    s["out"].copy_(o[b, r - start[b]])


def run(s):
    if own:
        from paged_kv_cache_228_gb300 import pa
    if s["op"] == "append":
        if own:
            pa.pa_append_slots_device(s["lens"], s["new"], s["table"], s["free_ids"], s["num_free"], s["block"], s["slots"],
                                      s["q_start"], s["seq_lens"], s["num_free_out"], s["done"])
        else:
            _append(s)
        return {k: s[k] for k in ("table", "slots", "q_start", "seq_lens", "num_free_out", "done")}
    if s["op"] == "trim":
        if own:
            pa.pa_trim_slots_device(s["lens"], s["new_lens"], s["table"], s["free_ids"], s["num_free"], s["block"],
                                    s["seq_lens"], s["num_free_out"])
        else:
            _trim(s)
        return {k: s[k] for k in ("free_ids", "seq_lens", "num_free_out")}
    if not own:
        _attend(s)
    elif s["op"] == "prefill":
        pa.pa_prefill(s["q"], s["k"], s["v"], s["table"], s["q_start"], s["kv_lens"], s["scale"], s["out"], s["workspace"],
                      k_scale=s["k_scale"], v_scale=s["v_scale"])
    else:
        # one token a sequence needs no offsets
        pa.pa_cross_attention(s["q"], s["k"], s["v"], s["table"], None if s["single"] else s["q_start"], s["kv_lens"],
                              s["scale"], s["out"], s["workspace"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return s["out"]


# ------------------------------------------------------------- exact, work ---
def _exact_slots(s):
    table, lens, bs = s["table"].tolist(), s["lens"].tolist(), s["block"]
    free_ids, n = s["free_ids"].tolist(), int(s["num_free"])
    if s["op"] == "trim":
        for b, (was, now) in enumerate(zip(lens, s["new_lens"].tolist())):
            for j in range(_cdiv(now, bs), _cdiv(was, bs)):
                free_ids[n] = table[b][j]
                n += 1
        return {"free_ids": torch.tensor(free_ids, dtype=torch.int32), "seq_lens": s["new_lens"].clone(),
                "num_free_out": torch.tensor([n], dtype=torch.int32)}
    places, start, after, done, stopped = [], [0], [], 0, False
    for b, (was, new) in enumerate(zip(lens, s["new"].tolist())):
        need = _cdiv(was + new, bs) - _cdiv(was, bs)
        stopped = stopped or need > n or was + new > len(table[b]) * bs
        if stopped:
            places += [-1] * new
        else:
            for j in range(_cdiv(was, bs), _cdiv(was + new, bs)):
                n -= 1
                table[b][j] = free_ids[n]
            places += [table[b][p // bs] * bs + p % bs for p in range(was, was + new)]
            done += 1
        after.append(was if stopped else was + new)
        start.append(start[-1] + new)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return {"table": i32(table), "slots": torch.tensor(places, dtype=torch.int64), "q_start": i32(start), "seq_lens": i32(after),
            "num_free_out": i32([n]), "done": i32([done])}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("append", "trim"):
        return _exact_slots(s)
    q, bs, group = s["q"].double(), s["block"], case["heads"] // case["kv_heads"]
    out = torch.zeros_like(q)
    start, lens, table = s["q_start"].tolist(), s["kv_lens"].tolist(), s["table"].long()

    def rows(cache, scale, b, h, n):
        ids = table[b, :_cdiv(n, bs)]
        x = cache[ids, h]
        x = x.double() if scale is None else x.view(torch.float8_e4m3fn).double() * scale[ids, h].double()[:, None, None]
        return x.reshape(-1, x.shape[-1])[:n]

    for b, n in enumerate(lens):
        lo, hi = start[b], start[b + 1]
        if n == 0 or lo == hi:
            continue
        hidden = None
        if case["op"] == "prefill":
            place = n - (hi - lo) + torch.arange(hi - lo, device=q.device)
            hidden = torch.arange(n, device=q.device)[None, :] > place[:, None]
        for h in range(case["kv_heads"]):
            k, v = rows(s["k"], s["k_scale"], b, h, n), rows(s["v"], s["v_scale"], b, h, n)
            for i in range(h * group, (h + 1) * group):
                a = q[lo:hi, i] @ k.T * s["scale"]
                if hidden is not None:
                    a = a.masked_fill(hidden, -math.inf)
                out[lo:hi, i] = torch.softmax(a, -1) @ v
    return out


def work(case):
    if case["op"] == "append":
        new, ctx = lengths(case)
        blocks = sum(_cdiv(c + n, case["block"]) - _cdiv(c, case["block"]) for n, c in zip(new, ctx))
        # lengths, growth, tail entries, offsets, new lengths; the blocks' ids read and written; the slots
        return {"bytes": 20 * case["seqs"] + 8 * blocks + 8 * sum(new) + 16, "flops": 0}
    if case["op"] == "trim":
        was, now = trimmed(case)
        blocks = sum(_cdiv(a, case["block"]) - _cdiv(b, case["block"]) for a, b in zip(was, now))
        return {"bytes": 12 * case["seqs"] + 8 * blocks + 8, "flops": 0}
    new, ctx = lengths(case)
    row = case["dim"] * (2 if case["kv"] == "bf16" else 1)
    causal = case["op"] == "prefill"
    states = sum(c + (n if causal else 0) for n, c in zip(new, ctx))
    blocks = sum(_cdiv(c + (n if causal else 0), case["block"]) for n, c in zip(new, ctx))
    pairs = sum(n * c + (n * (n + 1) // 2 if causal else 0) for n, c in zip(new, ctx))
    cache = 2 * case["kv_heads"] * states * row + 4 * blocks
    if case["kv"] == "fp8":
        cache += 8 * case["kv_heads"] * blocks
    return {"bytes": cache + 4 * sum(new) * case["heads"] * case["dim"], "flops": 4 * pairs * case["heads"] * case["dim"]}
