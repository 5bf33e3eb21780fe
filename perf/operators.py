"""Serving from a paged key/value cache: the operators' plain forms and the calls of this package that replace
them, with the cases they are measured at.

Three operators that a serving step makes in this order:

* slots   -- cu_seqlens, cache lengths, positions and cache slots of a step's new tokens from the requests' lengths,
             with the pages they need taken off a free list and entered in the block table;
* append  -- the step's K and V rows written to their slots, as bf16 or as e4m3 codes under a scale per head;
* attn    -- attention of the new tokens (one per request when decoding, a chunk when a prompt is read in pieces)
             over the pages of their requests, causal, aligned to the end of the cache.

A case names the operator, the number of requests, the ranges their lengths are drawn from, the head shape, the page
size and the cache's type. Lengths follow from the case alone; values follow from the seed. Cache slots that no request
owns hold NaN, as memory that was never written may.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------------------------- cases

def _attn(name, B, q_lo, q_hi, ctx_lo, ctx_hi, Hq, Hkv, d_qk, page, cache, lse=False, lens=1):
    return {"name": name, "op": "attn", "B": B, "q_lo": q_lo, "q_hi": q_hi, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "Hq": Hq,
            "Hkv": Hkv, "d_qk": d_qk, "page": page, "cache": cache, "lse": lse, "lens": lens}


def _append(name, B, q_lo, q_hi, ctx_lo, ctx_hi, Hkv, d_qk, page, cache, lens=1):
    return {"name": name, "op": "append", "B": B, "q_lo": q_lo, "q_hi": q_hi, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
            "Hq": 4 * Hkv if d_qk == 128 else Hkv, "Hkv": Hkv, "d_qk": d_qk, "page": page, "cache": cache, "lens": lens}


def _slots(name, B, q_lo, q_hi, ctx_lo, ctx_hi, page, pad, lens=1):
    return {"name": name, "op": "slots", "B": B, "q_lo": q_lo, "q_hi": q_hi, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
            "page": page, "pad": pad, "lens": lens}


def listed():
    return [
        # one decoding step of a small batch, padded to the batch a graph was captured for
        _slots("slots_decode", 13, 1, 1, 60, 2000, 16, 3),
        # a full step of a busy server: decoding requests and chunks of prompts together
        _slots("slots_mixed", 512, 1, 63, 0, 8000, 16, 117),
        # K and V of one decoding step
        _append("append_decode", 48, 1, 1, 10, 4000, 8, 128, 16, "bf16"),
        # K and V of a long prompt step into an e4m3 cache
        _append("append_prompt_e4m3", 9, 900, 2700, 0, 5000, 8, 128, 64, "e4m3"),
        # one request decoding, 7B-style heads: latency
        _attn("decode_one", 1, 1, 1, 4095, 4095, 32, 8, 128, 16, "bf16"),
        # a batch of decoding requests of very different ages
        _attn("decode_batch", 64, 1, 1, 5, 16000, 32, 8, 128, 64, "bf16"),
        # long contexts from an e4m3 cache, with the log-sum-exp
        _attn("decode_long_e4m3", 24, 1, 1, 9000, 32000, 32, 8, 128, 64, "e4m3", lse=True),
        # drafted tokens checked in one step: a few tokens per request
        _attn("verify_drafts", 32, 3, 9, 100, 9000, 32, 8, 128, 16, "bf16"),
        # a long prompt read in chunks of 4096: the last chunk of 32768
        _attn("chunk_long", 1, 4096, 4096, 28672, 28672, 32, 8, 128, 128, "bf16"),
        # ragged chunks of several prompts, some at their start, with the log-sum-exp
        _attn("chunk_ragged", 7, 1, 1500, 0, 6000, 32, 8, 128, 16, "bf16", lse=True),
        # the same from an e4m3 cache
        _attn("chunk_e4m3", 4, 500, 1300, 2000, 12000, 32, 8, 128, 64, "e4m3"),
        # the 192/128 head shape, a chunk of two prompts
        _attn("chunk_mla", 2, 1000, 1700, 3000, 9000, 16, 16, 192, 64, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["slots", "append", "decode", "decode", "verify", "chunk", "chunk"])
    lens = rng.randrange(1, 1 << 20)
    page = rng.choice([16, 32, 48, 64, 128, 256])
    if kind == "slots":
        B = _log_int(rng, 1, 512)
        c = _slots("", B, 1, _log_int(rng, 1, 63), 0, _log_int(rng, 16, 8000), page, rng.randrange(0, 200), lens)
    elif kind == "append":
        B = _log_int(rng, 1, 48)
        q_hi = _log_int(rng, 1, max(1, 16000 // B))
        d_qk = rng.choice([128, 128, 192])
        c = _append("", B, 1, q_hi, 0, 4000, rng.choice([1, 2, 5, 8]), d_qk, page, rng.choice(["bf16", "e4m3"]), lens)
    else:
        Hq, Hkv, d_qk = rng.choice([(32, 8, 128), (32, 8, 128), (16, 16, 192), (28, 4, 128), (8, 1, 128), (15, 5, 128)])
        cache, lse = rng.choice(["bf16", "e4m3"]), rng.random() < 0.3
        if kind == "decode":
            B = _log_int(rng, 1, 64)
            ctx = _log_int(rng, 64, min(32000, 500000 // B))
            c = _attn("", B, 1, 1, ctx // 4, ctx, Hq, Hkv, d_qk, page, cache, lse, lens)
        elif kind == "verify":
            B = _log_int(rng, 1, 32)
            ctx = _log_int(rng, 64, min(20000, 250000 // B))
            c = _attn("", B, 1, rng.randrange(2, 17), ctx // 8, ctx, Hq, Hkv, d_qk, page, cache, lse, lens)
        else:
            B = rng.randrange(1, 7)
            q = _log_int(rng, 20, 3000 // B)
            c = _attn("", B, max(1, q // 4), q, 0, _log_int(rng, 50, 12000), Hq, Hkv, d_qk, page, cache, lse, lens)
    del c["name"]
    return c


def _lengths(case):
    """(cached tokens, new tokens) of every request."""
    rng = random.Random(case["lens"] * 7919 + case["B"])
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    new = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(case["B"])]
    return ctx, new


def work(case):
    ctx, new = _lengths(case)
    T = sum(new)
    if case["op"] == "slots":
        taken = sum(-(-(c + n) // case["page"]) - -(-c // case["page"]) for c, n in zip(ctx, new))
        held = sum(1 + (c + n - 1) // case["page"] - c // case["page"] for c, n in zip(ctx, new))
        return {"bytes": 4.0 * (4 * case["B"] + 2 * (T + case["pad"]) + 2 * taken + held), "flops": 0.0}
    d_v, esz = 128, 2 if case["cache"] == "bf16" else 1
    per_token = case["Hkv"] * (case["d_qk"] + d_v)
    if case["op"] == "append":
        return {"bytes": float(T * per_token * (2 + esz) + 4 * T), "flops": 0.0}
    pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new))
    kv = sum(c + n for c, n in zip(ctx, new))
    bytes_ = kv * per_token * esz + 2 * T * case["Hq"] * (case["d_qk"] + d_v) + (4 * T * case["Hq"] if case["lse"] else 0)
    return {"bytes": float(bytes_), "flops": 2.0 * case["Hq"] * (case["d_qk"] + d_v) * pairs}


# ---------------------------------------------------------------------------------------------- inputs

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _tables(case, g, ctx, tail):
    """A block table over randomly ordered pages for `ctx` tokens of each request, with `tail` more entries per
    row that hold no page (-1), and the pages that no request has."""
    ps = case["page"]
    need = [-(-c // ps) for c in ctx]
    width = max(1, max(need)) + tail
    pool = sum(need) + sum(need) // 8 + 4
    order = torch.randperm(pool, generator=g, device=DEV, dtype=torch.int32)
    table = torch.full((case["B"], width), -1, dtype=torch.int32, device=DEV)
    at = _ints([0] + need).cumsum(0)
    col = torch.arange(width, device=DEV)
    has = col[None, :] < _ints(need)[:, None]
    table[has] = order[: sum(need)]
    return table, order[sum(need):].contiguous(), pool, at, col


def _slot_of(table, ps, b, pos):
    return table[b, pos // ps].long() * ps + pos % ps


def _gain(g, *shape):
    return torch.exp(0.5 * torch.randn(*shape, generator=g, device=DEV))


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    ctx, new = _lengths(case)
    B, ps, T = case["B"], case["page"], sum(new)
    if case["op"] == "slots":
        # the pages of the cached tokens are in the table; those of the new ones come off the free list, of which
        # an earlier step has taken some
        more = max(-(-(c + n) // ps) - -(-c // ps) for c, n in zip(ctx, new))
        table, spare, pool, _, _ = _tables(case, g, ctx, more + 2)
        taken = sum(-(-(c + n) // ps) - -(-c // ps) for c, n in zip(ctx, new))
        head = 1 + int(seed) % 5
        free = torch.randperm(taken + head + 9, generator=g, device=DEV, dtype=torch.int32) + pool
        return {"case": case, "table": table, "ctx": _ints(ctx), "new": _ints(new), "total": T + case["pad"], "free": free,
                "head": _ints([head])}
    kv = [c + n for c, n in zip(ctx, new)]
    table, _, pool, _, _ = _tables(case, g, kv, 2)
    Hq, Hkv, d_qk, d_v = case["Hq"], case["Hkv"], case["d_qk"], 128
    b_of = torch.repeat_interleave(torch.arange(B, device=DEV), _ints(new).long(), output_size=T)
    cu = _ints([0] + new).cumsum(0).to(torch.int32)
    # one projection's output holds the step's Q, K and V
    qkv = torch.randn(T, Hq * d_qk + Hkv * (d_qk + d_v), generator=g, device=DEV)
    kg, qg = _gain(g, Hkv, d_qk), _gain(g, Hq, d_qk)
    qkv[:, : Hq * d_qk] *= qg.reshape(-1)
    qkv[:, Hq * d_qk: (Hq + Hkv) * d_qk] *= kg.reshape(-1)
    qkv = qkv.to(torch.bfloat16)
    q, k, v = qkv.split([Hq * d_qk, Hkv * d_qk, Hkv * d_v], 1)
    q, k, v = q.view(T, Hq, d_qk), k.view(T, Hkv, d_qk), v.view(T, Hkv, d_v)
    used = torch.zeros(pool * ps, dtype=torch.bool, device=DEV)
    ends = _ints([0] + kv).cumsum(0)
    kv_b = torch.repeat_interleave(torch.arange(B, device=DEV), _ints(kv).long(), output_size=sum(kv))
    kv_pos = torch.arange(sum(kv), device=DEV) - ends[kv_b]
    used[_slot_of(table, ps, kv_b, kv_pos)] = True
    caches, scales = [], []
    for d, gain in ((d_qk, kg), (d_v, torch.ones(Hkv, d_v, device=DEV))):
        x = torch.randn(pool * ps, Hkv, d, generator=g, device=DEV)
        x *= gain
        if case["cache"] == "e4m3":
            scale = x.abs().amax((0, 2)) / 448.0
            x = (x / scale[None, :, None]).clamp_(-448.0, 448.0)
            scales.append(scale)
        x[~used] = math.nan
        caches.append(x.to(torch.bfloat16 if case["cache"] == "bf16" else torch.float8_e4m3fn).view(pool, ps, Hkv, d))
        del x
    s = {"case": case, "q": q, "k": k, "v": v, "k_cache": caches[0], "v_cache": caches[1], "table": table, "cu": cu,
         "kv_lens": _ints(kv), "max_q": max(new), "k_scale": scales[0] if scales else None,
         "v_scale": scales[1] if scales else None}
    if case["op"] == "append":
        pos = _ints(ctx)[b_of] + torch.arange(T, device=DEV) - cu[b_of]
        s["slots"] = _slot_of(table, ps, b_of, pos).to(torch.int32)
        if scales:  # what the scales were set for may be exceeded by a step's values
            s["k_scale"], s["v_scale"] = scales[0] * 0.9, scales[1] * 0.9
    return s


# ---------------------------------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        import bf16_causal_prefill_fwd_b200 as b2

        if op == "slots":
            cu, kv_lens, positions, slots, head = b2.paged_slots(
                state["table"], state["ctx"], state["new"], state["total"], state["case"]["page"],
                free_pages=state["free"], free_head=state["head"])
            return {"cu": cu, "kv_lens": kv_lens, "positions": positions, "slots": slots, "table": state["table"], "head": head}
        if op == "append":
            b2.paged_append_kv(state["k"], state["v"], state["k_cache"], state["v_cache"], state["slots"],
                               k_scale=state["k_scale"], v_scale=state["v_scale"])
            return {"k_cache": state["k_cache"], "v_cache": state["v_cache"]}
        got = b2.attn_paged_fwd(state["q"], state["k_cache"], state["v_cache"], state["table"], state["cu"], state["kv_lens"],
                                max_seqlen_q=state["max_q"], k_scale=state["k_scale"], v_scale=state["v_scale"],
                                return_lse=state["case"]["lse"])
        return {"o": got[0], "lse": got[1]} if state["case"]["lse"] else {"o": got}
    return {"slots": _plain_slots, "append": _plain_append, "attn": _plain_attn}[op](state)


def _plain_slots(s):
    ps, total, dev = s["case"]["page"], s["total"], s["table"].device
    ctx, new, table = s["ctx"].long(), s["new"].long(), s["table"]
    B, width = table.shape
    cu = torch.zeros(B + 1, dtype=torch.int64, device=dev)
    cu[1:] = new.cumsum(0)
    kv = ctx + new
    held, want = (ctx + ps - 1) // ps, (kv + ps - 1) // ps
    fresh = want - held
    before = s["head"].long() + fresh.cumsum(0) - fresh
    col = torch.arange(width, device=dev)[None, :]
    is_new = (col >= held[:, None]) & (col < want[:, None])
    at = (before[:, None] + col - held[:, None]).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(is_new, s["free"][at], table))
    t = torch.arange(total, device=dev)
    b = torch.searchsorted(cu[1:], t, right=True)
    real = b < B
    b = b.clamp(max=B - 1)
    pos = torch.where(real, ctx[b] + t - cu[b], 0)
    page = table[b, (pos // ps).clamp(max=width - 1)].long()
    slots = torch.where(real, page * ps + pos % ps, -1)
    head = s["head"] + fresh.sum()
    return {"cu": cu.to(torch.int32), "kv_lens": kv.to(torch.int32), "positions": pos.to(torch.int32),
            "slots": slots.to(torch.int32), "table": table, "head": head.to(torch.int32)}


def _plain_store(x, cache, slots, scale):
    if scale is not None:
        x = (x.float() / scale[None, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        cache = cache.view(torch.uint8)
    cache.view(-1, *cache.shape[2:]).index_copy_(0, slots, x)


def _plain_append(s):
    slots = s["slots"].long()
    _plain_store(s["k"], s["k_cache"], slots, s["k_scale"])
    _plain_store(s["v"], s["v_cache"], slots, s["v_scale"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_gather(cache, table, valid, scale):
    """[B, Hkv, keys, d] in 32 bits; what no request owns reads as zero."""
    x = cache.view(torch.uint8 if scale is not None else cache.dtype)[table.clamp(min=0).long()]
    x = (x.view(torch.float8_e4m3fn) if scale is not None else x).flatten(1, 2).float()
    x = torch.where(valid[:, :, None, None], x, 0.0)
    if scale is not None:
        x = x * scale[None, None, :, None]
    return x.transpose(1, 2)


def _plain_attn(s):
    c, q, cu, kv_lens = s["case"], s["q"], s["cu"].long(), s["kv_lens"].long()
    dev, nq, Hkv = q.device, s["max_q"], c["Hkv"]
    T, Hq, d_qk = q.shape
    B, G = kv_lens.numel(), Hq // Hkv
    q_lens = cu[1:] - cu[:-1]
    keys = torch.arange(s["table"].shape[1] * c["page"], device=dev)
    valid = keys[None, :] < kv_lens[:, None]
    k = _plain_gather(s["k_cache"], s["table"], valid, s["k_scale"])
    v = _plain_gather(s["v_cache"], s["table"], valid, s["v_scale"])
    i = torch.arange(nq, device=dev)
    rows = (cu[:-1, None] + i[None, :]).clamp(max=T - 1)
    qp = q[rows].float().view(B, nq, Hkv, G, d_qk).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * nq, d_qk)
    scores = torch.matmul(qp, k.transpose(2, 3)).view(B, Hkv, G, nq, -1)
    scores *= d_qk ** -0.5
    last = kv_lens[:, None] - q_lens[:, None] + i[None, :]  # the last key that new token i of a request sees
    scores.masked_fill_((keys[None, None, :] > last[:, :, None])[:, None, None], -math.inf)
    m = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    p = scores.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, G * nq, -1), v).view(B, Hkv, G, nq, -1) / l
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(cu[1:], t, right=True)
    at = t - cu[b]
    out = {"o": o.permute(0, 3, 1, 2, 4)[b, at].reshape(T, Hq, -1).to(torch.bfloat16)}
    if c["lse"]:
        lse = (m + l.log()).squeeze(-1)
        out["lse"] = lse.permute(0, 3, 1, 2)[b, at].reshape(T, Hq).t().contiguous()
    return out


# ---------------------------------------------------------------------------------------------- in 64 bits

def _e4m3_64(x):
    """x rounded to the nearest e4m3 value (3 mantissa bits, exponents -6 .. 8, ties to even), held at +-448."""
    x = x.clamp(-448.0, 448.0)
    _, e = torch.frexp(x)
    quantum = torch.ldexp(torch.ones_like(x), e.clamp(min=-5) - 4)
    return torch.round(x / quantum) * quantum


def exact(case, seed):
    if case["op"] == "slots":
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        got = {}
        for name, x, scale in (("k_cache", s["k"], s["k_scale"]), ("v_cache", s["v"], s["v_scale"])):
            cache = s[name].double().flatten(0, 1)
            x = x.double()
            if scale is not None:
                x = _e4m3_64(x / scale.double().view(1, -1, 1))
            cache[s["slots"].long()] = x
            got[name] = cache.view(s[name].shape)
        return got
    ctx, new = _lengths(case)
    T, Hq, d_qk = s["q"].shape
    G, ps = Hq // case["Hkv"], case["page"]
    o = torch.zeros(T, Hq, 128, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(Hq, T, dtype=torch.float64, device=s["q"].device)
    t0 = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        at = torch.arange(c + n, device=o.device)
        pages = s["table"][b].long()[at // ps]
        for h in range(case["Hkv"]):
            k = s["k_cache"][pages, at % ps, h].double()
            v = s["v_cache"][pages, at % ps, h].double()
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            for hq in range(h * G, (h + 1) * G):
                x = s["q"][t0:t0 + n, hq].double() @ k.T / math.sqrt(d_qk)
                x[at[None, :] > c + torch.arange(n, device=o.device)[:, None]] = -math.inf
                z = torch.logsumexp(x, 1)
                o[t0:t0 + n, hq] = torch.exp(x - z[:, None]) @ v
                lse[hq, t0:t0 + n] = z
        t0 += n
    return {"o": o, "lse": lse} if case["lse"] else {"o": o}
