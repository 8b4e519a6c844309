"""Workloads of the paged 8-bit cache: block tables and slot maps, rotary + append, attention.

Each case is one call that a serving step makes of one of the three operators:

  tables  moe.kv_tables      block tables, free stack, slot map and page runs from request lengths
  append  moe.rope_append    rotary positions of Q and K, K and V written into the E4M3 cache with one
                             scale per page and head (a page that holds older tokens is rescaled)
  attend  moe.kv_attention   causal (optionally windowed) attention over that cache, few query rows
                             per request (decode, verification) or whole prompts and chunks

With `own` false, `run` computes the same outputs in their plain form: elementary torch operations
in fp32 (whole-number operations for the tables), rounded once at the end.
"""

import math

import numpy as np
import torch

own = False

FP8_MAX = 448.0
SCALE_FLOOR = float(np.float32(1.0 / (448.0 * 512.0)))
FMT_FP32, FMT_POW2 = 0, 1
HALF, INTERLEAVED = 0, 1
DEV = "cuda"


# ------------------------------------------------------------------------------------------ cases
def _tables(name, B, P, ctx_lo, ctx_hi, mix, prompt):
    # mix: every `mix`-th request is a prompt of up to `prompt` tokens, as many have finished, as many
    # are rolled back by a few tokens; 0: every request adds one token
    return dict(name=name, op="tables", B=B, P=P, ctx_lo=ctx_lo, ctx_hi=ctx_hi, mix=mix, prompt=prompt)


def _append(name, B, q_lo, q_hi, ctx_lo, ctx_hi, Hq, Hkv, D, P, rot, layout, fmt):
    return dict(name=name, op="append", B=B, q_lo=q_lo, q_hi=q_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi, Hq=Hq,
                Hkv=Hkv, D=D, P=P, rot=rot, layout=layout, fmt=fmt)


def _attend(name, B, q_lo, q_hi, ctx_lo, ctx_hi, Hq, Hkv, D, P, window):
    return dict(name=name, op="attend", B=B, q_lo=q_lo, q_hi=q_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi, Hq=Hq,
                Hkv=Hkv, D=D, P=P, window=window)


def listed():
    return [
        # a handful of requests, one new token each: what a step costs when it is all latency
        _tables("tables decode 8", 8, 16, 100, 4000, 0, 0),
        # a full server's step: decoding, prompts admitted, requests finished and rolled back
        _tables("tables mixed 1024", 1024, 64, 1, 32000, 16, 1500),
        # one decode step of a medium batch
        _append("append decode 32", 32, 1, 1, 10, 8000, 32, 8, 128, 64, 128, HALF, FMT_FP32),
        # one decode step of a large batch, rotation of half the head in interleaved pairs, an odd
        # number of query heads per cache head, small pages
        _append("append decode 253 partial", 253, 1, 1, 3, 6000, 40, 8, 128, 16, 64, INTERLEAVED, FMT_POW2),
        # prompts of a batch, some of them continuing in a page that already holds tokens
        _append("append prompts 4", 4, 700, 4096, 5, 2000, 32, 8, 128, 64, 128, HALF, FMT_FP32),
        # the smallest attention call: one request, a short context
        _attend("decode 1 x 4k", 1, 1, 1, 4095, 4095, 32, 8, 128, 64, 0),
        # one request with a long context: few heads, so the cache's length is the only parallel axis
        _attend("decode 1 x 128k", 1, 1, 1, 131000, 131000, 32, 8, 128, 128, 0),
        # a ragged batch, from a few tokens to thousands, small pages, five query heads per cache head
        _attend("decode 61 ragged", 61, 1, 1, 6, 8190, 40, 8, 128, 16, 0),
        # a large decode batch over long contexts: the bandwidth of the cache
        _attend("decode 128 x 8k-16k", 128, 1, 1, 8000, 16300, 64, 8, 128, 64, 0),
        # verification of drafted tokens, narrow heads, a sliding window
        _attend("verify 16 x 4 window", 16, 4, 4, 500, 20000, 32, 4, 64, 32, 4096),
        # prompts of a batch, ragged, without a context
        _attend("prompts 5", 5, 300, 4000, 0, 0, 32, 8, 128, 64, 0),
        # a chunk of a long prompt: its tokens see the chunks before it
        _attend("chunk 4096 after 28k", 1, 4096, 4096, 28000, 28000, 32, 8, 128, 64, 0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "append", "attend", "attend", "attend"])
    P = rng.choice([16, 32, 64, 128])
    if op == "tables":
        B = _log(rng, 8, 1024)
        c = _tables("", B, P, _log(rng, 1, 500), _log(rng, 1000, 32000),
                    rng.choice([0, 5, 16]), _log(rng, 20, 1500))
        c["prompt"] = min(c["prompt"], 60000 // max(1, B // max(1, c["mix"] or B)))
    else:
        Hkv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 6, 8, 16])
        D = rng.choice([64, 128, 128])
        if op == "append":
            decode = rng.random() < 0.5
            q_hi = 1 if decode else _log(rng, 33, 4096)
            B = _log(rng, 8, 256) if decode else _log(rng, 1, max(1, 10000 // q_hi))
            c = _append("", B, 1 if decode else max(1, q_hi // 6), q_hi, rng.randrange(0, 100),
                        _log(rng, 101, 8000), Hkv * g if Hkv * g <= 64 else 64, Hkv, D, P,
                        rng.choice([D, D // 2, D // 4]), rng.choice([HALF, INTERLEAVED]),
                        rng.choice([FMT_FP32, FMT_POW2]))
        elif rng.random() < 0.65:                    # few rows per request
            q = rng.choice([1, 1, 1, 2, 3, 4])
            ctx = _log(rng, 1000, 131000)
            most = 1_000_000_000 // (ctx * Hkv * D)  # padded cache values of the plain form
            B = _log(rng, 1, max(1, min(256, most)))
            c = _attend("", B, q, q, ctx if B == 1 else max(1, ctx // _log(rng, 2, 300)), ctx, Hkv * g, Hkv,
                        D, P, rng.choice([0, 0, 0, _log(rng, 100, 5000)]))
        else:                                        # prompts and chunks
            q_hi = _log(rng, 65, 4096)
            ctx = rng.choice([0, 0, _log(rng, 10, 16000)])
            most = 3_000_000_000 // (q_hi * (ctx + q_hi) * Hkv * g)   # scores of the plain form
            B = _log(rng, 1, max(1, min(32, most)))
            c = _attend("", B, max(1, q_hi // _log(rng, 1, 20)), q_hi, ctx // 3, ctx, Hkv * g, Hkv, D, P,
                        rng.choice([0, 0, _log(rng, 100, 5000)]))
    del c["name"]
    return c


def _spread(lo, hi, n):
    """n lengths from lo to hi, evenly spread over their logarithm."""
    if n == 1:
        return [hi]
    a = math.log(lo + 1.0)
    b = math.log(hi + 1.0)
    return [int(round(math.exp(a + (b - a) * i / (n - 1)) - 1)) for i in range(n)]


def _lengths(case):
    """(older tokens, new length) of each request, before the seed's order."""
    B = case["B"]
    ctx = _spread(case["ctx_lo"], case["ctx_hi"], B)
    if case["op"] != "tables":
        q = _spread(case["q_lo"], case["q_hi"], B)[::-1]
        return ctx, [c + n for c, n in zip(ctx, q)]
    new = [c + 1 for c in ctx]
    m = case["mix"]
    if m:
        for i in range(B):
            if i % m == 1:                           # admitted
                ctx[i], new[i] = 0, 1 + (i * 7919) % case["prompt"]
            elif i % m == 2:                         # finished
                new[i] = 0
            elif i % m == 3:                         # rejected drafts
                new[i] = max(0, ctx[i] - 5)
    return ctx, new


def _pages(n, P):
    return (n + P - 1) // P


def _sizes(case):
    """(tokens added, capacity of runs, table width, pages of the pool)"""
    P = case["P"]
    ctx, new = _lengths(case)
    T = sum(max(0, b - a) for a, b in zip(ctx, new))
    width = _pages(max(max(ctx), max(new)), P) + 3
    pool = sum(_pages(max(a, b), P) for a, b in zip(ctx, new))
    pool += max(8, pool // (8 if case["op"] == "tables" else 50))
    return T, min(T, T // P + 2 * case["B"]), width, pool


# ---------------------------------------------------------------------------------------- prepare
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 2 + 1)
    return g


def _i32(v):
    return torch.as_tensor(np.asarray(v, dtype=np.int32)).to(DEV)


def _fill_cache(g, pages, Hkv, P, D, gain):
    """E4M3 codes and scales of normal values with a few wide channels (as K and V have), as an
    earlier step's append left them."""
    codes = torch.empty((pages, Hkv, P, D), dtype=torch.uint8, device=DEV)
    scale = torch.empty((pages, Hkv), dtype=torch.float32, device=DEV)
    wide = 1.0 + 3.0 * (torch.rand((Hkv, 1, D), generator=g, device=DEV) > 0.97).float()
    step = max(1, (1 << 27) // (Hkv * P * D))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        x = torch.randn((n, Hkv, P, D), generator=g, device=DEV).mul_(wide * gain)
        s = (x.abs().amax((2, 3)) / FP8_MAX).clamp_min(SCALE_FLOOR)
        codes[a:a + n] = (x / s[:, :, None, None]).clamp_(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        scale[a:a + n] = s
    return codes, scale


def _rope_table(rows, rot):
    """cos and sin of every position, fp32 [rows, rot / 2, 2]."""
    inv = 10000.0 ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    a = np.arange(rows, dtype=np.float64)[:, None] * inv
    return torch.from_numpy(np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)).to(DEV)


def prepare(case, seed):
    P = case["P"]
    g = _gen(seed)
    order = np.random.RandomState(seed % (1 << 31)).permutation(case["B"])
    ctx, new = (np.asarray(v, dtype=np.int64)[order] for v in _lengths(case))
    T, runs, width, pool = _sizes(case)
    B = case["B"]
    ids = torch.randperm(pool, generator=g, device=DEV).to(torch.int32).cpu().numpy()
    held = _pages(ctx, P)
    table = np.full((B, width), -1, np.int32)
    at = np.concatenate([[0], np.cumsum(held)])
    for i in range(B):
        table[i, :held[i]] = ids[at[i]:at[i + 1]]
    free = np.zeros(pool, np.int32)
    free[:pool - at[-1]] = ids[at[-1]:]
    st = {"case": dict(case), "P": P, "T": T, "runs": runs,
          "cur": _i32(ctx), "new": _i32(new), "table": _i32(table), "free": _i32(free),
          "count": _i32([pool - at[-1]])}
    if case["op"] == "tables":
        e = lambda *shape: torch.empty(shape, dtype=torch.int32, device=DEV)  # noqa: E731
        # the second set of tables, which a program that prepares a step ahead keeps
        st["out"] = dict(block_table=e(B, width), free_list=e(pool), free_count=e(1), kv_len=e(B),
                         tok_start=e(B + 1), slot=e(T), position=e(T), request=e(T), run_tok=e(runs),
                         run_len=e(runs), info=e(4))
        return st
    # the tables of this step, as kv_tables leaves them
    st["tables"] = _plain_tables(st)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    qkv = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device=DEV)
    qkv = (qkv * (1.0 + 2.0 * (torch.rand(qkv.shape[1], generator=g, device=DEV) > 0.98))).to(torch.bfloat16)
    q, k, v = qkv.split([Hq * D, Hkv * D, Hkv * D], dim=1)
    k_codes, k_scale = _fill_cache(g, pool, Hkv, P, D, 1.0)
    v_codes, v_scale = _fill_cache(g, pool, Hkv, P, D, 0.7)
    st["cache"] = (k_codes, v_codes, k_scale, v_scale)
    if case["op"] == "append":
        # Q, K and V are slices of one projection's output, as a decoder layer has them
        st["q"], st["k"], st["v"] = q.unflatten(1, (Hq, D)), k.unflatten(1, (Hkv, D)), v.unflatten(1, (Hkv, D))
        if case["fmt"] == FMT_POW2:
            for s in (k_scale, v_scale):
                s.copy_(_pow2_up(s))
        st["rope"] = _rope_table(width * P, case["rot"])
        st["q_out"] = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=DEV)
    else:
        st["q"] = q.unflatten(1, (Hq, D)).contiguous()
        st["out"] = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=DEV)
        st["workspace"] = torch.zeros(32 << 20, dtype=torch.uint8, device=DEV)
        st["max_q"] = int((new - ctx).max())
        st["max_kv"] = int(new.max())
    return st


# ------------------------------------------------------------------------------------------ plain
def _excl(x):
    return torch.cumsum(x, 0) - x


def _plain_tables(st):
    """Whole-number operations on padded arrays: see kv_tables for what each output is."""
    P, T, R = st["P"], st["T"], st["runs"]
    table, free = st["table"].long(), st["free"].long()
    B, W = table.shape
    pool = free.shape[0]
    cur, want, count = st["cur"].long().clamp(0, W * P), st["new"].long().clamp(min=0), st["count"].long()
    ok = want <= W * P
    pc, pw = (cur + P - 1) // P, (want + P - 1) // P
    rel = torch.where(ok, (pc - pw).clamp(min=0), 0)
    need = torch.where(ok, (pw - pc).clamp(min=0), 0)
    j = torch.arange(W, device=DEV)[None, :]
    # released pages onto the stack, in request order
    leaves = ok[:, None] & (j >= pw[:, None]) & (j < pc[:, None])
    to = torch.where(leaves, count + _excl(rel)[:, None] + j - pw[:, None], pool)
    stack = torch.cat([free, free.new_zeros(1)])
    stack[to.clamp(max=pool).reshape(-1)] = table.reshape(-1)
    stack = stack[:pool]
    count = count + rel.sum()
    # granted pages from its top, in stored order
    before = _excl(need)
    ok = ok & ((need == 0) | (before + need <= count))
    granted = torch.where(ok, need, 0).sum()
    joins = ok[:, None] & (j >= pc[:, None]) & (j < pw[:, None])
    take = (count - granted + before[:, None] + j - pc[:, None]).clamp(0, pool - 1)
    kv = torch.where(ok, want, cur)
    pk = (kv + P - 1) // P
    out = torch.where(joins, stack[take], torch.where(j < torch.minimum(pc, pk)[:, None], table, -1))
    # tokens
    n = torch.where(want <= W * P, (want - cur).clamp(min=0), 0)
    start = torch.cat([n.new_zeros(1), torch.cumsum(n, 0)])
    t = torch.arange(T, device=DEV)
    req = torch.searchsorted(start[1:], t, right=True).clamp(max=B - 1)
    live = t < start[-1]
    pos = cur[req] + t - start[req]
    page = out[req, (pos // P).clamp(0, W - 1)]
    slot = torch.where(live & ok[req], page * P + pos % P, -1)
    # runs: the tokens of a request that share a page
    nr = torch.where(ok & (n > 0), (want - 1).clamp(min=0) // P - cur // P + 1, 0)
    rs = torch.cat([nr.new_zeros(1), torch.cumsum(nr, 0)])
    r = torch.arange(R, device=DEV)
    rq = torch.searchsorted(rs[1:], r, right=True).clamp(max=B - 1)
    rl = r < rs[-1]
    p0 = (cur[rq] // P + r - rs[rq]) * P
    a, b = torch.maximum(p0, cur[rq]), torch.minimum(p0 + P, want[rq])
    info = torch.stack([start[-1], rs[-1], (~ok).sum(), granted])
    z = lambda m, x: torch.where(m, x, 0)  # noqa: E731
    got = dict(block_table=out, free_list=stack, free_count=(count - granted).reshape(1), kv_len=kv,
               tok_start=start, slot=slot, position=z(live, pos), request=torch.where(live, req, -1),
               run_tok=z(rl, start[rq] + a - cur[rq]), run_len=z(rl, b - a), info=info)
    return {k: v.to(torch.int32) for k, v in got.items()}


def _rotate(x, rope, layout):
    """x fp32 [T, heads, D]; the first rot values of each head are rotated."""
    c, s = rope[:, None, :, 0], rope[:, None, :, 1]
    rot = 2 * c.shape[-1]
    if layout == HALF:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat([a * c - b * s, b * c + a * s, x[..., rot:]], -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    r = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([r, x[..., rot:]], -1)


def _pow2_up(s):
    b = s.view(torch.int32)
    return torch.where((b & 0x7FFFFF) != 0, (b & ~0x7FFFFF) + 0x800000, b).view(torch.float32)


def _plain_write(st, x, codes, scale):
    """x fp32 [T, Hkv, D] into the touched pages of one cache."""
    P, fmt, t = st["P"], st["case"]["fmt"], st["tables"]
    live = t["run_len"] > 0
    first, n = t["run_tok"].long(), t["run_len"].long()
    slot = t["slot"].long()[first]
    page, off = slot // P, slot % P
    i = torch.arange(P, device=DEV)[None, :]
    src = (first[:, None] + i - off[:, None]).clamp(0, x.shape[0] - 1)
    fresh = (i >= off[:, None]) & (i < (off + n)[:, None])                       # [R, P]
    xb = x[src].transpose(1, 2)                                                   # [R, Hkv, P, D]
    amax = torch.where(fresh[:, None, :, None], xb.abs(), 0.0).amax((2, 3))
    s = (amax / torch.full_like(amax, FP8_MAX)).clamp_min(SCALE_FLOOR)   # a division, not a product
    if fmt == FMT_POW2:
        s = _pow2_up(s)
    was = scale[page]
    s = torch.where(off[:, None] > 0, torch.maximum(s, was), s)
    ratio = torch.where(off[:, None] > 0, was / s, 1.0)
    prev = codes[page]
    older = prev.view(torch.float8_e4m3fn).float()
    older = (older * ratio[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    new = (xb / s[:, :, None, None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    is_old = (i < off[:, None])[:, None, :, None]
    block = torch.where(fresh[:, None, :, None], new, torch.where(is_old, older, prev))
    codes[page[live]] = block[live]
    scale[page[live]] = s[live]


def _plain_append(st):
    kc, vc, ks, vs = st["cache"]
    rope = st["rope"][st["tables"]["position"].long()]
    q = _rotate(st["q"].float(), rope, st["case"]["layout"]).to(torch.bfloat16)
    _plain_write(st, _rotate(st["k"].float(), rope, st["case"]["layout"]), kc, ks)
    _plain_write(st, st["v"].float(), vc, vs)
    return q


def _plain_attend(st):
    c, t = st["case"], st["tables"]
    kc, vc, ks, vs = st["cache"]
    Hq, Hkv, D, P = c["Hq"], c["Hkv"], c["D"], c["P"]
    G, NQ, L = Hq // Hkv, st["max_q"], st["max_kv"]
    start, kv = t["tok_start"].long(), t["kv_len"].long()
    B = kv.shape[0]
    n = start[1:] - start[:-1]
    W = (L + P - 1) // P
    pages = t["block_table"][:, :W].long().clamp(min=0)
    j = torch.arange(W * P, device=DEV)
    inside = (j[None, :] < kv[:, None])[:, None, :, None]

    def values(codes, scale):
        x = codes[pages].view(torch.float8_e4m3fn).float() * scale[pages][..., None, None]
        return torch.where(inside, x.transpose(1, 2).reshape(B, Hkv, W * P, D), 0.0)

    i = torch.arange(NQ, device=DEV)
    at = (start[:-1, None] + i).clamp(max=st["T"] - 1)
    q = st["q"].float()[at].view(B, NQ, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * NQ, D)
    s = torch.matmul(q, values(kc, ks).transpose(-1, -2)) * (D ** -0.5)
    pos = (kv - n)[:, None] + i
    seen = j[None, None, :] <= pos[..., None]
    if c["window"]:
        seen &= j[None, None, :] > pos[..., None] - c["window"]
    s = s.view(B, Hkv, G, NQ, W * P)
    s = torch.where(seen[:, None, None], s, float("-inf"))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == float("-inf"), 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, G * NQ, W * P), values(vc, vs)).view(B, Hkv, G, NQ, D)
    o = o / torch.where(total == 0.0, 1.0, total)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, NQ, Hq, D).to(torch.bfloat16)
    req = t["request"].long()
    return o[req, torch.arange(st["T"], device=DEV) - start[req]]


# -------------------------------------------------------------------------------------------- run
def run(state):
    op = state["case"]["op"]
    if own:
        import block_fp8_mixture_gb300 as moe
        if op == "tables":
            return moe.kv_tables(state["cur"], state["new"], state["table"], state["free"], state["count"],
                                 page_size=state["P"], out=moe.KVTables(**state["out"]))._asdict()
        t = moe.KVTables(**state["tables"])
        cache = moe.KVCache(*state["cache"])
        if op == "append":
            q = moe.rope_append(state["q"], state["k"], state["v"], state["rope"], t, cache,
                                layout=state["case"]["layout"], scale_fmt=state["case"]["fmt"],
                                q_out=state["q_out"])
        else:
            return moe.kv_attention(state["q"], cache, t.block_table, t.kv_len, t.tok_start,
                                    state["workspace"], max_q=state["max_q"],
                                    window=state["case"]["window"], out=state["out"])
    elif op == "tables":
        return _plain_tables(state)
    elif op == "append":
        q = _plain_append(state)
    else:
        return _plain_attend(state)
    kc, vc, ks, vs = state["cache"]
    return {"q": q, "k": kc.view(torch.float8_e4m3fn), "v": vc.view(torch.float8_e4m3fn), "k_scale": ks,
            "v_scale": vs}


# ------------------------------------------------------------------------------------------- work
def work(case):
    P, B = case["P"], case["B"]
    T, runs, width, pool = _sizes(case)
    ctx, new = _lengths(case)
    if case["op"] == "tables":
        # lengths, both tables, both stacks, three words a token, two a run
        return {"bytes": 4.0 * (5 * B + 2 * B * width + 2 * pool + 3 * T + 2 * runs + 8), "flops": 0}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "append":
        b = T * (Hq * D * 4 + 2 * Hkv * D * 3 + case["rot"] * 4 + 8) + runs * (8 + 8 * Hkv)
        return {"bytes": float(b), "flops": 3.0 * T * (Hq + Hkv) * case["rot"] + 4.0 * T * Hkv * D}
    w = case["window"]
    pairs = tokens = 0
    for c, l in zip(ctx, new):
        n = l - c
        full = n * c + n * (n + 1) // 2
        if w:
            # positions from c to l - 1 see min(position + 1, w) tokens
            short = max(0, min(l, w) - c)            # positions below w
            full = short * c + short * (short + 1) // 2 + (n - short) * w
            tokens += min(l, n + w - 1)
        else:
            tokens += l
        pairs += full
    b = tokens * Hkv * 2 * D + 8.0 * Hkv * tokens / P + 4 * T * Hq * D + 4 * (tokens // P + 2 * B)
    return {"bytes": float(b), "flops": 4.0 * D * Hq * pairs}


# ------------------------------------------------------------------------------------------ exact
def _exact_tables(st):
    P, T, R = st["P"], st["T"], st["runs"]
    cur, new = st["cur"].tolist(), st["new"].tolist()
    table, free, count = st["table"].tolist(), st["free"].tolist(), int(st["count"])
    B, W = len(table), len(table[0])
    out = {k: [] for k in ("kv_len", "slot", "position", "request", "run_tok", "run_len")}
    start, refused, rows = [0], 0, [list(r) for r in table]
    for i in range(B):                               # what is given up
        while rows[i] and len(rows[i]) > _pages(cur[i], P):
            rows[i].pop()
        gone = rows[i][_pages(new[i], P):]
        rows[i] = rows[i][:_pages(new[i], P)]
        for page in gone:
            free[count] = page
            count += 1
    need = [max(0, _pages(new[i], P) - _pages(cur[i], P)) for i in range(B)]
    total, fits = 0, []
    for i in range(B):
        total += need[i]
        fits.append(need[i] == 0 or total <= count)
    granted = sum(x for x, f in zip(need, fits) if f)
    top = free[count - granted:count]
    count -= granted
    for i in range(B):
        if fits[i]:
            rows[i] += [top.pop(0) for _ in range(need[i])]
        else:
            refused += 1
        out["kv_len"].append(new[i] if fits[i] else cur[i])
        last = None
        for pos in range(cur[i], new[i]):
            if fits[i] and pos // P != last:
                last = pos // P
                out["run_tok"].append(len(out["slot"]))
                out["run_len"].append(0)
            if fits[i]:
                out["run_len"][-1] += 1
            out["slot"].append(rows[i][pos // P] * P + pos % P if fits[i] else -1)
            out["position"].append(pos)
            out["request"].append(i)
        start.append(len(out["slot"]))
        rows[i] += [-1] * (W - len(rows[i]))
    info = [start[-1], len(out["run_tok"]), refused, granted]
    for k in ("run_tok", "run_len"):
        out[k] += [0] * (R - len(out[k]))
    out.update(block_table=rows, free_list=free, free_count=[count], tok_start=start, info=info)
    return {k: torch.tensor(v, dtype=torch.int32) for k, v in out.items()}


def _exact_append(case, st):
    P, fmt, rot = st["P"], case["fmt"], case["rot"]
    pos = st["tables"]["position"].double()
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    z = torch.polar(torch.ones_like(pos)[:, None] * torch.ones_like(inv), pos[:, None] * inv)[:, None]

    def turn(x):                                     # pairs as complex numbers
        x = x.double().clone()
        if case["layout"] == HALF:
            y = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * z
            x[..., :rot // 2], x[..., rot // 2:rot] = y.real, y.imag
        else:
            y = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * z
            x[..., 0:rot:2], x[..., 1:rot:2] = y.real, y.imag
        return x

    kc, vc, ks, vs = st["cache"]
    first, length = st["tables"]["run_tok"].tolist(), st["tables"]["run_len"].tolist()
    slots = st["tables"]["slot"].tolist()

    def q8(y):                                       # nearest E4M3 value, ties to even
        e = torch.frexp(y.abs().clamp_min(2.0 ** -6)).exponent.double()
        step = torch.exp2(e - 4)
        return (torch.round(y / step) * step).clamp(-448.0, 448.0)

    def f32(y):                                      # quotients are fp32 numbers by definition: many
        return y.float().double()                    # are ties between two codes, which go to even

    def write(x, codes, scale):
        val = codes.view(torch.float8_e4m3fn).double()
        sc = scale.double()
        for a, n in zip(first, length):
            if n:
                page, off = divmod(slots[a], P)
                xb = x[a:a + n].transpose(0, 1)
                s = (xb.abs().amax((1, 2)) / 448.0).clamp_min(1.0 / (448.0 * 512.0))
                if fmt == FMT_POW2:
                    m, e = torch.frexp(s)
                    s = torch.exp2(torch.where(m == 0.5, e - 1, e).double())
                s = f32(s)                           # a scale is the fp32 number that is stored
                if off:
                    s = torch.maximum(s, sc[page])
                    val[page, :, :off] = q8(f32(val[page, :, :off] * f32(sc[page] / s)[:, None, None]))
                val[page, :, off:off + n] = q8(f32(xb / s[:, None, None]))
                sc[page] = s
        return val, sc

    k, k_scale = write(turn(st["k"]), kc, ks)
    v, v_scale = write(st["v"].double(), vc, vs)
    return {"q": turn(st["q"]), "k": k, "v": v, "k_scale": k_scale, "v_scale": v_scale}


def _exact_attend(case, st):
    kc, vc, ks, vs = st["cache"]
    Hq, Hkv, D, P, w = case["Hq"], case["Hkv"], case["D"], case["P"], case["window"]
    G = Hq // Hkv
    kv, start = st["tables"]["kv_len"].tolist(), st["tables"]["tok_start"].tolist()
    out = torch.zeros((st["T"], Hq, D), dtype=torch.float64, device=DEV)
    for b, L in enumerate(kv):
        a, n = start[b], start[b + 1] - start[b]
        first = max(0, L - n - w + 1) // P if w else 0
        pages = st["tables"]["block_table"][b, first:_pages(L, P)].long()
        pos = torch.arange(L - n, L, device=DEV)[:, None]
        j = torch.arange(first * P, L, device=DEV)[None, :]
        hide = (j > pos) | ((j <= pos - w) if w else (j < 0))
        for h in range(Hkv):
            k, v = ((c[pages, h].view(torch.float8_e4m3fn).double() * s[pages, h].double()[:, None, None])
                    .reshape(-1, D)[:L - first * P] for c, s in ((kc, ks), (vc, vs)))
            q = st["q"][a:a + n, h * G:(h + 1) * G].double().transpose(0, 1)
            p = torch.softmax((q @ k.T / math.sqrt(D)).masked_fill_(hide, float("-inf")), -1)
            out[a:a + n, h * G:(h + 1) * G] = (p @ v).transpose(0, 1)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "tables":
        return _exact_tables(st)
    return _exact_append(case, st) if case["op"] == "append" else _exact_attend(case, st)
