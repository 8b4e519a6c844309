"""CPU statement of the paged 8-bit cache: tables by plain loops, the rotary write in the fp32 steps
that define it (bit for bit), attention in 64 bits."""

from __future__ import annotations

import numpy as np

from .formats import e4m3_decode, e4m3_encode
from .moe_ref import group_scale

F32 = np.float32


def pages(n, P):
    return -(-n // P)


def kv_tables(cur_len, new_len, block_table, free_list, free_count, P, max_tokens, max_runs):
    """One request after another: pages given up, pages granted, tokens, runs."""
    table = np.array(block_table, np.int64)
    free = [int(v) for v in free_list]
    B, W = table.shape
    cur = [min(max(int(c), 0), W * P) for c in cur_len]
    want = [max(int(n), 0) for n in new_len]
    count = min(max(int(free_count), 0), len(free))
    fits = [w <= W * P for w in want]
    for b in range(B):
        if fits[b]:
            for j in range(pages(want[b], P), pages(cur[b], P)):
                if count < len(free):
                    free[count] = int(table[b, j])
                count += 1
    needs = [max(0, pages(w, P) - pages(c, P)) if f else 0 for c, w, f in zip(cur, want, fits)]
    total, tokens, ok = 0, 0, []
    for b in range(B):
        total += needs[b]
        add = max(0, want[b] - cur[b]) if fits[b] else 0
        tokens += add
        ok.append(fits[b] and (needs[b] == 0 or total <= count) and (add == 0 or tokens <= max_tokens))
    granted = sum(n for n, o in zip(needs, ok) if o)
    top = free[count - granted:count]
    out = np.full((B, W), -1, np.int64)
    kv, start, slot, pos, req, run_tok, run_len = [], [0], [], [], [], [], []
    for b in range(B):
        held = [int(v) for v in table[b, :pages(cur[b], P)]]
        if ok[b]:
            held = held[:pages(want[b], P)]
            held += [top.pop(0) for _ in range(needs[b])]
        kv.append(want[b] if ok[b] else cur[b])
        out[b, :len(held)] = held
        last = -1
        for p in range(cur[b], want[b] if fits[b] else 0):
            if ok[b]:
                if p // P != last:
                    last = p // P
                    run_tok.append(len(slot))
                    run_len.append(0)
                run_len[-1] += 1
            slot.append(held[p // P] * P + p % P if ok[b] else -1)
            pos.append(p)
            req.append(b)
        start.append(len(slot))
    info = [len(slot), len(run_tok), sum(not o for o in ok), granted]

    def fit(v, n, fill):
        return np.array((v + [fill] * n)[:n], np.int32)

    return dict(block_table=out.astype(np.int32), free_list=np.array(free, np.int32),
                free_count=np.array([count - granted], np.int32), kv_len=np.array(kv, np.int32),
                tok_start=np.array(start, np.int32), slot=fit(slot, max_tokens, -1),
                position=fit(pos, max_tokens, 0), request=fit(req, max_tokens, -1),
                run_tok=fit(run_tok, max_runs, 0), run_len=fit(run_len, max_runs, 0),
                info=np.array(info, np.int32))


def rope_frequencies(rot, base=10000.0, scaling=0, factor=1.0, low=1.0, high=32.0, original_len=4096):
    f = float(base) ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if scaling == 1:
        f = f / factor
    if scaling == 2:
        w = np.clip((original_len * f / (2 * np.pi) - low) / (high - low), 0.0, 1.0)
        f = f * (w + (1 - w) / factor)
    return f


def rope_table(max_pos, rot, magnitude=1.0, **scaling):
    """float64 [max_pos, rot / 2, 2]"""
    a = np.arange(max_pos, dtype=np.float64)[:, None] * rope_frequencies(rot, **scaling)
    return magnitude * np.stack([np.cos(a), np.sin(a)], -1)


def rotate(x, rope, positions, layout):
    """x fp32 [T, H, D]; fp32 products and sums, each rounded."""
    x = np.array(x, F32)
    if rope is None:
        return x
    cs = np.asarray(rope, F32)[np.asarray(positions)][:, None]
    c, s = cs[..., 0], cs[..., 1]
    half = c.shape[-1]
    ia = slice(0, half) if layout == 0 else slice(0, 2 * half, 2)
    ib = slice(half, 2 * half) if layout == 0 else slice(1, 2 * half, 2)
    a, b = x[..., ia].copy(), x[..., ib].copy()
    x[..., ia] = a * c - b * s
    x[..., ib] = b * c + a * s
    return x


def cache_write(x, codes, scale, slot, run_tok, run_len, P, fmt):
    """x fp32 [T, Hkv, D] into codes uint8 [pages, Hkv, P, D] and scale fp32 [pages, Hkv], in place."""
    for t0, n in zip(run_tok, run_len):
        if n <= 0 or slot[t0] < 0:
            continue
        page, off = divmod(int(slot[t0]), P)
        for h in range(codes.shape[1]):
            rows = x[t0:t0 + n, h]
            s = group_scale(np.abs(rows).max().astype(F32), fmt)
            if off:
                was = F32(scale[page, h])
                s = max(F32(s), was)
                if s > was:
                    old = e4m3_decode(codes[page, h, :off]).astype(F32)
                    codes[page, h, :off] = e4m3_encode((old * F32(was / s)).astype(F32))
            codes[page, h, off:off + n] = e4m3_encode((rows / F32(s)).astype(F32))
            scale[page, h] = s


def attention(q, codes, scale, block_table, kv_len, tok_start, sm_scale, window=0):
    """q [T, Hq, D]; codes, scale: (K, V) pairs.  Returns out and sum_j p_j |v_j|, float64."""
    (kc, vc), (ks, vs) = codes, scale
    T, Hq, D = q.shape
    _, Hkv, P, _ = kc.shape
    G = Hq // Hkv
    out, mag = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    for b in range(len(kv_len)):
        L, a, n = int(kv_len[b]), int(tok_start[b]), int(tok_start[b + 1] - tok_start[b])
        if n == 0 or L == 0:
            continue
        ids = np.asarray(block_table[b, :pages(L, P)])
        pos = np.arange(L - n, L)[:, None]
        j = np.arange(L)[None, :]
        seen = j <= pos
        if window > 0:
            seen &= j > pos - window
        for h in range(Hkv):
            # tokens that no row sees may hold anything
            used = seen.any(0)[:, None]

            def values(c, s):
                x = e4m3_decode(c[ids, h]) * s[ids, h].astype(np.float64)[:, None, None]
                return np.where(used, x.reshape(-1, D)[:L], 0.0)

            k, v = values(kc, ks), values(vc, vs)
            for g in range(h * G, (h + 1) * G):
                s = np.where(seen, q[a:a + n, g].astype(np.float64) @ k.T * sm_scale, -np.inf)
                top = s.max(1, keepdims=True)
                p = np.exp(s - np.where(np.isinf(top), 0.0, top))
                total = p.sum(1, keepdims=True)
                p /= np.where(total == 0, 1.0, total)
                out[a:a + n, g] = p @ v
                mag[a:a + n, g] = p @ np.abs(v)
    return out, mag
