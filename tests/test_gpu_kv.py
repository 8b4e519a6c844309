"""GPU parity of the paged 8-bit cache against its CPU statement (oracle/kv_ref.py).

Tables, codes and scales are compared bit for bit (the oracle takes the same fp32 steps); the rotated
queries too.  Attention outputs: |gpu - ref| <= 2^-8 |ref| + 2^-9 sum_j p_j |v_j|.  The first term is
the BF16 rounding of the result (2^-9) with room for fp32 sums; the second covers a relative error of
each probability of at most 2^-9: its rounding for the matrix product (2^-11), the ratio of the pages'
scales (2^-11), and a score error of 2^-11 (the query's split into E4M3 terms, 2^-17 of its largest
value times sum |k| sm_scale <= 100, and fp32 sums).
"""

import numpy as np
import pytest

import oracle
from oracle import kv_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import block_fp8_mixture_gb300 as moe  # noqa: E402


@pytest.fixture(autouse=True)
def _library():
    moe.load_library(build_if_missing=True)


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def bf16(rng, *shape):
    """Random BF16 values as (device tensor, the same values in fp32)."""
    x = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16)
    return x.cuda(), x.float().numpy()


# ------------------------------------------------------------------------------------------ tables
def random_state(rng, B, P, W, N):
    """A table whose requests hold what their lengths need, the rest of the pool on the stack."""
    ids = rng.permutation(N)
    cur = np.zeros(B, np.int64)
    table = np.full((B, W), -1, np.int32)
    at = 0
    for b in range(B):
        n = int(rng.integers(0, W * P + 1))
        if at + kv_ref.pages(n, P) > N:
            n = 0
        k = kv_ref.pages(n, P)
        table[b, :k] = ids[at:at + k]
        cur[b], at = n, at + k
    free = rng.integers(0, N, N).astype(np.int32)       # entries past the count hold anything
    free[:N - at] = ids[at:]
    return cur.astype(np.int32), table, free, N - at


def run_tables(cur, new, table, free, count, P, T, R=None):
    B, W = table.shape
    out = moe.alloc_kv_tables(B, W, len(free), P, T)
    if R is not None:
        out = out._replace(run_tok=torch.full((R,), 77, dtype=torch.int32, device="cuda"),
                           run_len=torch.full((R,), 77, dtype=torch.int32, device="cuda"))
    for t in out:
        t.fill_(-77)
    ins = [dev(np.asarray(v, np.int32)) for v in (cur, new, table, free, [count])]
    keep = [t.clone() for t in ins]
    got = moe.kv_tables(*ins, page_size=P, out=out)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ins, keep))
    return got


@pytest.mark.parametrize("B,P,W,N,grow", [
    (1, 16, 1, 1, 16), (1, 128, 5, 8, 200), (7, 16, 9, 60, 30), (33, 64, 12, 300, 100),
    (513, 32, 6, 2000, 40), (1024, 16, 20, 12000, 3), (2500, 16, 3, 4000, 20), (4096, 64, 2, 5000, 64),
])
def test_tables_match_the_oracle(B, P, W, N, grow):
    rng = np.random.default_rng(B * 1000 + P)
    cur, table, free, count = random_state(rng, B, P, W, N)
    kind = rng.integers(0, 4, B)
    new = np.where(kind == 0, 0, np.where(kind == 1, np.maximum(cur - rng.integers(0, 9, B), 0),
                                          np.minimum(cur + rng.integers(0, grow + 1, B), W * P)))
    T = int(np.maximum(new - cur, 0).sum()) + 3
    got = run_tables(cur, new, table, free, count, P, T)
    ref = kv_ref.kv_tables(cur, new, table, free, count, P, T, got.run_tok.shape[0])
    for name, t in got._asdict().items():
        assert np.array_equal(t.cpu().numpy(), ref[name]), name


def test_tables_short_pool_bad_lengths_and_small_capacities():
    rng = np.random.default_rng(1)
    P, B, W, N = 16, 40, 6, 90
    cur, table, free, count = random_state(rng, B, P, W, N)
    new = np.minimum(cur + 40, W * P).astype(np.int64)
    new[5], new[9], new[11] = W * P + 1, -4, 2 ** 31 - 1     # too long, negative, far too long
    cur = cur.copy()
    cur[20] = -3                                             # clamped
    table[20] = -1
    new[20] = 7
    total = int(sum(max(0, n - max(c, 0)) for c, n in zip(cur, new) if n <= W * P))
    for T, R in ((total, 200), (total // 2, 3), (0, 0)):
        got = run_tables(cur, new, table, free, count, P, T, R)
        ref = kv_ref.kv_tables(cur, new, table, free, count, P, T, R)
        assert ref["info"][2] > 3                            # the pool ran out too
        for name, t in got._asdict().items():
            assert np.array_equal(t.cpu().numpy(), ref[name]), name


def test_tables_growing_and_giving_back_restores_the_stack():
    P, B, W, N = 32, 20, 10, 220
    free = np.random.default_rng(0).permutation(N).astype(np.int32)
    zero, want = np.zeros(B, np.int32), np.arange(B, dtype=np.int32) * 16
    a = run_tables(zero, want, np.full((B, W), -1, np.int32), free, N, P, int(want.sum()))
    b = moe.kv_tables(a.kv_len, dev(zero), a.block_table, a.free_list, a.free_count, page_size=P, max_tokens=4)
    assert np.array_equal(b.free_list.cpu().numpy(), free) and int(b.free_count) == N
    assert int(b.block_table.max()) == -1 and int(b.tok_start.abs().max()) == 0


# -------------------------------------------------------------------------------------------- rope
@pytest.mark.parametrize("kw", [
    {}, dict(base=500000.0), dict(scaling=1, factor=4.0), dict(magnitude=1.25),
    dict(scaling=2, factor=8.0, low=1.0, high=4.0, original_len=8192),
])
@pytest.mark.parametrize("max_pos,rot", [(1, 16), (77, 128), (70000, 64)])
def test_rope_table(max_pos, rot, kw):
    got = moe.rope_table(max_pos, rot, **kw).cpu().numpy()
    ref = kv_ref.rope_table(max_pos, rot, **kw)
    # one rounding to fp32, half a unit in the last place of each value, and the angle's error in 64
    # bits: 2^-52 of angles below 2^17
    assert (np.abs(got - ref) <= 0.5 * np.spacing(np.abs(ref).astype(np.float32)) + 2.0 ** -34).all()


# ------------------------------------------------------------------------------------------ append
def make_batch(rng, ctx, add, P, Hkv, D, extra_tokens=0, spare=3):
    """Tables of a step that takes requests from ctx to ctx + add tokens, with a random cache."""
    ctx, add = np.asarray(ctx, np.int32), np.asarray(add, np.int32)
    B, W = len(ctx), int(kv_ref.pages((ctx + add).max(), P)) + 1
    N = int(sum(kv_ref.pages(int(c + a), P) for c, a in zip(ctx, add))) + spare
    ids = rng.permutation(N).astype(np.int32)
    table = np.full((B, W), -1, np.int32)
    at = 0
    for b in range(B):
        k = kv_ref.pages(int(ctx[b]), P)
        table[b, :k] = ids[at:at + k]
        at += k
    free = np.zeros(N, np.int32)
    free[:N - at] = ids[at:]
    T = int(add.sum()) + extra_tokens
    t = moe.kv_tables(dev(ctx), dev(ctx + add), dev(table), dev(free), dev(np.array([N - at], np.int32)),
                      page_size=P, max_tokens=T)
    x = rng.standard_normal((2, N, Hkv, P, D)).astype(np.float32) * 1.5
    scale = (np.abs(x).max((3, 4)) / 448).astype(np.float32)
    codes = oracle.e4m3_encode((x / scale[..., None, None]).astype(np.float32))
    return t, codes, scale, T


def host(t):
    return {k: v.cpu().numpy() for k, v in t._asdict().items()}


@pytest.mark.parametrize("layout", [moe.ROPE_HALF, moe.ROPE_INTERLEAVED])
@pytest.mark.parametrize("P,D,Hq,Hkv,rot,fmt,ctx,add", [
    (16, 128, 8, 2, 128, 0, [0, 5, 31, 32, 100], [1, 1, 1, 1, 1]),
    (16, 64, 3, 3, 32, 1, [0, 15, 16, 40], [17, 1, 33, 5]),
    (32, 128, 5, 1, 64, 1, [7, 0, 63], [100, 32, 1]),
    (64, 128, 4, 4, 128, 0, [0, 63, 64, 200, 10], [64, 1, 65, 3, 300]),
    (64, 64, 4, 2, 16, 0, [9], [500]),
    (128, 128, 2, 1, 128, 1, [0, 100, 127, 5], [128, 200, 2, 1]),
    (128, 64, 2, 2, 64, 0, [3, 250], [126, 7]),
])
def test_append_matches_the_oracle(P, D, Hq, Hkv, rot, fmt, ctx, add, layout):
    rng = np.random.default_rng(P + D + rot + layout)
    t, codes, scale, T = make_batch(rng, ctx, add, P, Hkv, D, extra_tokens=2)
    # half of the old scales small enough that the step has to raise them
    scale[:, ::2] /= 4
    if fmt:
        scale = oracle.pow2_ceil(scale)
    qkv, x = bf16(rng, T, (Hq + 2 * Hkv) * D)
    q, k, v = (a.unflatten(1, (-1, D)) for a in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
    xq, xk, xv = (a.reshape(T, -1, D) for a in np.split(x, [Hq * D, (Hq + Hkv) * D], 1))
    rope = moe.rope_table(1024, rot)
    cache = moe.KVCache(*(dev(a) for a in (codes[0], codes[1], scale[0], scale[1])))
    got = moe.rope_append(q, k, v, rope, t, cache, layout=layout, scale_fmt=fmt)
    h = host(t)
    cs = rope.cpu().numpy()
    rq = kv_ref.rotate(xq, cs, h["position"], layout)
    kv_ref.cache_write(kv_ref.rotate(xk, cs, h["position"], layout), codes[0], scale[0], h["slot"],
                       h["run_tok"], h["run_len"], P, fmt)
    kv_ref.cache_write(xv, codes[1], scale[1], h["slot"], h["run_tok"], h["run_len"], P, fmt)
    assert np.array_equal(got.float().cpu().numpy(), oracle.bf16_round(rq))
    for name, a, b in (("k_codes", cache.k_codes, codes[0]), ("v_codes", cache.v_codes, codes[1]),
                       ("k_scale", cache.k_scale, scale[0]), ("v_scale", cache.v_scale, scale[1])):
        assert np.array_equal(a.cpu().numpy(), b), name


def test_append_variants():
    """No rotation; q in place; cache write only; refused requests and padding write nothing."""
    rng = np.random.default_rng(0)
    P, D, Hkv = 16, 64, 2
    t, codes, scale, T = make_batch(rng, [3, 20], [5, 2], P, Hkv, D, extra_tokens=4)
    q, xq = bf16(rng, T, 3, D)
    k, xk = bf16(rng, T, Hkv, D)
    fresh = lambda: moe.KVCache(*(dev(a) for a in (codes[0], codes[1], scale[0], scale[1])))  # noqa: E731
    a, b = fresh(), fresh()
    assert torch.equal(moe.rope_append(q, k, k, None, t, a), q)
    assert moe.rope_append(None, k, k, None, t, b) is None
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    rope = moe.rope_table(64, 32)
    want = moe.rope_append(q, k, k, rope, t, fresh())
    mine = q.clone()
    assert moe.rope_append(mine, k, k, rope, t, fresh(), q_out=mine) is mine and torch.equal(mine, want)
    c = fresh()
    nothing = t._replace(slot=torch.full_like(t.slot, -1))
    moe.rope_append(None, k, k, rope, nothing, c)
    assert all(torch.equal(x, y) for x, y in zip(c, fresh()))
    # runs and slots that point outside are skipped
    far = t._replace(run_tok=torch.full_like(t.run_tok, T), slot=torch.full_like(t.slot, 1 << 30))
    moe.rope_append(None, k, k, rope, far, c)
    moe.rope_append(None, k, k, rope, t._replace(slot=far.slot), c)
    assert all(torch.equal(x, y) for x, y in zip(c, fresh()))


def test_append_extreme_values():
    """Zeros get the scale's floor; an infinity saturates; a NaN stays a NaN and leaves the scale alone."""
    rng = np.random.default_rng(2)
    P, D = 16, 64
    t, codes, scale, T = make_batch(rng, [0, 0, 0], [2, 2, 2], P, 1, D)
    x = torch.zeros((T, 1, D), dtype=torch.bfloat16, device="cuda")
    x[2:] = 3.5
    x[2, 0, 5], x[4, 0, 7] = float("nan"), float("inf")
    cache = moe.KVCache(*(dev(a) for a in (codes[0], codes[1], scale[0], scale[1])))
    moe.rope_append(None, x, x, None, t, cache)
    page = [int(t.block_table[b, 0]) for b in range(3)]
    val = cache.v_codes.view(torch.float8_e4m3fn).float().cpu().numpy()
    s = cache.v_scale.cpu().numpy()
    assert s[page[0], 0] == np.float32(1.0 / 229376.0) and (val[page[0], 0, :2] == 0).all()
    assert s[page[1], 0] == np.float32(3.5) / np.float32(448) and np.isnan(val[page[1], 0, 0, 5])
    assert np.isnan(val[page[1], 0, :2]).sum() == 1 and val[page[1], 0, 1, 0] == 448
    assert np.isinf(s[page[2], 0])


# --------------------------------------------------------------------------------------- attention
def check_attention(q, xq, cache, codes, scale, t, max_q, window=0, sm_scale=None, ws=None, out=None, what=""):
    Hq, D = xq.shape[1:]
    Hkv = codes[0].shape[1]
    if ws is None:
        ws = moe.alloc_kv_attention_workspace(Hq, Hkv, D, max_q)
    got = moe.kv_attention(q, cache, t.block_table, t.kv_len, t.tok_start, ws, max_q=max_q, window=window,
                           sm_scale=sm_scale, out=out)
    assert moe.last_device_status(ws) == moe.MOE_OK
    h = host(t)
    ref, mag = kv_ref.attention(xq, codes, scale, h["block_table"], h["kv_len"], h["tok_start"],
                                D ** -0.5 if sm_scale is None else sm_scale, window)
    n = int(h["tok_start"][-1])
    g = got.float().cpu().numpy()[:n].astype(np.float64)
    err = np.abs(g - ref[:n]) - (2.0 ** -8 * np.abs(ref[:n]) + 2.0 ** -9 * mag[:n])
    assert np.isfinite(g).all(), what
    assert err.max(initial=-1) <= 0, f"{what}: {np.argwhere(err > 0)[:4]} of {err.shape}, by {err.max()}"
    return got


def attention_case(rng, ctx, add, P, Hq, Hkv, D, extra_tokens=0, poison=True):
    t, codes, scale, T = make_batch(rng, ctx, add, P, Hkv, D, extra_tokens)
    if poison:
        # everything that no request holds is NaN: other pages, rows past the end of the last page
        live = np.zeros((codes.shape[1], P), bool)
        h = host(t)
        for b, n in enumerate(h["kv_len"]):
            for j in range(n):
                live[h["block_table"][b, j // P], j % P] = True
        codes = np.where(live[None, :, None, :, None], codes, np.uint8(0x7F))
        scale = np.where(live.any(1)[None, :, None], scale, np.float32(np.nan))
    q, xq = bf16(rng, T, Hq, D)
    cache = moe.KVCache(*(dev(a) for a in (codes[0], codes[1], scale[0], scale[1])))
    return q, xq, cache, codes, scale, t


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P,Hq,Hkv,ctx,add", [
    (16, 8, 1, [0, 1, 14, 15, 16, 130], [1] * 6),              # one token to a few tiles
    (16, 5, 1, [127, 128, 129, 255, 256, 700], [1] * 6),       # odd group, around the tiles' edges
    (32, 4, 4, [50, 1000, 3], [1, 1, 1]),                      # no shared heads
    (64, 16, 2, [2049], [1]),                                  # one request, split over the cache
    (128, 32, 2, [300, 4000], [1, 1]),                         # 16 heads a group
    (16, 24, 1, [10, 900], [1, 1]),                            # 24 rows
    (64, 64, 1, [77, 1500], [1, 1]),                           # 64 rows
    (16, 4, 2, [0, 9, 120, 500], [3, 5, 8, 2]),                # several tokens a request
    (32, 8, 1, [0, 40, 1000], [4, 1, 8]),                      # 64 rows of 8 tokens
])
def test_attention_few_rows(P, Hq, Hkv, ctx, add, D):
    rng = np.random.default_rng(P * 10 + Hq + D)
    case = attention_case(rng, ctx, add, P, Hq, Hkv, D, extra_tokens=1)
    check_attention(*case, max_q=max(add))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P,Hq,Hkv,ctx,add", [
    (16, 2, 2, [0], [129]),
    (16, 4, 1, [0, 0, 0, 0], [1, 127, 128, 300]),              # prompts with a single token among them
    (64, 6, 2, [1000, 0, 63], [70, 200, 129]),                 # chunks after a context
    (128, 3, 1, [250], [515]),
    (32, 8, 1, [5, 2000, 600], [100, 1, 2]),                   # chunks and single tokens in one call
    (64, 40, 1, [0, 100], [30, 11]),                           # 40 heads a group
])
@pytest.mark.parametrize("window", [0, 100])
def test_attention_prompts(P, Hq, Hkv, ctx, add, D, window):
    rng = np.random.default_rng(P * 10 + Hq + D)
    case = attention_case(rng, ctx, add, P, Hq, Hkv, D, extra_tokens=1)
    check_attention(*case, max_q=max(add), window=window)


@pytest.mark.parametrize("window", [1, 2, 17, 128, 1000, 5000])
@pytest.mark.parametrize("add", [1, 4])
def test_attention_window(window, add):
    rng = np.random.default_rng(window)
    case = attention_case(rng, [0, 5, 127, 1111, 3000], [add] * 5, 16, 4, 2, 128)
    check_attention(*case, max_q=add, window=window)


def test_attention_window_reads_nothing_before_it():
    """Pages that lie wholly before the window have been given away: their table entries are -1 or
    point to pages full of NaN."""
    rng = np.random.default_rng(9)
    for add in (1, 200):
        q, xq, cache, codes, scale, t = attention_case(rng, [1500], [add], 16, 4, 2, 64)
        first = (1500 - 100 + 1) // 16
        table = t.block_table.clone()
        gone = table[0, :first].cpu().numpy()
        codes[:, gone] = 0x7F
        scale[:, gone] = np.nan
        cache = moe.KVCache(*(dev(a) for a in (codes[0], codes[1], scale[0], scale[1])))
        table[0, :first:2] = -1
        ref = host(t)
        ws = moe.alloc_kv_attention_workspace(4, 2, 64, add)
        got = moe.kv_attention(q, cache, table, t.kv_len, t.tok_start, ws, max_q=add, window=100)
        want, mag = kv_ref.attention(xq, codes, scale, ref["block_table"], ref["kv_len"], ref["tok_start"],
                                     0.125, 100)
        g = got.float().cpu().numpy()
        assert np.isfinite(g).all()
        assert (np.abs(g - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * mag).all()


@pytest.mark.parametrize("max_q", [1, 200])
def test_attention_empty_rows(max_q):
    """kv_len 0, kv_len below the number of query tokens, requests without query tokens: rows that see
    nothing are zero, rows past the tokens are left alone."""
    rng = np.random.default_rng(4)
    n = np.array([1, 0, 1, 1] if max_q == 1 else [200, 0, 5, 150], np.int32)
    q, xq, cache, codes, scale, t = attention_case(rng, [0, 40, 0, 33], n, 16, 4, 2, 128, extra_tokens=3)
    kv = t.kv_len.clone()
    kv[0] = 0 if max_q == 1 else 90
    kv[2] = 0
    t = t._replace(kv_len=kv)
    out = torch.full((q.shape[0], 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    got = check_attention(q, xq, cache, codes, scale, t, max_q, out=out)
    assert (got[int(n.sum()):] == 7.0).all()
    start = t.tok_start.cpu().tolist()
    assert (got[start[2]:start[3]] == 0).all()
    if max_q > 1:
        assert (got[:110] == 0).all()


@pytest.mark.parametrize("add", [1, 130])
def test_attention_strides_stream_and_repeats(add):
    """Query heads inside a fused projection, an output with padding between tokens, another stream, a
    captured graph, the same bits on every call."""
    rng = np.random.default_rng(6)
    q, xq, cache, codes, scale, t = attention_case(rng, [70, 500], [add, add], 32, 6, 2, 64)
    T = q.shape[0]
    fused = torch.zeros((T, 10, 64), dtype=torch.bfloat16, device="cuda")
    fused[:, 2:8] = q
    wide = torch.zeros((T, 8, 64), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = check_attention(fused[:, 2:8], xq, cache, codes, scale, t, add, out=wide[:, 1:7])
    torch.cuda.synchronize()
    assert (wide[:, 0] == 0).all() and (wide[:, 7] == 0).all()
    ws = moe.alloc_kv_attention_workspace(6, 2, 64, add)
    out = torch.empty_like(q)
    call = lambda: moe.kv_attention(q, cache, t.block_table, t.kv_len, t.tok_start, ws, max_q=add, out=out)  # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, a)


@pytest.mark.parametrize("add", [1, 150])
def test_attention_wide_ranges(add):
    """A sink token far above a long tail, scores far apart, page scales that differ by 2^20, a large
    softmax scale: the running maximum, the probabilities' range and the scales' ratios at their ends."""
    rng = np.random.default_rng(8)
    P, D, L = 16, 128, 6000
    for kind in ("sink", "spread", "scales", "sharp"):
        q, xq, cache, codes, scale, t = attention_case(rng, [L], [add], P, 4, 2, D, poison=False)
        table = host(t)["block_table"][0]
        if kind == "sink":                       # token 37 scores about 11 above the others
            codes[0, table[37 // P], :, 37 % P] = 0x38
            scale[0, table[37 // P]] = 1.0
            scale[0, table[:37 // P]] = scale[0, table[37 // P + 1:]] = 1e-4
            x = np.abs(xq) * 0.15
            q = torch.from_numpy(x).to(torch.bfloat16).cuda()
            xq = q.float().cpu().numpy()
        if kind == "scales":
            scale[1] = np.exp2(rng.integers(-20, 1, scale[1].shape)).astype(np.float32) / 100
        cache = moe.KVCache(*(dev(a) for a in (codes[0], codes[1], scale[0], scale[1])))
        sm = dict(spread=0.5, sharp=4.0).get(kind)
        if kind == "sharp":                      # scores over +-1000: the largest token decides
            x = np.sign(xq)
            q = torch.from_numpy(x).to(torch.bfloat16).cuda()
            xq = x
        check_attention(q, xq, cache, codes, scale, t, add, sm_scale=sm, what=kind)


def test_attention_many_requests_and_long_cache():
    rng = np.random.default_rng(11)
    ctx = rng.integers(0, 260, 300)
    case = attention_case(rng, ctx, [1] * 300, 16, 4, 1, 64)
    check_attention(*case, max_q=1)
    case = attention_case(rng, [70001], [1], 128, 2, 1, 64, poison=False)
    check_attention(*case, max_q=1)


@pytest.mark.parametrize("Hq,Hkv,D,ctx,add", [
    (3, 1, 128, [12000], [1]),               # 3 rows, about 95 parts
    (8, 1, 128, [9000, 21000], [1, 1]),      # 8 rows, items that start inside a group of parts
    (16, 1, 64, [17000], [1]),               # 16 rows
    (12, 2, 128, [9000, 30], [3, 2]),        # 18 rows: two sets of 16
    (64, 1, 64, [13000], [1]),               # 64 rows
    (5, 1, 64, [700, 24000, 10, 8000], [1, 0, 1, 2]),
])
def test_attention_long_items_are_joined_in_two_steps(Hq, Hkv, D, ctx, add):
    """Items whose parts are more than one step of additions takes; the counters must be back at zero
    after each call and the order of the additions fixed, so a second call repeats the first."""
    rng = np.random.default_rng(Hq + D)
    case = attention_case(rng, ctx, add, 32, Hq, Hkv, D, poison=False)
    ws = moe.alloc_kv_attention_workspace(Hq, Hkv, D, max(add))
    first = check_attention(*case, max_q=max(add), ws=ws).clone()
    assert torch.equal(check_attention(*case, max_q=max(add), ws=ws), first)


@pytest.mark.parametrize("D,P,Hq,Hkv,ctx,add,window", [
    (128, 64, 8, 2, [3000, 0, 40], [700, 130, 1], 0),      # fewer blocks than pairs, each over several of them
    (64, 16, 64, 8, [2000], [1000], 0),                    # one round of whole blocks, a last one poured over pairs
    (128, 32, 64, 8, [1800, 100], [700, 450], 0),          # unequal loads before the last round
    (64, 32, 3, 3, [6000, 5000], [300, 200], 0),           # parts that some rows do not see
    (128, 16, 4, 1, [0] * 90 + [1900], [140] * 90 + [200], 300),   # short blocks, odd rounds, not poured
    (128, 128, 40, 8, [0], [900], 0),
])
def test_attention_prompts_shared_by_pairs(D, P, Hq, Hkv, ctx, add, window):
    rng = np.random.default_rng(P + Hq)
    case = attention_case(rng, ctx, add, P, Hq, Hkv, D, extra_tokens=3)
    first = check_attention(*case, max_q=max(add), window=window).clone()
    again = moe.kv_attention(case[0], case[2], case[5].block_table, case[5].kv_len, case[5].tok_start,
                             moe.alloc_kv_attention_workspace(Hq, Hkv, D, max(add)), max_q=max(add), window=window)
    n = sum(add)
    assert torch.equal(again[:n], first[:n])


def test_attention_one_workspace_for_all_row_counts():
    """A workspace for the largest max_q serves calls with any smaller one, in any order: what one variant
    leaves behind must not be another's counters."""
    rng = np.random.default_rng(31)
    Hq, Hkv, D, P = 8, 1, 64, 32
    ws = moe.alloc_kv_attention_workspace(Hq, Hkv, D, 300)
    cases = {n: attention_case(rng, [9000, 700], [n, 1], P, Hq, Hkv, D, poison=False) for n in (1, 2, 4, 8, 300)}
    first = {}
    for n in (1, 8, 1, 4, 1, 2, 300, 1, 300, 8, 2, 4, 1):
        if n not in first:
            first[n] = check_attention(*cases[n], max_q=n, ws=ws, what=n).clone()
        else:
            q, _, cache, _, _, t = cases[n]
            got = moe.kv_attention(q, cache, t.block_table, t.kv_len, t.tok_start, ws, max_q=n)
            assert torch.equal(got, first[n]), n


# ------------------------------------------------------------------------------- the pieces together
def test_paged_attention_over_steps():
    """PagedAttention over steps that add, finish, refill and roll back requests, on two layers: every
    step's attention against the CPU statement over the cache as the library left it, and the tables
    against theirs."""
    rng = np.random.default_rng(21)
    B, P, W, N, T, Hq, Hkv, D = 4, 16, 8, 20, 150, 4, 2, 64
    attn = moe.PagedAttention(num_layers=2, num_pages=N, page_size=P, num_heads=Hq, num_kv_heads=Hkv, head_dim=D,
                              max_requests=B, max_pages=W, max_tokens=T, max_q=T, rope=moe.rope_table(W * P, D),
                              scale_fmt=moe.SCALE_FP32_POW2)
    held = dict(block_table=np.full((B, W), -1), free_list=np.arange(N), free_count=[N], kv_len=np.zeros(B, int))
    for new in ([90, 0, 20, 1], [91, 30, 21, 2], [92, 31, 0, 3], [85, 32, 100, 4], [86, 0, 101, 120], [87, 5, 102, 0]):
        t = attn.advance(dev(np.array(new, np.int32)))
        ref = kv_ref.kv_tables(held["kv_len"], new, held["block_table"], held["free_list"], held["free_count"][0],
                               P, T, t.run_tok.shape[0])
        for name, x in t._asdict().items():
            assert np.array_equal(x.cpu().numpy(), ref[name]), name
        held = ref
        for layer in range(2):
            qkv, x = bf16(rng, T, (Hq + 2 * Hkv) * D)
            q, k, v = (a.unflatten(1, (-1, D)) for a in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
            got = attn(layer, q, k, v).float().cpu().numpy().astype(np.float64)
            assert moe.last_device_status(attn.workspace) == moe.MOE_OK
            c = attn.caches[layer]
            xq = oracle.bf16_round(kv_ref.rotate(np.split(x, [Hq * D], 1)[0].reshape(T, Hq, D), attn.rope.cpu().numpy(),
                                                 ref["position"], 0))
            want, mag = kv_ref.attention(xq, [a.cpu().numpy() for a in c[:2]], [a.cpu().numpy() for a in c[2:]],
                                         ref["block_table"], ref["kv_len"], ref["tok_start"], D ** -0.5)
            # a refused request's rows stand at positions that it does not hold: the caller drops them
            n = int(ref["tok_start"][-1])
            keep = ref["slot"][:n] >= 0
            err = np.abs(got[:n] - want[:n]) - (2.0 ** -8 * np.abs(want[:n]) + 2.0 ** -9 * mag[:n])
            assert err[keep].max(initial=-1) <= 0


def test_decoder_block_example():
    """The example runs, and the 8-bit cache stays near unquantized attention: a code is within 2^-4 of its
    value (half a unit in the last of 4 bits), so keys move scores by at most 2^-4 sum |q k| sm_scale (below
    0.2 here, 0.05 rms) and values move the output by 2^-4 / sqrt(3) rms relative: 0.1 bounds both."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_block.py")
    spec = importlib.util.spec_from_file_location("decoder_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    assert mod.main(seed=3, verbose=False) < 0.1
