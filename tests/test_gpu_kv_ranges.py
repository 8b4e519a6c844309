"""GPU: the paged 8-bit cache where its ranges end, against the CPU statement (oracle/kv_ref.py).  The bounds
are those of test_gpu_kv.py."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import block_fp8_mixture_gb300 as moe  # noqa: E402
from oracle import kv_ref  # noqa: E402
from test_gpu_kv import attention_case, check_attention, dev, host  # noqa: E402


@pytest.fixture(autouse=True)
def _library():
    moe.load_library(build_if_missing=True)


def device_cache(codes, scale):
    return moe.KVCache(*(dev(a) for a in (codes[0], codes[1], scale[0], scale[1])))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P,Hq,Hkv,add", [
    (16, 4, 2, 1), (32, 8, 1, 1), (64, 16, 1, 1), (16, 24, 1, 1), (32, 8, 2, 8), (16, 64, 1, 1), (32, 4, 2, 150),
])
@pytest.mark.parametrize("ratio", [-12, -20, -30, 25])
def test_attention_weight_on_a_page_with_another_v_scale(ratio, P, Hq, Hkv, add, D):
    """Even heads put all their weight on one page, odd ones on all others, and that page's V scale is
    2^ratio of the others'.  The scores of the two kinds of pages are 64 (D = 128: 90) apart in natural
    units: exp(-64) = 2^-92, so what is not meant adds nothing even at ratio -30."""
    rng = np.random.default_rng(P + Hq + D)
    L = 330
    q, xq, _, codes, scale, t = attention_case(rng, [L], [add], P, Hq, Hkv, D)
    table = host(t)["block_table"][0]
    page = table[kv_ref.pages(L, P) // 2]
    codes[0][page] = 0x38                                 # keys of the page: ones
    scale[0][page] = 1.0
    others = [x for x in table[:kv_ref.pages(L + add, P)] if x != page]
    scale[0][others] = 2.0 ** -20
    scale[1][others] = 2.0 ** -7
    scale[1][page] = 2.0 ** (ratio - 7)
    xq = np.full(xq.shape, 8.0, np.float32)
    xq[:, 1::2] = -8.0
    q = torch.from_numpy(xq).to(torch.bfloat16).cuda()
    check_attention(q, xq, device_cache(codes, scale), codes, scale, t, add)


@pytest.mark.parametrize("Hq,Hkv,max_q,n", [
    (8, 1, 1, [3, 1, 2]),                 # 8 rows: three tokens would not fit
    (8, 2, 2, [5, 1, 3]),
    (4, 4, 3, [4, 0, 9]),                 # 8 rows hold four tokens too
    (8, 1, 8, [20, 8, 9]),                # 64 rows
    (4, 2, 70, [150, 3, 71]),             # prompts with a short request among them
])
@pytest.mark.parametrize("window", [0, 40])
def test_attention_cuts_requests_to_max_q(Hq, Hkv, max_q, n, window):
    """The first max_q rows of a longer request are those of the whole request, the later ones are left as
    they were, and cached tokens that only those would see may hold anything."""
    rng = np.random.default_rng(Hq + max_q)
    D, P = 64, 16
    q, xq, _, codes, scale, t = attention_case(rng, [200, 30, 0], n, P, Hq, Hkv, D, extra_tokens=2)
    h = host(t)
    ref, mag = kv_ref.attention(xq, codes, scale, h["block_table"], h["kv_len"], h["tok_start"], D ** -0.5, window)
    keep = np.zeros(q.shape[0], bool)
    codes = codes.copy()
    for b, (m, L) in enumerate(zip(n, h["kv_len"])):
        a = h["tok_start"][b]
        keep[a:a + min(m, max_q)] = True
        for j in range(L - m + min(m, max_q), L):
            codes[:, h["block_table"][b, j // P], :, j % P] = 0x7F
    out = torch.full((q.shape[0], Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = moe.alloc_kv_attention_workspace(Hq, Hkv, D, max_q)
    moe.kv_attention(q, device_cache(codes, scale), t.block_table, t.kv_len, t.tok_start, ws, max_q=max_q,
                     window=window, out=out)
    assert moe.last_device_status(ws) == moe.MOE_OK
    got = out.float().cpu().numpy().astype(np.float64)
    assert (got[~keep] == 7.0).all()
    assert (np.abs(got - ref)[keep] <= (2.0 ** -8 * np.abs(ref) + 2.0 ** -9 * mag)[keep]).all()


@pytest.mark.parametrize("add", [1, 4, 130])
@pytest.mark.parametrize("which", [0, 1])
def test_attention_nan_scale_is_seen(which, add):
    """A page whose K or V scale is NaN: every row that sees a token of it is NaN, other requests are not."""
    rng = np.random.default_rng(add)
    P, Hq, Hkv, D = 32, 4, 2, 64
    q, xq, _, codes, scale, t = attention_case(rng, [300, 90], [add, add], P, Hq, Hkv, D)
    h = host(t)
    want = kv_ref.attention(xq, codes, scale, h["block_table"], h["kv_len"], h["tok_start"], D ** -0.5)
    scale = scale.copy()
    scale[which, h["block_table"][0, 3], 1] = np.nan          # head 1 of the first request
    ws = moe.alloc_kv_attention_workspace(Hq, Hkv, D, add)
    got = moe.kv_attention(q, device_cache(codes, scale), t.block_table, t.kv_len, t.tok_start, ws, max_q=add)
    g = got.float().cpu().numpy().astype(np.float64)
    assert np.isnan(g[:add, 2:]).all()
    ok = np.abs(g - want[0]) <= 2.0 ** -8 * np.abs(want[0]) + 2.0 ** -9 * want[1]
    assert ok[add:].all() and ok[:add, :2].all()


@pytest.mark.parametrize("pages", [(8, 15), (0, 29)])
@pytest.mark.parametrize("which", [0, 1])
def test_attention_nan_scales_in_parts_of_cut_blocks(which, pages):
    """Some or all of the tiles that a cut block sees have NaN scales.  A part of it that holds nothing else has
    no maximum; it must not be taken for one whose tokens the row does not see."""
    rng = np.random.default_rng(5)
    P, Hq, Hkv, D, add = 128, 8, 2, 128, 700
    q, _, _, codes, scale, t = attention_case(rng, [3000], [add], P, Hq, Hkv, D)
    scale = scale.copy()
    scale[which, host(t)["block_table"][0, slice(*pages)], 0] = np.nan
    ws = moe.alloc_kv_attention_workspace(Hq, Hkv, D, add)
    got = moe.kv_attention(q, device_cache(codes, scale), t.block_table, t.kv_len, t.tok_start, ws, max_q=add)
    assert torch.isnan(got[:, :4].float()).all() and torch.isfinite(got[:, 4:].float()).all()


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("k_exp", [0, -30])
@pytest.mark.parametrize("Hq,add", [(4, 1), (24, 1), (4, 130)])
def test_attention_query_that_is_not_finite(Hq, add, k_exp, value):
    """A row of q with an infinity or a NaN has no softmax: it is NaN, whatever the size of K, and no other row
    is touched."""
    rng = np.random.default_rng(Hq)
    D = 128
    q, _, _, codes, scale, t = attention_case(rng, [500], [add], 16, Hq, 1, D)
    scale = scale.copy()
    scale[0] *= 2.0 ** k_exp
    cache = device_cache(codes, scale)
    ws = moe.alloc_kv_attention_workspace(Hq, 1, D, add)
    call = lambda: moe.kv_attention(q, cache, t.block_table, t.kv_len, t.tok_start, ws, max_q=add)  # noqa: E731
    plain = call()
    q[add // 2, 1, 77] = value
    got = call()
    assert torch.isnan(got[add // 2, 1].float()).all()
    got[add // 2, 1] = plain[add // 2, 1]
    assert torch.equal(got, plain)


@pytest.mark.parametrize("value", [0.0, 2.0 ** -120])
@pytest.mark.parametrize("Hq,add", [(4, 1), (24, 1), (4, 130)])
def test_attention_of_queries_without_size(Hq, add, value):
    """Queries of zeros, or of values whose scores vanish: the mean of the values seen."""
    rng = np.random.default_rng(Hq)
    _, xq, cache, codes, scale, t = attention_case(rng, [500], [add], 16, Hq, 1, 128)
    xq = np.full(xq.shape, value, np.float32)
    check_attention(torch.from_numpy(xq).to(torch.bfloat16).cuda(), xq, cache, codes, scale, t, add)
