"""GPU: steps of the paged 8-bit cache that add more tokens than the token list holds."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import block_fp8_mixture_gb300 as moe  # noqa: E402
from oracle import kv_ref  # noqa: E402
from test_gpu_kv import bf16, dev, random_state, run_tables  # noqa: E402


@pytest.fixture(autouse=True)
def _library():
    moe.load_library(build_if_missing=True)


@pytest.mark.parametrize("B,P,W,N", [(5, 16, 4, 30), (300, 32, 6, 900), (2000, 64, 3, 4000)])
@pytest.mark.parametrize("share", [0.0, 0.01, 0.5, 0.99, 1.0])
def test_tables_refuse_what_does_not_fit_the_token_list(B, P, W, N, share):
    rng = np.random.default_rng(B)
    cur, table, free, count = random_state(rng, B, P, W, N)
    kind = rng.integers(0, 4, B)
    new = np.where(kind == 0, 0, np.where(kind == 1, cur, np.minimum(cur + rng.integers(0, 40, B), W * P)))
    total = int(np.maximum(new - cur, 0).sum())
    T = int(total * share)
    got = run_tables(cur, new, table, free, count, P, T)
    ref = kv_ref.kv_tables(cur, new, table, free, count, P, T, got.run_tok.shape[0])
    assert share == 1.0 or ref["info"][2] > 0
    for name, t in got._asdict().items():
        assert np.array_equal(t.cpu().numpy(), ref[name]), name


def test_paged_attention_after_a_step_that_was_too_large():
    """A step of 24 + 20 + 20 tokens on a capacity of 32 takes the first request only; the steps after it add
    the others, and every row sees its own tokens and nothing else."""
    rng = np.random.default_rng(3)
    B, P, W, N, T, Hq, Hkv, D = 3, 16, 4, 12, 32, 4, 2, 64
    attn = moe.PagedAttention(num_layers=1, num_pages=N, page_size=P, num_heads=Hq, num_kv_heads=Hkv, head_dim=D,
                              max_requests=B, max_pages=W, max_tokens=T, max_q=T)
    for c in attn.caches[0]:                              # what earlier owners of the pages left
        c.copy_(torch.full_like(c, 0x7F) if c.dtype == torch.uint8 else torch.full_like(c, float("nan")))
    for new, lengths, refused in (([24, 20, 20], [24, 0, 0], 2), ([25, 20, 0], [25, 20, 0], 0),
                                  ([26, 21, 20], [26, 21, 20], 0)):
        t = attn.advance(dev(np.array(new, np.int32)))
        assert t.kv_len.tolist() == lengths and int(t.info[2]) == refused
        q, xq = bf16(rng, T, Hq, D)
        k, _ = bf16(rng, T, Hkv, D)
        v, _ = bf16(rng, T, Hkv, D)
        got = attn(0, q, k, v).float().cpu().numpy().astype(np.float64)
        assert moe.last_device_status(attn.workspace) == moe.MOE_OK
        c = [a.cpu().numpy() for a in attn.caches[0]]
        h = {n: a.cpu().numpy() for n, a in t._asdict().items()}
        live = h["slot"] >= 0
        start = np.minimum(h["tok_start"], live.sum())    # the requests that were taken come first
        want, mag = kv_ref.attention(xq, c[:2], c[2:], h["block_table"], h["kv_len"], start, D ** -0.5)
        assert np.isfinite(got[live]).all()
        assert (np.abs(got - want)[live] <= (2.0 ** -8 * np.abs(want) + 2.0 ** -9 * mag)[live]).all()
