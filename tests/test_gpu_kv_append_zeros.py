"""GPU: the codes of the 8-bit cache to the bit where the values are zeros of either sign, or become zero."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import block_fp8_mixture_gb300 as moe  # noqa: E402
import oracle  # noqa: E402
from oracle import kv_ref  # noqa: E402
from test_gpu_kv import dev, host, make_batch  # noqa: E402


@pytest.fixture(autouse=True)
def _library():
    moe.load_library(build_if_missing=True)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("P,D,ctx,add", [(16, 64, [0, 5, 15], [1, 1, 1]), (64, 128, [3, 60], [150, 70])])
def test_zeros_keep_their_sign(P, D, ctx, add, fmt):
    rng = np.random.default_rng(P + fmt)
    t, codes, scale, T = make_batch(rng, ctx, add, P, 2, D)
    if fmt:
        scale = oracle.pow2_ceil(scale)
    x = rng.choice([0.0, -0.0, 1.5, -2.0, 2.0 ** -100, -(2.0 ** -100)], (2, T, 2, D)).astype(np.float32)
    k, v = (torch.from_numpy(a).to(torch.bfloat16).cuda() for a in x)
    cache = moe.KVCache(*(dev(a) for a in (codes[0], codes[1], scale[0], scale[1])))
    moe.rope_append(None, k, v, None, t, cache, scale_fmt=fmt)
    h = host(t)
    for i in range(2):
        kv_ref.cache_write(x[i], codes[i], scale[i], h["slot"], h["run_tok"], h["run_len"], P, fmt)
        assert np.array_equal(cache[i].cpu().numpy(), codes[i]) and np.array_equal(cache[2 + i].cpu().numpy(), scale[i])
