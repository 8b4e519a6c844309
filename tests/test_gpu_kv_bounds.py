"""GPU: tables that hold anything at all.  What points outside is skipped, also where 32-bit sums wrap round."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import block_fp8_mixture_gb300 as moe  # noqa: E402
from test_gpu_kv import attention_case, dev  # noqa: E402

BIG = 2 ** 31 - 1


@pytest.fixture(autouse=True)
def _library():
    moe.load_library(build_if_missing=True)


@pytest.mark.parametrize("add", [1, 4])
def test_append_skips_runs_that_wrap_round(add):
    rng = np.random.default_rng(add)
    q, _, cache, _, _, t = attention_case(rng, [30, 5], [add, add], 16, 4, 2, 64)
    kv = q[:, :2]
    keep = [x.clone() for x in cache]
    for at in (BIG, BIG - 2, q.shape[0], -1, -BIG - 1):
        bad = t._replace(run_tok=torch.full_like(t.run_tok, at), run_len=torch.full_like(t.run_len, 16))
        moe.rope_append(None, kv, kv, None, bad, cache)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(cache, keep)), at


@pytest.mark.parametrize("max_q", [1, 8, 100])
@pytest.mark.parametrize("start", [[BIG, -BIG - 1, BIG], [BIG, -BIG, 0], [-1, 0, -BIG - 1], [1, -BIG - 1, BIG],
                                   [-BIG - 1, BIG, -5]])
def test_attention_skips_requests_that_wrap_round(start, max_q):
    rng = np.random.default_rng(max_q)
    q, _, cache, _, _, t = attention_case(rng, [30, 300], [max_q, max_q], 16, 4, 2, 64)
    ws = moe.alloc_kv_attention_workspace(4, 2, 64, max_q)
    out = torch.full_like(q, 7.0)
    for kv_len in (t.kv_len, dev(np.array([BIG, -BIG - 1], np.int32))):
        moe.kv_attention(q, cache, t.block_table, kv_len, dev(np.array(start, np.int64).astype(np.int32)), ws,
                         max_q=max_q, out=out)
        assert moe.last_device_status(ws) == moe.MOE_OK and bool((out == 7.0).all())
