"""GPU: the paged cache's calls on a stream that is not torch's current one.  What they allocate has to belong
to that stream: memory of the current stream may be handed out again, or still be filled, while they run."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import block_fp8_mixture_gb300 as moe  # noqa: E402
from test_gpu_kv import bf16, dev, host  # noqa: E402


@pytest.fixture(autouse=True)
def _library():
    moe.load_library(build_if_missing=True)


class Handle:
    """A stream as other libraries hand it over."""

    def __init__(self, stream):
        self.cuda_stream = stream.cuda_stream


def owner(t):
    """The stream whose pool a tensor's memory is from."""
    p = t.data_ptr()
    return next(s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= p < s["address"] + s["total_size"])


@pytest.mark.parametrize("as_handle", [False, True])
def test_what_a_call_allocates_belongs_to_its_stream(monkeypatch, as_handle):
    rng = np.random.default_rng(1)
    B, P, W, N, T, Hq, Hkv, D = 3, 16, 4, 12, 40, 4, 2, 64
    attn = moe.PagedAttention(num_layers=1, num_pages=N, page_size=P, num_heads=Hq, num_kv_heads=Hkv, head_dim=D,
                              max_requests=B, max_pages=W, max_tokens=T, max_q=T, rope=moe.rope_table(W * P, D))
    twin = moe.PagedAttention(num_layers=1, num_pages=N, page_size=P, num_heads=Hq, num_kv_heads=Hkv, head_dim=D,
                              max_requests=B, max_pages=W, max_tokens=T, max_q=T, rope=attn.rope)
    q, k, v = (bf16(rng, T, h, D)[0] for h in (Hq, Hkv, Hkv))
    new = dev(np.array([20, 0, 13], np.int32))
    side = torch.cuda.Stream()
    s = Handle(side) if as_handle else side
    side.wait_stream(torch.cuda.current_stream())
    seen = []
    attention = moe.kv.kv_attention
    monkeypatch.setattr(moe.kv, "kv_attention", lambda q, *a, **kw: seen.append(owner(q)) or attention(q, *a, **kw))
    t = attn.advance(new, stream=s)
    got = attn(0, q, k, v, stream=s)
    assert seen == [side.cuda_stream] and owner(got) == side.cuda_stream
    rope = moe.rope_table(W * P, D, stream=s)
    more = moe.kv_tables(t.kv_len, new, t.block_table, t.free_list, t.free_count, page_size=P, max_tokens=8, stream=s)
    assert owner(rope) == side.cuda_stream and all(owner(x) == side.cuda_stream for x in more)
    side.synchronize()
    twin.advance(new)
    want = twin(0, q, k, v)
    assert torch.equal(got[:33], want[:33]) and torch.equal(rope, attn.rope)
    assert seen[1] == torch.cuda.current_stream().cuda_stream
    h = host(more)
    assert h["info"].tolist() == [0, 0, 0, 0] and np.array_equal(h["block_table"], host(t)["block_table"])
