"""GPU: each argument of the paged cache's binding in host memory, all others on the device: refused."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import block_fp8_mixture_gb300 as moe  # noqa: E402


@pytest.fixture(autouse=True)
def _library():
    moe.load_library(build_if_missing=True)


def refused(call):
    with pytest.raises(moe.MoeError) as e:
        call()
    assert e.value.status == moe.MOE_ERR_INVALID_ARG


def each_on_the_host(args):
    for i in range(len(args)):
        yield [a.cpu() if i == j else a for j, a in enumerate(args)]


def test_one_argument_on_the_host_is_refused():
    B, W, N, P, T = 2, 4, 6, 16, 8
    t, out = moe.alloc_kv_tables(B, W, N, P, T), moe.alloc_kv_tables(B, W, N, P, T)
    first = [t.kv_len, torch.zeros_like(t.kv_len), t.block_table, t.free_list, t.free_count]
    for ins in each_on_the_host(first):
        refused(lambda: moe.kv_tables(*ins, page_size=P, out=out))
    for outs in each_on_the_host(list(out)):
        refused(lambda: moe.kv_tables(*first, page_size=P, out=moe.KVTables(*outs)))
    cache = moe.alloc_kv_cache(N, 2, P, 64)
    q = torch.zeros(T, 4, 64, dtype=torch.bfloat16, device="cuda")
    kv = q[:, :2]
    rope = moe.rope_table(W * P, 64)
    used = [t.position, t.slot, t.run_tok, t.run_len]
    for x in each_on_the_host([q, kv, kv, rope, torch.empty_like(q), *used, *cache]):
        mine = t._replace(position=x[5], slot=x[6], run_tok=x[7], run_len=x[8])
        refused(lambda: moe.rope_append(*x[:4], mine, moe.KVCache(*x[9:]), q_out=x[4]))
    ws = moe.alloc_kv_attention_workspace(4, 2, 64, T)
    for x in each_on_the_host([q, t.block_table, t.kv_len, t.tok_start, ws, torch.empty_like(q), *cache]):
        refused(lambda: moe.kv_attention(x[0], moe.KVCache(*x[6:]), *x[1:5], max_q=T, out=x[5]))
    # a workspace whose elements are not all its own
    refused(lambda: moe.kv_attention(q, cache, t.block_table, t.kv_len, t.tok_start, ws[:1].expand(ws.numel()), max_q=T))
    refused(lambda: moe.rope_table(16, 32, out=torch.empty(16, 16, 2)))
