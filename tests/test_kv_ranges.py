"""The paged cache's capacities and argument checks, without a GPU: the CPU statement by hand, refusals on
the host."""

import ctypes

import numpy as np
import pytest

import block_fp8_mixture_gb300 as moe
from oracle import kv_ref


def test_tables_refuse_what_does_not_fit_the_token_list():
    """Requests 1 and 3 end past 32 added tokens; 2 gives a page back, 4 stays as it is; 5 is too late as well,
    though it needs no page.  What 1 would have needed goes to nobody, and the next step finds it."""
    table = np.full((6, 3), -1)
    table[2, :2], table[4, 0], table[5, 0] = [7, 8], 9, 6
    cur, free = [0, 0, 20, 0, 4, 3], [0, 1, 2, 3, 4, 5, 0, 0, 0, 0]
    t = kv_ref.kv_tables(cur, [20, 17, 16, 1, 4, 5], table, free, 6, 16, 32, 8)
    assert t["kv_len"].tolist() == [20, 0, 16, 0, 4, 3]
    assert t["info"].tolist() == [40, 2, 3, 2] and t["free_count"].tolist() == [5]
    assert t["tok_start"].tolist() == [0, 20, 37, 37, 38, 38, 40]
    assert t["block_table"].tolist() == [[5, 8, -1], [-1] * 3, [7, -1, -1], [-1] * 3, [9, -1, -1], [6, -1, -1]]
    assert (t["slot"][:20] >= 0).all() and (t["slot"][20:] == -1).all()
    assert t["run_len"].tolist() == [16, 4, 0, 0, 0, 0, 0, 0]
    u = kv_ref.kv_tables(t["kv_len"], [20, 17, 16, 1, 4, 5], t["block_table"], t["free_list"], 5, 16, 32, 8)
    assert u["kv_len"].tolist() == [20, 17, 16, 1, 4, 5] and u["info"].tolist() == [20, 4, 0, 3]


# Arguments of a tables call whose buffers lie apart: fake device addresses, refused before anything uses them.
TABLES = dict(B=4, max_pages=8, num_pages=64, page_size=16, max_tokens=32, max_runs=8)
BUFFERS = ("cur_len", "new_len", "block_table", "free_list", "free_count", "out_block_table", "out_free_list",
           "out_free_count", "kv_len", "tok_start", "slot", "position", "request", "run_tok", "run_len", "info")
SIZES = dict(cur_len=4, new_len=4, block_table=32, free_list=64, free_count=1, out_block_table=32, out_free_list=64,
             out_free_count=1, kv_len=4, tok_start=5, slot=32, position=32, request=32, run_tok=8, run_len=8, info=4)


def tables_args(**kw):
    where = {n: (i + 1) << 12 for i, n in enumerate(BUFFERS)}
    return moe.KVTablesArgs(**{**TABLES, **where, **kw})


@pytest.mark.parametrize("out", BUFFERS[5:])
def test_tables_refuse_outputs_that_share_memory_with_inputs(lib, out):
    """With every input: the same address, its last entry, and its first entry as the output's last."""
    where = {n: getattr(tables_args(), n) for n in BUFFERS}
    for other in BUFFERS[:5]:
        for at in (where[other], where[other] + 4 * (SIZES[other] - 1), where[other] - 4 * (SIZES[out] - 1)):
            args = tables_args(**{out: at})
            assert lib.moe_kv_tables(ctypes.byref(args), None) == moe.MOE_ERR_INVALID_ARG, (out, other, at)


@pytest.mark.parametrize("name", BUFFERS)
def test_tables_refuse_missing_and_misaligned_buffers(lib, name):
    for at in (None, getattr(tables_args(), name) + 2):
        args = tables_args(**{name: at})
        assert lib.moe_kv_tables(ctypes.byref(args), None) == moe.MOE_ERR_INVALID_ARG, at


def test_binding_refuses_tensors_of_the_host(lib):
    """Tensors in host memory, right in all else: refused before their addresses reach the library."""
    torch = pytest.importorskip("torch")
    cache = moe.alloc_kv_cache(4, 2, 16, 64, device="cpu")
    t = moe.alloc_kv_tables(2, 4, 4, 16, 8, device="cpu")
    q = torch.zeros(8, 4, 64, dtype=torch.bfloat16)
    kv = torch.zeros(8, 2, 64, dtype=torch.bfloat16)
    ws = torch.zeros(moe.kv_attention_workspace_bytes(4, 2, 64, 8), dtype=torch.uint8)
    attn = moe.PagedAttention(num_layers=1, num_pages=4, page_size=16, num_heads=4, num_kv_heads=2, head_dim=64,
                              max_requests=2, max_pages=4, max_tokens=8, max_q=8, device="cpu")
    for call in (
            lambda: moe.kv_tables(t.kv_len, t.kv_len, t.block_table, t.free_list, t.free_count, page_size=16,
                                  max_tokens=8),
            lambda: moe.rope_table(16, 32, device="cpu"),
            lambda: moe.rope_append(q, kv, kv, None, t, cache),
            lambda: moe.kv_attention(q, cache, t.block_table, t.kv_len, t.tok_start, ws, max_q=8),
            lambda: attn.advance(t.kv_len),
            lambda: attn(0, q, kv, kv)):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.status == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("page_size", [16, 32, 64])
def test_attention_refuses_caches_whose_last_tile_passes_32_bits(lib, page_size):
    at = {n: (i + 1) << 12 for i, n in enumerate(("q", "k_codes", "v_codes", "k_scale", "v_scale", "block_table",
                                                  "kv_len", "tok_start", "out"))}
    need = lib.moe_kv_attention_workspace_bytes(4, 1, 128, 1)
    a = moe.KVAttentionArgs(**at, q_token_stride=512, q_head_stride=128, out_token_stride=512, out_head_stride=128,
                            T=4, B=1, Hq=4, Hkv=1, D=128, page_size=page_size, num_pages=64,
                            max_pages=(2 ** 31 - 128) // page_size + 1, max_q=1, window=0, sm_scale=0.1)
    assert lib.moe_kv_attention(ctypes.byref(a), 1 << 20, need, None) == moe.MOE_ERR_UNSUPPORTED_SHAPE


@pytest.mark.parametrize("name", ["max_tokens", "max_runs"])
def test_tables_refuse_lists_whose_loops_pass_32_bits(lib, name):
    far = {n: (i + 1) << 40 for i, n in enumerate(BUFFERS)}
    args = tables_args(**far, **{name: 2 ** 31 - 2 ** 20})
    assert lib.moe_kv_tables(ctypes.byref(args), None) == moe.MOE_ERR_UNSUPPORTED_SHAPE


def test_append_refuses_more_units_than_32_bits_count(lib):
    at = {n: (i + 1) << 40 for i, n in enumerate(("q", "k", "v", "q_out", "rope", "position", "slot", "run_tok",
                                                  "run_len", "k_codes", "v_codes", "k_scale", "v_scale"))}
    a = moe.RopeAppendArgs(**at, q_token_stride=512, q_head_stride=128, k_token_stride=131072, k_head_stride=128,
                           v_token_stride=131072, v_head_stride=128, qo_token_stride=512, qo_head_stride=128, T=4,
                           Hq=4, Hkv=1024, D=128, page_size=16, num_pages=64, max_runs=2 ** 21 + 1, rot_dim=128,
                           max_pos=100, layout=0, scale_fmt=0)
    assert lib.moe_rope_append(ctypes.byref(a), None) == moe.MOE_ERR_UNSUPPORTED_SHAPE
