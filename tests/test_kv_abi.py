"""The paged cache's C ABI without a GPU: every declared symbol is exported and bound, and arguments
are refused on the host before anything is launched."""

import ctypes
import os
import re

import pytest

import block_fp8_mixture_gb300 as moe

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe_kv.h")


def test_declared_symbols_are_exported_and_bound(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^(?:moe_status|size_t)\s+(moe_[a-z0-9_]+)\s*\(", text, re.M))
    assert {"moe_kv_tables", "moe_rope_table", "moe_rope_append", "moe_kv_attention"} <= names
    for n in names:
        assert hasattr(lib, n) and n in moe.SIGNATURES, n


def _fill(cls, base, kw):
    base = dict(base)
    base.update(kw)
    return cls(**base)


PTR = 1 << 12     # an aligned, fake device address: never dereferenced on these paths
TABLES = dict(cur_len=PTR, new_len=PTR, block_table=PTR, free_list=PTR, free_count=PTR,
              out_block_table=2 * PTR, out_free_list=2 * PTR, out_free_count=2 * PTR, kv_len=PTR,
              tok_start=PTR, slot=PTR, position=PTR, request=PTR, run_tok=PTR, run_len=PTR, info=PTR,
              B=4, max_pages=8, num_pages=64, page_size=16, max_tokens=32, max_runs=8)
APPEND = dict(q=PTR, k=PTR, v=PTR, q_out=PTR, rope=PTR, position=PTR, slot=PTR, run_tok=PTR,
              run_len=PTR, k_codes=PTR, v_codes=PTR, k_scale=PTR, v_scale=PTR, q_token_stride=512,
              q_head_stride=128, k_token_stride=128, k_head_stride=128, v_token_stride=128,
              v_head_stride=128, qo_token_stride=512, qo_head_stride=128, T=4, Hq=4, Hkv=1, D=128,
              page_size=16, num_pages=64, max_runs=4, rot_dim=128, max_pos=100, layout=0, scale_fmt=0)
ATTEND = dict(q=PTR, k_codes=PTR, v_codes=PTR, k_scale=PTR, v_scale=PTR, block_table=PTR, kv_len=PTR,
              tok_start=PTR, out=PTR, q_token_stride=512, q_head_stride=128, out_token_stride=512,
              out_head_stride=128, T=4, B=4, Hq=4, Hkv=1, D=128, page_size=16, num_pages=64,
              max_pages=8, max_q=1, window=0, sm_scale=0.1)
INV, SHAPE = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED_SHAPE


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), INV), (dict(B=5000), SHAPE), (dict(max_pages=0), INV), (dict(page_size=24), SHAPE),
    (dict(num_pages=-1), INV), (dict(max_tokens=-1), INV), (dict(cur_len=None), INV),
    (dict(block_table=None), INV), (dict(slot=None), INV), (dict(run_len=None), INV), (dict(info=2), INV),
    (dict(out_block_table=PTR), INV), (dict(out_free_list=PTR), INV), (dict(out_free_count=PTR), INV),
    (dict(max_pages=1 << 26), SHAPE), (dict(num_pages=1 << 27), SHAPE),
])
def test_tables_refusals(lib, kw, status):
    assert lib.moe_kv_tables(ctypes.byref(_fill(moe.KVTablesArgs, TABLES, kw)), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INV), (dict(Hkv=0), INV), (dict(D=96), SHAPE), (dict(D=256), SHAPE),
    (dict(page_size=48), SHAPE), (dict(rot_dim=24), SHAPE), (dict(rot_dim=144), SHAPE),
    (dict(layout=2), INV), (dict(scale_fmt=2), INV), (dict(scale_fmt=-1), INV), (dict(rope=None), INV),
    (dict(max_pos=0), INV), (dict(q=None), INV), (dict(k=None), INV), (dict(k=PTR + 8), INV),
    (dict(k_codes=PTR + 4), INV), (dict(v_scale=None), INV), (dict(q_token_stride=516), INV),
    (dict(v_head_stride=-128), INV), (dict(position=None), INV), (dict(run_tok=None), INV),
])
def test_append_refusals(lib, kw, status):
    assert lib.moe_rope_append(ctypes.byref(_fill(moe.RopeAppendArgs, APPEND, kw)), None) == status


def test_append_of_nothing_is_ok(lib):
    a = _fill(moe.RopeAppendArgs, APPEND, dict(T=0, q=None, k=None))
    assert lib.moe_rope_append(ctypes.byref(a), None) == moe.MOE_OK


@pytest.mark.parametrize("args,status", [
    ((PTR, 10, 24, 1e4, 0, 1.0, 1.0, 2.0, 10, 1.0), SHAPE), ((PTR, 10, 256, 1e4, 0, 1.0, 1.0, 2.0, 10, 1.0), SHAPE),
    ((PTR, -1, 64, 1e4, 0, 1.0, 1.0, 2.0, 10, 1.0), INV), ((None, 10, 64, 1e4, 0, 1.0, 1.0, 2.0, 10, 1.0), INV),
    ((PTR, 10, 64, 1.0, 0, 1.0, 1.0, 2.0, 10, 1.0), INV), ((PTR, 10, 64, 1e4, 3, 1.0, 1.0, 2.0, 10, 1.0), INV),
    ((PTR, 10, 64, 1e4, 1, 0.5, 1.0, 2.0, 10, 1.0), INV), ((PTR, 10, 64, 1e4, 2, 4.0, 2.0, 2.0, 10, 1.0), INV),
    ((PTR, 10, 64, 1e4, 2, 4.0, 1.0, 2.0, 0, 1.0), INV), ((PTR, 10, 64, 1e4, 0, 1.0, 1.0, 2.0, 10, float("inf")), INV),
])
def test_rope_table_refusals(lib, args, status):
    assert lib.moe_rope_table(*args, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INV), (dict(B=0), INV), (dict(B=4097), SHAPE), (dict(Hq=6, Hkv=4), SHAPE),
    (dict(Hq=65), SHAPE), (dict(D=80), SHAPE), (dict(page_size=8), SHAPE), (dict(max_q=0), INV),
    (dict(window=-1), INV), (dict(sm_scale=0.0), INV), (dict(sm_scale=float("nan")), INV),
    (dict(sm_scale=float("inf")), INV), (dict(q=None), INV), (dict(out=PTR + 2), INV),
    (dict(kv_len=None), INV), (dict(block_table=None), INV), (dict(k_codes=PTR + 8), INV),
    (dict(q_head_stride=4), INV), (dict(max_pages=0), INV),
])
def test_attention_refusals(lib, kw, status):
    need = lib.moe_kv_attention_workspace_bytes(4, 1, 128, 1)
    a = _fill(moe.KVAttentionArgs, ATTEND, kw)
    assert lib.moe_kv_attention(ctypes.byref(a), PTR, need, None) == status


def test_attention_workspace(lib):
    need = lib.moe_kv_attention_workspace_bytes(4, 1, 128, 1)
    ref = ctypes.byref(_fill(moe.KVAttentionArgs, ATTEND, {}))
    assert need >= 256
    assert lib.moe_kv_attention(None, PTR, need, None) == INV
    assert lib.moe_kv_attention(ref, None, need, None) == INV
    assert lib.moe_kv_attention(ref, PTR + 16, need, None) == INV
    assert lib.moe_kv_attention(ref, PTR, need - 1, None) == moe.MOE_ERR_WORKSPACE_TOO_SMALL
    empty = ctypes.byref(_fill(moe.KVAttentionArgs, ATTEND, dict(T=0, q=None)))
    assert lib.moe_kv_attention(empty, PTR, need, None) == moe.MOE_OK
    for bad in ((0, 1, 128, 1), (4, 3, 128, 1), (65, 1, 128, 1), (4, 1, 96, 1), (4, 1, 128, 0)):
        assert lib.moe_kv_attention_workspace_bytes(*bad) == 0


def test_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    cache = moe.alloc_kv_cache(4, 2, 16, 64, device="cpu")
    t = moe.alloc_kv_tables(2, 4, 4, 16, 8, device="cpu")
    q = torch.zeros(8, 4, 64, dtype=torch.bfloat16)
    kv = torch.zeros(8, 2, 64, dtype=torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8)
    for bad in (q.float(), q[:4], q.transpose(1, 2).contiguous().transpose(1, 2)):
        with pytest.raises(moe.MoeError):
            moe.rope_append(bad, kv, kv, None, t, cache)
    with pytest.raises(moe.MoeError):
        moe.rope_append(q, kv, kv, torch.zeros(10, 8), t, cache)
    with pytest.raises(moe.MoeError):
        moe.rope_append(q, kv, kv, None, t, cache._replace(k_scale=cache.k_scale.double()))
    with pytest.raises(moe.MoeError):
        moe.kv_attention(q, cache, t.block_table, t.kv_len.long(), t.tok_start, ws, max_q=1)
    with pytest.raises(moe.MoeError):
        moe.kv_attention(q, cache, t.block_table, t.kv_len, t.tok_start[:-1], ws, max_q=1)
    with pytest.raises(moe.MoeError):
        moe.kv_tables(t.kv_len, t.kv_len, t.block_table, t.free_list, t.free_count, page_size=16)


def test_packed_arguments_match_the_structures():
    """The binding packs its arguments with struct formats; they have to be the C structures' layouts."""
    from block_fp8_mixture_gb300 import kv
    for cls, fmt in ((moe.KVTablesArgs, kv._PACK_TABLES), (moe.RopeAppendArgs, kv._PACK_APPEND),
                     (moe.KVAttentionArgs, kv._PACK_ATTENTION)):
        values = [i + 1 for i in range(len(cls._fields_))]
        got = cls.from_buffer_copy(fmt.pack(*values))
        assert fmt.size == ctypes.sizeof(cls)
        assert [getattr(got, n) for n, _ in cls._fields_] == values
