"""Binding of include/moe_kv.h: the paged 8-bit key/value cache, its tables, the rotary write and the
attention that reads it.  As in the rest of the package these functions only marshal arguments; the
work is done by the library's CUDA kernels on `stream` (default: torch's current stream).  What a call
allocates is allocated on that stream too, so that its memory is not handed out again while the kernels use it;
as everywhere in torch, a tensor that another stream uses needs record_stream before it is dropped.
"""

from __future__ import annotations

import ctypes
import math
import struct
from typing import NamedTuple

import torch

from . import MOE_ERR_INVALID_ARG, SCALE_FP32, MoeError, _check, load_library
from . import _stream as _given_stream

ROPE_HALF = 0
ROPE_INTERLEAVED = 1
ROPE_SCALE_NONE = 0
ROPE_SCALE_LINEAR = 1
ROPE_SCALE_RAMP = 2
PAGE_SIZES = (16, 32, 64, 128)

_VP, _SZ, _I, _L, _F, _D = (ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64,
                            ctypes.c_float, ctypes.c_double)


class KVTablesArgs(ctypes.Structure):
    _fields_ = [(n, _VP) for n in (
        "cur_len", "new_len", "block_table", "free_list", "free_count", "out_block_table",
        "out_free_list", "out_free_count", "kv_len", "tok_start", "slot", "position", "request",
        "run_tok", "run_len", "info")] + [(n, _I) for n in (
            "B", "max_pages", "num_pages", "page_size", "max_tokens", "max_runs")]


class RopeAppendArgs(ctypes.Structure):
    _fields_ = [(n, _VP) for n in (
        "q", "k", "v", "q_out", "rope", "position", "slot", "run_tok", "run_len", "k_codes", "v_codes",
        "k_scale", "v_scale")] + [(n, _L) for n in (
            "q_token_stride", "q_head_stride", "k_token_stride", "k_head_stride", "v_token_stride",
            "v_head_stride", "qo_token_stride", "qo_head_stride")] + [(n, _I) for n in (
                "T", "Hq", "Hkv", "D", "page_size", "num_pages", "max_runs", "rot_dim", "max_pos",
                "layout", "scale_fmt")]


class KVAttentionArgs(ctypes.Structure):
    _fields_ = [(n, _VP) for n in (
        "q", "k_codes", "v_codes", "k_scale", "v_scale", "block_table", "kv_len", "tok_start",
        "out")] + [(n, _L) for n in (
            "q_token_stride", "q_head_stride", "out_token_stride", "out_head_stride")] + [
                (n, _I) for n in ("T", "B", "Hq", "Hkv", "D", "page_size", "num_pages", "max_pages",
                                  "max_q", "window")] + [("sm_scale", _F)]


# The C structures' layouts for struct.pack: a decode step is a handful of short calls, and packing the
# fields is several times quicker than filling a ctypes structure (tests hold the two layouts together).
_PACK_TABLES = struct.Struct("@16P6i")
_PACK_APPEND = struct.Struct("@13P8q11i0P")
_PACK_ATTENTION = struct.Struct("@9P4q10if0P")

SIGNATURES = {
    "moe_kv_tables": (_I, [_VP, _VP]),
    "moe_rope_table": (_I, [_VP, _I, _I, _D, _I, _D, _D, _D, _I, _F, _VP]),
    "moe_rope_append": (_I, [_VP, _VP]),
    "moe_kv_attention_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "moe_kv_attention": (_I, [_VP, _VP, _SZ, _VP]),
}


class KVTables(NamedTuple):
    """One step's tables (int32 device tensors), as moe_kv_tables writes them."""
    block_table: object   # [B, max_pages]
    free_list: object     # [num_pages]
    free_count: object    # [1]
    kv_len: object        # [B]
    tok_start: object     # [B + 1]
    slot: object          # [max_tokens]
    position: object      # [max_tokens]
    request: object       # [max_tokens]
    run_tok: object       # [max_runs]
    run_len: object       # [max_runs]
    info: object          # [4] added tokens, runs, refused requests, granted pages


class KVCache(NamedTuple):
    """The cache's four tensors: codes uint8 (or float8_e4m3fn) [num_pages, Hkv, page_size, D], scales
    fp32 [num_pages, Hkv]."""
    k_codes: object
    v_codes: object
    k_scale: object
    v_scale: object


def _stream(stream, dev: int):
    """The stream's handle, for tensors on device `dev`, which has to be the current one; torch's current
    stream through the raw handle, without building an object (3 us of a call that takes 10)."""
    if dev != _current_device():
        _bad(f"the tensors are on device {dev}, the current device is {_current_device()}")
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev)
    return _given_stream(stream)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# (there are tensors on a device when this is asked, so torch need not look whether CUDA is initialised)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _allocate(stream, make, *args, **kw):
    """make(...) with the call's stream as torch's current one."""
    if stream is None:
        return make(*args, **kw)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    with torch.cuda.stream(stream):
        return make(*args, **kw)


def _bad(what: str):
    raise MoeError(MOE_ERR_INVALID_ARG, what)


def _device(name: str, t) -> int:
    """The CUDA device that a call's first tensor is on, and so all others have to be."""
    dev = t.get_device()
    if dev < 0:
        _bad(f"{name}: a CUDA tensor is needed")
    return dev


def _i32(name: str, t, shape, dev: int):
    if t.dtype is not torch.int32 or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _bad(f"{name}: a contiguous int32 tensor of shape {shape} on device {dev} is needed")
    return t.data_ptr()


def max_runs(max_tokens: int, page_size: int, num_requests: int) -> int:
    """A capacity of the run list that always suffices."""
    return min(max_tokens, max_tokens // page_size + 2 * num_requests)


def alloc_kv_cache(num_pages: int, num_kv_heads: int, page_size: int, head_dim: int,
                   device="cuda") -> KVCache:
    shape = (num_pages, num_kv_heads, page_size, head_dim)
    code = [torch.zeros(shape, dtype=torch.uint8, device=device) for _ in range(2)]
    scale = [torch.zeros(shape[:2], dtype=torch.float32, device=device) for _ in range(2)]
    return KVCache(*code, *scale)


def alloc_kv_tables(num_requests: int, max_pages: int, num_pages: int, page_size: int,
                    max_tokens: int, device="cuda") -> KVTables:
    """A set of tables for `num_requests` requests and steps of up to `max_tokens` tokens: all pages
    free, no request holds any."""
    i32 = dict(dtype=torch.int32, device=device)
    runs = max_runs(max_tokens, page_size, num_requests)
    return KVTables(
        block_table=torch.full((num_requests, max_pages), -1, **i32),
        free_list=torch.arange(num_pages, **i32), free_count=torch.full((1,), num_pages, **i32),
        kv_len=torch.zeros(num_requests, **i32), tok_start=torch.zeros(num_requests + 1, **i32),
        slot=torch.full((max_tokens,), -1, **i32), position=torch.zeros(max_tokens, **i32),
        request=torch.full((max_tokens,), -1, **i32), run_tok=torch.zeros(runs, **i32),
        run_len=torch.zeros(runs, **i32), info=torch.zeros(4, **i32))


def kv_tables(cur_len, new_len, block_table, free_list, free_count, *, page_size: int,
              max_tokens: int | None = None, out: KVTables | None = None, stream=None) -> KVTables:
    """Block tables, free stack, slot map and page runs that take the requests from cur_len to new_len
    cached tokens (moe_kv_tables).  The inputs are left as they are; `out` is the second set of tables
    (allocated for `max_tokens` added tokens when it is not given)."""
    B, W = block_table.shape
    N = free_list.shape[0]
    if out is None:
        if max_tokens is None:
            _bad("kv_tables: max_tokens or out is needed")
        out = _allocate(stream, alloc_kv_tables, B, W, N, page_size, max_tokens, block_table.device)
    o_table, o_free, o_count, kv_len, tok_start, slot, position, request, run_tok, run_len, info = out
    T, R = slot.shape[0], run_tok.shape[0]
    if max_tokens is not None and max_tokens != T:
        _bad("kv_tables: out holds another number of tokens than max_tokens")
    d = _device("block_table", block_table)
    b, t, r, one, table, pool = (B,), (T,), (R,), (1,), (B, W), (N,)
    a = _PACK_TABLES.pack(
        _i32("cur_len", cur_len, b, d), _i32("new_len", new_len, b, d), _i32("block_table", block_table, table, d),
        _i32("free_list", free_list, pool, d), _i32("free_count", free_count, one, d),
        _i32("out.block_table", o_table, table, d), _i32("out.free_list", o_free, pool, d),
        _i32("out.free_count", o_count, one, d), _i32("out.kv_len", kv_len, b, d),
        _i32("out.tok_start", tok_start, (B + 1,), d), _i32("out.slot", slot, t, d),
        _i32("out.position", position, t, d), _i32("out.request", request, t, d),
        _i32("out.run_tok", run_tok, r, d), _i32("out.run_len", run_len, r, d),
        _i32("out.info", info, (4,), d), B, W, N, page_size, T, R)
    _check(load_library().moe_kv_tables(a, _stream(stream, d)), "moe_kv_tables")
    return out


def rope_table(max_pos: int, rot_dim: int, base: float = 10000.0, *, scaling: int = ROPE_SCALE_NONE,
               factor: float = 1.0, low: float = 1.0, high: float = 32.0, original_len: int = 4096,
               magnitude: float = 1.0, out=None, device="cuda", stream=None):
    """cos and sin of every position, fp32 [max_pos, rot_dim / 2, 2] (moe_rope_table)."""
    if out is None:
        out = _allocate(stream, torch.empty, (max_pos, rot_dim // 2, 2), dtype=torch.float32, device=device)
    elif out.dtype != torch.float32 or tuple(out.shape) != (max_pos, rot_dim // 2, 2) or not out.is_contiguous():
        _bad("rope_table: out is a contiguous fp32 tensor [max_pos, rot_dim / 2, 2]")
    _check(load_library().moe_rope_table(out.data_ptr(), max_pos, rot_dim, base, scaling, factor, low,
                                         high, original_len, magnitude, _stream(stream, _device("out", out))),
           "moe_rope_table")
    return out


def _heads(name: str, t, T: int, H: int, D: int, dev: int):
    """Pointer, token stride and head stride of a BF16 tensor [T, H, D] with contiguous heads."""
    if t.dtype is not torch.bfloat16 or t.shape != (T, H, D) or t.get_device() != dev:
        _bad(f"{name}: a bfloat16 tensor of shape {(T, H, D)} on device {dev} is needed")
    st, sh, sd = t.stride()
    if sd != 1:
        _bad(f"{name}: the values of a head have to be contiguous")
    return t.data_ptr(), st, sh


def _cache(cache: KVCache):
    """Pointers of the cache's tensors, (num_pages, Hkv, page_size, D) and the device."""
    kc, vc, ks, vs = cache
    shape = kc.shape
    dev = _device("cache", kc)
    if (len(shape) != 4 or vc.shape != shape or kc.element_size() != 1 or vc.element_size() != 1
            or ks.shape != shape[:2] or vs.shape != ks.shape or ks.dtype is not torch.float32
            or vs.dtype is not torch.float32
            or not (vc.get_device() == ks.get_device() == vs.get_device() == dev)
            or not (kc.is_contiguous() and vc.is_contiguous()
                    and ks.is_contiguous() and vs.is_contiguous())):
        _bad("cache: contiguous codes [num_pages, Hkv, page_size, D] and fp32 scales [num_pages, Hkv] "
             "on one device are needed")
    return kc.data_ptr(), vc.data_ptr(), ks.data_ptr(), vs.data_ptr(), shape, dev


def rope_append(q, k, v, rope, tables: KVTables, cache: KVCache, *, layout: int = ROPE_HALF,
                scale_fmt: int = SCALE_FP32, q_out=None, stream=None):
    """Rotate q and k [T, heads, D] by the tables' positions, write k and v to the cache and return the
    rotated q (moe_rope_append).  rope: rope_table's result, or None for no rotation; q None: cache
    write only; q_out may be q.  T is the tables' token capacity."""
    kc, vc, ks, vs, (N, Hkv, P, D), d = _cache(cache)
    T, R = tables.slot.shape[0], tables.run_tok.shape[0]
    rot = max_pos = 0
    rp = 0
    if rope is not None:
        if (rope.dtype is not torch.float32 or rope.dim() != 3 or rope.shape[2] != 2 or rope.get_device() != d
                or not rope.is_contiguous()):
            _bad(f"rope: a contiguous fp32 tensor [max_pos, rot_dim / 2, 2] on device {d} is needed")
        max_pos, rot, rp = rope.shape[0], 2 * rope.shape[1], rope.data_ptr()
    Hq = qp = op = qt = qh = ot = oh = 0
    if q is not None:
        Hq = q.shape[1]
        if q_out is None:
            q_out = _allocate(stream, torch.empty, (T, Hq, D), dtype=torch.bfloat16, device=q.device)
        qp, qt, qh = _heads("q", q, T, Hq, D, d)
        op, ot, oh = _heads("q_out", q_out, T, Hq, D, d)
    kp, kt, kh = _heads("k", k, T, Hkv, D, d)
    vp, vt, vh = _heads("v", v, T, Hkv, D, d)
    t, r = (T,), (R,)
    a = _PACK_APPEND.pack(qp, kp, vp, op, rp, _i32("position", tables.position, t, d),
                          _i32("slot", tables.slot, t, d), _i32("run_tok", tables.run_tok, r, d),
                          _i32("run_len", tables.run_len, r, d), kc, vc, ks, vs, qt, qh, kt, kh, vt, vh,
                          ot, oh, T, Hq, Hkv, D, P, N, R, rot, max_pos, layout, scale_fmt)
    _check(load_library().moe_rope_append(a, _stream(stream, d)), "moe_rope_append")
    return q_out


def kv_attention_workspace_bytes(num_heads: int, num_kv_heads: int, head_dim: int, max_q: int) -> int:
    return load_library().moe_kv_attention_workspace_bytes(num_heads, num_kv_heads, head_dim, max_q)


def alloc_kv_attention_workspace(num_heads: int, num_kv_heads: int, head_dim: int, max_q: int,
                                 device="cuda"):
    """A zeroed workspace for kv_attention calls with these heads and up to max_q tokens a request."""
    n = kv_attention_workspace_bytes(num_heads, num_kv_heads, head_dim, max_q)
    return torch.zeros(max(256, n), dtype=torch.uint8, device=device)


def kv_attention(q, cache: KVCache, block_table, kv_len, tok_start, workspace, *, max_q: int,
                 sm_scale: float | None = None, window: int = 0, out=None, stream=None):
    """Causal attention of q [T, Hq, D] over the cache (moe_kv_attention): the tokens of request b are
    rows [tok_start[b], tok_start[b+1]) of q and the last ones of its kv_len[b] cached tokens.  max_q
    bounds the tokens of one request; sm_scale defaults to D^-0.5; window > 0 limits how far back a
    token sees."""
    kc, vc, ks, vs, (N, Hkv, P, D), d = _cache(cache)
    T, Hq = q.shape[0], q.shape[1]
    B, W = block_table.shape
    if out is None:
        out = _allocate(stream, torch.empty, (T, Hq, D), dtype=torch.bfloat16, device=q.device)
    qp, qt, qh = _heads("q", q, T, Hq, D, d)
    op, ot, oh = _heads("out", out, T, Hq, D, d)
    if workspace.get_device() != d or not workspace.is_contiguous():
        _bad(f"workspace: a contiguous tensor on device {d} is needed")
    b = (B,)
    a = _PACK_ATTENTION.pack(qp, kc, vc, ks, vs, _i32("block_table", block_table, (B, W), d),
                             _i32("kv_len", kv_len, b, d), _i32("tok_start", tok_start, (B + 1,), d), op, qt, qh,
                             ot, oh, T, B, Hq, Hkv, D, P, N, W, max_q, window,
                             1.0 / math.sqrt(D) if sm_scale is None else sm_scale)
    _check(load_library().moe_kv_attention(a, workspace.data_ptr(), workspace.numel(), _stream(stream, d)),
           "moe_kv_attention")
    return out


class PagedAttention:
    """Rotary embedding, 8-bit paged cache and attention of a model's layers, for up to `max_requests`
    requests at a time.  The layers share the tables, which advance() moves one step on; each layer has
    its own cache.  Steps are built in the second of two sets of tables, so advance() may be called (on
    another stream, ordered after the step before it) while kernels of that step still read the first.  The
    object itself is made on the current stream: a first step on another one has to wait for that.

    rope: rope_table's result or None; max_tokens: capacity of a step's added tokens (q, k and v always
    have that many rows; rows past a step's tokens are ignored); max_q: most tokens a request adds at once
    (of more than that only the first max_q get an output).
    """

    def __init__(self, *, num_layers: int, num_pages: int, page_size: int, num_heads: int, num_kv_heads: int,
                 head_dim: int, max_requests: int, max_pages: int, max_tokens: int, max_q: int, rope=None,
                 layout: int = ROPE_HALF, scale_fmt: int = SCALE_FP32, sm_scale: float | None = None,
                 window: int = 0, device="cuda"):
        self.caches = [alloc_kv_cache(num_pages, num_kv_heads, page_size, head_dim, device)
                       for _ in range(num_layers)]
        self.tables, self._next = (alloc_kv_tables(max_requests, max_pages, num_pages, page_size, max_tokens,
                                                   device) for _ in range(2))
        self.workspace = alloc_kv_attention_workspace(num_heads, num_kv_heads, head_dim, max_q, device)
        self.page_size, self.max_q, self.rope, self.layout = page_size, max_q, rope, layout
        self.scale_fmt, self.sm_scale, self.window = scale_fmt, sm_scale, window

    def advance(self, new_len, stream=None) -> KVTables:
        """Take every request to new_len cached tokens (int32 device tensor; 0: finished).  tables.info says
        on the device how many tokens were added and how many requests were refused, because the pool or
        max_tokens did not suffice: those keep the length they had."""
        t = self.tables
        kv_tables(t.kv_len, new_len, t.block_table, t.free_list, t.free_count, page_size=self.page_size,
                  out=self._next, stream=stream)
        self.tables, self._next = self._next, t
        return self.tables

    def __call__(self, layer: int, q, k, v, out=None, stream=None):
        """Write the step's k and v [max_tokens, Hkv, D] to the layer's cache and return the attention of
        q [max_tokens, Hq, D] over it."""
        t, cache = self.tables, self.caches[layer]
        q = rope_append(q, k, v, self.rope, t, cache, layout=self.layout, scale_fmt=self.scale_fmt, stream=stream)
        return kv_attention(q, cache, t.block_table, t.kv_len, t.tok_start, self.workspace, max_q=self.max_q,
                            sm_scale=self.sm_scale, window=self.window, out=out, stream=stream)
