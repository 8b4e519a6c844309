"""Binding of include/moe_step.h: the norm in front of attention and experts, the routing to experts and the
verification of drafted tokens.  As in the rest of the package these functions only marshal arguments; the
work is done by the library's CUDA kernels on `stream` (default: torch's current stream), and what a call
allocates is allocated on that stream too.
"""

from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple

import torch

from . import NUMERICS_DIVIDE, SCALE_FP32, SCALE_FP32_POW2, SCALE_UE8M0, FwdArgs, _check, load_library
from .kv import _allocate, _bad, _device, _i32, _stream

# (names of this module are found quicker than torch's attributes; a short call is bound by its checks)
_BF16, _FP32, _U8, _E4M3 = torch.bfloat16, torch.float32, torch.uint8, torch.float8_e4m3fn

ROUTE_SOFTMAX = 0
ROUTE_SIGMOID = 1

_VP, _SZ, _I, _L, _F, _D = (ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                            ctypes.c_double)


class RmsNormArgs(ctypes.Structure):
    _fields_ = [(n, _VP) for n in (
        "x", "residual", "weight", "d_num_tokens", "residual_out", "out", "codes", "scales")] + [(n, _L) for n in (
            "x_stride", "residual_stride", "residual_out_stride", "out_stride", "codes_stride",
            "scales_stride")] + [("eps", _D)] + [(n, _I) for n in (
                "M_cap", "H", "weight_fp32", "weight_plus_one", "scale_fmt", "numerics")]


class RouteArgs(ctypes.Structure):
    _fields_ = [(n, _VP) for n in ("logits", "bias", "d_num_tokens", "topk_ids", "topk_weights")] + [
        ("logits_stride", _L)] + [(n, _I) for n in (
            "M_cap", "E", "topk", "logits_bf16", "scoring", "num_groups", "topk_groups", "group_best",
            "renormalize")] + [("scale", _F)]


class VerifyDraftsArgs(ctypes.Structure):
    _fields_ = [(n, _VP) for n in (
        "target", "draft", "tokens", "tok_start", "kv_len", "slot", "uniform", "uniform_next", "accepted",
        "next_token", "kept_len")] + [("target_stride", _L), ("draft_stride", _L)] + [
            (n, _I) for n in ("T", "B", "V", "bf16")]


# The C structures' layouts for struct.pack, as in kv.py (tests hold the two layouts together).
_PACK_NORM = struct.Struct("@8P6qd6i0P")
_PACK_ROUTE = struct.Struct("@5Pq9if0P")
_PACK_VERIFY = struct.Struct("@11P2q4i0P")

SIGNATURES = {
    "moe_rms_norm": (_I, [_VP, _VP]),
    "moe_place_act": (_I, [_VP, _L, _VP, _L, _VP, _I, _I, _I, _I, _I, _I, _VP, _SZ, _VP]),
    "moe_fp8_block_forward_codes": (_I, [ctypes.POINTER(FwdArgs), _VP, _L, _VP, _L, _VP, _SZ, _VP]),
    "moe_route": (_I, [_VP, _VP]),
    "moe_verify_drafts": (_I, [_VP, _VP]),
}


class _Outputs(NamedTuple):
    out: object        # bf16 [M, H]
    residual: object   # bf16 [M, H]
    codes: object      # float8_e4m3fn (or uint8) [M, H]
    scales: object     # [ceil(H / 128), M] fp32, or uint8 UE8M0


class Normed(_Outputs):
    """rms_norm's outputs; those not asked for are None.  quant and numerics say how the codes were made, so that a layer
    can refuse those of another format; None where there are no codes, or a caller has put them together."""
    quant = None
    numerics = None

    def _replace(self, **kw):
        new = super()._replace(**kw)
        new.quant, new.numerics = self.quant, self.numerics
        return new


class Verified(NamedTuple):
    """verify_drafts' outputs, int32 [B]."""
    accepted: object
    next_token: object
    kept_len: object


def _rows(name: str, t, dtype, shape, dev: int):
    """Pointer and row stride of a matrix of that shape with contiguous rows."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _bad(f"{name}: a {dtype} tensor of shape {tuple(shape)} on device {dev} is needed")
    sr, sc = t.stride()
    if sc != 1 and shape[1] > 1:
        _bad(f"{name}: the values of a row have to be contiguous")
    return t.data_ptr(), sr


def _vector(name: str, t, dtype, n: int, dev: int):
    if t.dtype is not dtype or t.shape != (n,) or t.get_device() != dev or not t.is_contiguous():
        _bad(f"{name}: a contiguous {dtype} tensor of shape {(n,)} on device {dev} is needed")
    return t.data_ptr()


def _count(d_num_tokens, dev: int) -> int:
    if d_num_tokens is None:
        return 0
    t = d_num_tokens
    if t.dtype is not torch.int32 or t.numel() < 1 or t.get_device() != dev:
        _bad(f"d_num_tokens: an int32 tensor on device {dev} is needed")
    return t.data_ptr()


def rms_norm(x, weight, *, eps: float = 1e-6, residual=None, residual_out=None, weight_plus_one: bool = False,
             quant: int | None = None, numerics: int = NUMERICS_DIVIDE, write_out: bool = True, out=None, codes=None,
             scales=None, d_num_tokens=None, stream=None) -> Normed:
    """Root-mean-square norm of x [M, H] (bf16), or of x + residual, which is written to residual_out (by default
    to residual itself) (moe_rms_norm).  weight: bf16 or fp32 [H], with weight_plus_one its difference from
    one.  quant: SCALE_FP32, SCALE_FP32_POW2 or SCALE_UE8M0 for the normed rows as E4M3 codes with 1x128 scales too,
    or with write_out false instead."""
    d = _device("x", x)
    if x.dim() != 2:
        _bad("x: a bfloat16 tensor [M, H] is needed")
    shape = M, H = x.shape
    xp, xs = _rows("x", x, _BF16, shape, d)
    wide = weight.dtype is _FP32
    wp = _vector("weight", weight, _FP32 if wide else _BF16, H, d)
    rp = rs = rop = ros = op = os = cp = cs = sp = ss = 0
    if residual is not None:
        rop, ros = rp, rs = _rows("residual", residual, _BF16, shape, d)
        if residual_out is None:
            residual_out = residual
        else:
            rop, ros = _rows("residual_out", residual_out, _BF16, shape, d)
    elif residual_out is not None:
        _bad("residual_out: there is no residual")
    if write_out:
        if out is None:
            out = _allocate(stream, torch.empty, (M, H), dtype=_BF16, device=x.device)
        op, os = _rows("out", out, _BF16, shape, d)
    elif out is not None:
        _bad("out: write_out is false")
    if quant is not None:
        if quant not in (SCALE_FP32, SCALE_FP32_POW2, SCALE_UE8M0):
            _bad("quant: SCALE_FP32, SCALE_FP32_POW2 or SCALE_UE8M0")
        groups = (H + 127) // 128
        kind = _U8 if quant == SCALE_UE8M0 else _FP32
        if codes is None:
            codes = _allocate(stream, torch.empty, (M, H), dtype=_E4M3, device=x.device)
        if scales is None:
            scales = _allocate(stream, torch.empty, (groups, M), dtype=kind, device=x.device)
        cp, cs = _rows("codes", codes, _U8 if codes.dtype is _U8 else _E4M3, shape, d)
        sp, ss = _rows("scales", scales, kind, (groups, M), d)
    elif codes is not None or scales is not None:
        _bad("codes and scales: quant says their format")
    a = _PACK_NORM.pack(xp, rp, wp, _count(d_num_tokens, d), rop, op, cp, sp, xs, rs, ros, os, cs, ss, eps, M, H,
                        wide, bool(weight_plus_one), quant or 0, numerics)
    _check(load_library().moe_rms_norm(a, _stream(stream, d)), "moe_rms_norm")
    got = Normed(out, residual_out, codes, scales)
    if quant is not None:
        got.quant, got.numerics = quant, numerics
    return got


def _codes(codes, scales, act_fmt: int, dev: int):
    """Pointers and strides of quantized rows [M, H] and their scales [H / 128, M]."""
    if codes.dim() != 2 or codes.dtype not in (_E4M3, _U8):
        _bad("codes: a tensor [M, H] of E4M3 codes is needed")
    M, H = codes.shape
    cp, cs = _rows("codes", codes, codes.dtype, (M, H), dev)
    sp, ss = _rows("scales", scales, _U8 if act_fmt == SCALE_UE8M0 else _FP32, ((H + 127) // 128, M), dev)
    return cp, cs, sp, ss


def _workspace(workspace, dev: int):
    if workspace.get_device() != dev or not workspace.is_contiguous() or workspace.element_size() != 1:
        _bad(f"workspace: a contiguous tensor of bytes on device {dev} is needed")
    return workspace.data_ptr(), workspace.numel()


def place_act(codes, scales, topk: int, E: int, I: int, workspace, *, d_num_tokens=None, act_fmt: int = SCALE_FP32,
              stream=None):
    """Quantized rows (rms_norm's) to the experts' workspace, in quant_act's place (moe_place_act)."""
    d = _device("codes", codes)
    cp, cs, sp, ss = _codes(codes, scales, act_fmt, d)
    M, H = codes.shape
    _check(load_library().moe_place_act(cp, cs, sp, ss, _count(d_num_tokens, d), M, E, H, I, topk, act_fmt,
                                        *_workspace(workspace, d), _stream(stream, d)), "moe_place_act")


def forward_codes(args: FwdArgs, codes, scales, workspace, stream=None):
    """The whole layer on quantized rows (moe_fp8_block_forward_codes)."""
    d = _device("codes", codes)
    if codes.shape != (args.M_cap, args.H):
        _bad(f"codes: a tensor of shape {(args.M_cap, args.H)} is needed")
    cp, cs, sp, ss = _codes(codes, scales, args.act_scale_fmt, d)
    _check(load_library().moe_fp8_block_forward_codes(ctypes.byref(args), cp, cs, sp, ss, *_workspace(workspace, d),
                                                      _stream(stream, d)), "moe_fp8_block_forward_codes")


def route(logits, topk: int, *, scoring: int = ROUTE_SOFTMAX, bias=None, num_groups: int = 1, topk_groups: int = 1,
          group_best: int = 2, renormalize: bool = True, scale: float = 1.0, ids=None, weights=None,
          d_num_tokens=None, stream=None):
    """Experts (int32 [M, topk]) and weights (fp32 [M, topk]) of each token, as MoELayer takes them, from the
    router's logits [M, E], fp32 or bf16 (moe_route).  bias: fp32 [E], added for the choice only; with
    num_groups > 1 only the experts of the topk_groups best groups are chosen from."""
    d = _device("logits", logits)
    if logits.dim() != 2:
        _bad("logits: a tensor [M, E] is needed")
    M, E = logits.shape
    if topk < 1:
        _bad("topk: at least one expert")
    half = logits.dtype is _BF16
    lp, ls = _rows("logits", logits, _BF16 if half else _FP32, (M, E), d)
    bp = 0 if bias is None else _vector("bias", bias, _FP32, E, d)
    if ids is None:
        ids = _allocate(stream, torch.empty, (M, topk), dtype=torch.int32, device=logits.device)
    if weights is None:
        weights = _allocate(stream, torch.empty, (M, topk), dtype=_FP32, device=logits.device)
    if (weights.dtype is not _FP32 or weights.shape != (M, topk) or weights.get_device() != d
            or not weights.is_contiguous()):
        _bad(f"weights: a contiguous fp32 tensor of shape {(M, topk)} on device {d} is needed")
    a = _PACK_ROUTE.pack(lp, bp, _count(d_num_tokens, d), _i32("ids", ids, (M, topk), d), weights.data_ptr(), ls, M,
                         E, topk, half, scoring, num_groups, topk_groups, group_best, bool(renormalize), scale)
    _check(load_library().moe_route(a, _stream(stream, d)), "moe_route")
    return ids, weights


def verify_drafts(target, tokens, tok_start, kv_len, uniform, uniform_next, *, draft=None, slot=None,
                  out: Verified | None = None, stream=None) -> Verified:
    """How many of each request's drafted tokens stay, the token that follows them and the cached tokens to
    keep (moe_verify_drafts): PagedAttention.advance(kept_len) gives the others' pages back.  target [T, V]: the
    probabilities after each of a step's rows (fp32 or bf16); tokens [T]: what was fed at them; tok_start, kv_len and
    slot: the step's tables; draft [T, V]: the probabilities that the drafts were drawn from, None for certain
    ones; uniform [T] and uniform_next [B]: random numbers in [0, 1)."""
    d = _device("target", target)
    if target.dim() != 2:
        _bad("target: a tensor [T, V] is needed")
    T, V = target.shape
    if kv_len.dim() != 1:
        _bad("kv_len: a tensor [B] is needed")
    B = kv_len.shape[0]
    half = target.dtype is _BF16
    kind = _BF16 if half else _FP32
    tp, ts = _rows("target", target, kind, (T, V), d)
    dp, ds = (0, 0) if draft is None else _rows("draft", draft, kind, (T, V), d)
    if out is None:
        out = Verified(*(_allocate(stream, torch.empty, B, dtype=torch.int32, device=target.device) for _ in range(3)))
    accepted, next_token, kept_len = out
    b, t = (B,), (T,)
    a = _PACK_VERIFY.pack(tp, dp, _i32("tokens", tokens, t, d), _i32("tok_start", tok_start, (B + 1,), d),
                          _i32("kv_len", kv_len, b, d), 0 if slot is None else _i32("slot", slot, t, d),
                          _vector("uniform", uniform, _FP32, T, d),
                          _vector("uniform_next", uniform_next, _FP32, B, d),
                          _i32("accepted", accepted, b, d), _i32("next_token", next_token, b, d),
                          _i32("kept_len", kept_len, b, d), ts, ds, T, B, V, half)
    _check(load_library().moe_verify_drafts(a, _stream(stream, d)), "moe_verify_drafts")
    return out
