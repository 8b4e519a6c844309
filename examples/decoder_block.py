"""A decoder block served step by step: paged 8-bit attention, then the block-FP8 experts.

Requests of different lengths are prefilled in one step and decoded for a few more; one finishes on the
way, and its pages serve a new request.  Weights and inputs are random.  The attention of every step is
checked against a plain fp32 computation over the same rotated keys and values, unquantized, so the
difference printed is what the 8-bit cache costs.

    python examples/decoder_block.py
"""

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_fp8_mixture_gb300 as moe  # noqa: E402
import synth  # noqa: E402

HQ, HKV, D, PAGE = 8, 2, 64, 16          # heads, key/value heads, head size, tokens per page
B, MAX_TOKENS = 3, 96


def rotate(x, rope, pos):
    """Half layout, fp32."""
    c, s = rope[pos][:, None, :, 0], rope[pos][:, None, :, 1]
    a, b = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def main(seed: int = 0, verbose: bool = True) -> float:
    moe.load_library(build_if_missing=True)
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = synth.SHAPES["tiny"]          # 8 experts, hidden 512, top-2
    H = shape.H

    def rand(*size):
        return torch.randn(*size, generator=g, device="cuda")

    w_qkv = (rand(H, (HQ + 2 * HKV) * D) / H ** 0.5).to(torch.bfloat16)
    w_out = (rand(HQ * D, H) / (HQ * D) ** 0.5).to(torch.bfloat16)
    w_gate = rand(H, shape.E) / H ** 0.5
    w = synth.make_case("tiny", 16).weights
    experts = moe.MoELayer(*(torch.from_numpy(a).cuda() for a in (w.w13, w.s13, w.w2, w.s2)),
                           max_tokens=MAX_TOKENS, topk=shape.topk)
    attention = moe.PagedAttention(num_layers=1, num_pages=24, page_size=PAGE, num_heads=HQ, num_kv_heads=HKV,
                                   head_dim=D, max_requests=B, max_pages=8, max_tokens=MAX_TOKENS, max_q=MAX_TOKENS,
                                   rope=moe.rope_table(128, D))

    lengths = [40, 7, 23]
    steps = [lengths, [41, 8, 24], [42, 0, 25], [43, 12, 26], [44, 13, 27]]   # request 1 finishes, a new one joins
    past = [[], [], []]                    # rotated keys and values of each request, for the check
    worst = 0.0
    have = [0] * B
    for new in steps:
        t = attention.advance(torch.tensor(new, dtype=torch.int32, device="cuda"))
        x = rand(MAX_TOKENS, H).to(torch.bfloat16)
        q, k, v = (a.unflatten(1, (-1, D)) for a in (x @ w_qkv).split([HQ * D, HKV * D, HKV * D], 1))
        o = attention(0, q, k, v)
        x = x + o.flatten(1) @ w_out
        weight, ids = torch.softmax(x.float() @ w_gate, -1).topk(shape.topk)
        y = x + experts(x, ids.to(torch.int32), weight, d_num_tokens=t.info[:1])
        assert moe.last_device_status(attention.workspace) == moe.MOE_OK
        assert moe.last_device_status(experts.workspace) == moe.MOE_OK
        added, _, refused, _ = t.info.tolist()
        assert refused == 0 and bool(torch.isfinite(y[:added].float()).all())
        # plain attention over the same tokens
        rope, start = attention.rope, t.tok_start.tolist()
        for b in range(B):
            if new[b] <= have[b]:
                past[b] = past[b] if new[b] else []
                continue
            rows = slice(start[b], start[b + 1])
            pos = torch.arange(have[b], new[b], device="cuda")
            past[b].append((rotate(k[rows].float(), rope, pos), v[rows].float()))
            kk, vv = (torch.cat(c).repeat_interleave(HQ // HKV, 1) for c in zip(*past[b]))
            s = torch.einsum("ihd,jhd->hij", rotate(q[rows].float(), rope, pos), kk) * D ** -0.5
            s.masked_fill_(torch.arange(new[b], device="cuda")[None, None] > pos[None, :, None], float("-inf"))
            ref = torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), vv)
            err = float((o[rows].float() - ref).norm() / ref.norm())
            worst = max(worst, err)
        have = new
        if verbose:
            print(f"lengths {new}: {added} tokens added, {int(t.free_count)} pages free, attention within "
                  f"{worst:.3f} of unquantized fp32 (relative)")
    return worst


if __name__ == "__main__":
    assert np.isfinite(main())
