"""Pins of the paged cache's CPU statement to something other than itself: hand-worked tables,
invariants of the free stack, rotations as complex products, a dense softmax."""

import numpy as np
import pytest

import oracle
from oracle import kv_ref


def test_tables_by_hand():
    # request 0 grows over a page edge, 1 finishes, 2 arrives, 3 rolls back inside its page
    table = [[7, -1, -1], [3, 5, -1], [-1, -1, -1], [2, -1, -1]]
    t = kv_ref.kv_tables([15, 20, 0, 9], [18, 0, 33, 4], table, [9, 8, 0, 0, 0, 0, 0, 0, 0, 0], 2, 16, 40, 8)
    # stack 9 8 3 5; four pages granted, the whole stack in stored order
    assert t["block_table"].tolist() == [[7, 9, -1], [-1, -1, -1], [8, 3, 5], [2, -1, -1]]
    assert t["free_count"].tolist() == [0] and t["info"].tolist() == [36, 5, 0, 4]
    assert t["kv_len"].tolist() == [18, 0, 33, 4] and t["tok_start"].tolist() == [0, 3, 3, 36, 36]
    assert t["slot"][:4].tolist() == [7 * 16 + 15, 9 * 16, 9 * 16 + 1, 8 * 16]
    assert t["slot"][35] == 5 * 16 and t["slot"][36:].tolist() == [-1] * 4
    assert t["run_tok"].tolist() == [0, 1, 3, 19, 35, 0, 0, 0]
    assert t["run_len"].tolist() == [1, 2, 16, 16, 1, 0, 0, 0]


def test_tables_refuse_in_order():
    table = np.full((3, 4), -1)
    t = kv_ref.kv_tables([0, 0, 0], [16, 33, 16], table, [4, 5, 6], 3, 16, 65, 8)
    assert t["kv_len"].tolist() == [16, 0, 0] and t["info"].tolist() == [65, 1, 2, 1]
    assert t["free_count"].tolist() == [2] and t["block_table"][0, 0] == 6
    assert (t["slot"][16:] == -1).all() and t["request"][20] == 1


def test_growing_and_giving_back_restores_the_stack():
    rng = np.random.default_rng(3)
    P, B, W, N = 16, 9, 12, 120
    free = rng.permutation(N).astype(np.int32)
    zero = [0] * B
    want = rng.integers(0, W * P, B)
    a = kv_ref.kv_tables(zero, want, np.full((B, W), -1), free, N, P, 2000, 400)
    used = a["block_table"][a["block_table"] >= 0]
    left = a["free_list"][:a["free_count"][0]]
    assert sorted(used.tolist() + left.tolist()) == list(range(N))
    b = kv_ref.kv_tables(want, zero, a["block_table"], a["free_list"], a["free_count"][0], P, 0, 0)
    assert np.array_equal(b["free_list"], free) and b["free_count"][0] == N


@pytest.mark.parametrize("layout", [0, 1])
def test_rotation_is_a_complex_product(layout):
    rng = np.random.default_rng(layout)
    x = rng.standard_normal((5, 2, 64)).astype(np.float32)
    pos = np.array([0, 1, 17, 1000, 40])
    rope = kv_ref.rope_table(1001, 32)
    got = kv_ref.rotate(x, rope, pos, layout)
    f = 10000.0 ** (-np.arange(16) / 16)
    z = np.exp(1j * pos[:, None] * f)[:, None]
    a, b = (x[..., :16], x[..., 16:32]) if layout == 0 else (x[..., 0:32:2], x[..., 1:32:2])
    y = (a + 1j * b) * z
    ga, gb = (got[..., :16], got[..., 16:32]) if layout == 0 else (got[..., 0:32:2], got[..., 1:32:2])
    # three fp32 roundings of values up to |x| <= 6
    assert np.abs(ga - y.real).max() < 3 * 6 * 2.0 ** -24 * 2 and np.abs(gb - y.imag).max() < 36 * 2.0 ** -24
    assert np.array_equal(got[..., 32:], x[..., 32:])


def test_ramp_keeps_fast_pairs_and_interpolates_slow_ones():
    plain = kv_ref.rope_frequencies(64)
    ramp = kv_ref.rope_frequencies(64, scaling=2, factor=8.0, low=1.0, high=4.0, original_len=8192)
    turns = 8192 * plain / (2 * np.pi)
    assert np.array_equal(ramp[turns >= 4], plain[turns >= 4])
    assert np.allclose(ramp[turns <= 1], plain[turns <= 1] / 8, rtol=1e-15)
    assert np.all(np.diff(ramp) < 0)


def test_cache_write_rescales_older_tokens():
    codes = np.zeros((2, 1, 16, 64), np.uint8)
    scale = np.zeros((2, 1), np.float32)
    small = np.full((3, 1, 64), 0.5, np.float32)
    kv_ref.cache_write(small, codes, scale, [16, 17, 18], [0], [3], 16, oracle.SCALE_FP32_POW2)
    assert scale[1, 0] == 2.0 ** -9 and (oracle.e4m3_decode(codes[1, 0, :3]) == 256).all()
    big = np.full((1, 1, 64), 4.0, np.float32)
    kv_ref.cache_write(big, codes, scale, [19], [0], [1], 16, oracle.SCALE_FP32_POW2)
    assert scale[1, 0] == 2.0 ** -6
    assert (oracle.e4m3_decode(codes[1, 0, :3]) == 32).all()       # 32 * 2^-6 = 0.5 still
    assert (oracle.e4m3_decode(codes[1, 0, 3]) == 256).all() and (codes[1, 0, 4:] == 0).all()


@pytest.mark.parametrize("window", [0, 3])
def test_attention_against_a_dense_softmax(window):
    rng = np.random.default_rng(5)
    P, Hkv, D, L, n = 16, 2, 64, 21, 4
    x = rng.standard_normal((2, 2, Hkv, P, D)).astype(np.float32)
    codes = [oracle.e4m3_encode(v) for v in x]
    scale = [np.full((2, Hkv), 0.25, np.float32)] * 2
    q = rng.standard_normal((n, 4, D))
    out, mag = kv_ref.attention(q, codes, scale, np.array([[1, 0]]), [L], [0, n], 0.1, window)
    k, v = ((oracle.e4m3_decode(c)[[1, 0]] * 0.25).transpose(1, 0, 2, 3).reshape(Hkv, 32, D)[:, :L] for c in codes)
    for i in range(n):
        p = L - n + i
        lo = max(0, p - window + 1) if window else 0
        for h in range(4):
            e = np.exp(k[h // 2, lo:p + 1] @ q[i, h] * 0.1)
            assert np.allclose(out[i, h], (e / e.sum()) @ v[h // 2, lo:p + 1], rtol=1e-12, atol=1e-14)
    assert (mag >= np.abs(out) - 1e-12).all()


def test_attention_rows_that_see_nothing_are_zero():
    codes = [np.full((1, 1, 16, 64), 0x7F, np.uint8)] * 2          # NaN codes everywhere
    scale = [np.ones((1, 1), np.float32)] * 2
    out, _ = kv_ref.attention(np.ones((3, 1, 64)), codes, scale, np.array([[0], [0]]), [0, 0], [0, 1, 3], 1.0)
    assert (out == 0).all()
