"""GPU: random calls of norm, routing and verification against their CPU statement in 64 bits: odd sizes, strides, ties,
masks, infinities, tables out of range, values far from one.  Each test is a seed; `python tests/test_gpu_step_random.py
<first seed> <seconds>` runs as many as fit."""

import sys
import time

import numpy as np
import pytest

if __name__ == "__main__":
    import os
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import oracle  # noqa: E402
from oracle import step_ref  # noqa: E402

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import block_fp8_mixture_gb300 as moe  # noqa: E402
from test_gpu_kv import dev  # noqa: E402
from test_gpu_step import check_norm, check_route, check_verify, f32, step  # noqa: E402


@pytest.fixture(autouse=True)
def _library():
    moe.load_library(build_if_missing=True)


def some_route(rng):
    G = int(rng.choice([1, 1, 1, 2, 3, 4, 8, 8, 16, 32]))
    lanes = 1 << (G - 1).bit_length()
    size = min(int(rng.integers(1, 301)), 1024 // lanes)
    E, best = G * size, int(rng.integers(1, G + 1))
    k, M = int(rng.integers(1, min(16, size * best) + 1)), int(rng.integers(1, 300))
    x = rng.choice([0.1, 1.0, 2.0, 10.0, 40.0]) * rng.standard_normal((M, E)) + rng.choice([0, 0, -5, 5, -60, -95])
    x = x.astype(np.float32)
    mode = rng.integers(0, 7)
    if mode == 0:
        x = np.round(x * 2) / 2                                        # ties
    elif mode == 1:                                                    # neighbours
        x = (np.repeat(x, 3, 1)[:, :E].copy().view(np.int32) + rng.integers(-2, 3, x.shape)).astype(np.int32).view(np.float32)
    elif mode == 2:
        x[rng.random(x.shape) < rng.choice([0.3, 0.95])] = -np.inf
    elif mode == 3:
        x[rng.random(x.shape) < 0.01] = rng.choice([np.nan, np.inf, -np.inf, 0.0, -0.0])
    elif mode == 4:
        x[rng.random(x.shape) < rng.choice([0.3, 0.95])] = rng.choice([-1e4, -100, -90])
    bias = None
    if rng.random() < 0.6:
        bias = (rng.choice([0.01, 0.3, 3.0]) * rng.standard_normal(E)).astype(np.float32)
        if rng.random() < 0.2:
            bias = np.round(bias * 4) / 4
        if rng.random() < 0.1:
            bias[rng.integers(0, E)] = rng.choice([np.inf, -np.inf, np.nan])
    check_route(x, k, scoring=int(rng.integers(0, 2)), bias=bias, num_groups=G, topk_groups=best,
                group_best=int(rng.integers(1, 3)), half=bool(rng.random() < 0.4), pad=int(rng.choice([0, 0, 1, 4, 8])),
                renormalize=bool(rng.random() < 0.7))


def some_norm(rng):
    M, H = int(rng.integers(1, 80)), int(rng.choice([rng.integers(1, 600), rng.integers(1, 9000), 8 * rng.integers(1, 1024),
                                                     rng.integers(8193, 32769)]))
    M = min(M, 12) if H > 9000 else M
    quant = [None, 0, 1, 2][rng.integers(0, 4)]
    check_norm(M, H, bool(rng.random() < .5), bool(rng.random() < .5), bool(rng.random() < .5), quant,
               live=None if rng.random() < .7 else int(rng.integers(-2, M + 3)), pad=int(rng.choice([0, 0, 1, 3, 4, 8, 16])),
               numerics=int(rng.integers(0, 2)), seed=int(rng.integers(0, 1 << 30)), gain=float(2.0 ** rng.integers(-30, 30)),
               write_out=quant is None or bool(rng.random() < .7))


def some_far_norm(rng):
    """Rows, weights and eps of any magnitude.  Results below 2^-100, and values below that share of the root, are left out:
    fewer bits are promised there."""
    M, H = int(rng.integers(1, 200)), int(rng.choice([rng.integers(1, 40), rng.integers(1, 600), 8 * rng.integers(1, 600)]))
    x = rng.standard_normal((M, H)) * 2.0 ** rng.integers(-90, 125, (M, 1))
    if rng.random() < .3:
        x *= 2.0 ** rng.integers(-40, 1, x.shape)
    x = oracle.bf16_round(x.astype(np.float32))
    w = (rng.standard_normal(H) * 2.0 ** rng.integers(-100, 118)).astype(np.float32)
    wide = bool(rng.random() < .5)
    w = w if wide else oracle.bf16_round(w)
    eps = float(10.0 ** rng.uniform(-20, 38))
    got = f32(moe.rms_norm(dev(x).to(torch.bfloat16), dev(w) if wide else dev(w).to(torch.bfloat16), eps=eps).out)
    want = step_ref.rms_norm(x, w, eps)[0]
    x64 = x.astype(np.float64)
    root = np.sqrt((x64 * x64).mean(-1, keepdims=True) + eps)
    ok = (np.abs(want) >= 2.0 ** -100) & (np.abs(x64) >= 2.0 ** -100 * root)
    assert np.array_equal(got[ok], want[ok]) and not np.isnan(got).any()


def some_verify(rng):
    B = int(rng.integers(1, 40))
    V = int(rng.choice([rng.integers(1, 40), rng.integers(1, 3000), rng.integers(1, 60000), 1024 * rng.integers(1, 40),
                        1024 * rng.integers(1, 40) + 1]))
    n = rng.integers(0, int(rng.choice([2, 4, 9])), B)
    if n.sum() * V > 4e6:
        n = n[:max(1, int(4e6 / V / 5))]
    if n.sum() == 0:
        n[0] = 2
    B, mode = len(n), int(rng.integers(0, 5))
    a = list(step(rng, n, V, certain=bool(rng.random() < .4), near=float(rng.choice([0, .1, .5, 3]))))
    T = a[0].shape[0]
    if mode == 1:                                                      # coarse numbers: sums and products are exact
        a[:2] = [None if z is None else rng.integers(0, 4, (T, V)).astype(np.float32) / 64 for z in a[:2]]
        a[5], a[6] = (rng.integers(0, 17, s).astype(np.float32) / 16 for s in (T, B))
    elif mode == 2:
        a[0][rng.random(a[0].shape) < .9] = 0
        if a[1] is not None and rng.random() < .5:
            a[1] = a[0].copy()
        a[0][rng.random(T) < .2] = 0
    elif mode == 3:
        for z in a[:2]:
            if z is not None:
                m = rng.random(z.shape) < min(.01, 3.0 / V)
                z[m] = rng.choice(np.float32([np.nan, np.inf, -np.inf, -1, -0.0, 1.0, 1e-45]), m.sum())
        a[5][rng.random(T) < .2] = rng.choice(np.float32([np.nan, -1, 2, np.inf]))
        a[6][rng.random(B) < .2] = rng.choice(np.float32([np.nan, -1, 2, np.inf]))
        a[2][rng.random(T) < .1] = rng.choice([-1, V, V + 7, -2 ** 31, 2 ** 31 - 1])
    elif mode == 4:
        a[3] = np.array(a[3])
        a[3][rng.integers(0, len(a[3]))] = rng.choice([-5, T + 9, 0, 2 ** 31 - 1])
    slot = None
    if rng.random() < .5:
        slot = rng.integers(0, 100, T)
        slot[rng.random(T) < .2] = -1
    check_verify(*a, half=bool(rng.random() < .4), pad=int(rng.choice([0, 0, 1, 3, 4, 8])), slot=slot)


CALLS = (some_route, some_norm, some_far_norm, some_verify)


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("seed", range(4))
def test_random_calls(call, seed):
    for i in range(30):
        call(np.random.default_rng([seed, i]))


if __name__ == "__main__":
    first, until, counts = int(sys.argv[1]), time.time() + float(sys.argv[2]), [0] * len(CALLS)
    moe.load_library(build_if_missing=True)
    while time.time() < until:
        for c, call in enumerate(CALLS):
            seed = [1000 + first, counts[c]]
            try:
                call(np.random.default_rng(seed))
            except Exception:
                print("failed:", call.__name__, seed)
                raise
            counts[c] += 1
    print({call.__name__: n for call, n in zip(CALLS, counts)})
