"""GPU: norm and routing of values far from one, against the CPU statement in 64 bits.

The kernels carry some 40 bits up to the roundings that the header names, so whole numbers and BF16 values equal the
statement's but where that stands within 2^-40 of a border between two results.  Values are drawn a few million at a
time, so that an error of 2^-28 before the rounding to BF16 (borders 2^-8 apart) shows in some of them.
"""

import numpy as np
import pytest

import oracle
from oracle import step_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import block_fp8_mixture_gb300 as moe  # noqa: E402
from test_gpu_kv import dev  # noqa: E402
from test_gpu_step import same_bits  # noqa: E402


@pytest.fixture(autouse=True)
def _library():
    moe.load_library(build_if_missing=True)


def check(x, k, rel, bias=None, scale=1.0, **kw):
    """ids to the bit; weights within rel of their value, and half of fp32's smallest step."""
    ids, weights = moe.route(dev(x), k, bias=None if bias is None else dev(bias), scale=scale, **kw)
    want, w = step_ref.route(x, k, bias=bias, scale=scale, **{"groups" if a == "num_groups" else a: b for a, b in kw.items()})
    assert np.array_equal(ids.cpu().numpy(), want)
    got = weights.cpu().numpy().astype(np.float64)
    assert (np.abs(got - w) <= rel * np.abs(w) + 2.0 ** -150).all()


def test_route_order_of_neighbours_with_small_scores():
    """Scores that both round to 4.964734e-38; two of 22 bits; each pair once in either order."""
    for row in ([0.10412609577, 0.10412610322, 86.0], [0.0, -0.27704, -0.164926, -95.027985, -95.02769]):
        x = np.float32([row, row[::-1]])
        check(x, len(row), 2.0 ** -18)


@pytest.mark.parametrize("scoring", [0, 1])
@pytest.mark.parametrize("G", [1, 4])
def test_route_order_of_small_scores(scoring, G):
    """A few logits at the top and pairs some 2^-11 to 2^-24 apart far below, so that the choice hangs on how scores round that
    are small, or below fp32's normal numbers."""
    rng = np.random.default_rng(7 + G)
    M, E = 4000, 32
    x = np.repeat(rng.uniform(-104, -70, (M, E // 2)), 2, 1)
    x[:, ::2] += rng.choice([2.0 ** -16, 2.0 ** -13, 2.0 ** -11, 2.0 ** -9], (M, E // 2))
    if scoring == 0:
        x[:, ::8] = rng.uniform(-1, 0, (M, 4))          # one in each group, so that a group's value is one of these
    x = x.astype(np.float32)
    kw = dict(scoring=scoring, num_groups=G, topk_groups=G)
    check(x, 16, 2.0 ** -18, renormalize=False, **kw)
    check(x, 16, 2.0 ** -18, **kw)
    check(x, 16, 2.0 ** -18, bias=np.zeros(E, np.float32), **kw)
    if G > 1:
        check(x, 10, 2.0 ** -18, scoring=scoring, num_groups=G, topk_groups=2)


# Scores below 2^-104 that equal the statement's: what joins them are 4 additions over the lanes, a division and a product,
# 2^-24 of the value each.
FEW = 6 * 2.0 ** -24


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("k", [1, 3, 8, 16])
def test_route_renormalizes_small_sums(bias, k):
    """Sigmoid scores whose sum is below fp32's normal numbers: weights are still shares of it."""
    rng = np.random.default_rng(k)
    x = rng.uniform(-103.5, -91, (500, 48)).astype(np.float32)
    x[0], x[1] = -103.0, -92.0
    x[2, 1:] = -200.0
    x[3] = -200.0
    b = (rng.integers(0, 4, 48) / 8).astype(np.float32) if bias else None
    check(x, k, FEW, bias=b, scoring=1)
    check(x, k, FEW, bias=b, scoring=1, scale=2.5)


@pytest.mark.parametrize("scoring", [0, 1])
@pytest.mark.parametrize("G", [1, 4])
def test_route_weights_of_small_scores_that_a_bias_chose(scoring, G):
    """The bias chooses experts whose scores have few bits left, or none: their weights are shares of those scores."""
    rng = np.random.default_rng(3)
    x = rng.uniform(-106, -86, (600, 64)).astype(np.float32)
    b = (np.arange(64) % 16 / 16).astype(np.float32)
    x[:, 16 * np.arange(4)] = 1.0                        # the top of the softmax, which no bias helps
    b[16 * np.arange(4)] = -3.0
    x[5, 1::2] = -1e4                                    # finite masks
    kw = dict(scoring=scoring, bias=b, num_groups=G, topk_groups=G)
    check(x, 8, FEW, **kw)
    check(x, 8, FEW, renormalize=False, **kw)
    check(x, 12, FEW, scale=0.75, **kw)


# ------------------------------------------------------------------------------------------------ norm
def norm(xv, w, eps, wide, **kw):
    """The kernel's rows and the statement's."""
    wt = dev(w) if wide else dev(w).to(torch.bfloat16)
    got = moe.rms_norm(dev(xv).to(torch.bfloat16), wt, eps=eps, **kw).out
    return got, step_ref.rms_norm(xv, w, eps)[0]


def rows(rng, M, H, exponent):
    return oracle.bf16_round((rng.standard_normal((M, H)) * 2.0 ** exponent).astype(np.float32))


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("H", [8, 264, 4096, 4100])
def test_norm_of_far_products(wide, H):
    """The value times its weight leaves fp32's range where the normed value does not."""
    rng = np.random.default_rng(H)
    w = oracle.bf16_round(rng.standard_normal(H).astype(np.float32))
    for h_exponent, w_exponent, eps in ((50, 83, 1e-6), (66, 62, 1e-6), (30, 100, 1e-6), (120, 20, 1e-6), (-30, -95, 1e-20),
                                        (-20, -80, 1e-6), (-60, -60, 1e-20)):
        v = w * np.float32(2.0 ** w_exponent)
        if wide:
            v = (v * (1 + 2.0 ** -12 * rng.random(H))).astype(np.float32)
        got, want = norm(rows(rng, 700, H, h_exponent), v, eps, wide)
        assert np.isfinite(want).all()
        same_bits(got, want)
    got, _ = norm(np.full((2, H), 1e15, np.float32), np.full(H, 1e25, np.float32), 1e-6, True)
    same_bits(got, np.full((2, H), oracle.bf16_round(np.float32([1e25]))[0]))


@pytest.mark.parametrize("wide", [False, True])
def test_norm_of_results_beyond_the_largest_number(wide):
    """Infinite where the value times its weight is, with the value's sign; finite beside it."""
    w = np.full(64, 3e38, np.float32)
    w[1::2] = -1.0
    xv = rows(np.random.default_rng(0), 300, 64, 3)
    got, want = norm(xv, oracle.bf16_round(w), 1e-6, wide)
    assert np.isinf(want).any() and np.isfinite(want).any() and not np.isnan(want).any()
    same_bits(got, want)


@pytest.mark.parametrize("exponent", [40, 50, 56, 59, 61, 62])
@pytest.mark.parametrize("wide", [False, True])
def test_norm_of_large_rows_keeps_its_bits(exponent, wide):
    """Sums of squares below fp32's largest number, whose root's square is near its smallest."""
    rng = np.random.default_rng(exponent)
    w = rng.standard_normal(8).astype(np.float32)
    w = w if wide else oracle.bf16_round(w)
    got, want = norm(rows(rng, 1 << 18, 8, exponent), w, 1e-6, wide)
    same_bits(got, want)


@pytest.mark.parametrize("eps", [1e20, 1e30, 1e36, 1e38, 3.4e38])
@pytest.mark.parametrize("exponent", [0, 55, 62, 65, 70])
def test_norm_of_a_large_eps(eps, exponent):
    """eps counts in every row, whatever its values: in one whose squares leave fp32's range too."""
    rng = np.random.default_rng(exponent)
    w = rng.standard_normal(8).astype(np.float32)
    xv = rows(rng, 1 << 17, 8, exponent)
    same_bits(*norm(xv, w, eps, True))
    xv = rows(rng, 9, 4096, exponent)
    same_bits(*norm(xv, rng.standard_normal(4096).astype(np.float32), eps, True))
