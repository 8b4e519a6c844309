"""GPU: a layer takes a norm's codes only where the norm made them as the layer would."""

import pytest

import synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import block_fp8_mixture_gb300 as moe  # noqa: E402
from test_gpu_step_experts import layer_of  # noqa: E402


@pytest.fixture(autouse=True)
def _library():
    moe.load_library(build_if_missing=True)


WAYS = [(fmt, numerics) for fmt in (moe.SCALE_FP32, moe.SCALE_FP32_POW2, moe.SCALE_UE8M0) for numerics in (0, 1)]


@pytest.mark.parametrize("act_fmt,numerics", WAYS)
def test_layer_refuses_codes_of_another_format(act_fmt, numerics):
    case = synth.make_case("tiny", 16)
    sh = case.shape
    layer = layer_of(case, 16, act_fmt, numerics)
    x = torch.randn(16, sh.H, device="cuda").to(torch.bfloat16)
    w = torch.ones(sh.H, device="cuda")
    ids, weights = moe.route(torch.randn(16, sh.E, device="cuda"), sh.topk)
    for quant, way in WAYS:
        n = moe.rms_norm(x, w, quant=quant, numerics=way)
        assert (n.quant, n.numerics) == (quant, way) and len(n) == 4
        for given in (n, n._replace(out=None)):
            if quant == act_fmt and (way == numerics or quant != moe.SCALE_FP32):     # powers of two: the same either way
                assert torch.equal(layer(given, ids, weights), layer(n.out, ids, weights))
            else:
                with pytest.raises(moe.MoeError) as e:
                    layer(given, ids, weights)
                assert e.value.status == moe.MOE_ERR_INVALID_ARG
    # what a caller has put together from codes of its own is taken as it is
    own = moe.rms_norm(x, w, quant=act_fmt, numerics=numerics)
    assert torch.equal(layer(moe.Normed(None, None, own.codes, own.scales), ids, weights), layer(own, ids, weights))
    assert moe.rms_norm(x, w).quant is None
