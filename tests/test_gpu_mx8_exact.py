"""The routed experts on operands whose fp32 sums are exact (mx8_exact.py): h bit for bit and the
results of down within its own bound, by every way that a call can take.
Each test prints the case it runs (flushed) before touching the GPU.
"""
import pytest

import mx8_exact as ex
from test_gpu_mx4 import DT, awq, say  # noqa: F401
from test_gpu_mx8 import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("case", range(len(ex.LAYERS)))
def test_experts_h(awq, case, dt):
    """The 8-bit h of every pair, shown by a down product of single ones: the definition's, whatever
    the way and Y's type."""
    say("experts' h", *ex.LAYERS[case], dt)
    layer = ex.Layer(*ex.LAYERS[case], case, True)
    Y = awq.mx4_experts(*dev(*layer.arrays()), dtype=DT[dt])
    off = layer.check(Y.cpu().double().numpy(), dt)
    say("err/bound", off)
    assert off <= 1


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("case", range(len(ex.LAYERS)))
def test_experts_sums(awq, case, dt):
    say("experts' sums", *ex.LAYERS[case], dt)
    layer = ex.Layer(*ex.LAYERS[case], 100 + case, False)
    Y = awq.mx4_experts(*dev(*layer.arrays()), dtype=DT[dt])
    off = layer.check(Y.cpu().double().numpy(), dt, ex.some_tokens(layer.shape[0], 8))
    say("err/bound", off)
    assert off <= 1
