"""examples/experts_layer.py: lookup, router and experts' products together, both directions."""
import importlib.util
import os

import pytest

from quantized_weight_out_gb300 import inputs

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# The activations between the calls are bf16: x, gate, up, h and y, and on the way back dy's
# products, each off by at most 2^-8 (rms 2^-8 / sqrt(3), 2.3e-3) of a value; the operands' fp16
# roundings are an eighth of that.  Five of them on the way to y in root sum of squares are
# 5e-3, eight on the way to dx 6.4e-3; silu's slope, up to 1.1 over a value's own size, and
# products of two rounded factors are within a factor of three.
@pytest.mark.parametrize("name,tokens", [("q4_k", 300), ("q8_0", 40), ("mxfp4", 200), ("bf16", 97)])
def test_experts_layer(name, tokens):
    spec = importlib.util.spec_from_file_location("experts_layer", os.path.join(ROOT, "examples", "experts_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    inner = 1024 if name == "mxfp4" else 768
    y, dx, da, decoded = mod.run(inputs.NAME_TO_TYPE[name], tokens=tokens, inner=inner, verbose=False)
    assert y <= 1.5e-2 and decoded <= 1.5e-2
    assert dx <= 2e-2 and da <= 2e-2
