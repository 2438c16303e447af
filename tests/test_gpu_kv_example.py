"""examples/attention_layer.py: projections, cache and attention together."""
import importlib.util
import os

import pytest

from quantized_weight_out_gb300 import inputs

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# The layer's projections round their inputs and decoded weights to fp16 (2^-11 each), which
# alone is well below 5e-3 of the result.  A cached value is off by at most half a step of its
# block, uniformly: rms step / sqrt(12).  A block of 32 normal values has its largest near 2.2
# deviations, so a Q8_0 step is about 2.2 / 127 and a Q4_0 step 2.2 / 8 of one: 0.5 % and 8 %
# rms of the values, about the same of the attention's mean over them, and some more through
# the scores; a factor of two above their sum.
@pytest.mark.parametrize("name,bound", [("f16", 5e-3), ("bf16", 2e-2), ("q8_0", 3e-2), ("q4_0", 0.35)])
def test_attention_layer(name, bound):
    spec = importlib.util.spec_from_file_location("attention_layer", os.path.join(ROOT, "examples", "attention_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    assert mod.run(inputs.NAME_TO_TYPE[name], prompts=(37, 1, 130, 64), steps=3, verbose=False) <= bound
