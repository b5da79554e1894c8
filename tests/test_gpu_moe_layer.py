"""The example of a mixture-of-experts layer: decode, prefill and training
through the library's calls, against plain torch."""
import importlib.util
import os

import pytest

from _gpu import require_gpu

pytestmark = pytest.mark.gpu
EXAMPLE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer.py")


def test_example_layer():
    require_gpu()
    spec = importlib.util.spec_from_file_location("moe_layer", EXAMPLE)
    layer = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(layer)
    worst = layer.main()
    # BF16 roundings (2^-9 on average): two in the decoding chain's products and one of its sum, one elsewhere
    assert worst["decode, 1 tokens"] < 8e-3 and worst["decode, 7 tokens"] < 8e-3
    assert worst["prefill, combine"] < 4e-3
    assert worst["gradient of the experts' rows"] < 4e-3
    assert worst["gradient of the logits"] < 1e-4  # FP32 throughout
    assert worst["prefill, FP8 against FP32 weights"] < 8e-2  # E4M3 operands: 2^-4 steps, on average a third of that
