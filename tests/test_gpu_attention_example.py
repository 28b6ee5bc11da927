"""The example of linear attention and the paged cache runs, its decoding continues its prefill, and its gradients are right."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_attention_mixers():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_mixers.py")
    spec = importlib.util.spec_from_file_location("attention_mixers", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    linear, attention, gradient = module.main()
    # outputs are bf16 (2^-8 of an element each), scores and states enter products as bf16, and the output projection adds as much
    assert linear <= 4 * 2.0 ** -8 and attention <= 4 * 2.0 ** -8
    # a central difference of step 1e-2 is off by a sixth of 1e-4 times the third derivative (here of the order of the first)
    # and by fp32 sums (2^-24 of the terms) over 2e-2
    assert gradient <= 1e-3
