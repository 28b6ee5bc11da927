"""The example that runs the operators together: decoding continues a prefill, and training lowers the loss.

Both sides of the continuation round every operator's output to bf16 (unit roundoff 2^-8) at about eight places in a row
(projection, convolution, norm, mixer, output, and the chunk kernels' 16-bit operands): 8 * 2^-8 = 3.1e-2.
"""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu


def test_hybrid_mixer():
    from gated_delta_rule_gdn_gb300 import build
    build.build()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import hybrid_mixer
    errors, losses = hybrid_mixer.main()
    assert max(errors) <= 3.1e-2, errors
    assert losses[-1] < 0.7 * losses[0], losses
