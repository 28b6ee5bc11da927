"""The extension module's handling of arguments that no caller should pass."""
import pytest
import torch

import gated_delta_rule_gdn_gb300 as gdn
from gated_delta_rule_gdn_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    gdn.load()


@pytest.mark.parametrize("name", ["\ud800", "x\udfff", "straße", "a" * 1000])
def test_keywords_of_any_text_are_refused(name):
    """Names without a UTF-8 form among them (a lone surrogate)."""
    x = torch.zeros(1, 4, 8)
    for call in (gdn.glr_scan_fwd, gdn.gdn_qk_norm_fwd, gdn.gdn_short_conv_fwd):
        with pytest.raises(TypeError, match="unexpected keyword"):
            call(x, x, **{name: 1})
    with pytest.raises(TypeError, match="multiple values for argument 'x'"):
        gdn.glr_scan_fwd(x, x, x=x)
    with pytest.raises(TypeError, match="missing argument 'g'"):
        gdn.glr_scan_fwd(x)


@pytest.mark.gpu
@pytest.mark.parametrize("norm", ["\ud800", "L2", "", 2, b"l2"])
def test_norms_of_any_text_are_refused(norm):
    q = torch.zeros(2, 3, 4, 8, device="cuda")
    with pytest.raises(ValueError, match="norm must be"):
        gdn.gdn_qk_norm_fwd(q, q, norm=norm)
