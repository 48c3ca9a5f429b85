"""add_rms_norm refuses addresses inside an element (no GPU needed; none of these reaches a launch)."""
import pytest

from test_norm_overlaps import M, P, _call


@pytest.mark.parametrize("kw,name", [(dict(x=P + 1), "x"), (dict(dtype=1, x=P + 2, x_stride=256), "x"), (dict(residual=P + M + 1), "residual"),
                                     (dict(residual_out=P + 3 * M + 1), "residual_out"), (dict(out=P + 4 * M + 1), "out"),
                                     (dict(weight=P + 2 * M + 1), "weight"), (dict(scales=P + 6 * M + 2), "scales"),
                                     (dict(dtype=1, weight=P + 2 * M + 2), "weight")])
def test_refused(kw, name):
    from gated_mla_b200 import _lib as L
    status, message = _call(**kw)
    assert status == L.GMLA_ERR_INVALID_ARG and name in message and "aligned" in message
