"""The norm and rotation at the edges of its sizes: what a call refuses (made-up device addresses)."""
import pytest

from test_norm_boundary import INVALID, KD, QD, call, lib, message  # noqa: F401


@pytest.mark.parametrize("sizes", [dict(S=0), dict(B=0)])
@pytest.mark.parametrize("side,dw", [("q", QD), ("k", KD)])
def test_weight_gradients_of_no_rows_are_aligned(lib, sizes, side, dw):  # noqa: F811
    """They are written (zeros) all the same."""
    assert call(lib, "bwd", **sizes, **{side: dict(dw=dw + 2)}) == INVALID
    assert "aligned" in message(lib)
