"""nm_kv4_attention refuses a scale that is no number (no GPU)."""
import ctypes
import math

import pytest

from tests.test_kv4_refusals import P, cache, nm  # noqa: F401


@pytest.mark.parametrize("scale,ok", [(math.nan, False), (math.inf, False), (-math.inf, False), (0.0, True), (-0.7, True)])
def test_scale_is_finite(nm, scale, ok):
    """Checked before the kernels, which would take a NaN for next to nothing. Without tokens there is nothing to run."""
    c = cache(nm)
    got = nm.lib().nm_kv4_attention(ctypes.byref(c), 0, None, None, 0, 0, 1, P, 512, 4, scale, P, 512, None, None)
    assert got == (nm.NM_OK if ok else nm.NM_ERR_INVALID_ARG)
