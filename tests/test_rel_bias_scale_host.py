"""The bias is taken over the softmax scale: a scale at which that overflows is refused."""
import ctypes

import pytest

from test_rel_bias_host import INVALID, _fill, abi  # noqa: F401


@pytest.mark.parametrize("scale,fine", [(2.0 ** -111, True), (2.0 ** -112, False), (1e-37, False), (1e-39, False), (1e30, True)])
def test_scales(abi, scale, fine):  # noqa: F811
    p = abi.AttnFwdParams()
    _fill(p, abi)
    p.softmax_scale = scale
    lib = abi.load()
    assert (lib.attn_fwd_workspace_size(ctypes.byref(p)) > 2 * 4 * 100 * 64 * 2 + 1024) == fine  # V's copy and the bias
    if not fine:
        assert lib.attn_fwd(ctypes.byref(p), None, 0, None) == INVALID
