"""Host-side checks at the borders of what the entry points take, on made-up addresses."""
import ctypes

import pytest

import muon_newton_schulz_04_b200 as mb
from test_model_ops_cpu import BASE, attention, built, check, grad, heads, wgrad  # noqa: F401


@pytest.mark.parametrize("rows,cols,want", [(1 << 30, 1, "OK"), (1, 1 << 30, "OK"), ((1 << 30) + 1, 1, "ERR_UNSUPPORTED"),
                                            (1, (1 << 30) + 1, "ERR_UNSUPPORTED"), ((1 << 31) - 1, 1, "ERR_UNSUPPORTED"),
                                            (1, (1 << 31) - 100, "ERR_UNSUPPORTED"), (1 << 16, 1 << 15, "ERR_INVALID"),
                                            (1 << 30, 2, "ERR_INVALID")])
def test_weight_grad_of_very_long_rows(rows, cols, want):
    """Rows and columns up to 2^30, as checkpoints have them: sizes are rounded up to tiles in 32 bits."""
    want = getattr(mb, "MUON_" + want)
    far = 1 << 44
    a = wgrad(tokens=5, rows=rows, cols=cols, dy=far, dy_stride=rows, codes=2 * far, scales=3 * far, G=4 * far,
              workspace=5 * far, workspace_bytes=1 << 43)
    need = ctypes.c_size_t(0)
    assert mb.lib().muon_weight_grad_workspace(ctypes.byref(a), ctypes.byref(need)) == want
    assert mb.lib().muon_validate_weight_grad(ctypes.byref(a)) == want
    assert need.value < 1 << 36
