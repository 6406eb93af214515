"""Host-side checks at the borders of what the entry points take, on made-up addresses."""
import ctypes
import random

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


def taken(base, rows, rs, n, hs, d):
    return {base + r * rs + h * hs + e for r in range(rows) for h in range(n) for e in range(d)}


def test_overlap_by_counting():
    """q and out as views of one array: what is accepted shares no element, and views at the same strides that share
    none are accepted: vectors of the heads side by side, interleaved head by head, rows padded, heads first."""
    rng = random.Random(3)
    seen = {True: 0, False: 0}
    for _ in range(4000):
        rows, n, d = rng.randint(1, 4), rng.randint(1, 4), 8 * rng.randint(1, 2)
        inner, pad = 8 * rng.randint(d // 8, 6), 8 * rng.choice((0, 0, 1, 2))
        first, second = (n, rows) if rng.random() < 0.5 else (rows, n)      # counts of the inner and the outer dimension
        outer = inner * rng.randint(first, first + 2) + pad
        strides = (outer, inner) if first == n else (inner, outer)          # of rows, of heads
        other = strides
        if rng.random() < 0.3:
            other = (8 * rng.randint(0, 20), 8 * rng.randint(0, 20))
        shift = 8 * rng.randint(-30, 30)
        q = mb._Heads(BASE, *strides)
        out = mb._Heads(BASE + 2 * shift, *other)
        a = attention(n_heads=n, n_kv_heads=n, head_dim=d, total_q=rows, q=q, out=out,
                      k=heads(2, 4096, 64), v=heads(3, 4096, 64))
        got = check(a)
        itself = len(taken(0, rows, other[0], n, other[1], d)) == rows * n * d
        shares = bool(taken(0, rows, strides[0], n, strides[1], d) & taken(shift, rows, other[0], n, other[1], d))
        if got == mb.MUON_OK:
            assert itself and not shares, (rows, n, d, strides, other, shift)
        elif other == strides:
            assert shares, (rows, n, d, strides, shift)
        seen[got == mb.MUON_OK] += 1
    assert min(seen.values()) > 400, seen


def test_gradients_interleaved_head_by_head():
    """dq, dk and dv of a fused projection whose heads lie as q, k, v, q, k, v, ..., also with a single row, and with
    rows longer than their heads."""
    d, n = 64, 4
    p = BASE + 0x80000000
    for rows, row in ((100, 3 * d * n), (1, 3 * d * n), (100, 3 * d * n + 40)):
        part = [mb._Heads(p + 2 * d * i, row, 3 * d) for i in range(3)]
        fwd = attention(n_kv_heads=n, total_q=rows, total_k=rows, k=heads(1, 256, 64), v=heads(2, 256, 64))
        g = grad(fwd, dq=part[0], dk=part[1], dv=part[2])
        assert mb.lib().muon_validate_attention_grad(ctypes.byref(g)) == mb.MUON_OK
        g = grad(fwd, dq=part[0], dk=part[1], dv=mb._Heads(p + 2 * d * 2 - 16, row, 3 * d))
        assert mb.lib().muon_validate_attention_grad(ctypes.byref(g)) == mb.MUON_ERR_INVALID
