"""Host-side checks of the attention, checkpoint and weight-gradient entry points: every
refusal is decided before anything is launched, so it is tested without a GPU on made-up
addresses."""
import ctypes

import pytest

import muon_newton_schulz_04_b200 as mb
from muon_newton_schulz_04_b200 import build as mbuild


@pytest.fixture(scope="module", autouse=True)
def built():
    mbuild.build()


BASE = 0x100000000


def heads(place, rs, hs):
    return mb._Heads(BASE + place * 0x10000000, rs, hs)


def attention(**kw):
    d = dict(n_seqs=2, n_heads=4, n_kv_heads=2, head_dim=64, total_q=100, total_k=100, cu_seqlens_q=0x1000,
             cu_seqlens_k=0x1000, scale=0.125, q=heads(0, 256, 64), k=heads(1, 128, 64), v=heads(2, 128, 64),
             out=heads(3, 256, 64), lse=BASE + 4 * 0x10000000, max_logits=BASE + 5 * 0x10000000)
    d.update(kw)
    return mb._AttentionArgs(*[d[n] for n, _ in mb._AttentionArgs._fields_])


def check(a):
    return mb.lib().muon_validate_attention(ctypes.byref(a))


def test_attention_accepts():
    for kw in (dict(), dict(max_logits=None), dict(n_seqs=0, cu_seqlens_q=None, cu_seqlens_k=None),
               dict(total_q=0, q=mb._Heads(), out=mb._Heads(), lse=None), dict(total_k=0, k=mb._Heads(), v=mb._Heads()),
               dict(head_dim=8), dict(q=heads(0, 64, 6400), out=heads(3, 64, 6400)),        # heads first
               dict(q=heads(0, 1024, 64)), dict(total_q=1, q=heads(0, 0, 64), out=heads(3, 3, 64)),
               dict(n_heads=1, n_kv_heads=1, q=heads(0, 64, 0))):
        assert check(attention(**kw)) == mb.MUON_OK, kw
    # q, k and v side by side in one array, out in the next columns of it
    row, p = 512 * 2, BASE
    fused = dict(q=mb._Heads(p, row, 64), k=mb._Heads(p + 256 * 2, row, 64), v=mb._Heads(p + 384 * 2, row, 64),
                 out=mb._Heads(p + 512 * 2, row, 64))
    assert check(attention(**fused)) == mb.MUON_OK


@pytest.mark.parametrize("kw", [
    dict(n_seqs=-1), dict(n_heads=0), dict(n_kv_heads=3), dict(head_dim=0), dict(total_q=-1), dict(scale=0.0),
    dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(cu_seqlens_q=None),
    dict(cu_seqlens_k=0x1002), dict(q=mb._Heads(None, 256, 64)), dict(lse=None), dict(lse=BASE + 0x40000002),
    dict(q=heads(0, 64, 64)), dict(k=heads(1, 0, 64)), dict(q=heads(0, -256, 64)), dict(q=heads(0, 256, 32)),
    dict(out=heads(0, 256, 64)), dict(out=mb._Heads(BASE + 512, 256, 64)), dict(lse=BASE + 0x10000000),
    dict(max_logits=BASE + 4 * 0x10000000 + 64), dict(max_logits=0x1004),
])
def test_attention_refuses(kw):
    assert check(attention(**kw)) == mb.MUON_ERR_INVALID


@pytest.mark.parametrize("kw", [dict(head_dim=12), dict(head_dim=136, q=heads(0, 600, 136)),
                                dict(q=mb._Heads(BASE + 8, 256, 64)), dict(q=heads(0, 260, 64)),
                                dict(q=heads(0, 1024, 68)), dict(n_heads=65536, n_kv_heads=2)])
def test_attention_does_not_support(kw):
    assert check(attention(**kw)) == mb.MUON_ERR_UNSUPPORTED


@pytest.mark.parametrize("scale,want", [(2.0 ** -64, mb.MUON_OK), (2.0 ** 64, mb.MUON_OK),
                                        (2.0 ** -65, mb.MUON_ERR_UNSUPPORTED), (2.0 ** 65, mb.MUON_ERR_UNSUPPORTED)])
def test_attention_scales(scale, want):
    assert check(attention(scale=scale)) == want


def grad(fwd=None, **kw):
    d = dict(forward=fwd if fwd is not None else attention(), grad_out=heads(6, 256, 64), dq=heads(7, 256, 64),
             dk=heads(8, 128, 64), dv=heads(9, 128, 64), delta=BASE + 10 * 0x10000000)
    d.update(kw)
    return mb._AttentionGradArgs(*[d[n] for n, _ in mb._AttentionGradArgs._fields_])


def test_attention_grad():
    L = mb.lib()
    ok = [grad(), grad(grad_out=heads(3, 256, 64)),      # read twice
          grad(dk=mb._Heads(BASE + 0x80000000, 256, 64), dv=mb._Heads(BASE + 0x80000000 + 256, 256, 64))]
    for g in ok:
        assert L.muon_validate_attention_grad(ctypes.byref(g)) == mb.MUON_OK
    for kw in (dict(delta=None), dict(delta=BASE + 2), dict(dq=heads(0, 256, 64)), dict(dk=heads(9, 128, 64)),
               dict(dv=mb._Heads(None, 128, 64)), dict(grad_out=heads(7, 256, 64)), dict(delta=BASE + 4 * 0x10000000),
               dict(fwd=attention(scale=0.0))):
        g = grad(**kw)
        assert L.muon_validate_attention_grad(ctypes.byref(g)) == mb.MUON_ERR_INVALID, kw
    assert L.muon_validate_attention_grad(None) == mb.MUON_ERR_INVALID
    assert L.muon_validate_attention(None) == mb.MUON_ERR_INVALID


def wgrad(**kw):
    d = dict(tokens=100, rows=64, cols=96, dy=BASE, dy_stride=64, codes=BASE + 0x10000000, scales=BASE + 0x20000000,
             G=BASE + 0x30000000, grad_dtype=mb.MUON_FP32, accumulate=0, workspace=BASE + 0x40000000,
             workspace_bytes=1 << 27)
    d.update(kw)
    return mb._WeightGradArgs(*[d[n] for n, _ in mb._WeightGradArgs._fields_])


def test_weight_grad_checks():
    L = mb.lib()
    for kw in (dict(), dict(tokens=0, dy=None, codes=None, scales=None), dict(grad_dtype=mb.MUON_BF16, accumulate=1),
               dict(tokens=1, dy_stride=0), dict(dy_stride=71), dict(dy=BASE + 2), dict(rows=63, cols=97),
               dict(tokens=20000, rows=768, cols=768, dy_stride=768)):
        a = wgrad(**kw)
        need = ctypes.c_size_t(0)
        assert L.muon_weight_grad_workspace(ctypes.byref(a), ctypes.byref(need)) == mb.MUON_OK, kw
        assert L.muon_validate_weight_grad(ctypes.byref(a)) == mb.MUON_OK, kw
        if need.value:
            for w in (dict(workspace=None), dict(workspace_bytes=need.value - 1), dict(workspace=BASE + 0x40000008)):
                b = wgrad(**{**kw, **w})
                assert L.muon_validate_weight_grad(ctypes.byref(b)) == mb.MUON_ERR_INVALID
    for kw in (dict(tokens=-1), dict(rows=0), dict(cols=0), dict(dy=None), dict(codes=None), dict(scales=None),
               dict(G=None), dict(grad_dtype=2), dict(accumulate=2), dict(dy_stride=63), dict(dy=BASE + 1),
               dict(codes=BASE + 0x10000008), dict(G=BASE + 0x30000002), dict(G=BASE), dict(rows=1 << 16, cols=1 << 16)):
        a = wgrad(**kw)
        assert L.muon_validate_weight_grad(ctypes.byref(a)) == mb.MUON_ERR_INVALID, kw
    assert L.muon_validate_weight_grad(None) == mb.MUON_ERR_INVALID
    assert L.muon_weight_grad_workspace(None, ctypes.byref(ctypes.c_size_t())) == mb.MUON_ERR_INVALID
    a = wgrad()
    assert L.muon_weight_grad_workspace(ctypes.byref(a), None) == mb.MUON_ERR_INVALID


def test_null_handles():
    L = mb.lib()
    assert L.muon_attention(None, ctypes.byref(attention()), None) == mb.MUON_ERR_INVALID
    assert L.muon_attention_backward(None, ctypes.byref(grad()), None) == mb.MUON_ERR_INVALID
    assert L.muon_weight_grad(None, ctypes.byref(wgrad()), None) == mb.MUON_ERR_INVALID
    assert L.muon_checkpoint_store(None, BASE, 0, 1, 1, 1, BASE, BASE, None) == mb.MUON_ERR_INVALID
    assert L.muon_checkpoint_load(None, BASE, BASE, 1, 1, BASE, 0, 1, None) == mb.MUON_ERR_INVALID
    assert L.muon_qk_clip_grouped(None, BASE, BASE, BASE, 1, 1, 1, 1, 1.0, None) == mb.MUON_ERR_INVALID
