"""8-bit activation checkpoints and the weight gradient taken from them, against their
definitions in 64 bits; QK-Clip of grouped heads; and one layer's run through all of
them and the Muon step.

Tolerances.  A checkpoint's values are exact (codes, units and their products have at
most 8 significant bits), so they are compared bit for bit.  weight_grad: products of two
bf16 values are exact in fp32 and t of them are summed in fp32, each sum off by at most
2^-23 of the running magnitude; for random-sign terms the relative norm grows like the
root of t at the most: 2^-23 * sqrt(16384) = 1.6e-5; bf16 outputs add 2^-8.
"""
import math

import numpy as np
import pytest
import torch

import muon_newton_schulz_04_b200 as mb
from muon_newton_schulz_04_b200 import build as mbuild

pytestmark = pytest.mark.gpu

TOL_FP32 = 1.6e-5
TOL_BF16 = 2.0 ** -8


@pytest.fixture(scope="module")
def opt():
    mbuild.build()
    o = mb.Muon(mb.config())
    yield o
    o.close()


def normal(seed, *shape, dtype=torch.float32):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


def define(x):
    """codes, E and values of a checkpoint by the definition: the smallest E >= 0 whose rounded codes fit."""
    x = x.double().cpu().numpy()
    rows, cols = x.shape
    b = np.zeros((rows, -(-cols // 32) * 32))
    b[:, :cols] = x
    b = b.reshape(rows, -1, 32)
    E = np.zeros(b.shape[:2], dtype=np.int64)
    codes = np.zeros(b.shape, dtype=np.int64)
    for r in range(rows):
        for i in range(b.shape[1]):
            v = b[r, i]
            if not np.isfinite(v).all():
                E[r, i] = 255
                continue
            e = max(0, int(np.frexp(np.abs(v).max())[1]) + 124)
            while e < 254 and np.abs(np.rint(v * 2.0 ** (133 - e))).max() > 127:
                e += 1
            while e > 0 and np.abs(np.rint(v * 2.0 ** (133 - e + 1))).max() <= 127:
                e -= 1
            E[r, i] = e
            codes[r, i] = np.clip(np.rint(v * 2.0 ** (133 - e)), -127, 127)
    values = np.where(E[..., None] == 255, np.nan, codes * 2.0 ** (E[..., None] - 133.0))
    return codes.reshape(rows, -1), E, values.reshape(rows, -1)[:, :cols]


def awkward(dtype):
    """Blocks at the borders: zeros, subnormals, the largest values, ties, infinities and NaN, and ordinary ones."""
    x = normal(1, 12, 70)
    x[0] = 0
    x[1] = x[1] * 1e-41
    x[2] = x[2].sign() * 3.3e38
    x[3, :32] = torch.arange(32, device="cuda") + 0.5       # codes exactly between two integers
    x[3, 31] = 127.0
    x[4, :32] = 0
    x[4, 5] = 127.5                                         # rounds to 128: the next unit
    x[5, 40] = math.inf
    x[6, 69] = math.nan
    x[7] *= 1e30
    x[8] *= 1e-30
    x[9, :32] = 127.49
    x[10] = x[10] * 2.0 ** -126
    x[11] = 1.1754944e-38 * (1 - 2.0 ** -9)                 # the largest subnormals
    return x.to(dtype)


def units(c):
    """2^(E - 133) of every block."""
    return torch.tensor([2.0 ** (e - 133) for e in range(256)], dtype=torch.float64, device="cuda")[c.scales.long()]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_checkpoint_by_the_definition(opt, dtype):
    x = awkward(dtype)
    c = opt.checkpoint(x)
    back32 = opt.checkpoint_load(c, out=torch.empty(12, 70, device="cuda"))
    back16 = opt.checkpoint_load(c)
    opt.sync()
    codes, E, values = define(x)
    assert np.array_equal(c.scales.cpu().numpy(), E)
    assert np.array_equal(c.codes.cpu().numpy()[:, :70], codes[:, :70]) and not c.codes[:, 70:].any()
    assert np.array_equal(back32.double().cpu().numpy(), values, equal_nan=True)
    assert np.array_equal(back16.double().cpu().numpy(), values, equal_nan=True)


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 31), (3, 33), (5, 8), (200, 771), (64, 4096), (1000, 100)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_checkpoint_sizes_and_strides(opt, rows, cols, dtype):
    wide = normal(rows + cols, rows, cols + 3, dtype=dtype)
    for x in (wide[:, :cols].contiguous(), wide[:, 1:cols + 1]):
        c = opt.checkpoint(x)
        room = torch.full((rows, cols + 5), 9.0, dtype=dtype, device="cuda")
        opt.checkpoint_load(c, out=room[:, 2:2 + cols])
        opt.sync()
        _, E, values = define(x[:8])
        assert np.array_equal(room[:8, 2:2 + cols].double().cpu().numpy(), values)
        assert bool((room[:, :2] == 9).all()) and bool((room[:, 2 + cols:] == 9).all())
        # half a unit: 2^(E - 134) a value
        unit = units(c)
        off = (room[:, 2:2 + cols].double() - x.double()).abs()
        assert bool((off <= 0.5 * unit.repeat_interleave(32, 1)[:, :cols]).all())


def values_of(c):
    return c.codes.double() * units(c).repeat_interleave(32, 1)


WG = [(1, 1, 1), (1, 40, 33), (17, 128, 64), (64, 256, 256), (65, 257, 255), (200, 96, 771), (513, 768, 768),
      (2048, 64, 64), (4099, 130, 200), (1000, 1600, 300), (333, 8, 2000), (16384, 256, 128)]


@pytest.mark.parametrize("t,r,n", WG)
@pytest.mark.parametrize("dtype,accumulate", [(torch.float32, False), (torch.bfloat16, True), (torch.float32, True)])
def test_weight_grad(opt, t, r, n, dtype, accumulate):
    c = opt.checkpoint(normal(t + n, t, n, dtype=torch.bfloat16))
    dy = normal(t + r, t, r, dtype=torch.bfloat16)
    G = normal(r + n, r, n, dtype=dtype)
    before = G.double()
    assert opt.weight_grad(dy, c, G, accumulate=accumulate) is G
    opt.sync()
    want = dy.double().t() @ values_of(c)[:, :n] + (before if accumulate else 0)
    err = float((G.double() - want).norm() / want.norm())
    assert err <= (TOL_FP32 if dtype == torch.float32 else TOL_FP32 + TOL_BF16), err


def test_weight_grad_strides_and_no_tokens(opt):
    c = opt.checkpoint(normal(1, 300, 200, dtype=torch.bfloat16))
    wide = normal(2, 300, 140, dtype=torch.bfloat16)
    for first, r in ((0, 96), (8, 100), (3, 97), (1, 64)):
        dy = wide[:, first:first + r]
        G = torch.empty(r, 200, device="cuda")
        opt.weight_grad(dy, c, G)
        want = dy.double().t() @ values_of(c)[:, :200]
        assert float((G.double() - want).norm() / want.norm()) <= TOL_FP32
    # behind rows of a larger gradient, at an address that is 4 bytes off 16
    flat = torch.full((1 + 50 * 200 + 3,), 9.0, device="cuda")
    G = flat[1:1 + 50 * 200].view(50, 200)
    opt.weight_grad(wide[:, :50], c, G)
    want = wide[:, :50].double().t() @ values_of(c)[:, :200]
    assert float((G.double() - want).norm() / want.norm()) <= TOL_FP32
    assert float(flat[0]) == 9 and bool((flat[-3:] == 9).all())
    empty = mb.Checkpoint.empty(0, 200, "cuda")
    G = torch.full((8, 200), 5.0, device="cuda")
    opt.weight_grad(torch.empty(0, 8, dtype=torch.bfloat16, device="cuda"), empty, G, accumulate=True)
    assert bool((G == 5).all())
    opt.weight_grad(torch.empty(0, 8, dtype=torch.bfloat16, device="cuda"), empty, G)
    opt.sync()
    assert not G.any()


def test_strides_past_32_bits(opt):
    """Rows 2^20 elements apart, the last one past 2^32 elements: the same bits as from dense arrays."""
    n = 4100
    wide = torch.empty(n, 1 << 20, dtype=torch.bfloat16, device="cuda")
    x, dy, back = wide[:, :200], wide[:, 256:356], wide[:, 512:712]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(35)
    dense_x = torch.randn(n, 200, generator=gen, device="cuda").to(torch.bfloat16)
    dense_dy = torch.randn(n, 100, generator=gen, device="cuda").to(torch.bfloat16)
    x.copy_(dense_x)
    dy.copy_(dense_dy)
    a, b = opt.checkpoint(x), opt.checkpoint(dense_x)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    opt.checkpoint_load(a, out=back)
    assert torch.equal(back, opt.checkpoint_load(b))
    G = [opt.weight_grad(y, a, torch.empty(100, 200, device="cuda")) for y in (dy, dense_dy)]
    opt.sync()
    assert torch.equal(*G)


def test_weight_grad_same_bits_and_non_finite(opt):
    x = normal(3, 5000, 160, dtype=torch.bfloat16)
    dy = normal(4, 5000, 128, dtype=torch.bfloat16)
    c = opt.checkpoint(x)
    a = opt.weight_grad(dy, c, torch.empty(128, 160, device="cuda"))
    b = opt.weight_grad(dy, c, torch.empty(128, 160, device="cuda"))
    x[4000, 40] = math.nan                  # its block of 32 columns comes out NaN, the others as before
    bad = opt.weight_grad(dy, opt.checkpoint(x), torch.empty(128, 160, device="cuda"))
    opt.sync()
    assert torch.equal(a, b)
    assert bool(torch.isnan(bad[:, 32:64]).all())
    assert torch.equal(bad[:, :32], a[:, :32]) and torch.equal(bad[:, 64:], a[:, 64:])


def test_weight_grad_captured_and_on_two_streams(opt):
    c = [opt.checkpoint(normal(5 + i, 3000, 128, dtype=torch.bfloat16)) for i in range(2)]
    dy = [normal(7 + i, 3000, 192, dtype=torch.bfloat16) for i in range(2)]
    want = [opt.weight_grad(dy[i], c[i], torch.empty(192, 128, device="cuda")).clone() for i in range(2)]
    G = [torch.empty(192, 128, device="cuda") for _ in range(2)]
    graphs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            opt.weight_grad(dy[i], c[i], G[i])
        graphs.append(g)
    for _ in range(3):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    assert torch.equal(G[0], want[0]) and torch.equal(G[1], want[1])
    for i in range(2):
        opt.weight_grad(dy[i], c[i], G[i], stream=streams[i])
    torch.cuda.synchronize()
    assert torch.equal(G[0], want[0]) and torch.equal(G[1], want[1])
    del graphs


@pytest.mark.parametrize("hq,hk,d,cols", [(12, 12, 64, 768), (8, 2, 64, 100), (6, 1, 5, 7), (32, 8, 128, 512)])
def test_qk_clip_grouped(opt, hq, hk, d, cols):
    """Each element is off by at most the four fp32 roundings of its factor and one of the product: 5 * 2^-23."""
    Wq, Wk = normal(1, hq * d, cols), normal(2, hk * d, cols)
    S = torch.exp(normal(3, hq)) * 80
    S[0] = math.nan if hq > hk else S[0]
    tau = 100.0
    wq, wk = Wq.clone(), Wk.clone()
    opt.qk_clip_grouped(wq, wk, S, d, tau)
    opt.sync()
    g = torch.where(S.double() > tau, tau / S.double(), 1.0)
    root = g.view(hk, -1).amin(1).sqrt()
    fq, fk = g / root.repeat_interleave(hq // hk), root
    want_q, want_k = Wq.double() * fq.repeat_interleave(d)[:, None], Wk.double() * fk.repeat_interleave(d)[:, None]
    for got, want in ((wq, want_q), (wk, want_k)):
        assert float(((got.double() - want).abs() / (want.abs() + 1e-30)).max()) <= 5 * 2.0 ** -23
    if hq == hk:                            # one query head a key head: the ungrouped call
        a, b = Wq.clone(), Wk.clone()
        opt.qk_clip(a, b, S, d, tau)
        opt.sync()
        assert float(((a - wq).abs() / (a.abs() + 1e-30)).max()) <= 6 * 2.0 ** -23
        assert float(((b - wk).abs() / (b.abs() + 1e-30)).max()) <= 6 * 2.0 ** -23


def test_one_layer_from_its_input_to_its_step(opt):
    """x in 8 bits; q, k, v; attention; gradients; weight gradients from the checkpoint into a Muon step; QK-Clip with
    the logits that the attention saw.  The weight gradients equal those of the same chain in 64 bits on x^ for the
    product of attention's and the projections' bf16 roundings (three, 2^-8 each, on top of the gradient's)."""
    t, width, hq, hk, d, lens = 260, 256, 4, 2, 64, [100, 160]
    x = normal(1, t, width, dtype=torch.bfloat16)
    W = {"q": normal(2, hq * d, width) * 0.1, "k": normal(3, hk * d, width) * 0.1, "v": normal(4, hk * d, width) * 0.06}
    cu = torch.tensor([0, 100, 260], dtype=torch.int32, device="cuda")
    ckpt = opt.checkpoint(x)
    y = {n: (x @ w.to(torch.bfloat16).t()).view(t, -1, d) for n, w in W.items()}
    top = torch.full((hq,), -math.inf, device="cuda")
    out, lse = opt.attention(y["q"], y["k"], y["v"], cu, max_logits=top)
    do = normal(5, t, hq, d, dtype=torch.bfloat16)
    grads = opt.attention_backward(do, y["q"], y["k"], y["v"], out, lse, cu)
    G = {n: opt.weight_grad(g.view(t, -1), ckpt, torch.empty_like(W[n])) for n, g in zip("qkv", grads)}
    opt.sync()
    # the chain in 64 bits
    p = {n: y[n].double().requires_grad_(True) for n in "qkv"}
    at = 0
    loss, logits = 0, []
    for n in lens:
        for h in range(hq):
            q, k, v = (p[s][at:at + n, h if s == "q" else h // 2] for s in "qkv")
            s = (q @ k.t() / math.sqrt(d)).masked_fill(~torch.ones(n, n, dtype=torch.bool, device="cuda").tril(), -math.inf)
            logits.append(s.detach().max())
            loss = loss + (torch.softmax(s, 1) @ v * do[at:at + n, h].double()).sum()
        at += n
    loss.backward()
    xv = values_of(ckpt)[:, :width]
    for n in "qkv":
        want = p[n].grad.reshape(t, -1).t() @ xv
        assert float((G[n].double() - want).norm() / want.norm()) <= 4 * 2.0 ** -8, n
    want_top = torch.stack(logits).view(2, hq).amax(0)
    assert float((top.double() - want_top).abs().max()) <= 1e-5
    # the step and the clip
    tau = float(top.max()) / 2
    B = {n: torch.zeros_like(w) for n, w in W.items()}
    before = {n: w.clone() for n, w in W.items()}
    opt.step([mb.Group(W=[W["q"]], G=[G["q"]], B=[B["q"]]),
              mb.Group(W=[W["k"], W["v"]], G=[G["k"], G["v"]], B=[B["k"], B["v"]])])
    stepped = {n: w.clone() for n, w in W.items()}
    opt.qk_clip_grouped(W["q"], W["k"], top, d, tau)
    opt.sync()
    for n in "qkv":
        assert bool((stepped[n] != before[n]).any()) and bool(torch.isfinite(W[n]).all())
        assert torch.equal(B[n], G[n])
    assert torch.equal(W["v"], stepped["v"])
    # logits of the clipped weights are those of the stepped ones times gamma
    gamma = torch.clamp(tau / top.double(), max=1.0)
    for h in range(hq):
        rows, krows = slice(h * d, (h + 1) * d), slice(h // 2 * d, (h // 2 + 1) * d)
        a = W["q"][rows].double().t() @ W["k"][krows].double()
        b = stepped["q"][rows].double().t() @ stepped["k"][krows].double()
        assert float((a - gamma[h] * b).norm() / b.norm()) <= 1e-6


def test_refusals(opt):
    x = normal(1, 8, 64, dtype=torch.bfloat16)
    c = opt.checkpoint(x)
    G = torch.empty(16, 64, device="cuda")
    dy = normal(2, 8, 16, dtype=torch.bfloat16)
    for call in (lambda: opt.checkpoint(x.half()), lambda: opt.weight_grad(dy.float(), c, G),
                 lambda: opt.weight_grad(dy, c, G.half())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: opt.checkpoint(x[0]), lambda: opt.checkpoint(x.t()), lambda: opt.checkpoint(x.cpu()),
                 lambda: opt.checkpoint(x, mb.Checkpoint.empty(8, 65, "cuda")),
                 lambda: opt.checkpoint_load(c, out=torch.empty(8, 63, device="cuda")),
                 lambda: opt.weight_grad(dy[:7], c, G), lambda: opt.weight_grad(dy, c, G[:, :32]),
                 lambda: opt.weight_grad(dy, mb.Checkpoint(c.codes, c.scales, 32), G[:, :32].contiguous()),
                 lambda: opt.qk_clip_grouped(G, G, torch.ones(4, device="cuda"), 3, 1.0)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: opt.qk_clip_grouped(G, G[:8], torch.ones(4, device="cuda"), 4, 1.0),
                 lambda: opt.qk_clip_grouped(G, G.clone()[:12], torch.ones(4, device="cuda"), 4, 1.0),
                 lambda: opt.qk_clip_grouped(G, G.clone()[:8], torch.ones(4, device="cuda"), 4, -1.0)):
        with pytest.raises(mb.MuonError) as e:
            call()
        assert e.value.status == mb.MUON_ERR_INVALID
    opt.sync()
