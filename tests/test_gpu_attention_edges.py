"""Attention, its gradients and what reads their results, at the values and layouts where the formulas
and the kernels can part: against the formulas in 64 bits, or bit for bit where the change must not be seen."""
import math

import pytest
import torch

import muon_newton_schulz_04_b200 as mb
from test_gpu_attention import TOL_GRAD, TOL_OUT, TOL_STAT, close, cu, inputs, opt, reference, run_both  # noqa: F401

pytestmark = pytest.mark.gpu

LARGE = 3.3e38          # finite in bf16; 2^-126 of it is 3.9


@pytest.mark.parametrize("hq,hk,d", [(2, 1, 128), (2, 2, 64), (1, 1, 40)])
@pytest.mark.parametrize("at", [1, 7, 63, 64, 100, 129, 200, 299])
def test_large_values_of_later_tokens_weigh_nothing(opt, at, hq, hk, d):
    """The weight of a key that a query does not see is 0, not a small number: finite values however large of tokens
    from `at` on leave earlier rows bit for bit as they were, and exactly 0 where the values that they see are 0."""
    q, k, v, _ = inputs(130 + at, 300, 300, hq, hk, d)
    want, lse = opt.attention(q, k, v, cu([300]))
    v[at:] = LARGE
    v[at::2] *= -1
    got, lse2 = opt.attention(q, k, v, cu([300]))
    v[:at] = 0
    none, _ = opt.attention(q, k, v, cu([300]))
    opt.sync()
    assert torch.equal(got[:at], want[:at]) and torch.equal(lse, lse2)
    assert not none[:at].any()


@pytest.mark.parametrize("d", [128, 64])
def test_weights_below_the_smallest_number_are_zero(opt, d):
    """Every key but the first has a logit 1024 or more below it (q = 1, k = 64 and -64): a weight of 2^-1477, 0 in
    any type of 32 bits whichever unit computes it.  Values of 3.3e38 behind such weights, and output gradients of
    that size, give 0 exactly."""
    n = 300
    q = torch.ones(n, 1, d, dtype=torch.bfloat16, device="cuda")
    k = torch.full_like(q, -64.0)
    k[0] = 64
    v = torch.full_like(q, LARGE)
    v[0] = 0
    out, lse = opt.attention(q, k, v, cu([n]))
    opt.sync()
    assert not out.any()
    dq, dk, dv = opt.attention_backward(v, q, k, torch.zeros_like(v), out, lse, cu([n]))
    opt.sync()
    assert not dv[1:].any() and not dq.any() and not dk.any()


@pytest.mark.parametrize("d", [128, 64])
def test_infinite_logits_count(opt, d):
    """A logit of +inf is the largest: finite q and k of 1e20 overflow.  One of -inf is none, and has weight 0; a row
    with a NaN among its logits is passed over."""
    n = 200
    q, k, v, _ = inputs(140 + d, n, n, 3, 3, d)
    q[:, :, 0] = k[:, :, 0] = 0
    c = cu([n])
    want = torch.full((3,), -math.inf, device="cuda")
    plain, _ = opt.attention(q, k, v, c, max_logits=want)
    # only the last row sees the last key; 0 times 1e20 leaves every other logit as it was
    q[-1, :2, 0] = 1e20
    k[-1, 0, 0] = 1e20
    k[-1, 1, 0] = -1e20
    q[-1, 2, 0] = math.nan
    top = torch.full((3,), -math.inf, device="cuda")
    out, lse = opt.attention(q, k, v, c, max_logits=top)
    opt.sync()
    assert float(top[0]) == math.inf
    ro, rl, rt = reference(q[:, 1:2], k[:, 1:2], v[:, 1:2], [n], [n], d ** -0.5)
    assert abs(float(top[1]) - float(rt)) <= TOL_STAT and abs(float(lse[1, -1]) - float(rl[0, -1])) <= TOL_STAT
    close(out[:, 1:2], ro, TOL_OUT, "out")
    _, _, rt = reference(q[:-1, 2:], k[:-1, 2:], v[:-1, 2:], [n - 1], [n - 1], d ** -0.5)
    assert abs(float(top[2]) - float(rt)) <= TOL_STAT
    assert torch.equal(out[:-1], plain[:-1])
    # a larger finite maximum of an earlier call is raised, too
    top = torch.full((3,), 1e30, device="cuda")
    opt.attention(q, k, v, c, max_logits=top)
    opt.sync()
    assert top.tolist() == [math.inf, float(torch.tensor(1e30)), float(torch.tensor(1e30))]


def test_clip_with_infinite_logits(opt):
    """A head whose logits overflowed has gamma = 0: its query rows become 0, and the other heads that share its key
    rows are clipped as without it.  Where every head of a group is like that, the key rows become 0 too, as in the
    call of ungrouped heads.  Finite elements: at most 5 * 2^-23 off (four roundings of a factor, one of the product)."""
    hq, hk, d, cols, tau = 8, 2, 16, 50, 100.0
    gen = torch.Generator(device="cuda")
    gen.manual_seed(150)
    Wq, Wk = (torch.randn(h * d, cols, generator=gen, device="cuda") for h in (hq, hk))
    top = torch.tensor([math.inf, 50.0, 400.0, 200.0] + [math.inf] * 4, device="cuda")
    wq, wk = Wq.clone(), Wk.clone()
    opt.qk_clip_grouped(wq, wk, top, d, tau)
    opt.sync()
    fq = torch.tensor([0, 2, 0.5, 1, 0, 0, 0, 0], dtype=torch.float64, device="cuda").repeat_interleave(d)[:, None]
    fk = torch.tensor([0.5, 0], dtype=torch.float64, device="cuda").repeat_interleave(d)[:, None]
    for got, old, f in ((wq, Wq, fq), (wk, Wk, fk)):
        want = old.double() * f
        assert bool(((got.double() - want).abs() <= 5 * 2.0 ** -23 * want.abs()).all())
    a, b = Wq.clone(), Wq.clone()
    opt.qk_clip_grouped(a, b, top, d, tau)
    c, e = Wq.clone(), Wq.clone()
    opt.qk_clip(c, e, top, d, tau)
    opt.sync()
    assert not a[4 * d:].any() and torch.equal(a == 0, c == 0) and torch.equal(b == 0, e == 0)


@pytest.mark.parametrize("hq,hk,d", [(2, 1, 128), (2, 2, 64), (2, 1, 40)])
@pytest.mark.parametrize("at", [1, 63, 100, 127, 128, 200, 299, 555])
def test_an_infinite_component_of_a_key_with_no_weight(opt, at, hq, hk, d):
    """One component of key `at` is infinite and every query's is negative there: the logit is -inf, the weight 0 and
    the log-sum finite.  By the formula dq of the queries that see the key has 0 * inf in that component, wherever the
    key lies in its tile; the other components, and the queries before, are as if the key were not there."""
    n = 600
    q, k, v, do = inputs(160 + at, n, n, hq, hk, d)
    q[:, :, 3] = -q[:, :, 3].abs() - 0.5
    want = [t.clone() for t in run_both(opt, q, k, v, do, cu([n]), cu([n]))]
    k[at, 0, 3] = math.inf
    out, lse, top, dq, dk, dv = run_both(opt, q, k, v, do, cu([n]), cu([n]))
    heads = hq // hk                                            # those that read key head 0
    assert torch.equal(dq[:at], want[3][:at]) and torch.equal(dq[:, heads:], want[3][:, heads:])
    assert bool(torch.isfinite(lse).all()) and bool(torch.isfinite(out).all())
    assert not bool(torch.isfinite(dq[at:, :heads, 3]).any())
    others = [e for e in range(d) if e != 3]
    assert bool(torch.isfinite(dq[:, :, others]).all())
    # key `at` of head 0 far away instead of infinitely far: the same weights
    k[at, 0, 3] = 1e30
    far = run_both(opt, q, k, v, do, cu([n]), cu([n]))
    assert torch.equal(dq[:, :, others], far[3][:, :, others]) and torch.equal(out, far[0]) and torch.equal(lse, far[1])


@pytest.mark.parametrize("d", [64, 128])
def test_padding_of_returned_buffers(opt, d):
    """Rows of no sequence in buffers that a call returns are 0 (lse: -inf), whatever the allocator's memory held, so
    that weight gradients, which sum over all rows, are those of the sequences' rows."""
    total, hq, hk = 330, 4, 2
    q, k, v, do = inputs(170 + d, total, total, hq, hk, d)
    c = torch.tensor([20, 120, 290], dtype=torch.int32, device="cuda")
    inside = torch.zeros(total, dtype=torch.bool, device="cuda")
    inside[20:290] = True
    for stream in (None, torch.cuda.Stream()):
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            stale = [torch.full_like(t, math.nan) for t in (q, q, k, k)] + [torch.full((hq, total), math.nan, device="cuda")]
            stale += [torch.full((hq, total), math.nan, device="cuda")]
            del stale
        out, lse = opt.attention(q, k, v, c, stream=stream)
        grads = opt.attention_backward(do, q, k, v, out, lse, c, stream=stream)
        torch.cuda.synchronize()
        for t in (out, *grads):
            assert not t[~inside].any() and bool(torch.isfinite(t).all()) and bool(t[inside].any())
        assert bool((lse[:, ~inside] == -math.inf).all()) and bool(torch.isfinite(lse[:, inside]).all())
    x = inputs(180, total, total, 1, 1, 128)[0].view(total, 128)
    for g in grads:
        dy = g.flatten(1)
        whole = opt.weight_grad(dy, opt.checkpoint(x), torch.empty(dy.shape[1], 128, device="cuda"))
        part = opt.weight_grad(dy[20:290], opt.checkpoint(x[20:290]), torch.empty(dy.shape[1], 128, device="cuda"))
        opt.sync()
        # the same sums of fp32 products in another grouping of the rows: 270 additions at most, 2^-24 each
        assert float((whole - part).norm()) <= 270 * 2.0 ** -24 * float(part.norm())


@pytest.mark.parametrize("bounds", [[0], [70], [0, 0], [70, 70, 70], [69, 70], [5, 6, 40, 70]])
@pytest.mark.parametrize("d", [16, 128])
def test_padding_only_and_in_front(opt, bounds, d):
    """No sequence at all, empty ones, a single row, padding in front: rows of no sequence are 0, lse -inf there, for
    the buffers that the call makes, and stay in those that it is given."""
    q, k, v, do = inputs(175, 70, 70, 4, 2, d)
    c = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    inside = torch.zeros(70, dtype=torch.bool, device="cuda")
    inside[bounds[0]:bounds[-1]] = True
    want = run_both(opt, q, k, v, do, c, c)
    torch.cuda.synchronize()
    stale = [torch.full_like(t, math.nan) for t in (q, q, k, k)] + [torch.full((4, 70), math.nan, device="cuda")] * 2
    del stale
    out, lse = opt.attention(q, k, v, c)
    grads = opt.attention_backward(do, q, k, v, out, lse, c)
    kept = torch.full_like(k, 7.0)
    dq, dk, dv = opt.attention_backward(do, q, k, v, out, lse, c, dk=kept)
    opt.sync()
    for t in (out, *grads, dq, dv):
        assert not t[~inside].any()
    assert bool((lse[:, ~inside] == -math.inf).all()) and dk is kept and bool((dk[~inside] == 7).all())
    for x, y in zip((out, *grads, dk), (want[0], *want[3:], want[4])):
        assert torch.equal(x[inside], y[inside])
    assert torch.equal(lse[:, inside], want[1][:, inside])


def test_fill_of_other_buffers_is_refused(opt):
    """`fill` names outputs of its own call only."""
    q, k, v, do = inputs(176, 8, 8, 1, 1, 64)
    c = cu([8])
    out, lse = opt.attention(q, k, v, c)
    fields = opt._attention_fields(q, k, v, c, None, None, out, lse, None)
    args = mb._AttentionArgs.from_buffer_copy(mb._ATTENTION_PACK.pack(*fields))
    for fill in (-1, mb.MUON_FILL_DQ, 64):
        assert mb.lib().muon_attention_fill(opt._h, args, fill, None) == mb.MUON_ERR_INVALID
    h = mb._heads("q", q, q.shape, opt.device)
    dq, dk, dv, delta = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q), torch.empty_like(lse)
    grad = mb._AttentionGradArgs.from_buffer_copy(mb._ATTENTION_GRAD_PACK.pack(
        *fields, *h, *(x for t in (dq, dk, dv) for x in mb._heads("t", t, q.shape, opt.device)), delta.data_ptr()))
    for fill in (-1, mb.MUON_FILL_OUT, 64):
        assert mb.lib().muon_attention_backward_fill(opt._h, grad, fill, None) == mb.MUON_ERR_INVALID
    opt.sync()


def test_rows_of_bad_sequences_stay(opt):
    """Bounds out of range: the forward and the gradient kernels leave the rows of such a sequence as they were,
    compute the good one to the same bits as alone, and report it."""
    q, k, v, do = inputs(190, 64, 64, 2, 1, 64)
    i32 = dict(dtype=torch.int32, device="cuda")
    for bad, good in (([0, 20, 65], (0, 20)), ([0, 30, 20], (0, 30)), ([-1, 20, 64], (20, 64))):
        want = run_both(opt, q, k, v, do, torch.tensor(good, **i32), torch.tensor(good, **i32))
        c = torch.tensor(bad, **i32)
        out, lse = torch.full_like(q, 7.0), torch.full((2, 64), 7.0, device="cuda")
        top = torch.full((2,), -math.inf, device="cuda")
        opt.attention(q, k, v, c, out=out, lse=lse, max_logits=top)
        with pytest.raises(mb.MuonError) as e:
            opt.sync()
        assert e.value.status == mb.MUON_ERR_INVALID
        grads = [torch.full_like(t, 7.0) for t in (q, k, v)]
        opt.attention_backward(do, q, k, v, out, lse, c, dq=grads[0], dk=grads[1], dv=grads[2])
        with pytest.raises(mb.MuonError) as e:
            opt.sync()
        assert e.value.status == mb.MUON_ERR_INVALID
        # (rows outside the good sequence hold 7 in `want`, too)
        for name, got, ref in zip(("out", "lse", "top", "dq", "dk", "dv"), [out, lse, top] + grads, want):
            assert torch.equal(got, ref), (name, bad)
    opt.sync()


@pytest.mark.parametrize("d", [64, 128])
def test_gradients_at_large_logits(opt, d):
    """dq and dk where S - lse cancels.  Logits / scale reach 2^13; five or nine accumulations of 16 columns, each off
    by at most 2^-23 of that, move S and lse by 9 * 2^-10 * scale <= 2^-9.8 each, so P, and with it dS, by a factor
    within 1 + 2^-8.8: on top of the other test's tolerance, 2^-8.8 of the sum of the terms' magnitudes."""
    n, scale = 300, d ** -0.5
    q, k, v, do = inputs(200 + d, n, n, 2, 2, d)
    q, k = (q.float() * 8).to(torch.bfloat16), (k.float() * 8).to(torch.bfloat16)
    out, lse, top, dq, dk, dv = run_both(opt, q, k, v, do, cu([n]), cu([n]))
    ro, rl, rt, rq, rk, rv = reference(q, k, v, [n], [n], scale, do)
    assert 150 < float(rt.max()) and float(rt.max()) / scale < 2.0 ** 13
    Q, K, V, G = (t.double().transpose(0, 1) for t in (q, k, v, do))
    S = (Q @ K.transpose(1, 2) * scale).masked_fill(~torch.ones(n, n, dtype=torch.bool, device="cuda").tril(), -math.inf)
    P = torch.softmax(S, 2)
    dS = (P * (G @ V.transpose(1, 2) - (G * (P @ V)).sum(2, keepdim=True))).abs() * scale
    # (`close` weighs what comes beside the gradient with 2^-8)
    more = 2.0 ** -0.8
    mq, mk = (dS @ K.abs()).transpose(0, 1) * more, (dS.transpose(1, 2) @ Q.abs()).transpose(0, 1) * more
    close(dq, (rq[0], rq[1] + mq), TOL_GRAD, "dq")
    close(dk, (rk[0], rk[1] + mk), TOL_GRAD, "dk")
    close(dv, (rv[0], 2.0 ** -0.8 * (P.transpose(1, 2) @ G.abs()).transpose(0, 1)), TOL_GRAD, "dv")


def test_clip_of_too_many_heads_is_refused(opt):
    """More heads than a grid has rows, up to sums of heads that leave 32 bits: refused before anything is launched."""
    w = torch.ones(64, device="cuda")
    p = w.data_ptr()
    for hq, hk in ((65535, 1), (32768, 32768), ((1 << 31) - 1, (1 << 31) - 1), ((1 << 31) - 1, 1), (1 << 30, 1 << 30)):
        st = mb.lib().muon_qk_clip_grouped(opt._h, p, p + 128, p + 64, hq, hk, 1, 1, 1.0, None)
        assert st == mb.MUON_ERR_UNSUPPORTED, (hq, hk)
    opt.sync()
    assert bool((w == 1).all())


@pytest.mark.parametrize("rows_first", [True, False])
@pytest.mark.parametrize("ql,h,d", [([150, 3, 260], 4, 64), ([77, 300], 3, 128), ([1], 5, 8)])
def test_views_interleaved_head_by_head(opt, ql, h, d, rows_first):
    """q, k and v (dq, dk and dv) of an array whose heads lie as q, k, v, q, k, v, ...: the same bits as dense ones, and
    nothing written beside them."""
    t = sum(ql)
    q, k, v, do = inputs(210 + d, t, t, h, h, d)
    want = run_both(opt, q, k, v, do, cu(ql), cu(ql))

    def parts():
        x = torch.full((t, h, 4, d) if rows_first else (h, t, 4, d), 7.0, dtype=q.dtype, device="cuda")
        return x, [(x if rows_first else x.transpose(0, 1))[:, :, i] for i in range(4)]

    fused, views = parts()
    for a, b in zip(views, (q, k, v)):
        a.copy_(b)
    out, lse = opt.attention(*views[:3], cu(ql), out=views[3])
    grads, g = parts()
    opt.attention_backward(do, *views[:3], out, lse, cu(ql), dq=g[0], dk=g[1], dv=g[2])
    opt.sync()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    for a, b in zip(g, want[3:]):
        assert torch.equal(a, b)
    for a, b in zip(views, (q, k, v)):
        assert torch.equal(a, b)
    assert bool((g[3] == 7).all())


def test_sizes_past_32_bits_are_refused(opt):
    """A row of 2^32 + 5 values is refused, not taken for one of 5."""
    n = (1 << 32) + 5
    x = torch.empty(1, n, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        opt.checkpoint(x)
    dy = torch.zeros(1, n, dtype=torch.bfloat16, device="cuda")
    c = opt.checkpoint(torch.ones(1, 1, device="cuda"))
    with pytest.raises(ValueError):
        opt.weight_grad(dy, c, x.view(n, 1))
    w = torch.empty(1, (1 << 32) + 5, device="cuda")
    with pytest.raises(ValueError):
        opt.qk_clip_grouped(w, w, torch.ones(1, device="cuda"), 1, 1.0)
    opt.sync()


def test_scales_and_widths_outside_their_types(opt):
    """A scale above fp32's range and heads without width are refused by the library, as other arguments are."""
    q, k, v, do = inputs(220, 8, 8, 1, 1, 64)
    c = cu([8])
    out, lse = opt.attention(q, k, v, c)
    e = torch.empty(8, 1, 0, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: opt.attention(q, k, v, c, scale=1e39), lambda: opt.attention(e, e, e, c),
                 lambda: opt.attention_backward(do, q, k, v, out, lse, c, scale=1e39),
                 lambda: opt.attention_backward(e, e, e, e, e, lse, c)):
        with pytest.raises(mb.MuonError) as err:
            call()
        assert err.value.status == mb.MUON_ERR_INVALID
    opt.sync()


@pytest.mark.parametrize("d,power", [(64, -61), (64, -20), (64, 30), (64, 67), (16, -62), (16, 66)])
def test_scales_at_their_limits(opt, d, power):
    """q times 2^-n with a scale 2^n times as large, up to the scales' limits 2^-64 and 2^64: every product, sum and
    rounding is the same times a power of two, so the same bits; dq is 2^n times as large."""
    n, base = [150, 43], d ** -0.5
    assert math.frexp(base)[0] == 0.5 and 2.0 ** -64 <= base * 2.0 ** power <= 2.0 ** 64
    q, k, v, do = inputs(230 + d, 193, 193, 4, 2, d)
    want = run_both(opt, q, k, v, do, cu(n), cu(n), scale=base)
    got = run_both(opt, (q.double() * 2.0 ** -power).to(torch.bfloat16), k, v, do, cu(n), cu(n), scale=base * 2.0 ** power)
    for name, i in (("out", 0), ("lse", 1), ("top", 2), ("dk", 4), ("dv", 5)):
        assert torch.equal(got[i], want[i]), name
    assert torch.equal(got[3].double(), want[3].double() * 2.0 ** power)


@pytest.mark.parametrize("size", [2.0 ** -128, 2.0 ** -120, 2.0 ** 120, 2.0 ** 125])
@pytest.mark.parametrize("t,r,n", [(300, 70, 100), (1100, 130, 40)])
def test_weight_grad_of_the_smallest_and_largest_activations(opt, t, r, n, size):
    """Activations whose blocks have units below 2^-126, where the values of a checkpoint are subnormal, and near the
    largest: as exact as any others.  The tolerance of the other tests: sums in fp32, 2^-23 * sqrt(tokens)."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(240 + t)
    x = torch.randn(t, n, generator=gen, device="cuda").clamp(-3.9, 3.9).double() * size
    dy = (torch.randn(t, r, generator=gen, device="cuda").double() / size).clamp(-1e38, 1e38).to(torch.bfloat16)
    c = opt.checkpoint(x.to(torch.bfloat16))
    G = opt.weight_grad(dy, c, torch.empty(r, n, device="cuda"))
    opt.sync()
    unit = torch.tensor([2.0 ** (e - 133) for e in range(255)], dtype=torch.float64, device="cuda")[c.scales.long()]
    values = (c.codes.double() * unit.repeat_interleave(32, 1))[:, :n]
    want = dy.double().t() @ values
    assert float(want.abs().max()) > 1e-3
    assert float((G.double() - want).norm() / want.norm()) <= 2.0 ** -23 * math.sqrt(16384)
