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
