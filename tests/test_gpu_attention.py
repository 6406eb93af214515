"""Packed causal attention with grouped heads, its largest logits and its gradients,
against the formulas in 64 bits.

Tolerances.  out, dq, dk and dv are rounded to bf16 once (2^-8 of the value at most,
relative norm below 2^-8), and the exponentials (dS in the backward pass) enter their
product rounded to bf16, which moves the sum by at most 2^-8 of the sum of its terms'
magnitudes; for the random-sign terms used here the moved part adds up like the sum
itself, so the relative norm stays below 2 * 2^-8 = 2^-7.  In the backward pass D_i is
formed from the rounded out: one more 2^-8 of the same kind, hence 3 * 2^-8.  Where the
gradients themselves cancel (a query that sees one key has dS = 0), that last part is not
small beside them: |error of D_i| <= 2^-8 sum_d |do_id out_id| = 2^-8 A_i moves dS_ij by
P_ij times that, so dq and dk get 2^-8 scale || sum P_ij A_i |k_j| || on top (`slack`).
lse and the largest logits are fp32 sums of at most 128 + 2^13 terms: 1e-5 absolute for
logits of order 10 leaves 8 fp32 steps of 2^-20 each.
"""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import muon_newton_schulz_04_b200 as mb
from muon_newton_schulz_04_b200 import build as mbuild

pytestmark = pytest.mark.gpu

TOL_OUT = 2.0 ** -7
TOL_GRAD = 3 * 2.0 ** -8
TOL_STAT = 1e-5


@pytest.fixture(scope="module")
def opt():
    mbuild.build()
    o = mb.Muon(mb.config())
    yield o
    o.close()


def cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def reference(q, k, v, ql, kl, scale, do=None):
    """out, lse, largest logits (and dq, dk, dv) of the packed rows, in 64 bits by the formulas."""
    q, k, v = q.double(), k.double(), v.double()
    hq, hk = q.shape[1], k.shape[1]
    out, lse, top = torch.zeros_like(q), torch.zeros(hq, q.shape[0], dtype=torch.float64, device=q.device), torch.full(
        (hq,), -math.inf, dtype=torch.float64, device=q.device)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    mq, mk = torch.zeros_like(q), torch.zeros_like(k)
    a = c = 0
    for lq, lk in zip(ql, kl):
        see = torch.arange(lk, device=q.device)[None, :] <= torch.arange(lq, device=q.device)[:, None] + lk - lq
        for h in range(hq):
            qs, ks, vs = q[a:a + lq, h], k[c:c + lk, h * hk // hq], v[c:c + lk, h * hk // hq]
            s = scale * qs @ ks.t()
            s = s.masked_fill(~see, -math.inf)
            m = s.amax(1, keepdim=True) if lk else s.new_full((lq, 1), -math.inf)
            e = torch.exp(s - torch.where(torch.isinf(m), 0.0, m))
            l = e.sum(1, keepdim=True)
            p = e / torch.where(l == 0, 1.0, l)
            out[a:a + lq, h] = p @ vs
            lse[h, a:a + lq] = (torch.where(torch.isinf(m), 0.0, m) + torch.log(l))[:, 0]
            if lq and lk:
                top[h] = torch.maximum(top[h], m.max())
            if do is not None:
                g = do[a:a + lq, h].double()
                dp = g @ vs.t()
                ds = p * (dp - (g * out[a:a + lq, h]).sum(1, keepdim=True))
                dq[a:a + lq, h] = scale * ds @ ks
                dk[c:c + lk, h * hk // hq] += scale * ds.t() @ qs
                dv[c:c + lk, h * hk // hq] += p.t() @ g
                pa = scale * p * (g * out[a:a + lq, h]).abs().sum(1, keepdim=True)
                mq[a:a + lq, h] = pa @ ks.abs()
                mk[c:c + lk, h * hk // hq] += pa.t() @ qs.abs()
        a, c = a + lq, c + lk
    return (out, lse, top) if do is None else (out, lse, top, (dq, mq), (dk, mk), (dv, 0 * dv))


def close(got, want, tol, what):
    want, slack = want if isinstance(want, tuple) else (want, 0 * want)
    got = got.double()
    assert torch.isfinite(got).all(), what
    err, most = float((got - want).norm()), tol * float(want.norm()) + 2.0 ** -8 * float(slack.norm())
    assert err <= most, f"{what}: {err:.3g} > {most:.3g}"


def inputs(seed, tq, tk, hq, hk, d):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    return r(tq, hq, d), r(tk, hk, d), r(tk, hk, d), r(tq, hq, d)


def run_both(opt, q, k, v, do, cq, ck, scale=None, **kw):
    out = torch.full_like(q, 7.0)
    lse = torch.full((q.shape[1], q.shape[0]), 7.0, device="cuda")
    top = torch.full((q.shape[1],), -math.inf, device="cuda")
    opt.attention(q, k, v, cq, out=out, lse=lse, max_logits=top, cu_seqlens_k=ck, scale=scale)
    dq, dk, dv = torch.full_like(q, 7.0), torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    opt.attention_backward(do, q, k, v, out, lse, cq, dq=dq, dk=dk, dv=dv, cu_seqlens_k=ck, scale=scale)
    opt.sync()
    return out, lse, top, dq, dk, dv


CASES = [
    # q lengths, k lengths (None: the same), heads, kv heads, head dim
    ([1], None, 1, 1, 64),
    ([1, 17, 63, 119], None, 12, 12, 64),
    ([128, 256, 127, 129, 255, 257], None, 2, 1, 128),
    ([300, 0, 1, 513], None, 6, 2, 128),
    ([0, 0, 5, 0], None, 3, 3, 8),
    ([700], None, 4, 4, 80),
    ([64, 65], [64, 65], 2, 2, 16),
    ([40, 1, 200], [300, 77, 200], 4, 1, 64),        # chunks at the end of longer prompts
    ([200, 130, 3, 9], [60, 129, 0, 300], 4, 2, 128),   # first rows that see nothing; no keys at all
    ([0, 5], [33, 0], 2, 2, 64),                     # keys without queries, queries without keys
    ([1500], None, 8, 1, 128),
    ([1100], [1357], 2, 1, 72),
    ([3] * 70 + [150], None, 2, 2, 64),              # more sequences than a warp has lanes
    ([33] * 9, None, 40, 8, 96),
]


@pytest.mark.parametrize("ql,kl,hq,hk,d", CASES)
def test_forward_and_gradients(opt, ql, kl, hq, hk, d):
    kl = ql if kl is None else kl
    q, k, v, do = inputs(sum(ql) + hq * d, sum(ql), sum(kl), hq, hk, d)
    scale = d ** -0.5
    out, lse, top, dq, dk, dv = run_both(opt, q, k, v, do, cu(ql), cu(kl))
    ro, rl, rt, rq, rk, rv = reference(q, k, v, ql, kl, scale, do)
    close(out, ro, TOL_OUT, "out")
    empty = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse), empty) and bool((out.transpose(0, 1)[empty] == 0).all())
    assert float((lse.double() - rl)[~empty].abs().max() if (~empty).any() else 0) <= TOL_STAT
    assert torch.equal(torch.isinf(top), torch.isinf(rt))
    seen = ~torch.isinf(rt)
    assert float((top.double() - rt)[seen].abs().max() if seen.any() else 0) <= TOL_STAT
    close(dq, rq, TOL_GRAD, "dq")
    close(dk, rk, TOL_GRAD, "dk")
    close(dv, rv, TOL_GRAD, "dv")


def test_gradients_against_differences(opt):
    """The directional derivative of L = <out, do> in 64-bit differences of the reference forward along a random
    direction equals <dq, direction> ...: the difference quotient with step 1e-4 is off by O(1e-8), the gradients
    by TOL_GRAD of the product of norms."""
    ql = [70, 131]
    q, k, v, do = inputs(5, 201, 201, 2, 1, 64)
    _, _, _, dq, dk, dv = run_both(opt, q, k, v, do, cu(ql), cu(ql))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(6)
    for x, g, place in ((q, dq, 0), (k, dk, 1), (v, dv, 2)):
        u = torch.randn(x.shape, generator=gen, device="cuda", dtype=torch.float64)
        value = []
        for sign in (1, -1):
            t = [q.double(), k.double(), v.double()]
            t[place] = t[place] + sign * 1e-4 * u
            value.append(float((reference(*t, ql, ql, 64 ** -0.5)[0] * do.double()).sum()))
        slope = (value[0] - value[1]) / 2e-4
        assert abs(slope - float((g.double() * u).sum())) <= TOL_GRAD * float(g.double().norm() * u.norm())


def test_rows_behind_and_between_sequences_stay(opt):
    """Rows of no sequence are not written, and what they hold (NaN) reaches nothing."""
    q, k, v, do = inputs(9, 400, 400, 4, 2, 64)
    c = torch.tensor([30, 130, 331], dtype=torch.int32, device="cuda")
    want = [t.clone() for t in run_both(opt, q, k, v, do, c, c)]
    inside = torch.zeros(400, dtype=torch.bool, device="cuda")
    inside[30:331] = True
    for t in (q, k, v, do):
        t[~inside] = math.nan
    got = run_both(opt, q, k, v, do, c, c)
    for name, a, b in zip(("out", "lse", "top", "dq", "dk", "dv"), got, want):
        assert torch.equal(a, b), name
    assert bool((got[0][~inside] == 7).all()) and bool((got[1][:, ~inside] == 7).all())
    for t in got[3:]:
        assert bool((t[~inside] == 7).all()) and bool(torch.isfinite(t).all())


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_one_sequence_never_reaches_another(opt, bad):
    ql = [100, 77, 140]
    q, k, v, do = inputs(10, 317, 317, 2, 2, 128)
    want = [t.clone() for t in run_both(opt, q, k, v, do, cu(ql), cu(ql))]
    for t in (q, k, v, do):
        t[100:177] = bad
    got = run_both(opt, q, k, v, do, cu(ql), cu(ql))
    for i in (0, 3, 4, 5):
        for part in (slice(0, 100), slice(177, 317)):
            assert torch.equal(got[i][part], want[i][part]), (i, part)
    assert torch.equal(got[1][:, :100], want[1][:, :100]) and torch.equal(got[1][:, 177:], want[1][:, 177:])


@pytest.mark.parametrize("hq,hk,d", [(2, 1, 128), (2, 2, 64)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("at", [0, 63, 100, 200, 299])
def test_later_tokens_never_reach_earlier_ones(opt, at, bad, hq, hk, d):
    """A non-finite value of v, or of all of token `at`, reaches the queries from `at` on and no earlier one, bit for
    bit; those from `at` on show it."""
    q, k, v, do = inputs(30 + at, 300, 300, hq, hk, d)
    want = [t.clone() for t in run_both(opt, q, k, v, do, cu([300]), cu([300]))]
    v2 = v.clone()
    v2[at, 0, 3] = bad
    out, lse = opt.attention(q, k, v2, cu([300]))
    opt.sync()
    assert torch.equal(out[:at], want[0][:at]) and torch.equal(lse, want[1])
    assert not bool(torch.isfinite(out[at:, 0, 3]).any())
    assert torch.equal(out[:, :, 4:], want[0][:, :, 4:]) and torch.equal(out[:, :, :3], want[0][:, :, :3])
    for t in (q, k, v):
        t[at] = bad
    got = run_both(opt, q, k, v, do, cu([300]), cu([300]))
    assert torch.equal(got[0][:at], want[0][:at]) and torch.equal(got[1][:, :at], want[1][:, :at])
    assert torch.equal(got[3][:at], want[3][:at])
    assert not bool(torch.isfinite(got[0][at]).any()) and not bool(torch.isfinite(got[3][at:]).any())


@pytest.mark.parametrize("hq,hk,d", [(2, 1, 128), (2, 2, 64)])
@pytest.mark.parametrize("at", [0, 70, 128, 299])
def test_gradients_of_keys_that_a_bad_query_does_not_see(opt, at, hq, hk, d):
    """A non-finite output gradient of query `at` reaches its dq and the keys up to `at`, and nothing else."""
    q, k, v, do = inputs(60 + at, 300, 300, hq, hk, d)
    want = [t.clone() for t in run_both(opt, q, k, v, do, cu([300]), cu([300]))]
    for bad in (math.nan, math.inf):
        do[at] = bad
        got = run_both(opt, q, k, v, do, cu([300]), cu([300]))
        for i in (4, 5):
            assert torch.equal(got[i][at + 1:], want[i][at + 1:]), i
        assert not bool(torch.isfinite(got[5][:at + 1]).any())
        keep = torch.arange(300, device="cuda") != at
        assert torch.equal(got[3][keep], want[3][keep])


def test_single_tokens_have_no_gradient_but_dv(opt):
    """A query that sees one key has P = 1: its out is v, and dq and dk are zero exactly."""
    for d, hq, hk in ((64, 4, 2), (128, 2, 2)):
        n = 140
        q, k, v, do = inputs(90 + d, n, n, hq, hk, d)
        out, lse, top, dq, dk, dv = run_both(opt, q, k, v, do, cu([1] * n), cu([1] * n))
        assert torch.equal(out, v.repeat_interleave(hq // hk, 1)) and not dq.any() and not dk.any()
        want = do.float().view(n, hk, -1, d).sum(2)
        assert float((dv.float() - want).abs().max()) <= 2.0 ** -8 * float(want.abs().max())


def test_views_of_one_fused_projection(opt):
    """q, k, v (and dq, dk, dv) as strided views of one array, and heads-first arrays: the same bits as dense ones."""
    ql, hq, hk, d = [150, 3, 260], 6, 2, 64
    t = sum(ql)
    q, k, v, do = inputs(11, t, t, hq, hk, d)
    want = run_both(opt, q, k, v, do, cu(ql), cu(ql))
    fused = torch.empty(t, hq + 2 * hk, d, dtype=torch.bfloat16, device="cuda")
    fq, fk, fv = fused[:, :hq], fused[:, hq:hq + hk], fused[:, hq + hk:]
    fq.copy_(q), fk.copy_(k), fv.copy_(v)
    grads = torch.zeros_like(fused)
    hf = lambda x: x.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    out, lse = opt.attention(fq, fk, fv, cu(ql), out=hf(torch.zeros_like(q)))
    opt.attention_backward(hf(do), fq, fk, fv, out, lse, cu(ql), dq=grads[:, :hq], dk=grads[:, hq:hq + hk],
                           dv=grads[:, hq + hk:])
    opt.sync()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert torch.equal(grads, torch.cat(want[3:], 1))


def test_offsets_past_32_bits(opt):
    """All eight arrays are column ranges of one array whose rows lie 2^20 elements apart: the last row starts past
    2^32 elements.  The same bits as from dense arrays."""
    n, h, d = 4100, 2, 64
    wide = torch.empty(n, 1 << 20, dtype=torch.bfloat16, device="cuda")
    views = [wide[:, 128 * i:128 * i + 128].view(n, h, d) for i in range(8)]
    q, k, v, do = inputs(33, n, n, h, h, d)
    for x, y in zip(views, (q, k, v, do)):
        x.copy_(y)
    c = cu([3000, 1100])
    out, lse = opt.attention(q, k, v, c)
    dense = (out, *opt.attention_backward(do, q, k, v, out, lse, c))
    _, lse2 = opt.attention(*views[:3], c, out=views[4])
    opt.attention_backward(views[3], *views[:3], views[4], lse2, c, dq=views[5], dk=views[6], dv=views[7])
    opt.sync()
    assert torch.equal(lse, lse2)
    for x, y in zip(views[4:], dense):
        assert torch.equal(x, y)


@pytest.mark.parametrize("d,hq", [(64, 2), (128, 2)])
def test_a_long_sequence(opt, d, hq):
    """40000 tokens: rows and keys picked from it, by the formulas (for keys with the call's own log-sums).  A row's sum
    is 313 additions of tiles' sums: 313 * 2^-24 = 1.9e-5 if all were off by half a step in one direction; of random
    sign they stay below a tenth of that, within TOL_STAT."""
    n = 40000
    q, k, v, do = inputs(34, n, n, hq, 1, d)
    c, scale = cu([n]), d ** -0.5
    out, lse = opt.attention(q, k, v, c)
    dq, dk, dv = opt.attention_backward(do, q, k, v, out, lse, c)
    opt.sync()
    q, k, v, do = (x.double() for x in (q, k[:, 0], v[:, 0], do))
    rows = [0, 1, 127, 128, 20001, n - 1]
    keys = [0, 63, 64, 19999, n - 130, n - 1]
    want = {"out": [], "dq": [], "dk": [], "dv": []}
    for i in rows:
        for h in range(hq):
            s = scale * (k[:i + 1] @ q[i, h])
            assert abs(float(torch.logsumexp(s, 0)) - float(lse[h, i])) <= TOL_STAT
            p = torch.softmax(s, 0)
            o, dp = p @ v[:i + 1], v[:i + 1] @ do[i, h]
            a = float((do[i, h] * o).abs().sum())
            want["out"].append((out[i, h], o, 0 * o))
            want["dq"].append((dq[i, h], scale * (p * (dp - do[i, h] @ o)) @ k[:i + 1], scale * a * (p @ k[:i + 1].abs())))
    delta = (do * out.double()).sum(2)
    for j in keys:
        gk = gv = 0
        for h in range(hq):
            p = torch.exp(scale * (q[j:, h] @ k[j]) - lse[h, j:].double())
            gv = gv + p @ do[j:, h]
            gk = gk + scale * (p * (do[j:, h] @ v[j] - delta[j:, h])) @ q[j:, h]
        want["dk"].append((dk[j, 0], gk, 0 * gk))
        want["dv"].append((dv[j, 0], gv, 0 * gv))
    for what, tol in (("out", TOL_OUT), ("dq", TOL_GRAD), ("dk", TOL_GRAD), ("dv", TOL_GRAD)):
        got, y, slack = (torch.stack([x[m] for x in want[what]]) for m in range(3))
        close(got, (y, slack), tol, what)


def test_max_logits_keep_the_largest(opt):
    """Micro-batches raise one running maximum; heads whose logits are all negative count too."""
    q, k, v, _ = inputs(12, 90, 90, 4, 4, 64)
    k[:, 1] = -q[:, 1].abs()
    q[:, 1] = q[:, 1].abs()
    top = torch.full((4,), -math.inf, device="cuda")
    opt.attention(q, k, v, cu([90]), max_logits=top)
    first = top.clone()
    _, _, rt = reference(q, k, v, [90], [90], 64 ** -0.5)
    assert rt[1] < 0 and float((first.double() - rt).abs().max()) <= TOL_STAT
    opt.attention((0.5 * q.float()).to(torch.bfloat16), k, v, cu([90]), max_logits=top)
    opt.sync()
    keep = torch.maximum(first, 0.5 * first)
    assert float((top - keep).abs().max()) <= TOL_STAT


def test_same_bits_every_time(opt):
    ql = [513, 40, 300]
    q, k, v, do = inputs(13, 853, 853, 8, 2, 128)
    a = run_both(opt, q, k, v, do, cu(ql), cu(ql))
    b = run_both(opt, q, k, v, do, cu(ql), cu(ql))
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_large_logits(opt):
    """Logits of several hundred: rows are dominated by one key, and nothing overflows."""
    q, k, v, do = inputs(14, 300, 300, 2, 2, 64)
    q, k = (q.float() * 8).to(torch.bfloat16), (k.float() * 8).to(torch.bfloat16)
    out, lse, top, dq, dk, dv = run_both(opt, q, k, v, do, cu([300]), cu([300]))
    ro, rl, rt, rq, rk, rv = reference(q, k, v, [300], [300], 0.125, do)
    assert float(rt.max()) > 150
    close(out, ro, TOL_OUT, "out")
    # fp32 logits of up to 2^9 carry 2^-15 of rounding each
    assert float((lse.double() - rl).abs().max()) <= 2.0 ** -13 and float((top.double() - rt).abs().max()) <= 2.0 ** -13
    close(dv, rv, TOL_GRAD, "dv")


def test_captured_calls_replay_on_new_inputs(opt):
    """Forward and backward captured at the first call, replayed on other inputs and lengths."""
    q, k, v, do = inputs(15, 260, 260, 4, 2, 64)
    c = cu([100, 160])
    out, lse, top = torch.zeros_like(q), torch.zeros(4, 260, device="cuda"), torch.full((4,), -math.inf, device="cuda")
    grads = [torch.zeros_like(t) for t in (q, k, v)]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        opt.attention(q, k, v, c, out=out, lse=lse, max_logits=top)
        opt.attention_backward(do, q, k, v, out, lse, c, dq=grads[0], dk=grads[1], dv=grads[2])
    for seed, ql in ((16, [100, 160]), (17, [37, 223]), (18, [1, 259])):
        for old, new in zip((q, k, v, do), inputs(seed, 260, 260, 4, 2, 64)):
            old.copy_(new)
        c.copy_(cu(ql))
        g.replay()
        torch.cuda.synchronize()
        ro, rl, _, rq, rk, rv = reference(q, k, v, ql, ql, 0.125, do)
        close(out, ro, TOL_OUT, "out")
        for name, a, b in zip(("dq", "dk", "dv"), grads, (rq, rk, rv)):
            close(a, b, TOL_GRAD, name)
    del g


def test_two_calls_on_two_streams(opt):
    a, b = inputs(19, 500, 500, 4, 4, 64), inputs(20, 700, 700, 4, 1, 128)
    ca, cb = cu([500]), cu([333, 367])
    want_a, want_b = run_both(opt, *a, ca, ca), run_both(opt, *b, cb, cb)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        oa, la = opt.attention(*a[:3], ca, stream=s1)
        ob, lb = opt.attention(*b[:3], cb, stream=s2)
        ga = opt.attention_backward(a[3], *a[:3], oa, la, ca, stream=s1)
        gb = opt.attention_backward(b[3], *b[:3], ob, lb, cb, stream=s2)
    torch.cuda.synchronize()
    for got, want in (((oa, la) + ga, want_a), ((ob, lb) + gb, want_b)):
        for x, y in zip(got, want[:2] + want[3:]):
            assert torch.equal(x, y)


def test_sequence_bounds_out_of_range_are_reported(opt):
    """The kernels check cu_seqlens: bad sequences are passed over and muon_sync says so; good ones are computed."""
    q, k, v, do = inputs(21, 64, 64, 2, 2, 64)
    for bad in ([0, 20, 65], [0, 30, 20], [-1, 20, 64]):
        c = torch.tensor(bad, dtype=torch.int32, device="cuda")
        out = torch.full_like(q, 7.0)
        opt.attention(q, k, v, c, out=out)
        with pytest.raises(mb.MuonError) as e:
            opt.sync()
        assert e.value.status == mb.MUON_ERR_INVALID
        opt.sync()
    assert bool((out[20:] != 7).any())


@pytest.mark.parametrize("n", [33, 1000, 1100])
def test_many_sequences(opt, n):
    """More sequences than one look of a warp covers, empty and long ones among them."""
    ql = [0 if i % 5 == 3 else 1 + i % 4 for i in range(n)]
    kl = [x + i % 3 for i, x in enumerate(ql)]
    ql[n // 2], kl[n // 2] = 300, 290
    ql[n - 2], kl[n - 2] = 130, 257
    q, k, v, do = inputs(31, sum(ql), sum(kl), 2, 1, 64)
    got = run_both(opt, q, k, v, do, cu(ql), cu(kl))
    want = reference(q, k, v, ql, kl, 0.125, do)
    seen = torch.isfinite(want[1])
    assert torch.equal(torch.isfinite(got[1]), seen)
    assert float((got[1].double() - want[1])[seen].abs().max()) <= TOL_STAT
    assert float((got[2].double() - want[2]).abs().max()) <= TOL_STAT
    for x, y, tol, what in zip((got[0],) + got[3:], (want[0],) + want[3:], (TOL_OUT,) + (TOL_GRAD,) * 3, ("out", "dq", "dk", "dv")):
        close(x, y, tol, what)


def test_bad_bounds_among_many_are_reported(opt):
    q, k, v, do = inputs(32, 400, 400, 2, 2, 64)
    c = torch.arange(0, 401, 4, dtype=torch.int32, device="cuda")       # 100 sequences of 4
    for at, bad in ((0, -1), (70, 100), (100, 401)):
        b = c.clone()
        b[at] = bad
        opt.attention(q, k, v, b)
        with pytest.raises(mb.MuonError) as e:
            opt.sync()
        assert e.value.status == mb.MUON_ERR_INVALID
    opt.attention(q, k, v, c)
    opt.sync()


FIRST_CALLS = """
import torch, muon_newton_schulz_04_b200 as mb
o = mb.Muon(mb.config())
q = torch.ones(70, 2, 64, device="cuda", dtype=torch.bfloat16)
do = torch.full_like(q, 0.5)
c = torch.tensor([0, 3, 70], dtype=torch.int32, device="cuda")
W = torch.ones(128, 24, device="cuda"); top = torch.full((2,), 400.0, device="cuda")
s = torch.cuda.Stream()
s.wait_stream(torch.cuda.current_stream())
g = torch.cuda.CUDAGraph()
with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
    out, lse = o.attention(q, q, q, c)
    grads = o.attention_backward(do, q, q, q, out, lse, c)
    ck = o.checkpoint(q.view(70, 128))
    back = o.checkpoint_load(ck)
    G = o.weight_grad(do.view(70, 128), ck, torch.empty(128, 128, device="cuda"))
    Wq, Wk = W.clone(), W.clone()
    o.qk_clip_grouped(Wq, Wk, top, 64, 100.0)
g.replay()
torch.cuda.synchronize()
o.sync()
assert torch.equal(out, q) and torch.equal(back, q.view(70, 128))
assert torch.equal(G, torch.full_like(G, 35.0))
assert torch.equal(Wq, W * 0.5) and torch.equal(Wk, W * 0.5)
assert float(grads[2].float().sum(0).sub(35.0).abs().max()) <= 35.0 * 2.0 ** -7
print("captured")
"""


def test_first_calls_of_a_process_inside_a_capture():
    """Every operator's first call in its process is a captured one."""
    mbuild.build()
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr


def test_nothing_to_do(opt):
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = opt.attention(e, e, e, cu([]))
    opt.attention_backward(e, e, e, e, out, lse, cu([0]))
    opt.sync()
    assert out.shape == e.shape


@pytest.mark.parametrize("d", [64, 128])
def test_one_side_is_empty(opt, d):
    """Queries without any key row in the call, and keys without any query row."""
    x = inputs(36, 5, 5, 2, 2, d)[0]
    e = torch.empty(0, 2, d, dtype=torch.bfloat16, device="cuda")
    c, none = cu([2, 3]), cu([0, 0])
    top = torch.full((2,), -math.inf, device="cuda")
    out, lse = opt.attention(x, e, e, c, cu_seqlens_k=none, max_logits=top)
    dq, dk, dv = opt.attention_backward(x, x, e, e, out, lse, c, cu_seqlens_k=none)
    assert not out.any() and not dq.any() and bool((lse == -math.inf).all()) and bool((top == -math.inf).all())
    assert dk.shape == e.shape and dv.shape == e.shape
    out, lse = opt.attention(e, x, x, none, cu_seqlens_k=c)
    dq, dk, dv = opt.attention_backward(e, e, x, x, out, lse, none, cu_seqlens_k=c)
    opt.sync()
    assert out.shape == e.shape and not dk.any() and not dv.any()


def test_refusals(opt):
    q, k, v, do = inputs(22, 16, 16, 4, 2, 64)
    c = cu([16])
    out, lse = opt.attention(q, k, v, c)
    for args, err in (((q.float(), k, v, c), TypeError), ((q, k[:, :, :32], v, c), ValueError),
                      ((q, k, v[:8], c), ValueError), ((q, k, v, c.long()), ValueError),
                      ((q, k, v, c.cpu()), ValueError), ((q[:, 0], k, v, c), ValueError)):
        with pytest.raises(err):
            opt.attention(*args)
    with pytest.raises(mb.MuonError) as e:                      # 4 query heads over 3 key heads
        opt.attention(q, torch.zeros(16, 3, 64, dtype=q.dtype, device="cuda"),
                      torch.zeros(16, 3, 64, dtype=q.dtype, device="cuda"), c)
    assert e.value.status == mb.MUON_ERR_INVALID
    with pytest.raises(mb.MuonError) as e:                      # written over an input
        opt.attention(q, k, v, c, out=q)
    assert e.value.status == mb.MUON_ERR_INVALID
    for d in (60, 136):
        x = torch.zeros(16, 2, d, dtype=q.dtype, device="cuda")
        with pytest.raises(mb.MuonError) as e:
            opt.attention(x, x, x, c)
        assert e.value.status == mb.MUON_ERR_UNSUPPORTED
    with pytest.raises(mb.MuonError):
        opt.attention(q, k, v, c, scale=0.0)
    with pytest.raises(mb.MuonError):
        opt.attention_backward(do, q, k, v, out, lse, c, dq=torch.empty_like(q), dk=k)
    opt.sync()
