"""sl_attention_plan, sl_attention_masked_fwd / _bwd against the formulas in 64 bits on the same bf16 inputs, the
gradient against differences, empty rows, strides, graphs and wrong plans.

Tolerances count the roundings to bf16 (2^-8 each, of the value): P before P V and P^T dO, dS before its two products,
the results themselves. The rest is fp32: scores (head_dim + 8 additions and roundings of 2^-24 of
scale sum |q||k|, which is at most 2^6 for these inputs: 2^-11 of P and of dS in the worst case), sums and lse.
  o:   (2^-8 + 2^-11) sum_j P |v|  + 2^-8 |o|
  dv:  (2^-8 + 2^-11) sum_i P |dO| + 2^-8 |dv|
  dS:  E = (2^-8 + 2^-11) |dS| + 2^-11 P (1 - tanh^2) (|dP| + sum_j P |dP|)  (D is a sum of P dP in fp32)
  dq:  scale E |k| + 2^-8 |dq|;  dk: scale E^T |q| + 2^-8 |dk|
  lse: 2^-11 in the worst case of a score; seen 1e-6. Bound used: 1e-4."""
import math

import pytest
import torch

from contextual_sparsity_lora_b200 import binding as B
from contextual_sparsity_lora_b200.packing import AttentionPlan, packed_rows

pytestmark = pytest.mark.gpu
DEV, BF = "cuda", torch.bfloat16
E8, E11 = 2.0 ** -8, 2.0 ** -11


def reference(q, k, v, do, lo, hi, n_seq, hq, hkv, hd, cap=0.0, slopes=None, scale=0.0):
    """fp64 values and error bounds: o, lse, dq, dk, dv as (value, bound)."""
    T = q.shape[0]
    S, per = T // n_seq, hq // hkv
    scale = scale or 1 / math.sqrt(hd)
    heads = lambda x, h: x.double().reshape(n_seq, S, h, hd).permute(0, 2, 1, 3)
    Q, K, V, G = heads(q, hq), heads(k, hkv), heads(v, hkv), heads(do, hq)
    K, V = (x.repeat_interleave(per, 1) for x in (K, V))
    raw = scale * Q @ K.transpose(2, 3)
    grad = torch.ones_like(raw)
    t = raw
    if cap:
        th = torch.tanh(raw / cap)
        t, grad = cap * th, 1 - th ** 2
    at = torch.arange(S, device=DEV)
    if slopes is not None:
        t = t - slopes.double().view(1, hq, 1, 1) * (at[:, None] - at[None, :]).abs()
    see = (at >= lo.view(n_seq, 1, S, 1)) & (at < hi.view(n_seq, 1, S, 1))
    t = torch.where(see, t, -math.inf)
    lse = torch.logsumexp(t, -1)
    P = torch.where(see, (t - torch.where(lse.isinf(), 0.0, lse)[..., None]).exp(), 0.0)
    O = P @ V
    Eo = (E8 + E11) * (P @ V.abs()) + E8 * O.abs()
    dP = G @ V.transpose(2, 3)
    dS = P * (dP - (G * O).sum(-1, keepdim=True)) * grad
    E = (E8 + E11) * dS.abs() + E11 * P * grad * (dP.abs() + (P * dP.abs()).sum(-1, keepdim=True))
    flat = lambda x: x.permute(0, 2, 1, 3).reshape(T, -1)
    group = lambda x: flat(x.reshape(n_seq, hkv, per, S, hd).sum(2))
    dq, dk, dv = scale * dS @ K, group(scale * dS.transpose(2, 3) @ Q), group(P.transpose(2, 3) @ G)
    out = dict(o=(flat(O), flat(Eo)), lse=(lse.permute(1, 0, 2).reshape(hq, T), 1e-4))
    out["dq"] = (flat(dq), flat(scale * E @ K.abs()) + E8 * flat(dq).abs())
    out["dk"] = (dk, group(scale * E.transpose(2, 3) @ Q.abs()) + E8 * dk.abs())
    out["dv"] = (dv, (E8 + E11) * group(P.transpose(2, 3) @ G.abs()) + E8 * dv.abs())
    return out


def hold(got, want):
    for name, (w, tol) in want.items():
        g = got[name].double()
        inf = w.isinf()
        assert torch.equal(g[inf], w[inf]), name
        err = (g - torch.where(inf, 0.0, w)).abs()[~inf]
        lim = (tol if isinstance(tol, float) else tol[~inf]) + 1e-7
        assert (err <= lim).all(), (name, int((~(err <= lim)).sum()), (err / lim).max().item())


def inputs(n_seq, S, hq, hkv, hd, seed, pad=0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    new = lambda h, s=1.0: (s * torch.randn(n_seq * S, h * hd + pad, generator=g)).to(BF).to(DEV)[:, : h * hd]
    return new(hq, spread), new(hkv), new(hkv), new(hq)


def call(q, k, v, do, plan, n_seq, hq, hkv, hd, ws=None, **kw):
    ws = ws or B.Workspace()
    T = q.shape[0]
    like = lambda t: torch.empty_strided(t.shape, t.stride(), dtype=BF, device=DEV).fill_(float("nan"))
    r = dict(o=like(q), lse=torch.full((hq, T), float("nan"), device=DEV), dq=like(q), dk=like(k), dv=like(v))
    B.sl_attention_masked_fwd(ws, q, k, v, n_seq, hq, hkv, hd, plan, r["o"], r["lse"], **kw)
    B.sl_attention_masked_bwd(ws, q, k, v, r["o"], do, r["lse"], n_seq, hq, hkv, hd, plan, r["dq"], r["dk"], r["dv"], **kw)
    torch.cuda.synchronize()
    assert ws.read_device_flag() == 0
    return r


def plan_of(lo, hi, n_seq, S):
    p = AttentionPlan(n_seq, S)
    p.set(lo, hi)
    return p.buf


def docs_of(n_seq, S, n_docs, pad, seed):
    g = torch.Generator().manual_seed(seed)
    live = S - min(pad, S)
    out = []
    for _ in range(n_seq):
        cuts = sorted({0, live} | set((torch.rand(n_docs - 1, generator=g) * live).long().tolist()))
        out.append([b - a for a, b in zip(cuts, cuts[1:])])
    return out


OPTIONS = {"plain": {}, "cap": dict(softcap=7.0), "bias": dict(slopes=True), "both": dict(softcap=4.0, slopes=True),
           "scale": dict(scale=0.3)}
SHAPES = [  # n_seq, S, hq, hkv, hd, documents, prefix, window, padding, ld padding
    (1, 1, 1, 1, 8, 1, 0, 0, 0, 0), (2, 2, 4, 2, 32, 1, 0, 0, 0, 0), (3, 64, 4, 2, 32, 3, 0, 0, 5, 0),
    (1, 127, 2, 1, 64, 2, 20, 0, 0, 8), (2, 128, 6, 3, 96, 1, 0, 0, 0, 0), (1, 129, 5, 1, 40, 2, 129, 0, 0, 0),
    (2, 300, 4, 1, 128, 4, 0, 0, 37, 16), (1, 257, 2, 2, 120, 1, 0, 1, 0, 0), (2, 513, 3, 3, 128, 3, 70, 90, 130, 0),
    (1, 1000, 8, 2, 64, 7, 0, 0, 400, 0), (9, 200, 2, 1, 16, 2, 30, 0, 0, 0),
    # more (head, query tile) units than a GPU has SMs, so that each CTA goes through several: three heads per group, four
    # of them, one tile per sequence, long and short documents
    (5, 333, 24, 8, 64, 3, 40, 0, 20, 0), (11, 200, 16, 4, 40, 2, 0, 60, 11, 8), (160, 40, 3, 1, 32, 2, 0, 0, 3, 0),
    (2, 700, 32, 8, 128, 3, 0, 0, 0, 0)]


@pytest.mark.parametrize("opt", OPTIONS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_intervals_and_scores(shape, opt):
    n_seq, S, hq, hkv, hd, docs, prefix, window, pad, ldpad = shape
    kw = dict(OPTIONS[opt])
    if kw.get("slopes"):
        kw["slopes"] = torch.tensor([2.0 ** -(h % 8 + 1) for h in range(hq)], device=DEV)
    lens = docs_of(n_seq, S, docs, pad, S)
    lo, hi, _ = packed_rows(lens, S, [[prefix] * len(d) for d in lens], window, DEV)
    q, k, v, do = inputs(n_seq, S, hq, hkv, hd, S + hd, ldpad, 2.0)
    got = call(q, k, v, do, plan_of(lo, hi, n_seq, S), n_seq, hq, hkv, hd, **kw)
    hold(got, reference(q, k, v, do, lo, hi, n_seq, hq, hkv, hd, kw.get("softcap", 0.0), kw.get("slopes"),
                        kw.get("scale", 0.0)))
    empty = (lo >= hi)
    assert (got["o"][empty] == 0).all() and (got["dq"][empty] == 0).all() and (got["lse"][:, empty] == -math.inf).all()


@pytest.mark.parametrize("n_seq,S,hq,hkv,hd", [(3, 517, 16, 4, 8), (2, 300, 4, 2, 64), (1, 4, 4, 2, 128), (8, 128, 6, 2, 120)])
def test_fine_gradients(n_seq, S, hq, hkv, hd):
    """Heads of up to 64 and sequences of up to 128 tokens: dq and dk are as exact as their own rounding to bf16. What is
    left of dS behind two bf16 is 2^-17 of it; were that 20 times as large against the output (sums that cancel), it would add
    2e-4 to the rounding's 1.7e-3: sqrt(1 + (0.2 / 1.7)^2) < 1.01 times the rounding's error, 1.05 allowed."""
    lo, hi, _ = packed_rows([[S]] * n_seq, S, None, 0, DEV)
    q, k, v, do = inputs(n_seq, S, hq, hkv, hd, S + hd, 0, 2.0)
    got = call(q, k, v, do, plan_of(lo, hi, n_seq, S), n_seq, hq, hkv, hd)
    want = reference(q, k, v, do, lo, hi, n_seq, hq, hkv, hd, 0.0, None, 0.0)
    for n in ("dq", "dk"):
        w = want[n][0]
        assert (got[n].double() - w).norm() <= 1.05 * (w.to(BF).double() - w).norm(), n


@pytest.mark.parametrize("n_seq,S,hq,hkv,hd", [(2, 300, 4, 2, 64), (1, 1500, 3, 1, 128), (40, 70, 2, 2, 32), (70, 130, 1, 1, 8)])
def test_random_intervals(n_seq, S, hq, hkv, hd):
    """Any intervals, not monotone, some empty, some out of range (clipped), whole tiles that see nothing."""
    g = torch.Generator().manual_seed(S)
    T = n_seq * S
    lo = torch.randint(-5, S, (T,), generator=g, dtype=torch.int32)
    hi = lo + torch.randint(-3, S, (T,), generator=g, dtype=torch.int32)
    lo[: min(140, S)] = hi[: min(140, S)] = 3
    lo[-1], hi[-1] = -2147483648, 2147483647
    lo, hi = lo.to(DEV), hi.to(DEV)
    q, k, v, do = inputs(n_seq, S, hq, hkv, hd, S, 0, 2.0)
    got = call(q, k, v, do, plan_of(lo, hi, n_seq, S), n_seq, hq, hkv, hd, softcap=5.0)
    hold(got, reference(q, k, v, do, lo, hi, n_seq, hq, hkv, hd, 5.0))


def test_nothing_seen_at_all_and_defaults():
    n_seq, S, hq, hkv, hd = 2, 150, 2, 1, 64
    q, k, v, do = inputs(n_seq, S, hq, hkv, hd, 1)
    zero = torch.zeros(n_seq * S, dtype=torch.int32, device=DEV)
    got = call(q, k, v, do, plan_of(zero, zero, n_seq, S), n_seq, hq, hkv, hd)
    assert all((got[n] == 0).all() for n in ("o", "dq", "dk", "dv")) and (got["lse"] == -math.inf).all()
    # the default plan is causal: the attention core's own results within both kernels' roundings
    pos = torch.arange(S, dtype=torch.int32, device=DEV).repeat(n_seq)
    got = call(q, k, v, do, AttentionPlan(n_seq, S).buf, n_seq, hq, hkv, hd)
    hold(got, reference(q, k, v, do, zero, pos + 1, n_seq, hq, hkv, hd))


@pytest.mark.parametrize("S,hd,kw", [(1, 8, {}), (77, 64, {}), (300, 128, dict(softcap=5.0)), (130, 96, dict(slopes=True))])
def test_rows_of_one_key_have_no_score_gradient(S, hd, kw):
    """P = 1, o = v, dq = dk = 0 exactly (not a rounding's rest), dv = do."""
    q, k, v, do = inputs(1, S, 2, 2, hd, S)
    at = torch.arange(S, dtype=torch.int32, device=DEV)
    if kw.get("slopes"):
        kw = dict(slopes=torch.tensor([0.5, 0.25], device=DEV))
    got = call(q, k, v, do, plan_of(at, at + 1, 1, S), 1, 2, 2, hd, **kw)
    assert (got["dq"] == 0).all() and (got["dk"] == 0).all() and torch.equal(got["o"], v)
    hold(got, reference(q, k, v, do, at, at + 1, 1, 2, 2, hd, kw.get("softcap", 0.0), kw.get("slopes")))


def test_large_scores_and_slopes():
    """Scores of several hundred (one key takes all) and slopes that leave only near keys."""
    n_seq, S, hq, hkv, hd = 1, 400, 4, 2, 64
    q, k, v, do = inputs(n_seq, S, hq, hkv, hd, 4)
    lo = torch.zeros(S, dtype=torch.int32, device=DEV)
    hi = torch.arange(1, S + 1, dtype=torch.int32, device=DEV)
    plan = plan_of(lo, hi, n_seq, S)
    slopes = torch.tensor([0.0, 3.0, 40.0, 1000.0], device=DEV)
    got = call(q, k, v, do, plan, n_seq, hq, hkv, hd, slopes=slopes)
    hold(got, reference(q, k, v, do, lo, hi, n_seq, hq, hkv, hd, 0.0, slopes))
    big = call((q.float() * 64).to(BF), k, v, do, plan, n_seq, hq, hkv, hd, softcap=30.0)
    hold(big, reference((q.float() * 64).to(BF), k, v, do, lo, hi, n_seq, hq, hkv, hd, 30.0))
    far = call((q.float() * 16).to(BF), k, v, do, plan, n_seq, hq, hkv, hd)
    assert all(torch.isfinite(far[n].float()).all() for n in far)


@pytest.mark.parametrize("n_seq,S,hq,hkv,docs,prefix,window,kw", [
    (8, 512, 32, 8, 3, 0, 0, {}), (1, 2500, 8, 2, 2, 300, 0, dict(softcap=20.0)), (1, 4096, 4, 1, 1, 0, 600, {})])
def test_larger(n_seq, S, hq, hkv, docs, prefix, window, kw):
    hd = 128
    lens = docs_of(n_seq, S, docs, S // 20, S)
    lo, hi, _ = packed_rows(lens, S, [[prefix] * len(d) for d in lens], window, DEV)
    q, k, v, do = inputs(n_seq, S, hq, hkv, hd, S, 0, 2.0)
    got = call(q, k, v, do, plan_of(lo, hi, n_seq, S), n_seq, hq, hkv, hd, **kw)
    per = hq // hkv
    for g in sorted({0, hkv - 1}):  # one group of heads at a time (the reference is S x S in 64 bits)
        hs = slice(g * per * hd, (g + 1) * per * hd)
        ks = slice(g * hd, (g + 1) * hd)
        want = reference(q[:, hs], k[:, ks], v[:, ks], do[:, hs], lo, hi, n_seq, per, 1, hd, kw.get("softcap", 0.0))
        hold(dict(o=got["o"][:, hs], dq=got["dq"][:, hs], dk=got["dk"][:, ks], dv=got["dv"][:, ks],
                  lse=got["lse"][g * per: (g + 1) * per]), want)


def test_forward_is_identical_between_runs_and_streams_and_follows_its_plan_in_a_graph():
    n_seq, S, hq, hkv, hd = 2, 300, 4, 2, 64
    q, k, v, do = inputs(n_seq, S, hq, hkv, hd, 8)
    plan = AttentionPlan(n_seq, S)
    ws = B.Workspace()
    want = call(q, k, v, do, plan.buf, n_seq, hq, hkv, hd, ws)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = call(q, k, v, do, plan.buf, n_seq, hq, hkv, hd, B.Workspace())
    s.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in ("o", "lse", "dq", "dk", "dv"))
    r = {n: torch.empty_like(t) for n, t in want.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.sl_attention_masked_fwd(ws, q, k, v, n_seq, hq, hkv, hd, plan.buf, r["o"], r["lse"])
        B.sl_attention_masked_bwd(ws, q, k, v, r["o"], do, r["lse"], n_seq, hq, hkv, hd, plan.buf, r["dq"], r["dk"], r["dv"])
    lo, hi, _ = packed_rows([[100, 150], [300]], S, device=DEV)
    for rows in ((None, None), (lo, hi)):  # the plan's buffer is read at replay
        plan.set(*rows)
        graph.replay()
        torch.cuda.synchronize()
        full = [torch.zeros_like(lo), torch.arange(1, S + 1, dtype=torch.int32, device=DEV).repeat(n_seq)]
        hold(r, reference(q, k, v, do, *(full if rows[0] is None else rows), n_seq, hq, hkv, hd))


def test_slices_of_one_projection_and_rows_behind_the_batch():
    """q, k, v as column slices of one tensor, outputs as the first rows of longer ones: what lies outside stays."""
    n_seq, S, hq, hkv, hd = 1, 150, 4, 2, 64
    g = torch.Generator().manual_seed(2)
    qkv = torch.randn(S, (hq + 2 * hkv) * hd, generator=g).to(BF).to(DEV)
    q, k, v = qkv[:, : hq * hd], qkv[:, hq * hd: (hq + hkv) * hd], qkv[:, (hq + hkv) * hd:]
    do = torch.randn(S, hq * hd, generator=g).to(BF).to(DEV)
    plan, ws = AttentionPlan(n_seq, S).buf, B.Workspace()
    o = torch.full((S + 9, hq * hd), 5.0, dtype=BF, device=DEV)
    lse = torch.empty(hq, S, device=DEV)
    grads = torch.full((S + 9, (hq + 2 * hkv) * hd), 5.0, dtype=BF, device=DEV)
    dq, dk, dv = grads[:S, : hq * hd], grads[:S, hq * hd: (hq + hkv) * hd], grads[:S, (hq + hkv) * hd:]
    B.sl_attention_masked_fwd(ws, q, k, v, n_seq, hq, hkv, hd, plan, o[:S], lse)
    B.sl_attention_masked_bwd(ws, q, k, v, o[:S], do, lse, n_seq, hq, hkv, hd, plan, dq, dk, dv)
    zero = torch.zeros(S, dtype=torch.int32, device=DEV)
    hold(dict(o=o[:S], lse=lse, dq=dq, dk=dk, dv=dv),
         reference(q, k, v, do, zero, torch.arange(1, S + 1, device=DEV), n_seq, hq, hkv, hd))
    assert (o[S:] == 5.0).all() and (grads[S:] == 5.0).all()


def test_wrong_plan_is_refused_on_the_device():
    """A buffer without a plan, or with one of other sizes: nothing is written, the error word says so."""
    n_seq, S, hq, hkv, hd = 2, 200, 2, 1, 64
    q, k, v, do = inputs(n_seq, S, hq, hkv, hd, 3)
    other = AttentionPlan(4, 100)
    for buf in (torch.zeros_like(AttentionPlan(n_seq, S).buf),
                torch.cat((other.buf, torch.zeros(8192, dtype=torch.uint8, device=DEV)))):
        ws = B.Workspace()
        o, lse = torch.full_like(q, 5.0), torch.full((hq, n_seq * S), 5.0, device=DEV)
        B.sl_attention_masked_fwd(ws, q, k, v, n_seq, hq, hkv, hd, buf, o, lse)
        assert ws.read_device_flag() != 0 and (o == 5.0).all() and (lse == 5.0).all()
        ws = B.Workspace()
        dk, dv = torch.full_like(k, 5.0), torch.full_like(v, 5.0)
        B.sl_attention_masked_bwd(ws, q, k, v, o, do, lse, n_seq, hq, hkv, hd, buf, torch.empty_like(q), dk, dv)
        assert ws.read_device_flag() != 0 and (dk == 5.0).all() and (dv == 5.0).all()


def test_formula_gradient_against_differences():
    """The formulas that the kernels are held to, in 64 bits: <do, o(x + h) - o(x - h)> / 2h against their gradients."""
    n_seq, S, hq, hkv, hd = 1, 40, 2, 1, 8
    g = torch.Generator().manual_seed(6)
    q, k, v, do = (torch.randn(S, h * hd, generator=g, dtype=torch.float64).to(DEV) for h in (hq, hkv, hkv, hq))
    lo, hi, _ = packed_rows([[15, 20]], S, [[5, 0]], device=DEV)
    slopes = torch.tensor([0.1, 0.3], device=DEV)
    f = lambda q, k, v: (do * reference(q, k, v, do, lo, hi, n_seq, hq, hkv, hd, 2.0, slopes)["o"][0]).sum()
    r = reference(q, k, v, do, lo, hi, n_seq, hq, hkv, hd, 2.0, slopes)
    e = [torch.randn(t.shape, generator=g, dtype=torch.float64).to(DEV) for t in (q, k, v)]
    h = 1e-5
    up, down = ([t + s * h * d for t, d in zip((q, k, v), e)] for s in (1, -1))
    diff = (f(*up) - f(*down)) / (2 * h)
    want = sum((r[n][0] * d).sum() for n, d in zip(("dq", "dk", "dv"), e))
    assert abs(diff - want) <= 1e-7 * sum((r[n][0] * d).abs().sum() for n, d in zip(("dq", "dk", "dv"), e))


@pytest.mark.parametrize("kw", [{}, dict(slopes=True), dict(softcap=5.0)], ids=["plain", "bias", "cap"])
def test_nan_and_infinite_scores_show_in_their_rows(kw):
    """A NaN in a key (at each place of a tile) or in a query: o and lse of the rows that see it are NaN throughout, the
    others are what they were. A score of +inf too (without a cap, whose tanh is 1 there). With a cap a warp's largest
    score chooses the form of its tanh, so the others' scores may change by both forms' errors, 5 x 2 x 2^-22 < 2^-18 (lse
    by that, P by a step of 2^-8 in the rows' sum of at most max |v|, o's own rounding by another)."""
    n_seq, S, hq, hkv, hd = 1, 300, 2, 1, 64
    if kw.get("slopes"):
        kw = dict(slopes=torch.tensor([0.5, 0.25], device=DEV))
    q, k, v, do = inputs(n_seq, S, hq, hkv, hd, 11)
    at = torch.arange(S, dtype=torch.int32, device=DEV)
    plan, ws = plan_of((at - 150).clamp(min=0), at + 1, n_seq, S), B.Workspace()

    def forward(q, k):
        o, lse = torch.empty_like(q), torch.empty(hq, S, device=DEV)
        B.sl_attention_masked_fwd(ws, q, k, v, n_seq, hq, hkv, hd, plan, o, lse, **kw)
        assert ws.read_device_flag() == 0
        return o, lse

    def same(got, want):
        if not kw.get("softcap"):
            return torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        return ((got[0] - want[0]).abs() <= 2.0 ** -7 * v.abs().max()).all() and \
            ((got[1] - want[1]).abs() <= 2.0 ** -18).all()

    o, lse = forward(q, k)
    for j in (*range(72), 127, 128, 190, 255, 299):
        bad = k.clone()
        bad[j, j % hd] = math.nan
        sees = (at >= j) & (at - 150 <= j)
        ob, lseb = forward(q, bad)
        assert ob[sees].isnan().all() and lseb[:, sees].isnan().all(), j
        assert same((ob[~sees], lseb[:, ~sees]), (o[~sees], lse[:, ~sees])), j
        bad = q.clone()
        bad[j, hd + 3] = math.nan               # of the second head
        ob, lseb = forward(bad, k)
        assert ob[j, hd:].isnan().all() and lseb[1, j].isnan()
        ob[j, hd:], lseb[1, j] = o[j, hd:], lse[1, j]
        assert same((ob, lseb), (o, lse)), j
        if not kw.get("softcap"):
            bad, one = k.clone(), q.clone()
            bad[j], one[:, :hd] = 0.0, q[:, :hd].abs()
            bad[j, 5] = math.inf
            one[j, 5] = 1.0
            want, (ob, lseb) = forward(one, k), forward(one, bad)
            hit = sees & (one[:, 5] > 0)
            assert hit[j] and ob[hit, :hd].isnan().all() and lseb[0, hit].isnan().all(), j
            assert same((ob[~sees], lseb[:, ~sees]), (want[0][~sees], want[1][:, ~sees])), j


def plan_parts(buf, n_seq, S):
    """What a plan's buffer holds: each part on 16 bytes, in the order in which the kernels' Plan names them."""
    n_t = (S + 127) // 128
    words, at, parts = buf.cpu().view(torch.int32), 16, {}
    for name, n, width in (("lo", n_seq * S, 1), ("hi", n_seq * S, 1), ("q", n_seq * n_t, 4), ("k", n_seq * n_t, 2),
                           ("q_order", n_seq * n_t, 4), ("k_order", n_seq * n_t, 4), ("q2", n_seq * ((n_t + 1) // 2), 2),
                           ("q2_order", n_seq * ((n_t + 1) // 2), 4)):
        parts[name] = words[at: at + n * width].view(n, width).long()
        at += -(-n * width // 4) * 4
    assert at == words.numel() and words[1:3].tolist() == [n_seq, S]
    return parts


@pytest.mark.parametrize("n_seq,S", [(1, 131072), (3, 16500), (150, 1), (2, 131071), (1, 16384), (1, 1 << 20)])
@pytest.mark.parametrize("kind", ["causal", "documents", "random"])
def test_plans_of_many_tiles(n_seq, S, kind):
    """Plans of more than 128 tiles (two kernels), up to the longest sequence: rows, ranges and orders."""
    g = torch.Generator().manual_seed(S)
    T, n_t = n_seq * S, (S + 127) // 128
    pos = torch.arange(S).repeat(n_seq)
    if kind == "causal":
        lo, hi = torch.zeros(T, dtype=torch.long), pos + 1
    elif kind == "documents":
        lens = docs_of(n_seq, S, 7, S // 30, S)
        lo, hi, _ = (t.long() for t in packed_rows(lens, S, [[90] * len(d) for d in lens], 2000))
    else:
        lo = torch.randint(0, S, (T,), generator=g)
        hi = lo + torch.randint(-40, min(S, 700) + 1, (T,), generator=g)
        lo[: min(200, S)] = hi[: min(200, S)] = 0
    rows = (None, None) if kind == "causal" else (lo.int().to(DEV), hi.int().to(DEV))
    parts = plan_parts(plan_of(*rows, n_seq, S), n_seq, S)
    empty = lo >= hi
    lo, hi = torch.where(empty, 0, lo), torch.where(empty, 0, hi.clamp(max=S))
    assert torch.equal(parts["lo"][:, 0], lo) and torch.equal(parts["hi"][:, 0], hi)
    pad = n_t * 128 - S
    tiles = lambda x, fill: torch.nn.functional.pad(x.view(n_seq, S), (0, pad), value=fill).view(n_seq * n_t, 128)
    full = torch.where(empty, S, lo), torch.where(empty, 0, lo), torch.where(empty, S, hi), hi
    l_min, l_max, h_min, h_max = (f(tiles(x, v), 1) for x, v, f in zip(full, (S, 0, S, 0), (torch.amin, torch.amax) * 2))
    nothing, holes = h_max == 0, tiles(empty, False).any(1)
    want = torch.stack((l_min // 128, (h_max + 127) // 128, (l_max + 127) // 128, h_min // 128), 1)
    want[holes, 2:] = 0
    want[nothing] = torch.tensor([0, 1, 0, 0])
    assert torch.equal(parts["q"], want)
    # key tiles: the first and the last query tile whose range holds them
    x, y = want[:, 0].view(n_seq, n_t, 1), want[:, 1].view(n_seq, n_t, 1)
    at = torch.arange(n_t)
    first, last = torch.full((n_seq, n_t), n_t), torch.zeros(n_seq, n_t, dtype=torch.long)
    for t in range(n_t):
        sees = (at >= x[:, t]) & (at < y[:, t])
        first, last = torch.where(sees, first.clamp(max=t), first), torch.where(sees, t + 1, last)
    first, last = torch.where(last == 0, 0, first), torch.where(last == 0, 1, last)
    assert torch.equal(parts["k"], torch.stack((first, last), 2).view(-1, 2))
    x, y = (torch.nn.functional.pad(v[..., 0], (0, n_t & 1), value=fill).view(n_seq, -1, 2) for v, fill in ((x, n_t), (y, 0)))
    assert torch.equal(parts["q2"], torch.stack((x.amin(2), y.amax(2)), 2).view(-1, 2))
    for name in ("q", "k", "q2"):
        order, ranges = parts[name + "_order"], parts[name]
        assert torch.equal(order[:, 0].sort().values, torch.arange(len(ranges)))
        assert torch.equal(order[:, 1:3], ranges[order[:, 0], :2])
        length = order[:, 2] - order[:, 1]
        assert (length[1:] <= length[:-1]).all()


@pytest.mark.parametrize("docs,window,prefix,kw", [(1, 0, 0, {}), (5, 900, 70, dict(softcap=9.0)), (2, 0, 0, dict(slopes=True))])
def test_long_sequences(docs, window, prefix, kw):
    """A sequence of more than 128 tiles, a head at a time (the reference is S x S in 64 bits)."""
    S, hq, hkv, hd = 16500, 3, 1, 64
    if kw.get("slopes"):
        kw = dict(slopes=torch.tensor([0.5, 0.01, 0.0], device=DEV))
    lens = docs_of(1, S, docs, S // 40, S)
    lo, hi, _ = packed_rows(lens, S, [[prefix] * len(d) for d in lens], window, DEV)
    q, k, v, do = inputs(1, S, hq, hkv, hd, S, 0, 2.0)
    got = call(q, k, v, do, plan_of(lo, hi, 1, S), 1, hq, hkv, hd, **kw)
    for h in (0, 2):
        hs = slice(h * hd, (h + 1) * hd)
        sl = kw["slopes"][h: h + 1] if "slopes" in kw else None
        want = reference(q[:, hs], k, v, do[:, hs], lo, hi, 1, 1, 1, hd, kw.get("softcap", 0.0), sl)
        hold(dict(o=got["o"][:, hs], dq=got["dq"][:, hs], lse=got["lse"][h: h + 1]),
             {n: want[n] for n in ("o", "dq", "lse")})
        del want
    one = {n: got[n].clone() for n in ("dk", "dv")}
    parts = [call(q[:, h * hd: (h + 1) * hd], k, v, do[:, h * hd: (h + 1) * hd], plan_of(lo, hi, 1, S), 1, 1, 1, hd,
                  **{**kw, **({"slopes": kw["slopes"][h: h + 1]} if "slopes" in kw else {})}) for h in range(hq)]
    for n in ("dk", "dv"):  # the group's sum against the heads' own, each rounded to bf16
        alone = torch.stack([p[n].double() for p in parts])
        tol = 2.0 ** -8 * (alone.abs().sum(0) + one[n].double().abs()) + 2.0 ** -16 * alone.abs().max()
        assert ((alone.sum(0) - one[n].double()).abs() <= tol).all(), n


@pytest.mark.parametrize("docs,window", [(1, 0), (170, 0), (1, 5), (60, 0)])
@pytest.mark.parametrize("S,hd", [(512, 128), (512, 96), (129, 72)])
def test_gradients_of_larger_heads(S, hd, docs, window):
    """Heads over 64 in sequences over 128 tokens, whose dS is rounded to bf16 once, for long documents, documents and windows
    of a few tokens: the rounding of dS and that of the result are of the same size and independent, so the error of dq and dk
    is sqrt(2) of the latter's alone; a tenth more allowed."""
    n_seq, hq, hkv = 2, 4, 2
    lens = docs_of(n_seq, S, docs, 0, S)
    lo, hi, _ = packed_rows(lens, S, None, window, DEV)
    q, k, v, do = inputs(n_seq, S, hq, hkv, hd, S + hd, 0, 2.0)
    got = call(q, k, v, do, plan_of(lo, hi, n_seq, S), n_seq, hq, hkv, hd)
    want = reference(q, k, v, do, lo, hi, n_seq, hq, hkv, hd)
    for n in ("dq", "dk"):
        w = want[n][0]
        assert (got[n].double() - w).norm() <= 1.1 * math.sqrt(2) * (w.to(BF).double() - w).norm(), n


def test_wrong_plan_leaves_every_output():
    """As in the test above of a wrong plan, dq among the outputs."""
    n_seq, S, hq, hkv, hd = 2, 200, 2, 1, 64
    q, k, v, do = inputs(n_seq, S, hq, hkv, hd, 3)
    ws, buf = B.Workspace(), torch.zeros_like(AttentionPlan(n_seq, S).buf)
    lse = torch.zeros(hq, n_seq * S, device=DEV)
    dq, dk, dv = (torch.full_like(t, 5.0) for t in (q, k, v))
    B.sl_attention_masked_bwd(ws, q, k, v, None, do, lse, n_seq, hq, hkv, hd, buf, dq, dk, dv)
    assert ws.read_device_flag() != 0 and all((t == 5.0).all() for t in (dq, dk, dv))
