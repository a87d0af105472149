"""sl_token_logprobs_fwd / _bwd against the formulas in 64 bits, the gradient against differences, alternatives exactly.

Tolerances, with x = z log2(e) - r of the kernels (r whole): x is right to half a unit (2^-24 |x|) and the constant
log2(e) to 2^-25 of z log2(e); 2^x (ex2.approx) to 2^-22; a sum passes an element through at most
ceil(V / 8192) * 8 + 32 additions of 2^-24 each, below 2^-17 of itself at these sizes (V <= 140000: 176 additions), so
log2 s is right to 2^-16.5 in the worst case. That bounds |logp| errors by ln 2 * 2^-16.5 + 2^-22 |logp - z range|; the
additions' errors have either sign, so a hundredth of it is seen. Bound used: 2^-17 + 2^-22 |logp|. The
entropy's: both log2 s and w / s, w a sum of terms p |x|: 2^-16 (1 + sum p |log p|). Gradients: p is right to
2^-17 + the error of x (2^-24 |x| ln 2, |x| <= 150 where p counts): 2^-16 (|g| + |gH| (|log p| + H)) p, plus
|gH| p times the errors of log p and of H themselves, 2^-17 + 2^-16 (1 + H) <= 2^-15 (1 + H) (where log p + H
cancels, as in a row of one token, this is all that is left), plus the type's rounding (bf16: 2^-8 of the value; fp32:
2^-22 of g at the target). 2^x below 2^-126 is 0: 2^-126 (|g| + 150 |gH|) < 1e-35 at most."""
import math

import pytest
import torch

from contextual_sparsity_lora_b200 import binding as B

pytestmark = pytest.mark.gpu
DEV, BF, F32 = "cuda", torch.bfloat16, torch.float32


def reference(z, t):
    z = z.double()
    lse = torch.logsumexp(z, 1, keepdim=True)
    logs = z - lse
    p = logs.exp()
    plogp = torch.where(p > 0, p * logs, 0.0)
    has = (t >= 0) & (t < z.shape[1])
    at = torch.where(has, t, 0).long()
    logp = torch.where(has, logs.gather(1, at[:, None])[:, 0], 0.0)
    return lse[:, 0], logs, p, plogp, -plogp.sum(1), logp, has, at


def best(z, k):
    """Indices of the k largest, equal ones by the lower index, NaN below every number."""
    z = torch.where(z.isnan(), -math.inf, z.double())
    return torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]


def run_fwd(z, t, k=0):
    N = z.shape[0]
    new = lambda *s: torch.full(s, float("nan"), device=DEV)
    logp, stats, ent = new(N), new(N, 2), new(N)
    ids = torch.full((N, k), -7, dtype=torch.int32, device=DEV) if k else None
    top = new(N, k) if k else None
    B.sl_token_logprobs_fwd(z, t, logp, stats, ent, ids, top)
    return logp, stats, ent, ids, top


def check(z, t, k, g, gh):
    N, V = z.shape
    lse, logs, p, plogp, H, logp_w, has, at = reference(z, t)
    logp, stats, ent, ids, top = run_fwd(z, t, k)
    assert ((logp - logp_w).abs() <= 2.0 ** -17 + 2.0 ** -22 * logp_w.abs()).all()
    assert ((stats.double().sum(1) * math.log(2) - lse).abs() <= 2.0 ** -17 + 2.0 ** -22 * lse.abs()).all()
    assert ((ent - H).abs() <= 2.0 ** -16 * (1 + H)).all()
    if k:
        want = best(z, k)
        assert torch.equal(ids.long(), want)
        assert ((top - logs.gather(1, want)).abs() <= 2.0 ** -17 + 2.0 ** -22 * logs.gather(1, want).abs()).all()
    plain = torch.empty(N, device=DEV), torch.empty(N, 2, device=DEV)
    B.sl_token_logprobs_fwd(z, t, *plain)  # without entropy and alternatives: the same sums
    assert torch.equal(plain[0], logp) and torch.equal(plain[1], stats)
    ld = -(-V // 8) * 8 + 8
    for with_h in (False, True):
        d = torch.full((N, ld), 3.0, dtype=z.dtype, device=DEV)
        B.sl_token_logprobs_bwd(z, t, stats, g, d[:, :V], gh if with_h else None, ent if with_h else None)
        gd, hd = torch.where(has, g.double(), 0.0)[:, None], (gh.double() if with_h else 0 * gh.double())[:, None]
        one = torch.zeros_like(p).scatter_(1, at[:, None], has.double()[:, None])
        want = gd * (one - p) - hd * torch.where(p > 0, p * (logs + H[:, None]), 0.0)
        mag = p * (gd.abs() + hd.abs() * (torch.where(p > 0, logs.abs(), 0.0) + H[:, None]))
        tol = 2.0 ** -16 * mag + 2.0 ** -22 * one * gd.abs() + (2.0 ** -8 * want.abs() if z.dtype == BF else 0) + 1e-35
        tol = tol + 2.0 ** -15 * p * hd.abs() * (1 + H[:, None])
        err = (d[:, :V].double() - want).abs()
        assert (err <= tol).all(), (with_h, (err / tol).max().item())
        assert (d[:, V:] == 3.0).all()
        if with_h:  # in the logits' place
            copy = torch.empty_strided(z.shape, z.stride(), dtype=z.dtype, device=DEV).copy_(z)
            B.sl_token_logprobs_bwd(copy, t, stats, g, copy, gh, ent)
            assert torch.equal(copy, d[:, :V])


def make(N, V, dtype, seed, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    ld = -(-V // 8) * 8
    z = (scale * torch.randn(N, ld, generator=g)).to(dtype).to(DEV)[:, :V]
    t = torch.randint(0, V, (N,), generator=g, dtype=torch.int32).to(DEV)
    return z, t, torch.randn(N, generator=g).to(DEV), torch.randn(N, generator=g).to(DEV)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N,V,k", [(1, 1, 1), (1, 2, 2), (3, 7, 5), (2, 16, 16), (5, 17, 3), (4, 40, 32), (33, 513, 20),
                                   (7, 8192, 1), (2, 8209, 32), (1, 131071, 20), (3, 70001, 32), (40, 32003, 5),
                                   (300, 5000, 8)])
def test_sizes(N, V, k, dtype):
    z, t, g, gh = make(N, V, dtype, N + V)
    t[::3] = -1
    check(z, t, k, g, gh)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_peaked_shifted_and_equal_rows(dtype):
    z, t, g, gh = make(6, 20001, dtype, 9)
    z[0] = 0.0                                  # all equal: alternatives 0 .. k - 1
    z[1, 77] = 90.0                             # one token has all
    z[2] += 5000.0
    z[3] -= 3000.0
    z[4, ::2] = -0.0
    z[4, 1::2] = 0.0                            # the two zeros are equal
    z[5] = torch.linspace(-40, 40, 20001, device=DEV).to(dtype)  # the maximum moves all along the row
    check(z, t, 20, g, gh)


@pytest.mark.parametrize("V", [100, 9000, 131072])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_masked_infinite_and_nan_rows(dtype, V):
    z, t, g, gh = make(9, V, dtype, V, 2.0)
    low = torch.finfo(dtype).min
    z[0, 3:] = -math.inf                        # three tokens left
    z[1, 5:] = low                              # masked by the type's lowest value: counts as -inf
    z[2, ::2] = -math.inf
    z[3] = -math.inf                            # nothing left
    z[4] = low                                  # nothing left
    t[4] = -1
    z[5, V - 1] = math.nan
    z[6] = -math.inf
    z[6, 8] = math.nan                          # NaN among masked ones
    z[7, 1] = math.inf
    z[8, 2] = 3e38
    t[0], t[1], t[2], t[5] = 1, 70, 1, 2
    k = 8
    logp, stats, ent, ids, top = run_fwd(z, t, k)
    d = torch.empty_strided(z.shape, z.stride(), dtype=z.dtype, device=DEV)
    B.sl_token_logprobs_bwd(z, t, stats, g, d, gh, ent)
    zc = torch.where(z < -1e37, -math.inf, z.double())
    lse, logs, p, plogp, H, logp_w, has, at = reference(zc, t)
    live = [0, 1, 2]
    assert ((ent - H).abs()[live] <= 2.0 ** -16 * (1 + H[live])).all()
    assert logp[1] == -math.inf and logp_w[1] == -math.inf
    for r in (0, 2):
        assert abs(logp[r] - logp_w[r]) <= 2.0 ** -17 + 2.0 ** -22 * abs(logp_w[r])
    assert torch.equal(ids[:5].long(), best(z, k)[:5])
    one = torch.zeros_like(p).scatter_(1, at[:, None], has.double()[:, None])
    for r in live:
        want = g[r].double() * (one[r] - p[r]) - gh[r].double() * torch.where(p[r] > 0, p[r] * (logs[r] + H[r]), 0.0)
        tol = (2.0 ** -16 * p[r] * (g[r].abs() + gh[r].abs() * (torch.where(p[r] > 0, logs[r].abs(), 0.0) + H[r]))
               + 2.0 ** -22 * g[r].abs() * one[r] + 2.0 ** -8 * want.abs() + 1e-35
               + 2.0 ** -15 * p[r] * gh[r].abs() * (1 + H[r]))
        assert ((d[r].double() - want).abs() <= tol).all()
        assert (d[r][(p[r] == 0) & (one[r] == 0)] == 0).all()
    for r in (3, 4):
        assert ent[r] == 0 and logp[r] == (-math.inf if r == 3 else 0.0) and (d[r] == 0).all()
        assert (top[r] == -math.inf).all() and stats[r, 0] == -math.inf
    for r in (5, 6, 7, 8):
        assert logp[r].isnan() and ent[r].isnan() and d[r].isnan().all()
    # NaN stands below every number among the alternatives
    assert torch.equal(ids[5].long(), best(z, k)[5])


def test_nan_rank_and_targets_out_of_range():
    z, t, g, gh = make(3, 40, F32, 1)
    z[0, 4:] = math.nan
    t[0], t[1], t[2] = -2147483648, 40, 2147483647  # no token: no logp, no gradient from it
    logp, stats, ent, ids, top = run_fwd(z, t, 5)
    assert (logp[1:] == 0).all() and logp[0] == 0
    assert set(ids[0, :4].tolist()) == {0, 1, 2, 3} and ids[0, 4] == 4 and top[0, 4].isnan()
    d = torch.full_like(z, 9.0)
    B.sl_token_logprobs_bwd(z[1:], t[1:], stats[1:], g[1:], d[1:])
    assert (d[1:] == 0).all() and (d[0] == 9.0).all()


def test_gradient_against_differences():
    """(f(z + h e) - f(z - h e)) / 2h of f = sum g logp + gH H in 64 bits against the kernel's gradient along e."""
    z, t, g, gh = make(4, 333, F32, 12)
    logp, stats, ent, _, _ = run_fwd(z, t)
    d = torch.empty_strided(z.shape, z.stride(), dtype=z.dtype, device=DEV)
    B.sl_token_logprobs_bwd(z, t, stats, g, d, gh, ent)
    e = torch.randn(z.shape, generator=torch.Generator().manual_seed(1), dtype=torch.float64).to(DEV)

    def f(z):
        lse, logs, p, plogp, H, logp, has, at = reference(z, t)
        return (g.double() * logp + gh.double() * H).sum()

    h = 1e-4
    diff = (f(z.double() + h * e) - f(z.double() - h * e)) / (2 * h)
    # the kernel's gradient is right to 2^-16 of its terms; the difference to h^2 times third derivatives (|g| + |gH| H per row)
    assert abs(diff - (d.double() * e).sum()) <= 2.0 ** -15 * (d.double() * e).abs().sum() + 1e-6


def test_other_stream_graph_and_identical_runs():
    z, t, g, gh = make(5, 50000, BF, 3)
    want = run_fwd(z, t, 20)
    again = run_fwd(z, t, 20)
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = run_fwd(z, t, 20)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    logp, stats = torch.empty(5, device=DEV), torch.empty(5, 2, device=DEV)
    d = torch.empty_strided(z.shape, z.stride(), dtype=z.dtype, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.sl_token_logprobs_fwd(z, t, logp, stats)
        B.sl_token_logprobs_bwd(z, t, stats, g, d)
    z.copy_(z.flip(1))
    graph.replay()
    want = run_fwd(z, t)
    dw = torch.empty_like(z)
    B.sl_token_logprobs_bwd(z, t, want[1], g, dw)
    assert torch.equal(logp, want[0]) and torch.equal(d, dw)


def test_refuses_what_is_not_rows():
    z, t, g, _ = make(4, 64, BF, 3)
    logp, stats = torch.empty(4, device=DEV), torch.empty(4, 2, device=DEV)
    ids, top = torch.empty(4, 5, dtype=torch.int32, device=DEV), torch.empty(4, 5, device=DEV)
    for call in (lambda: B.sl_token_logprobs_fwd(z[None], t, logp, stats),
                 lambda: B.sl_token_logprobs_fwd(z, t, logp, stats, None, ids, None),
                 lambda: B.sl_token_logprobs_fwd(z, t, logp, stats, None, None, top),
                 lambda: B.sl_token_logprobs_fwd(z, t, logp, stats, None, ids.flatten(), top.flatten()),
                 lambda: B.sl_token_logprobs_fwd(z.half(), t, logp, stats),
                 lambda: B.sl_token_logprobs_fwd(z, t.long(), logp, stats),
                 lambda: B.sl_token_logprobs_bwd(z[0], t[:1], stats[:1], g[:1], z[0]),
                 lambda: B.sl_token_logprobs_bwd(z, t, stats, g, z.float())):
        with pytest.raises(B.SparseLoRAError) as e:
            call()
        assert e.value.code == B.SL_ERR_INVALID_ARG


FILLS = (-1e4, -1e9, -1e10, -1e20, -1e30, -1e36)


@pytest.mark.parametrize("V", [100, 9000, 131072])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_finite_masks(dtype, V):
    """Rows masked by ordinary large numbers: whole chunks of them before, behind and between what is left, a whole
    CTA's part of a row that a cluster shares, and a target that is masked."""
    z, t, g, gh = make(5 * len(FILLS), V, dtype, V + 1, 2.0)
    for i, fill in enumerate(FILLS):
        a, b, c, d, e = range(5 * i, 5 * i + 5)
        z[a, : V // 3] = fill
        z[b, : V - 7] = fill
        z[c, V // 2:] = fill
        z[d, 5: V - 2] = fill
        z[e, 1:] = fill                         # one token has all
        t[a], t[e] = V // 3 - 1, 0
    check(z, t, 8, g, gh)
    check(z[:2], t[:2], 8, g[:2], gh[:2])       # few rows: clusters
    check(z[20:22], t[20:22], 8, g[20:22], gh[20:22])


def shifted_reference(z, t, plain=reference):
    """reference() about each row's maximum: beside 1e20 a 64-bit log-sum has lost log(V) (its unit is 2^14)."""
    top = z.double().amax(1, keepdim=True)
    lse, logs, p, plogp, H, logp, has, at = plain(z.double() - top, t)
    return lse + top[:, 0], logs, p, plogp, H, logp, has, at


@pytest.mark.parametrize("V", [1, 100, 9000, 131072])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_rows_of_far_logits(monkeypatch, dtype, V):
    """Rows whose maximum itself is large: all equal, masks of several kinds and nothing else, one above the rest, a
    maximum that comes in many places, neighbouring numbers (which fp32 cannot tell apart times log2 e)."""
    monkeypatch.setitem(globals(), "reference", shifted_reference)
    far = [s * v for v in (1e9, 1.4e9, 1.6e9, 1e10, 3e15, 1e20, 1e30, 1e36) for s in (1.0, -1.0)]
    z, t, g, gh = make(len(far) + 8, V, dtype, V + 2, 2.0)
    for i, v in enumerate(far):
        z[i] = v
    n = len(far)
    z[n] = -1e30
    z[n, V // 2:] = -1e10
    z[n + 1] = -1e10
    z[n + 1, ::3] = -1e20
    z[n + 2, V // 2] = 1e10                     # one far logit over ordinary ones
    z[n + 3, ::5] = 1e20
    for i, v in ((4, 3e9), (5, -3e9), (6, 2.2e9), (7, -1.2e10)):
        x = torch.full((V,), v, dtype=dtype)
        bits = x.view(torch.int16 if dtype == BF else torch.int32)
        bits += torch.arange(V, dtype=bits.dtype) % 7
        z[n + i] = x.to(DEV)
    t[: n] = torch.arange(n, dtype=torch.int32).to(DEV) % V
    t[n + 4:] = torch.arange(4, dtype=torch.int32).to(DEV) % V
    check(z, t, min(8, V), g, gh)
    check(z[2:4], t[2:4], min(8, V), g[2:4], gh[2:4])
    check(z[n + 5: n + 6], t[n + 5: n + 6], min(8, V), g[n + 5: n + 6], gh[n + 5: n + 6])


def test_far_logits_beside_nan_and_infinity():
    z, t, g, gh = make(4, 600, F32, 5)
    z[0], z[1], z[2], z[3] = -1e30, 1e20, -1e20, -1e30
    z[0, 300], z[1, 301] = math.nan, math.inf
    z[2, 302], z[3, 303] = 2e37, -math.inf      # above 2^123; -inf counts as nothing
    t[3] = 303
    logp, stats, ent, ids, top = run_fwd(z, t, 3)
    d = torch.empty_strided(z.shape, z.stride(), dtype=z.dtype, device=DEV)
    B.sl_token_logprobs_bwd(z, t, stats, g, d, gh, ent)
    assert logp[:3].isnan().all() and ent[:3].isnan().all() and d[:3].isnan().all()
    assert logp[3] == -math.inf and abs(ent[3] - math.log(599)) <= 2.0 ** -12 and d[3].isfinite().all()
    assert torch.equal(ids[3], torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV))
    assert (top[3] + math.log(599)).abs().max() <= 2.0 ** -16
