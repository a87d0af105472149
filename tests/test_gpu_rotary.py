"""sl_qk_norm_rope_fwd / _bwd against the formulas in 64 bits, and the gradient against differences.

Tolerances. Outputs are rounded to bf16 once: 2^-8 of the value. Before it, fp32: the norm, a cosine and a sine
(a few units of 2^-24 each, the angle's own rounding pi 2^-24 among them) and a sum of two products, together
below 32 units of 2^-24 of the largest element of the row's normalised head (backward: of the largest gradient
term). Gain gradients are sums in fp32: every term is right to 32 units of 2^-24, and no element passes through more
than 256 additions at these sizes, so the error stays within 288 * 2^-24 of the sum of magnitudes."""
import pytest
import torch

from contextual_sparsity_lora_b200 import binding as B

pytestmark = pytest.mark.gpu
DEV, BF, F32, F64 = "cuda", torch.bfloat16, torch.float32, torch.float64
ULP = 2.0 ** -24


def rows(g, T, n, pad=0, scale=1.0):
    t = (scale * torch.randn(T, n + pad, generator=g)).to(BF).to(DEV)
    return t[:, :n]


def split(x, rot, style):
    if style == B.SL_ROPE_PAIRS:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., : rot // 2], x[..., rot // 2: rot]


def turned(x, pos, freq, style, sign=1):
    """x [T, H, hd] (fp64) rotated by sign * pos * freq."""
    if freq is None:
        return x.clone()
    rot = 2 * freq.numel()
    t = sign * pos.double()[:, None, None] * freq.double()
    a, b = split(x, rot, style)
    y = x.clone()
    ya, yb = split(y, rot, style)
    ya.copy_(a * t.cos() - b * t.sin())
    yb.copy_(b * t.cos() + a * t.sin())
    return y


def ref_fwd(x, g, hd, pos, freq, style, eps):
    x = x.double().view(x.shape[0], -1, hd)
    n = x if g is None else x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * g.double()
    return turned(n, pos, freq, style), n


def ref_bwd(dy, x, g, hd, pos, freq, style, eps):
    dn = turned(dy.double().view(dy.shape[0], -1, hd), pos, freq, style, -1)
    if g is None:
        return dn, None, None, dn.abs().amax(-1, keepdim=True)
    x = x.double().view(x.shape[0], -1, hd)
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    terms = dn * x * r
    gd = dn * g.double()
    dx = r * gd - x * r ** 3 * (x * gd).mean(-1, keepdim=True)
    # largest term of a row: r |g dn| and |x| r^3 mean |x g dn|
    big = (r * gd.abs()).amax(-1, keepdim=True) + x.abs().amax(-1, keepdim=True) * r ** 3 * (x * gd).abs().mean(-1, keepdim=True)
    return dx, terms.sum((0, 1)), terms.abs().sum((0, 1)), big


def near(got, want, big):
    got, want = got.double().view_as(want), want
    bad = (got - want).abs() > 2.0 ** -8 * want.abs() + 32 * ULP * big
    assert not bad.any(), (int(bad.sum()), (got - want).abs().max().item())


CASES = [  # T, hq, hkv, hd, rot, norm, style, far, pad
    (1, 1, 1, 8, 8, True, 0, 0, 0), (1, 32, 8, 128, 128, True, 0, 131000, 0), (3, 4, 2, 64, 64, False, 1, 7, 8),
    (37, 6, 3, 96, 48, True, 1, 0, 16), (65, 5, 1, 40, 40, True, 0, 1 << 20, 0), (64, 3, 1, 256, 256, True, 0, 0, 0),
    (33, 2, 2, 248, 24, True, 0, 5, 0), (130, 8, 8, 128, 0, True, 0, 0, 8), (257, 4, 1, 32, 8, False, 0, -70000, 0),
    (5, 2, 1, 120, 8, True, 1, 0, 0), (700, 4, 2, 128, 64, False, 0, 2 ** 31 - 800, 0), (2, 2, 1, 256, 64, False, 1, 0, 0),
    (301, 40, 8, 16, 16, True, 1, 3, 0),
    # neither norm nor rotation: copies
    (9, 5, 1, 8, 0, False, 0, 0, 0), (70, 4, 2, 8, 0, False, 1, 0, 8), (3, 2, 2, 64, 0, False, 0, 9, 0)]


@pytest.mark.parametrize("T,hq,hkv,hd,rot,norm,style,far,pad", CASES)
def test_rotation_and_norm(T, hq, hkv, hd, rot, norm, style, far, pad):
    g = torch.Generator().manual_seed(T + hd)
    q, k = rows(g, T, hq * hd, pad, 3.0), rows(g, T, hkv * hd, pad)
    if T > 2:
        q[1] = 0  # a row of zeros: the norm's eps
    dyq, dyk = rows(g, T, hq * hd, pad), rows(g, T, hkv * hd, pad)
    pos = (torch.randint(0, 800, (T,), generator=g).clamp(max=799) + far).to(torch.int32).to(DEV)
    freq = torch.tensor([10000.0 ** (-2 * i / rot) for i in range(rot // 2)], dtype=F32, device=DEV) if rot else None
    gq, gk = ((1 + 0.2 * torch.randn(hd, generator=g)).to(BF).to(DEV) for _ in range(2)) if norm else (None, None)
    eps = 1e-5
    new = lambda n: torch.full((T, n + pad), 7.0, dtype=BF, device=DEV)[:, :n]
    yq, yk, dq, dk = new(hq * hd), new(hkv * hd), new(hq * hd), new(hkv * hd)
    B.sl_qk_norm_rope_fwd(q, k, pos if rot else None, freq, hd, yq, yk, gq, gk, eps, style)
    ws = B.Workspace()
    dgq, dgk = (torch.full((hd,), float("nan"), device=DEV) for _ in range(2)) if norm else (None, None)
    B.sl_qk_norm_rope_bwd(ws, dyq, dyk, q, k, pos if rot else None, freq, hd, dq, dk, gq, gk, eps, style, dgq, dgk)
    for x, y, dy, dx, gain, dg in ((q, yq, dyq, dq, gq, dgq), (k, yk, dyk, dk, gk, dgk)):
        want, n = ref_fwd(x, gain, hd, pos, freq, style, eps)
        near(y, want, n.abs().amax(-1, keepdim=True))
        want, dgain, mag, big = ref_bwd(dy, x, gain, hd, pos, freq, style, eps)
        near(dx, want, big)
        if norm:
            assert ((dg.double() - dgain).abs() <= 288 * ULP * mag + 1e-30).all()
        if pad:  # columns between the rows are left as they were
            full = y.as_strided((T, y.stride(0)), (y.stride(0), 1))
            assert (full[:, y.shape[1]:] == 7.0).all()


def test_backward_against_differences():
    """<dy, y(x + h) - y(x - h)> / 2h against <dx, h> in 64 bits of the formulas that the kernels are held to."""
    g = torch.Generator().manual_seed(3)
    T, hd = 9, 32
    x, dy, h = (torch.randn(T, 2 * hd, generator=g, dtype=F64).to(DEV) for _ in range(3))
    pos = torch.arange(T, device=DEV)
    freq = torch.tensor([3.0 ** -i for i in range(hd // 2)], device=DEV)
    gain = (1 + 0.1 * torch.randn(hd, generator=g)).to(DEV)
    f = lambda t: ref_fwd(t, gain, hd, pos, freq, 0, 1e-5)[0].flatten(1)
    step = 1e-5
    diff = (dy * (f(x + step * h) - f(x - step * h))).sum() / (2 * step)
    dx = ref_bwd(dy, x, gain, hd, pos, freq, 0, 1e-5)[0].flatten(1)
    assert abs(diff - (dx * h).sum()) <= 1e-7 * (dx * h).abs().sum()
    # and the kernel's gradient along the same direction, from bf16 inputs
    xb, dyb = x.to(BF), dy.to(BF)
    q, k = xb, xb[:, :hd].contiguous()
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    gb = gain.to(BF)
    B.sl_qk_norm_rope_bwd(B.Workspace(), dyb, dyb[:, :hd].contiguous(), q, k, pos.to(torch.int32), freq, hd, dq, dk, gb,
                          gb, 1e-5)
    f = lambda t: ref_fwd(t, gb, hd, pos, freq, 0, 1e-5)[0].flatten(1)
    diff = (dyb.double() * (f(xb.double() + step * h) - f(xb.double() - step * h))).sum() / (2 * step)
    # each dx element is right to 2^-8 of itself (and 32 fp32 units of its row)
    assert abs(diff - (dq.double() * h).sum()) <= (2.0 ** -8 + 1e-5) * (dq.double() * h).abs().sum()


def test_in_place_and_fused_slices():
    """Outputs in the inputs' place, q and k as column slices of one projection's output: bit-identical."""
    g = torch.Generator().manual_seed(5)
    T, hq, hkv, hd = 130, 4, 2, 64
    qkv = rows(g, T, (hq + 2 * hkv) * hd)
    q, k = qkv[:, : hq * hd], qkv[:, hq * hd: (hq + hkv) * hd]
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    freq = torch.tensor([10000.0 ** (-i / 32) for i in range(32)], device=DEV)
    gain = torch.ones(hd, dtype=BF, device=DEV)
    for norm in (None, gain):
        yq, yk = torch.empty(T, hq * hd, dtype=BF, device=DEV), torch.empty(T, hkv * hd, dtype=BF, device=DEV)
        B.sl_qk_norm_rope_fwd(q, k, pos, freq, hd, yq, yk, norm, norm)
        copy = qkv.clone()
        q2, k2 = copy[:, : hq * hd], copy[:, hq * hd: (hq + hkv) * hd]
        B.sl_qk_norm_rope_fwd(q2, k2, pos, freq, hd, q2, k2, norm, norm)
        assert torch.equal(q2, yq) and torch.equal(k2, yk) and torch.equal(copy[:, (hq + hkv) * hd:], qkv[:, (hq + hkv) * hd:])
        dq, dk = torch.empty_like(yq), torch.empty_like(yk)
        B.sl_qk_norm_rope_bwd(B.Workspace(), yq, yk, q, k, pos, freq, hd, dq, dk, norm, norm)
        B.sl_qk_norm_rope_bwd(B.Workspace(), yq, yk, q, k, pos, freq, hd, yq, yk, norm, norm)
        assert torch.equal(dq, yq) and torch.equal(dk, yk)


def test_nan_frequency_and_runs_are_identical():
    g = torch.Generator().manual_seed(6)
    q, k = rows(g, 2000, 128), rows(g, 2000, 64)
    pos = torch.arange(2000, dtype=torch.int32, device=DEV)
    gain = torch.ones(64, dtype=BF, device=DEV)
    freq = torch.rand(32, device=DEV)
    ws, got = B.Workspace(), []
    for _ in range(2):
        out = [torch.empty_like(q), torch.empty_like(k), torch.empty(64, device=DEV), torch.empty(64, device=DEV)]
        B.sl_qk_norm_rope_bwd(ws, q, k, q, k, pos, freq, 64, out[0], out[1], gain, gain, 1e-6, 0, out[2], out[3])
        got.append(out)
    assert all(torch.equal(a, b) for a, b in zip(*got))
    freq[3] = float("inf")
    yq, yk = torch.empty_like(q), torch.empty_like(k)
    B.sl_qk_norm_rope_fwd(q, k, pos, freq, 64, yq, yk)
    bad = yq.view(2000, 2, 64).isnan()
    assert bad[..., 3].all() and bad[..., 35].all() and bad.sum() == 2000 * 2 * 2


def test_other_stream_and_graph():
    g = torch.Generator().manual_seed(7)
    q, k = rows(g, 64, 256), rows(g, 64, 128)
    pos = torch.arange(64, dtype=torch.int32, device=DEV)
    freq = torch.rand(32, device=DEV)
    want = [torch.empty_like(q), torch.empty_like(k)]
    B.sl_qk_norm_rope_fwd(q, k, pos, freq, 64, *want)
    got = [torch.zeros_like(q), torch.zeros_like(k)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        B.sl_qk_norm_rope_fwd(q, k, pos, freq, 64, *got)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.sl_qk_norm_rope_fwd(q, k, pos, freq, 64, *got)
    pos += 11
    B.sl_qk_norm_rope_fwd(q, k, pos, freq, 64, *want)
    graph.replay()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
