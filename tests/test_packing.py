"""Intervals of packed batches, and the refusals of the packed-batch entry points: host side, no GPU (fake device
addresses are never touched)."""
import ctypes

import pytest
import torch

from contextual_sparsity_lora_b200 import binding as B
from contextual_sparsity_lora_b200.packing import packed_rows

P = ctypes.c_void_p
A, ODD = 0x10000, 0x10008


def brute(doc_lens, seq_len, prefix_lens, window):
    lo, hi, pos = [], [], []
    for s, lens in enumerate(doc_lens):
        start = 0
        for d, n in enumerate(lens):
            pre = min(n, prefix_lens[s][d]) if prefix_lens else 0
            for i in range(n):
                seen = [j for j in range(n) if (j <= i and (not window or j > i - window)) or (i < j < pre)]
                lo.append(start + min(seen))
                hi.append(start + max(seen) + 1)
                assert len(seen) == hi[-1] - lo[-1]
                pos.append(i)
            start += n
        for part in (lo, hi, pos):
            part += [0] * (seq_len - start)
    return lo, hi, pos


@pytest.mark.parametrize("docs,S,prefix,window", [([[5, 3], [8]], 8, None, 0), ([[4, 0, 2], []], 9, None, 0),
                                                   ([[6, 6]], 14, [[3, 9]], 0), ([[7, 5]], 12, None, 3),
                                                   ([[9, 4]], 13, [[4, 1]], 2), ([[1]], 1, [[1]], 1)])
def test_packed_rows_against_their_definition(docs, S, prefix, window):
    got = packed_rows(docs, S, prefix, window)
    for g, w in zip(got, brute(docs, S, prefix, window)):
        assert g.dtype == torch.int32 and g.tolist() == w


def test_packed_rows_refuses():
    for docs, S, window in (([[5, 4]], 8, 0), ([[-1]], 8, 0), ([[3]], 8, -1)):
        with pytest.raises(ValueError):
            packed_rows(docs, S, None, window)


@pytest.fixture(scope="module")
def lib():
    return B.lib()


def _ws(nbytes=1 << 40):
    return ctypes.byref(B.SlWorkspaceC(A, nbytes, 0))


def test_rotation_refuses(lib):
    f, g = lib.sl_qk_norm_rope_fwd, lib.sl_qk_norm_rope_bwd

    def fwd(q=A, ldq=256, pos=A, freq=A, rot=64, style=0, gq=A, gk=A, eps=1e-6, T=4, hq=4, hkv=2, hd=64, yk=A, ldyk=128):
        return f(q, ldq, A, 128, pos, freq, rot, style, gq, gk, eps, T, hq, hkv, hd, A, 256, yk, ldyk, None)

    assert fwd(q=None) == fwd(yk=None) == fwd(pos=None) == fwd(freq=None) == B.SL_ERR_INVALID_ARG
    assert fwd(gq=None) == fwd(style=2) == B.SL_ERR_INVALID_ARG
    assert fwd(T=0) == fwd(hq=0) == fwd(hkv=0) == fwd(hd=60) == fwd(hd=264) == fwd(hd=0) == B.SL_ERR_SHAPE
    assert fwd(rot=72) == fwd(rot=12) == fwd(rot=-8) == fwd(eps=-1.0) == fwd(eps=float("nan")) == B.SL_ERR_SHAPE
    assert fwd(q=ODD) == fwd(ldq=248) == fwd(ldq=260) == fwd(ldyk=100) == fwd(gq=ODD) == fwd(pos=A + 2) == \
        B.SL_ERR_ALIGNMENT

    def bwd(dyq=A, q=A, ldq=256, gq=A, gk=A, dgq=A, ws=_ws()):
        return g(dyq, 256, A, 128, q, ldq, A, 128, A, A, 64, 0, gq, gk, 1e-6, 4, 4, 2, 64, A, 256, A, 128, dgq, None, ws,
                 None)

    assert bwd(dyq=None) == bwd(q=None) == bwd(gq=None, gk=None) == B.SL_ERR_INVALID_ARG
    assert bwd(ldq=250) == bwd(dyq=ODD) == B.SL_ERR_ALIGNMENT
    assert bwd(ws=None) == bwd(ws=_ws(1 << 10)) == B.SL_ERR_WORKSPACE


def test_attention_plan_and_call_refuse(lib):
    assert lib.sl_attention_plan_bytes(0, 64) == lib.sl_attention_plan_bytes(1, 0) == 0
    assert lib.sl_attention_plan_bytes(1, (1 << 20) + 1) == lib.sl_attention_plan_bytes(1 << 20, 1 << 20) == 0
    n = lib.sl_attention_plan_bytes(2, 300)
    assert n >= 2 * 300 * 8
    plan = lib.sl_attention_plan
    assert plan(A, A, 2, 300, None, n, None) == B.SL_ERR_INVALID_ARG
    assert plan(A, A, 2, 300, A, n - 1, None) == plan(A, A, 0, 300, A, n, None) == B.SL_ERR_SHAPE
    assert plan(A, A, 2, 300, ODD, n, None) == plan(A + 1, A, 2, 300, A, n, None) == B.SL_ERR_ALIGNMENT
    f, g = lib.sl_attention_masked_fwd, lib.sl_attention_masked_bwd

    def fwd(q=A, ldq=256, S=300, hq=4, hkv=2, hd=64, scale=0.0, cap=0.0, pl=A, pb=n, o=A, lse=A, ws=_ws()):
        return f(q, ldq, A, 128, A, 128, 2, S, hq, hkv, hd, scale, cap, None, pl, pb, o, 256, lse, ws, None)

    def bwd(dv=A, lddv=128, S=300, hd=64, cap=0.0, pb=n, ws=_ws()):
        return g(A, 256, A, 128, A, 128, A, 256, A, 2, S, 4, 2, hd, 0.0, cap, None, A, pb, A, 256, A, 128, dv,
                 lddv, ws, None)

    assert fwd(q=None) == fwd(pl=None) == fwd(o=None) == fwd(lse=None) == bwd(dv=None) == B.SL_ERR_INVALID_ARG
    bad = float("nan")
    assert fwd(S=0) == fwd(S=301) == fwd(hkv=3) == fwd(hd=136) == fwd(hd=4) == fwd(hq=0) == B.SL_ERR_SHAPE
    assert fwd(scale=-1.0) == fwd(cap=-1.0) == fwd(cap=bad) == fwd(scale=float("inf")) == fwd(pb=n - 1) == B.SL_ERR_SHAPE
    assert bwd(S=301) == bwd(hd=12) == bwd(cap=bad) == bwd(pb=0) == B.SL_ERR_SHAPE
    assert fwd(q=ODD) == fwd(ldq=252) == fwd(ldq=248) == fwd(pl=ODD) == fwd(lse=A + 4) == bwd(lddv=120) == \
        B.SL_ERR_ALIGNMENT
    assert fwd(ws=None) == fwd(ws=_ws(16)) == bwd(ws=_ws(1 << 16)) == B.SL_ERR_WORKSPACE
    # more (head, query tile) pairs than the kernels count in 32 bits: 2^30 - 200 one-token sequences, two heads
    many = (1 << 30) - 200
    assert f(A, 16, A, 8, A, 8, many, 1, 2, 1, 8, 0.0, 0.0, None, A, lib.sl_attention_plan_bytes(many, 1), A, 16, A, _ws(),
             None) == B.SL_ERR_SHAPE


def test_token_logprobs_refuse(lib):
    f, g = lib.sl_token_logprobs_fwd, lib.sl_token_logprobs_bwd

    def fwd(t=0, z=A, ld=104, N=4, V=100, tg=A, logp=A, st=A, k=5, ids=A):
        return f(t, z, ld, N, V, tg, logp, st, None, k, ids, A, None)

    def bwd(t=0, z=A, ld=104, N=4, V=100, ent=A, d=A, ldd=104):
        return g(t, z, ld, N, V, A, A, A, A, ent, d, ldd, None)

    assert fwd(t=2) == fwd(z=None) == fwd(tg=None) == fwd(logp=None) == fwd(st=None) == fwd(ids=None) == \
        B.SL_ERR_INVALID_ARG
    assert bwd(ent=None) == bwd(d=None) == bwd(t=-1) == B.SL_ERR_INVALID_ARG
    assert fwd(N=0) == fwd(V=0) == fwd(k=33) == fwd(k=-1) == fwd(V=4) == fwd(V=1 << 25, ld=1 << 25) == B.SL_ERR_SHAPE
    assert bwd(N=0) == bwd(V=0) == B.SL_ERR_SHAPE
    assert fwd(z=ODD) == fwd(ld=96) == fwd(ld=100) == fwd(t=1, ld=102) == fwd(st=A + 4) == B.SL_ERR_ALIGNMENT
    assert bwd(d=ODD) == bwd(ldd=96) == bwd(ldd=108) == B.SL_ERR_ALIGNMENT
    # with alternatives, a vocabulary whose chunk maxima do not fit eight CTAs' shared memory
    assert fwd(V=1 << 24, ld=1 << 24) == B.SL_ERR_SHAPE


def test_wrappers_refuse_what_the_library_cannot_see():
    """Tensors of the CPU, of another type, shape or layout."""
    bf = torch.bfloat16
    x, g = torch.zeros(4, 64, dtype=bf), torch.zeros(4, dtype=torch.int32)
    for call in (lambda: B.sl_qk_norm_rope_fwd(x, x, g, None, 32, x, x),
                 lambda: B.sl_token_logprobs_fwd(x, g, torch.zeros(4), torch.zeros(4, 2)),
                 lambda: B.sl_attention_plan(g, g, 1, torch.zeros(4096, dtype=torch.uint8))):
        with pytest.raises(B.SparseLoRAError) as e:
            call()
        assert e.value.code == B.SL_ERR_INVALID_ARG
    with pytest.raises(B.SparseLoRAError):
        B.attention_plan_buffer(0, 64, "cpu")


def test_streams_without_torchs_private_names(monkeypatch):
    """Where torch has no _cuda_getDevice or _cuda_getCurrentRawStream, its public calls serve."""
    import importlib.util
    import types

    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: types.SimpleNamespace(cuda_stream=100 + device))
    spec = importlib.util.spec_from_file_location("binding_without_private_names", B.__file__)
    copy = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(copy)
    assert copy._current_device() == 3 and copy._raw_stream(3) == 103 and copy._stream().value == 103


def test_misaligned_32_bit_values_are_refused(lib):
    """Values that kernels read or write one by one (the others are in the tests above): an address off by two would
    fault them."""
    n, off = lib.sl_attention_plan_bytes(2, 300), A + 2
    bad = []
    for k in range(2):
        dg = [A, A]
        dg[k] = off
        bad.append(lib.sl_qk_norm_rope_bwd(A, 256, A, 128, A, 256, A, 128, A, A, 64, 0, A, A, 1e-6, 4, 4, 2, 64, A, 256, A, 128,
                                           *dg, _ws(), None))
    bad.append(lib.sl_attention_masked_fwd(A, 256, A, 128, A, 128, 2, 300, 4, 2, 64, 0.0, 0.0, off, A, n, A, 256, A, _ws(),
                                           None))
    bad.append(lib.sl_attention_masked_bwd(A, 256, A, 128, A, 128, A, 256, A, 2, 300, 4, 2, 64, 0.0, 0.0, off, A, n, A, 256,
                                           A, 128, A, 128, _ws(), None))
    for k in range(5):
        targets, logp, entropy, ids, top = (off if i == k else A for i in range(5))
        bad.append(lib.sl_token_logprobs_fwd(0, A, 104, 4, 100, targets, logp, A, entropy, 5, ids, top, None))
    for k in range(4):
        targets, g, gh, entropy = (off if i == k else A for i in range(4))
        bad.append(lib.sl_token_logprobs_bwd(0, A, 104, 4, 100, targets, A, g, gh, entropy, A, 104, None))
    assert bad == [B.SL_ERR_ALIGNMENT] * len(bad)


def test_scales_and_caps_that_32_bits_do_not_hold_are_refused(lib):
    """softcap log2(e) or scale / softcap as infinity, zero or a number without all its bits: NaN or 0 for any score. No
    workspace: a call that passes its checks ends there."""
    n = lib.sl_attention_plan_bytes(2, 300)

    def both(scale, cap):
        return (lib.sl_attention_masked_fwd(A, 256, A, 128, A, 128, 2, 300, 4, 2, 64, scale, cap, None, A, n, A, 256, A, None,
                                            None),
                lib.sl_attention_masked_bwd(A, 256, A, 128, A, 128, A, 256, A, 2, 300, 4, 2, 64, scale, cap, None, A, n, A, 256,
                                            A, 128, A, 128, None, None))

    for scale, cap in ((0.0, 3e38), (3e38, 0.0), (0.0, 1e38), (1.0, 1e-39), (1e38, 1e-3), (1e-40, 0.0)):
        assert both(scale, cap) == (B.SL_ERR_SHAPE,) * 2, (scale, cap)
    for scale, cap in ((0.0, 0.0), (0.0, 1e6), (1.0, 1e37), (1e-30, 0.0), (0.0, 1e-30)):
        assert both(scale, cap) == (B.SL_ERR_WORKSPACE,) * 2, (scale, cap)


def test_workspace_of_another_device_is_refused(monkeypatch):
    """Tensors of the current device 0 (stand-ins on the host) and a workspace of device 1, whose memory the kernels of
    device 0 may not reach."""

    class OnDevice0(torch.Tensor):
        def get_device(self):
            return 0

    here = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt).as_subclass(OnDevice0)
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    monkeypatch.setattr(B, "_raw_stream", lambda device: 0)
    ws = object.__new__(B.Workspace)
    ws.index, ws.device, ws.c = 1, "cuda:1", B.SlWorkspaceC(None, 0, 0)
    ws.ref = ctypes.byref(ws.c)
    x, lse, plan = here(4, 64), here(2, 4, dt=torch.float32), here(1 << 16, dt=torch.uint8)
    for call in (lambda: B.sl_attention_masked_fwd(ws, x, x, x, 1, 2, 2, 32, plan, x, lse),
                 lambda: B.sl_attention_masked_bwd(ws, x, x, x, x, x, lse, 1, 2, 2, 32, plan, x, x, x),
                 lambda: B.sl_qk_norm_rope_bwd(ws, x, x, x, x, None, None, 32, x, x, here(32), here(32),
                                               dgq=here(32, dt=torch.float32))):
        with pytest.raises(B.SparseLoRAError) as e:
            call()
        assert e.value.code == B.SL_ERR_INVALID_ARG
