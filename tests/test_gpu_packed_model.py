"""The packed-batch operators one behind the other, as a user runs them: a stack of decoder layers whose q and k are
normalised per head and rotated, attention over packed documents with capped and biased scores, and the loss,
log probabilities and alternatives at the head. Against the fp64 oracle of the same stack, whose attention is replaced
by a double-precision form with these options (its gradient by automatic differentiation), at the tolerance of the
stack without them (the options add two roundings to bf16 per layer, of q and of k, where it has dozens)."""
import math

import numpy as np
import pytest
import torch

import oracle
import oracle.sparselora_oracle as oracle_module
from contextual_sparsity_lora_b200 import binding as B
from contextual_sparsity_lora_b200.model import SparseLoRAModel
from contextual_sparsity_lora_b200.packing import AttentionPlan, packed_rows
from gpu_helpers import BF16_TOL, rel_fro
from test_gpu_model import build

pytestmark = pytest.mark.gpu
DEV = "cuda"


def attention64(lo, hi, pos, freq, style, gains, eps, cap, slopes):
    """(attention, attention_bwd) with the oracle's signatures."""
    lo, hi, pos = (torch.as_tensor(t).cpu().long() for t in (lo, hi, pos))

    def turn(x, hd, gain):
        x = x.view(x.shape[0], -1, hd)
        if gain is not None:
            x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * gain.double().cpu()
        if freq is None:
            return x
        t = pos.double()[:, None, None] * freq.double().cpu()
        rot = 2 * freq.numel()
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if style == B.SL_ROPE_PAIRS else (x[..., : rot // 2], x[..., rot // 2: rot])
        ya, yb = a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin()
        y = torch.stack((ya, yb), -1).flatten(-2) if style == B.SL_ROPE_PAIRS else torch.cat((ya, yb), -1)
        return torch.cat((y, x[..., rot:]), -1)

    def fwd(Q, K, V, n_seq, hq, hkv, hd):
        leaves = [torch.tensor(oracle.f64(t), requires_grad=True) for t in (Q, K, V)]
        gq, gk = gains if gains is not None else (None, None)
        q, k, v = turn(leaves[0], hd, gq), turn(leaves[1], hd, gk), leaves[2].view(-1, hkv, hd)
        S = q.shape[0] // n_seq
        q, k, v = (t.view(n_seq, S, -1, hd).transpose(1, 2) for t in (q, k, v))
        k, v = (t.repeat_interleave(hq // hkv, 1) for t in (k, v))
        t = q @ k.transpose(2, 3) / math.sqrt(hd)
        if cap:
            t = cap * torch.tanh(t / cap)
        at = torch.arange(S)
        if slopes is not None:
            t = t - slopes.double().cpu().view(1, hq, 1, 1) * (at[:, None] - at[None, :]).abs()
        see = (at >= lo.view(n_seq, 1, S, 1)) & (at < hi.view(n_seq, 1, S, 1))
        P = torch.where(see, torch.softmax(t.masked_fill(~see, -1e300), -1), 0.0)
        O = (P @ v).transpose(1, 2).reshape(n_seq * S, -1)
        return O.detach().numpy(), (O, leaves)

    def bwd(dO, Q, K, V, P, n_seq, hq, hkv, hd):
        O, leaves = P
        return tuple(g.numpy() for g in torch.autograd.grad(O, leaves, torch.tensor(oracle.f64(dO))))

    return fwd, bwd


def options(S, n_seq, hd, hq, style, norm, seed):
    g = torch.Generator().manual_seed(seed)
    lens = [[S - 21, 12], [9, S - 9]][:n_seq]  # documents; the first sequence ends in padding of 9 tokens
    lo, hi, pos = packed_rows(lens, S, [[5, 0], [0, 11]][:n_seq])
    freq = torch.tensor([1000.0 ** (-4 * i / hd) for i in range(hd // 4)])
    gains = tuple((1 + 0.2 * torch.randn(hd, generator=g)).to(torch.bfloat16) for _ in range(2)) if norm else None
    return lo, hi, pos, freq, gains, 3.0, torch.tensor([0.05 * (h + 1) for h in range(hq)])


@pytest.mark.parametrize("style,norm", [(B.SL_ROPE_HALVES, True), (B.SL_ROPE_PAIRS, False)])
def test_packed_step_matches_oracle(monkeypatch, style, norm):
    p = build([(1.0, 1.0), (0.5, 0.5)], seed=81)
    hq, hkv, hd = p["heads"]
    n_seq, T = p["n_seq"], len(p["perm"])
    S = T // n_seq
    lo, hi, pos, freq, gains, cap, slopes = options(S, n_seq, hd, hq, style, norm, 4)
    plan = AttentionPlan(n_seq, S)
    plan.set(lo.to(DEV), hi.to(DEV))
    model = SparseLoRAModel(p["frozen"], p["loras"], p["gammas"], [(1.0, 1.0), (0.5, 0.5)], p["perm"], p["C"], n_seq,
                            p["heads"], 8, 2.0, DEV, rope=(pos, freq, style), qk_norms=[gains, gains] if norm else None,
                            plan=plan, softcap=cap, slopes=slopes, loss="kernels")
    pt = torch.from_numpy(p["perm"])
    ids_cf, targets = p["ids"][pt].to(torch.int32).to(DEV), p["targets"].to(DEV)
    loss = float(model.forward_backward(ids_cf, targets))
    layers = []
    for i, lay in enumerate(model.layers):
        at, ff = lay.attn, lay.ffn
        full = {"q": at.Dq, "k": at.Dkv, "v": at.Dkv, "o": at.Dq}
        sig = {"q": at.sig_q, "k": at.sig_k, "v": at.sig_v, "o": at.sig_o}
        idx = {n: np.arange(full[n]) if at.dense else
               sig[n].cpu().numpy()[: at.ch[n].n_keep].astype(np.int64) for n in "qkvo"}
        idx["ffn"] = np.arange(ff.F) if ff.dense else ff.sigma.cpu().numpy()[: ff.n_keep].astype(np.int64)
        layers.append(dict(w={n: v.W for n, v in p["frozen"].items() if n not in ("embed", "lm_head", "gamma_f")},
                           lora=p["loras"][i], gammas=p["gammas"][i], idx=idx))
        assert lay.read_device_flag() == 0
    fwd, bwd = attention64(lo, hi, pos, freq, style, gains, 1e-5, cap, slopes)
    monkeypatch.setattr(oracle_module, "attention", fwd)
    monkeypatch.setattr(oracle_module, "attention_bwd", bwd)
    want, grads = oracle_module.model_step(p["ids"].numpy(), p["targets"].numpy(), p["ctx"], n_seq, p["frozen"]["embed"],
                                           p["frozen"]["lm_head"], p["frozen"]["gamma_f"], layers, 1e-5, 2.0, p["heads"])
    assert abs(loss - want) <= 2e-2 * abs(want)
    for i, lay in enumerate(model.layers):
        at, ff = lay.attn, lay.ffn
        for n in "qkvo":
            assert rel_fro(at.dA[n], grads[i]["dA_" + n]) < BF16_TOL, (i, n)
            assert rel_fro(at.dB[n], grads[i]["dB_" + n]) < BF16_TOL, (i, n)
        for n, a, b in (("gate", ff.dA_g, ff.dB_g), ("up", ff.dA_u, ff.dB_u), ("down", ff.dA_d, ff.dB_d)):
            assert rel_fro(a, grads[i]["dA_" + n]) < BF16_TOL, (i, n)
            assert rel_fro(b, grads[i]["dB_" + n]) < BF16_TOL, (i, n)


def test_loss_kernels_and_library_and_score():
    """The same stack without the options: the loss and the gradients of both heads, rows without a target, score()."""
    keep = [(0.5, 0.5)]
    p = build(keep, seed=82)
    lib = p["model"]
    ker = SparseLoRAModel(p["frozen"], p["loras"], p["gammas"], keep, p["perm"], p["C"], p["n_seq"], p["heads"], 8, 2.0,
                          DEV, loss="kernels")
    pt = torch.from_numpy(p["perm"])
    ids, targets = p["ids"][pt].to(torch.int32).to(DEV), p["targets"].to(DEV)
    a, b = float(lib.forward_backward(ids, targets)), float(ker.forward_backward(ids, targets))
    assert abs(a - b) <= 1e-5 * abs(a)  # the same bf16 logits, both sums in 32 bits
    # the logits' gradients differ by a rounding to bf16 at most (2^-8), so what follows by the order of that
    for n in "qkvo":
        assert rel_fro(ker.layers[0].attn.dA[n], lib.layers[0].attn.dA[n]) < 2.0 ** -7
    logp, ent, ids_top, top = ker.score(ids, targets, 3)
    assert abs(float(logp.mean()) + b) <= 1e-5 * abs(b)
    logits = ker._logits(ker._forward(ids)).double()
    logs = torch.log_softmax(logits, 1)
    assert torch.equal(ids_top.long(), torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :3])
    assert (top - logs.gather(1, ids_top.long())).abs().max() < 1e-5
    assert (ent + (logs * logs.exp()).sum(1)).abs().max() < 1e-4
    some = targets.clone()
    some[::3] = -1
    c = float(ker.forward_backward(ids, some))
    assert abs(c + float(logp[some >= 0].mean())) <= 1e-5 * abs(c)
    with pytest.raises(ValueError):
        SparseLoRAModel(p["frozen"], p["loras"], p["gammas"], keep, p["perm"], p["C"], p["n_seq"], p["heads"], 8, 2.0,
                        DEV, loss="other")


def test_default_layer_is_what_it_was():
    """Without the options the layer runs the attention core as before: two models, one built with explicit defaults."""
    keep = [(0.5, 0.5)]
    p = build(keep, seed=83)
    other = SparseLoRAModel(p["frozen"], p["loras"], p["gammas"], keep, p["perm"], p["C"], p["n_seq"], p["heads"], 8, 2.0,
                            DEV, rope=None, qk_norms=None, plan=None, softcap=0.0, slopes=None, loss="library")
    pt = torch.from_numpy(p["perm"])
    ids, targets = p["ids"][pt].to(torch.int32).to(DEV), p["targets"].to(DEV)
    a, b = p["model"].forward_backward(ids, targets), other.forward_backward(ids, targets)
    assert torch.equal(a, b) and other.layers[0].plan is None and other.layers[0].q_at is other.layers[0].q_nat


def test_options_that_do_not_fit_are_refused():
    keep = [(0.5, 0.5)]
    p = build(keep, seed=84)
    S = p["model"].layers[0].S
    for kw in (dict(softcap=-1.0), dict(softcap=math.nan), dict(plan=AttentionPlan(p["n_seq"], S + 1)),
               dict(plan=AttentionPlan(p["n_seq"] + 1, S))):
        with pytest.raises(ValueError):
            SparseLoRAModel(p["frozen"], p["loras"], p["gammas"], keep, p["perm"], p["C"], p["n_seq"], p["heads"], 8, 2.0,
                            DEV, **kw)


def test_rows_and_positions_change_from_batch_to_batch():
    """Two packed batches through one model, positions and rows as packed_rows gives them (on the CPU): the second gives
    what a model built for it gives; and back."""
    keep = [(1.0, 1.0), (0.5, 0.5)]
    p = build(keep, seed=85)
    hq, hkv, hd = p["heads"]
    n_seq, S = p["n_seq"], len(p["perm"]) // p["n_seq"]
    freq = torch.tensor([1000.0 ** (-4 * i / hd) for i in range(hd // 4)])
    batches = [packed_rows([[S - 21, 12], [9, S - 9]], S, [[5, 0], [0, 11]]), packed_rows([[7, 20, S - 27], [S]], S)]

    def model(batch):
        plan = AttentionPlan(n_seq, S)
        plan.set(batch[0].to(DEV), batch[1].to(DEV))
        return SparseLoRAModel(p["frozen"], p["loras"], p["gammas"], keep, p["perm"], p["C"], n_seq, p["heads"], 8, 2.0,
                               DEV, rope=(batch[2], freq, B.SL_ROPE_PAIRS), plan=plan, loss="kernels")

    pt = torch.from_numpy(p["perm"])
    ids, targets = p["ids"][pt].to(torch.int32).to(DEV), p["targets"].to(DEV)

    def step(m):
        loss = m.forward_backward(ids, targets).clone()
        return [loss, *(lay.attn.dA[n].clone() for lay in m.layers for n in "qkvo")]

    one = model(batches[0])
    assert one.layers[0].positions is one.layers[1].positions
    first, second = step(one), step(model(batches[1]))
    assert not torch.equal(first[0], second[0])
    one.set_rows(*batches[1])
    assert all(torch.equal(a, b) for a, b in zip(step(one), second))
    one.set_rows(*(t.to(DEV) for t in batches[0]))
    assert all(torch.equal(a, b) for a, b in zip(step(one), first))
    lo, hi, pos = batches[0]
    for args in ((lo, hi), (lo, hi, pos[1:]), (lo[1:], hi, pos), (lo, hi, pos.float())):
        with pytest.raises(ValueError):
            one.set_rows(*args)
    assert all(torch.equal(a, b) for a, b in zip(step(one), first))  # a refused call changes nothing
    with pytest.raises(ValueError):
        p["model"].set_rows(lo, hi)
    with pytest.raises(ValueError):
        p["model"].layers[0].set_positions(pos)


def test_score_options_without_a_plan_share_one():
    """softcap alone: the layers' causal plan is one, and set_rows changes it."""
    keep = [(0.5, 0.5), (0.5, 0.5)]
    p = build(keep, seed=86)
    m = SparseLoRAModel(p["frozen"], p["loras"], p["gammas"], keep, p["perm"], p["C"], p["n_seq"], p["heads"], 8, 2.0, DEV,
                        softcap=4.0)
    assert m.layers[0].plan is m.layers[1].plan is m.plan
    pt = torch.from_numpy(p["perm"])
    ids, targets = p["ids"][pt].to(torch.int32).to(DEV), p["targets"].to(DEV)
    causal = m.forward_backward(ids, targets).clone()
    S = m.layers[0].S
    lo, hi, _ = packed_rows([[S - 20, 20]] * p["n_seq"], S)
    m.set_rows(lo, hi)
    assert not torch.equal(m.forward_backward(ids, targets), causal)
    m.set_rows(None, None)
    assert torch.equal(m.forward_backward(ids, targets), causal)


def test_default_layer_runs_the_causal_core_and_the_library_loss():
    """Without the options, against what does not go through them: attention from the layer's own q, k and v by the causal
    core's entry points, forward and backward, bit for bit; the loss from the logits in 64 bits."""
    keep = [(0.5, 0.5)]
    p = build(keep, seed=87)
    m = p["model"]
    lay = m.layers[0]
    pt = torch.from_numpy(p["perm"])
    ids, targets = p["ids"][pt].to(torch.int32).to(DEV), p["targets"].to(DEV)
    loss = m.forward_backward(ids, targets).clone()
    at, ws = lay.attn, B.Workspace()
    a, lse = torch.empty_like(lay.a_nat), torch.empty_like(lay.lse)
    B.sl_attention_fwd(ws, lay.q_nat, lay.k_nat, lay.v_nat, lay.n_seq, at.hq, at.hkv, at.hd, a, lse)
    assert torch.equal(a, lay.a_nat) and torch.equal(lse, lay.lse)
    dk, dv = torch.empty_like(lay.dk_nat), torch.empty_like(lay.dv_nat)
    B.sl_attention_bwd(ws, lay.q_nat, lay.k_nat, lay.v_nat, a, lay.da_nat, lse, lay.n_seq, at.hq, at.hkv, at.hd,
                       torch.empty_like(lay.dq_nat), dk, dv)  # dq: sums of the causal core in no set order
    assert torch.equal(dk, lay.dk_nat) and torch.equal(dv, lay.dv_nat)
    logits = torch.matmul(m.hf[m.C:], m.lm_head.t()).double()
    want = -torch.log_softmax(logits, 1).gather(1, targets.long()[:, None]).mean()
    assert abs(float(loss) - float(want)) <= 1e-5 * abs(float(want))
