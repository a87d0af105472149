"""Measured cases of the packed-batch operators of a fine-tuning step, with their plain forms.

Three operators, each forward and backward, in the order in which a decoder layer and the head use them:

  rotate    per-head RMSNorm of q and k with gains, and the position rotation, in one pass
            (sl_qk_norm_rope_fwd, sl_qk_norm_rope_bwd);
  attend    grouped-query attention whose queries each see an interval of keys (packed documents, prefixes,
            windows, padding), with capped scores and a bias that falls with the distance
            (sl_attention_plan, sl_attention_masked_fwd, sl_attention_masked_bwd);
  score     log probabilities of given tokens, entropy and top alternatives from logits
            (sl_token_logprobs_fwd, sl_token_logprobs_bwd).

A case's "grad" says whether a pass is the forward alone (scoring) or forward and backward (a training step).
Where `own` is false, run() computes the formulas with elementary torch operations in 32 bits; where it is true it
calls the library as a user's program does.
"""
import math
import random

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one new token of each of four sequences, 32 / 8 heads of 128, far from the start: a call where latency counts
        dict(name="rotate 4 tokens", op="rotate", grad=False, n_tok=4, hq=32, hkv=8, hd=128, rot=128, norm=True,
             pairs=False, far=131000, base=500000.0),
        # q and k of one LLaMA3-8B layer, 8 x 512 tokens, a training step without the norm
        dict(name="rotate 4096 tokens train", op="rotate", grad=True, n_tok=4096, hq=32, hkv=8, hd=128, rot=128,
             norm=False, pairs=False, far=0, base=500000.0),
        # a long packed batch, norm with gains that train, a part of each head rotated, neighbouring pairs, odd length
        dict(name="rotate 20011 tokens train", op="rotate", grad=True, n_tok=20011, hq=24, hkv=6, hd=96, rot=48,
             norm=True, pairs=True, far=4096, base=10000.0),
        # the smallest layer of the tests: one short packed sequence, latency
        dict(name="attend 1x64 train", op="attend", grad=True, n_seq=1, seq=64, hq=4, hkv=2, hd=32, docs=3, prefix=0,
             window=0, pad=5, cap=0.0, bias=False),
        # LLaMA3-8B layer: 8 x 512 tokens packed from short documents, padded at the end
        dict(name="attend 8x512 train", op="attend", grad=True, n_seq=8, seq=512, hq=32, hkv=8, hd=128, docs=3,
             prefix=0, window=0, pad=19, cap=0.0, bias=False),
        # a long packed sequence with capped scores
        dict(name="attend 1x4096 cap train", op="attend", grad=True, n_seq=1, seq=4096, hq=32, hkv=8, hd=128, docs=2,
             prefix=0, window=0, pad=0, cap=50.0, bias=False),
        # scoring one long document: a prefix that sees itself whole, a bias by distance
        dict(name="attend 1x8192 prefix bias", op="attend", grad=False, n_seq=1, seq=8192, hq=32, hkv=8, hd=128,
             docs=1, prefix=1024, window=0, pad=0, cap=0.0, bias=True),
        # odd length, uneven head size and groups, prefixes in documents, a sliding window, all options at once
        dict(name="attend 3x333 all train", op="attend", grad=True, n_seq=3, seq=333, hq=6, hkv=3, hd=96, docs=2,
             prefix=33, window=200, pad=13, cap=30.0, bias=True),
        # the next token's alternatives for one sequence: latency over the whole vocabulary
        dict(name="score 1 row top20", op="score", grad=False, rows=1, vocab=128256, dtype="bf16", top=20, banned=0),
        # the loss of a training step: the output tokens of 8 sequences, 128 each
        dict(name="score 1024 rows train", op="score", grad=True, rows=1024, vocab=128256, dtype="bf16", top=0,
             banned=0),
        # scoring all tokens of a batch with their alternatives, some tokens banned
        dict(name="score 4096 rows top20", op="score", grad=False, rows=4096, vocab=128256, dtype="bf16", top=20,
             banned=256),
        # an odd vocabulary in 32 bits, entropy and its gradient too
        dict(name="score 301 rows fp32 train", op="score", grad=True, rows=301, vocab=32003, dtype="fp32", top=5,
             banned=3),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "attend", "attend", "score"])
    grad = rng.random() < 0.6
    if op == "rotate":
        hd = rng.choice([8, 32, 40, 64, 96, 128, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 3, 4, 5])
        tok = _spread(rng, 1, max(1, min(32768, 20011 * 30 * 96 // ((hq + hkv) * hd))))
        return dict(op=op, grad=grad, n_tok=tok, hq=hq, hkv=hkv, hd=hd, rot=rng.choice([hd, hd, hd // 16 * 8]),
                    norm=rng.random() < 0.6, pairs=rng.random() < 0.4, far=rng.choice([0, _spread(rng, 1, 1 << 20)]),
                    base=rng.choice([10000.0, 500000.0]))
    if op == "attend":
        hd = rng.choice([8, 32, 64, 96, 120, 128, 128])
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 4, 5])
        n_seq = rng.choice([1, 1, 2, 3, 8])
        most = math.sqrt((32 * 4096 ** 2 if grad else 32 * 8192 ** 2) / (hq * n_seq))
        seq = _spread(rng, 1, int(min(8192, most)))
        return dict(op=op, grad=grad, n_seq=n_seq, seq=seq, hq=hq, hkv=hkv, hd=hd,
                    docs=rng.choice([1, 1, 2, 5]), prefix=rng.choice([0, 0, seq // 7]),
                    window=rng.choice([0, 0, _spread(rng, 1, seq)]), pad=rng.choice([0, seq // 9]),
                    cap=rng.choice([0.0, 0.0, 20.0, 50.0]), bias=rng.random() < 0.4)
    vocab = _spread(rng, 40, 160000)
    rows = _spread(rng, 1, min(4096, max(1, (1024 if grad else 4096) * 128256 // vocab)))
    return dict(op=op, grad=grad, rows=rows, vocab=vocab, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                top=rng.choice([0, 1, 5, 20, 32]), banned=rng.choice([0, 0, vocab // 50]))


# ------------------------------------------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=F32)


def _rows(c):
    """For each token of a sequence, the first key that it sees and the key behind the last one. The lengths of the
    documents go by the case alone, so that its work does."""
    r, n_seq, seq = random.Random(7 * c["docs"] + c["seq"]), c["n_seq"], c["seq"]
    los, his = [], []
    for _ in range(n_seq):
        live = seq - min(c["pad"], seq - 1)
        cuts = sorted({0, live} | {r.randrange(1, live) for _ in range(c["docs"] - 1) if live > 1})
        lo, hi = [], []
        for a, e in zip(cuts, cuts[1:]):
            for t in range(a, e):
                lo.append(max(a, t + 1 - c["window"]) if c["window"] else a)
                hi.append(max(t + 1, min(e, a + c["prefix"])))
        los += lo + [0] * (seq - live)
        his += hi + [0] * (seq - live)
    return los, his


def _attend_pairs(c):
    lo, hi = _rows(c)
    return sum(h - l for l, h in zip(lo, hi))


def prepare(case, seed):
    c, g = case, _generator(seed)
    s = dict(c, seed=seed)
    if c["op"] == "rotate":
        T, nq, nk = c["n_tok"], c["hq"] * c["hd"], c["hkv"] * c["hd"]
        gain = _normal(g, 2, c["hd"])
        starts = torch.arange(T, device="cuda", dtype=torch.int32) % 1531  # documents one behind the other
        s.update(q=_normal(g, T, nq).to(BF16), k=(0.5 * _normal(g, T, nk)).to(BF16), positions=starts + c["far"],
                 inv_freq=torch.tensor([c["base"] ** (-2.0 * i / max(1, c["rot"])) for i in range(c["rot"] // 2)],
                                       device="cuda", dtype=F32),
                 gq=(1 + 0.1 * gain[0]).to(BF16), gk=(1 + 0.1 * gain[1]).to(BF16),
                 yq=torch.empty(T, nq, device="cuda", dtype=BF16), yk=torch.empty(T, nk, device="cuda", dtype=BF16))
        if c["grad"]:
            s.update(dyq=_normal(g, T, nq).to(BF16), dyk=_normal(g, T, nk).to(BF16), dq=torch.empty_like(s["yq"]),
                     dk=torch.empty_like(s["yk"]), dgq=torch.empty(c["hd"], device="cuda", dtype=F32),
                     dgk=torch.empty(c["hd"], device="cuda", dtype=F32))
        return s
    if c["op"] == "attend":
        T, nq, nk = c["n_seq"] * c["seq"], c["hq"] * c["hd"], c["hkv"] * c["hd"]
        lo, hi = _rows(c)
        s.update(q=(2 * _normal(g, T, nq)).to(BF16), k=_normal(g, T, nk).to(BF16), v=_normal(g, T, nk).to(BF16),
                 lo=torch.tensor(lo, device="cuda", dtype=torch.int32),
                 hi=torch.tensor(hi, device="cuda", dtype=torch.int32),
                 slopes=torch.tensor([2.0 ** (-8.0 * (h + 1) / c["hq"]) for h in range(c["hq"])], device="cuda",
                                     dtype=F32) if c["bias"] else None,
                 o=torch.empty(T, nq, device="cuda", dtype=BF16), lse=torch.empty(c["hq"], T, device="cuda", dtype=F32))
        if c["grad"]:
            s.update(d_o=_normal(g, T, nq).to(BF16), dq=torch.empty_like(s["q"]), dk=torch.empty_like(s["k"]),
                     dv=torch.empty_like(s["v"]))
        return s
    N, V, kind = c["rows"], c["vocab"], BF16 if c["dtype"] == "bf16" else F32
    ld = -(-V // 8) * 8  # rows start on 16 bytes
    z = 2.5 * _normal(g, N, ld)
    targets = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    rows = torch.arange(N, device="cuda")
    z[rows, targets.long()] += 6 * torch.rand(N, generator=g, device="cuda")  # a model that has learnt something
    if c["banned"]:
        z[:, torch.randint(0, V, (c["banned"],), generator=g, device="cuda")] = -math.inf
        targets[::5] = -1  # rows without a target
    s.update(logits=z.to(kind)[:, :V], targets=targets, logp=torch.empty(N, device="cuda"),
             stats=torch.empty(N, 2, device="cuda"), entropy=torch.empty(N, device="cuda"), top_ids=None, top_logp=None)
    if c["top"]:
        s.update(top_ids=torch.empty(N, c["top"], device="cuda", dtype=torch.int32),
                 top_logp=torch.empty(N, c["top"], device="cuda"))
    if c["grad"]:
        s.update(g_logp=-torch.rand(N, generator=g, device="cuda") / N, g_entropy=0.1 * _normal(g, N) / N,
                 dlogits=torch.zeros(N, ld, device="cuda", dtype=kind)[:, :V])
    return s


# ------------------------------------------------------------------------------------------------- plain forms

def _angles(s):
    a = s["positions"].double()[:, None] * s["inv_freq"].double()[None, :]
    return a.cos().to(F32)[:, None, :], a.sin().to(F32)[:, None, :]


def _halves(x, s):
    """The two members of each rotated pair, and what is not rotated."""
    rot = s["rot"]
    if s["pairs"]:
        return x[..., 0:rot:2], x[..., 1:rot:2], x[..., rot:]
    return x[..., : rot // 2], x[..., rot // 2: rot], x[..., rot:]


def _joined(a, b, rest, s):
    both = torch.stack((a, b), -1).flatten(-2) if s["pairs"] else torch.cat((a, b), -1)
    return torch.cat((both, rest), -1)


def _rotate_plain(x, gain, s, cos, sin):
    """(y, rstd, the normalised x) of x [T, heads * hd]."""
    x = x.float().view(x.shape[0], -1, s["hd"])
    rstd = None
    if s["norm"]:
        rstd = (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
        x = x * rstd
    a, b, rest = _halves(x * gain.float() if s["norm"] else x, s)
    y = _joined(a * cos - b * sin, b * cos + a * sin, rest, s)
    return y.flatten(1).to(BF16), rstd, x


def _rotate_plain_grad(dy, gain, s, cos, sin, rstd, x):
    dy = dy.float().view(dy.shape[0], -1, s["hd"])
    a, b, rest = _halves(dy, s)
    dn = _joined(a * cos + b * sin, b * cos - a * sin, rest, s)
    if not s["norm"]:
        return dn.flatten(1).to(BF16), None
    dgain = (dn * x).sum((0, 1))
    dn = dn * gain.float()
    dx = rstd * (dn - x * (dn * x).mean(-1, keepdim=True))
    return dx.flatten(1).to(BF16), dgain


def _rotate(s):
    cos, sin = _angles(s)
    yq, rq, xq = _rotate_plain(s["q"], s["gq"], s, cos, sin)
    yk, rk, xk = _rotate_plain(s["k"], s["gk"], s, cos, sin)
    if not s["grad"]:
        return [yq, yk]
    dq, dgq = _rotate_plain_grad(s["dyq"], s["gq"], s, cos, sin, rq, xq)
    dk, dgk = _rotate_plain_grad(s["dyk"], s["gk"], s, cos, sin, rk, xk)
    return [yq, yk, dq, dk] + ([dgq, dgk] if s["norm"] else [])


def _attend(s):
    n, S, hq, hkv, hd, cap = s["n_seq"], s["seq"], s["hq"], s["hkv"], s["hd"], s["cap"]
    wide = lambda x, h: x.float().view(n, S, hkv, h, hd).permute(0, 2, 3, 1, 4)  # [n, hkv, h, S, hd]
    flat = lambda x: x.permute(0, 3, 1, 2, 4).reshape(n * S, -1).to(BF16)
    q, k, v = wide(s["q"], hq // hkv), wide(s["k"], 1), wide(s["v"], 1)
    scale = 1 / math.sqrt(hd)
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(scale)
    tanh = None
    if cap:
        tanh = (p / cap).tanh_()
        p = tanh * cap
    at = torch.arange(S, device="cuda", dtype=torch.int32)
    if s["bias"]:
        p -= s["slopes"].view(hkv, -1, 1, 1) * (at[:, None] - at[None, :]).abs().float()
    lo, hi = s["lo"].view(n, 1, 1, S, 1), s["hi"].view(n, 1, 1, S, 1)
    p.masked_fill_((at < lo) | (at >= hi), -math.inf)
    top = p.amax(-1, keepdim=True)
    empty = top == -math.inf
    p = p.sub_(top.masked_fill(empty, 0)).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).masked_fill(empty, -math.inf)
    p /= total.masked_fill(empty, 1)
    o = torch.matmul(p, v)
    out = [flat(o), lse.permute(1, 2, 0, 3, 4).reshape(hq, n * S)]
    if not s["grad"]:
        return out
    do = wide(s["d_o"], hq // hkv)
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2, keepdim=True)
    ds = torch.matmul(do, v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    if cap:
        ds *= 1 - tanh * tanh
    dq = torch.matmul(ds, k) * scale
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2, keepdim=True) * scale
    return out + [flat(dq), flat(dk), flat(dv)]


def _score(s):
    z, t, V = s["logits"].float(), s["targets"].long(), s["vocab"]
    top = z.amax(1, keepdim=True)
    e = (z - top).exp()
    total = e.sum(1, keepdim=True)
    logs = (z - top) - total.log()
    p = e / total
    has = (t >= 0)[:, None]
    at = t.clamp(min=0)[:, None]
    logp = logs.gather(1, at).masked_fill(~has, 0)[:, 0]
    entropy = -torch.where(p > 0, p * logs, 0).sum(1)
    out = [logp, entropy]
    if s["top"]:  # larger first, of equal ones the lowest index: one whole number says both
        bits = (z + 0.0).view(torch.int32)
        bits = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long()
        ids = (bits << 32).add_(torch.arange(V - 1, -1, -1, device="cuda")).topk(s["top"], 1).indices
        out += [ids.to(torch.int32), logs.gather(1, ids)]
    if s["grad"]:
        d = -p * s["g_logp"].masked_fill(t < 0, 0)[:, None]
        d.scatter_add_(1, at, s["g_logp"].masked_fill(t < 0, 0)[:, None])
        d -= torch.where(p > 0, p * (logs + entropy[:, None]), 0) * s["g_entropy"][:, None]
        out.append(d.to(s["logits"].dtype))
    return out


# ------------------------------------------------------------------------------------------------- the library

def _kept(s, name, make):
    """What a program makes once and keeps next to its tensors."""
    if name not in s:
        s[name] = make()
    return s[name]


def _rotate_own(s):
    from contextual_sparsity_lora_b200 import binding as B

    kind = B.SL_ROPE_PAIRS if s["pairs"] else B.SL_ROPE_HALVES
    gq, gk = (s["gq"], s["gk"]) if s["norm"] else (None, None)
    freq = s["inv_freq"] if s["rot"] else None
    B.sl_qk_norm_rope_fwd(s["q"], s["k"], s["positions"], freq, s["hd"], s["yq"], s["yk"], gq, gk, 1e-6, kind)
    if not s["grad"]:
        return [s["yq"], s["yk"]]
    dgq, dgk = (s["dgq"], s["dgk"]) if s["norm"] else (None, None)
    B.sl_qk_norm_rope_bwd(_kept(s, "ws", B.Workspace), s["dyq"], s["dyk"], s["q"], s["k"], s["positions"], freq,
                          s["hd"], s["dq"], s["dk"], gq, gk, 1e-6, kind, dgq, dgk)
    return [s["yq"], s["yk"], s["dq"], s["dk"]] + ([dgq, dgk] if s["norm"] else [])


def _attend_own(s):
    from contextual_sparsity_lora_b200 import binding as B

    n, hq, hkv, hd = s["n_seq"], s["hq"], s["hkv"], s["hd"]
    ws = _kept(s, "ws", B.Workspace)
    plan = _kept(s, "plan", lambda: B.attention_plan_buffer(n, s["seq"]))
    B.sl_attention_plan(s["lo"], s["hi"], n, plan)
    B.sl_attention_masked_fwd(ws, s["q"], s["k"], s["v"], n, hq, hkv, hd, plan, s["o"], s["lse"], s["cap"], s["slopes"])
    if not s["grad"]:
        return [s["o"], s["lse"]]
    B.sl_attention_masked_bwd(ws, s["q"], s["k"], s["v"], s["o"], s["d_o"], s["lse"], n, hq, hkv, hd, plan, s["dq"],
                              s["dk"], s["dv"], s["cap"], s["slopes"])
    return [s["o"], s["lse"], s["dq"], s["dk"], s["dv"]]


def _score_own(s):
    from contextual_sparsity_lora_b200 import binding as B

    B.sl_token_logprobs_fwd(s["logits"], s["targets"], s["logp"], s["stats"], s["entropy"], s["top_ids"], s["top_logp"])
    out = [s["logp"], s["entropy"]] + ([s["top_ids"], s["top_logp"]] if s["top"] else [])
    if s["grad"]:
        B.sl_token_logprobs_bwd(s["logits"], s["targets"], s["stats"], s["g_logp"], s["dlogits"], s["g_entropy"],
                                s["entropy"])
        out.append(s["dlogits"])
    return out


def run(state):
    if own:
        return {"rotate": _rotate_own, "attend": _attend_own, "score": _score_own}[state["op"]](state)
    return {"rotate": _rotate, "attend": _attend, "score": _score}[state["op"]](state)


# ------------------------------------------------------------------------------------------------- floors

def work(case):
    c = case
    if c["op"] == "rotate":
        one = c["n_tok"] * (c["hq"] + c["hkv"]) * c["hd"]
        # forward: x in, y out; backward: dy (and x, which the norm's gradient needs) in, dx out
        return {"bytes": 4 * one + c["n_tok"] * 4 + c["grad"] * (4 + 2 * c["norm"]) * one,
                "flops": one * (3 + 4 * c["norm"]) * (1 + 2 * c["grad"])}
    if c["op"] == "attend":
        T, nq, nk = c["n_seq"] * c["seq"], c["hq"] * c["hd"], c["hkv"] * c["hd"]
        two = 2 * c["hq"] * c["hd"] * _attend_pairs(c)  # operations of one product over the seen pairs
        # two products forward; five backward (the scores again, dv, dp, dq, dk)
        return {"bytes": T * (4 * nq + 4 * nk + 8 + 4 * c["hq"]) + c["grad"] * T * (8 * nq + 8 * nk + 4 * c["hq"]),
                "flops": two * (7 if c["grad"] else 2)}
    one = c["rows"] * c["vocab"]
    size = 2 if c["dtype"] == "bf16" else 4
    return {"bytes": one * size * (3 if c["grad"] else 1) + c["rows"] * (24 + 8 * c["top"]),
            "flops": one * (9 if c["grad"] else 5)}


# ------------------------------------------------------------------------------------------------- in 64 bits

def _exact_rotate(s):
    T, hd, rot, half = s["n_tok"], s["hd"], s["rot"], s["rot"] // 2
    first = torch.arange(half, device="cuda") * (2 if s["pairs"] else 1)
    second = first + (1 if s["pairs"] else half)
    turn = torch.eye(hd, device="cuda", dtype=torch.float64).repeat(T, 1, 1)  # the rotation of a token as a matrix
    if rot:
        ang = torch.outer(s["positions"].double(), s["inv_freq"].double())
        turn[:, first, first] = ang.cos()
        turn[:, second, second] = ang.cos()
        turn[:, first, second] = -ang.sin()
        turn[:, second, first] = ang.sin()
    outs, grads, gains = [], [], []
    for x, gain, dy in ((s["q"], s["gq"], s.get("dyq")), (s["k"], s["gk"], s.get("dyk"))):
        x = x.double().view(T, -1, hd)
        w = gain.double() if s["norm"] else torch.ones(hd, device="cuda", dtype=torch.float64)
        r = torch.sqrt((x ** 2).sum(-1, keepdim=True) / hd + 1e-6) if s["norm"] else torch.ones_like(x[..., :1])
        outs.append(torch.bmm(x / r * w, turn.transpose(1, 2)).reshape(T, -1))
        if s["grad"]:
            back = torch.bmm(dy.double().view(T, -1, hd), turn)
            gains.append((back * x / r).sum((0, 1)))
            back = back * w
            dx = back / r - (x * (back * x).sum(-1, keepdim=True) / (hd * r ** 3) if s["norm"] else 0)
            grads.append(dx.reshape(T, -1))
    return outs + grads + (gains if s["norm"] and s["grad"] else [])


def _exact_attend(s):
    n, S, hq, hkv, hd = s["n_seq"], s["seq"], s["hq"], s["hkv"], s["hd"]
    T, per = n * S, hq // hkv
    f64 = dict(device="cuda", dtype=torch.float64)
    o, lse = torch.zeros(T, hq * hd, **f64), torch.zeros(hq, T, **f64)
    dq, dk, dv = torch.zeros(T, hq * hd, **f64), torch.zeros(T, hkv * hd, **f64), torch.zeros(T, hkv * hd, **f64)
    key = torch.arange(S, device="cuda")
    away = (key[:, None] - key[None, :]).abs().double()
    for b in range(n):
        rows = slice(b * S, (b + 1) * S)
        seen = (key[None, :] >= s["lo"][rows, None]) & (key[None, :] < s["hi"][rows, None])
        for h in range(hq):
            mine, kv = slice(h * hd, (h + 1) * hd), slice(h // per * hd, (h // per + 1) * hd)
            Q, K, V = s["q"][rows, mine].double(), s["k"][rows, kv].double(), s["v"][rows, kv].double()
            raw = Q @ K.T / hd ** 0.5
            x = s["cap"] * torch.tanh(raw / s["cap"]) if s["cap"] else raw
            slope = 1 - (x / s["cap"]) ** 2 if s["cap"] else None
            if s["bias"]:
                x = x - s["slopes"][h].double() * away
            x = torch.where(seen, x, -math.inf)
            norm = torch.logsumexp(x, 1)
            P = torch.where(seen, torch.exp(x - torch.where(norm == -math.inf, 0.0, norm)[:, None]), 0.0)
            o[rows, mine], lse[h, rows] = P @ V, norm
            if s["grad"]:
                G = s["d_o"][rows, mine].double()
                dv[rows, kv] += P.T @ G
                dP = G @ V.T
                dS = P * (dP - (P * dP).sum(1, keepdim=True))
                dS = dS * slope if s["cap"] else dS
                dq[rows, mine] = dS @ K / hd ** 0.5
                dk[rows, kv] += dS.T @ Q / hd ** 0.5
    return [o, lse] + ([dq, dk, dv] if s["grad"] else [])


def _exact_score(s):
    N, parts = s["rows"], []
    for r in range(0, N, 512):
        z, t = s["logits"][r:r + 512].double(), s["targets"][r:r + 512].long()
        logs = torch.log_softmax(z, 1)
        p = logs.exp()
        row = torch.arange(len(t), device="cuda")
        entropy = -torch.nan_to_num(p * logs, nan=0.0).sum(1)
        part = [torch.where(t >= 0, logs[row, t.clamp(min=0)], 0.0), entropy]
        if s["top"]:
            best = torch.sort(z, dim=1, descending=True, stable=True).values[:, : s["top"]]
            part.append(best - torch.logsumexp(z, 1, keepdim=True))
        if s["grad"]:
            one = torch.zeros_like(p)
            one[row[t >= 0], t[t >= 0]] = 1
            ga, gb = s["g_logp"][r:r + 512].double()[:, None], s["g_entropy"][r:r + 512].double()[:, None]
            d = torch.where((t >= 0)[:, None], one - p, 0.0) * ga
            part.append(d - gb * torch.nan_to_num(p * (logs + entropy[:, None]), nan=0.0))
        parts.append(part)
    out = [torch.cat(x) for x in zip(*parts)]
    return out[:2] + ([None] + out[2:] if s["top"] else out[2:])


def exact(case, seed):
    return {"rotate": _exact_rotate, "attend": _exact_attend, "score": _exact_score}[case["op"]](prepare(case, seed))
