"""A whole fine-tuning step of a LLaMA-style model with SparseLoRA ([WT] "Putting It All
Together"; "Layer Sensitivity Analysis" for the per-layer ratios; "Step Sensitivity and
Progressive Sparse Fine-Tuning" for the dense first steps):

    x = embedding[ids]; for each layer: x = DecoderLayer(x) with the layer's keep ratios;
    logits = RMSNorm(x) W_lm^T on the output rows; loss = cross-entropy(logits, targets);
    backward through every layer; AdamW on every LoRA matrix.

Per-layer keep ratios (attention q/k/v/o, FFN) come from a table; the first steps of a run are
dense (progressive schedule). Every projection, RMSNorm, residual, the embedding gather and
AdamW run in libsparselora's kernels; the frozen LM head's product and, by default, its
cross-entropy are torch library calls (like cuBLAS), outside the method's steps. With
loss="kernels" the cross-entropy and its gradient run in sl_token_logprobs_fwd / _bwd on the
product's bf16 logits; score() gives log probabilities, entropies and top alternatives.
Packed batches, rotation, q/k norms and capped or biased scores: see DecoderLayer's options."""
from __future__ import annotations

import math

import torch

from . import binding as B
from .blocks import AttnProjBlock, FFNBlock
from .layer import DecoderLayer
from .packing import AttentionPlan


def llama3_8b_math10k_keep(n_layers: int = 32):
    """Keep ratios per layer (attention, FFN) from the walkthrough's reading of the LLaMA3-8B /
    Math10K configuration ([WT] "Converting sensitivity curves to sparsity configurations"): FFN
    sparsity 99% on layers L3-L30, QKVO sparsity 75% on L14-L19, L21-L23, L25-L29, the other
    layers dense (layers numbered from 1)."""
    out = []
    for i in range(1, n_layers + 1):
        ffn = 0.01 if 3 <= i <= 30 else 1.0
        attn = 0.25 if (14 <= i <= 19 or 21 <= i <= 23 or 25 <= i <= 29) else 1.0
        out.append((attn, ffn))
    return out


def layerwise_keep(n_layers: int = 32, dense_layers: int = 8, mid_end: int = 20, mid_keep: float = 0.6,
                   deep_keep: float = 0.35):
    """A non-uniform keep table over a 32-layer LLaMA3-8B (layers numbered from 0): layers
    0-7 dense, 8-19 at keep 0.6, 20-31 at keep 0.35, the same ratio on the attention
    projections and the FFN ([WT] "Layer Sensitivity Analysis and Non-Uniform Sparsity":
    deeper layers tolerate more sparsity, so shallow layers stay dense)."""
    out = []
    for i in range(n_layers):
        k = 1.0 if i < dense_layers else (mid_keep if i < mid_end else deep_keep)
        out.append((k, k))
    return out


def cosine_lr(step: int, n_steps: int, peak: float, warmup_frac: float = 0.04) -> float:
    """Learning rate of 1-based `step` of `n_steps` ([WT] "Step Sensitivity and Progressive
    Sparse Fine-Tuning", the schedule of Table 11): linear warm-up to `peak` over the first
    ceil(warmup_frac * n_steps) steps, then cosine decay to 0 at the last step."""
    n_warm = math.ceil(warmup_frac * n_steps)
    if step <= n_warm:
        return peak * step / n_warm
    if n_steps == n_warm:
        return peak
    t = (step - n_warm) / (n_steps - n_warm)
    return 0.5 * peak * (1.0 + math.cos(math.pi * t))


class SparseLoRAModel:
    def __init__(self, frozen, loras, gammas, keep, perm, n_ctx, n_seq, heads, est_k, lora_scale, device="cuda",
                 eps=1e-5, rope=None, qk_norms=None, plan: AttentionPlan | None = None, softcap: float = 0.0,
                 slopes=None, loss: str = "library"):
        """frozen: dict with "embed" [V, D], "lm_head" [V, D], "gamma_f" [D] and the projection
        weights "q","k","v","o","gate","up","down" (SpectralWeight-like: .W, .W_A, .W_B), shared by
        every layer or a list of such dicts (one per layer); loras: per layer a dict of (A, B);
        gammas: per layer (g1, g2); keep: per layer (attn_keep, ffn_keep); perm: context-first
        row order of the batch (n_seq sequences); heads: (n_q_heads, n_kv_heads, head_dim).
        rope, plan, softcap, slopes: DecoderLayer's options, the same for every layer (one copy of the
        positions and one plan for all; set_rows changes both from batch to batch); qk_norms: per
        layer (gq, gk); loss: "library" or "kernels" (see above)."""
        if loss not in ("library", "kernels"):
            raise ValueError('loss is "library" or "kernels"')
        bf = torch.bfloat16
        self.device = device
        self.eps = eps
        self.n_layers = len(keep)
        self.keep = list(keep)
        hq, hkv, hd = heads
        T = len(perm)
        self.T, self.C = T, n_ctx
        self.embed = frozen["embed"].to(device=device, dtype=bf).contiguous()
        self.lm_head = frozen["lm_head"].to(device=device, dtype=bf).contiguous()
        self.gamma_f = frozen["gamma_f"].to(device=device, dtype=bf).contiguous()
        self.D = self.embed.shape[1]
        if rope is not None:
            rope = (torch.as_tensor(rope[0]).to(device=device, dtype=torch.int32).contiguous(), *rope[1:])
        if plan is None and (softcap > 0 or slopes is not None):
            plan = AttentionPlan(n_seq, T // n_seq, device)
        self.plan = plan
        self.layers = []
        for i in range(self.n_layers):
            w = frozen["layers"][i] if "layers" in frozen else frozen
            lo = loras[i]
            attn = AttnProjBlock(w["q"], w["k"], w["v"], w["o"], lo["q"], lo["k"], lo["v"], lo["o"], lora_scale, est_k,
                                 hq, hkv, hd, T, n_ctx, keep[i][0], device, io_layout="sigma")
            ffn = FFNBlock(w["gate"], w["up"], w["down"], lo["gate"], lo["up"], lo["down"], lora_scale, est_k, T, n_ctx,
                           keep[i][1], device)
            self.layers.append(DecoderLayer(attn, ffn, gammas[i][0], gammas[i][1], perm, n_seq, eps, rope,
                                            None if qk_norms is None else qk_norms[i], plan, softcap, slopes))
        # fp32 master copies of every LoRA matrix and their AdamW moments, in the blocks' flat layout
        self.opt = []
        for lay in self.layers:
            for blk in (lay.attn, lay.ffn):
                master = blk.params.flat.float()
                self.opt.append((blk, master, torch.zeros_like(master), torch.zeros_like(master)))
        e = lambda *sh, dt=bf: torch.empty(*sh, dtype=dt, device=device)
        self.x0 = e(T, self.D)
        self.hf, self.dhf, self.dx_top = e(T, self.D), e(T, self.D), e(T, self.D)
        self.rstd_f = e(T, dt=torch.float32)
        self.loss = torch.zeros((), dtype=torch.float32, device=device)
        self.loss_kernels = loss == "kernels"

    def set_rows(self, row_lo, row_hi, positions=None):
        """What the tokens of the next batches see and where they stand, as packed_rows gives it (whole numbers [T] in
        sequence order, on any device; row_lo or row_hi None: see AttentionPlan.set). A model that rotates needs the
        positions with them. Captured steps follow both."""
        lay = self.layers[0]
        if self.plan is None or (positions is None) != (lay.positions is None):
            raise ValueError("set_rows needs a model with a plan, and positions exactly when it rotates")
        rows = [None if r is None else torch.as_tensor(r).to(device=self.device, dtype=torch.int32).contiguous()
                for r in (row_lo, row_hi)]
        if any(r is not None and r.shape != (self.T,) for r in rows):
            raise ValueError("row_lo and row_hi are one number per token")
        if positions is not None:
            lay.set_positions(positions)
        self.plan.set(*rows)

    def set_dense(self, on: bool):
        for lay in self.layers:
            lay.attn.set_dense(on)
            lay.ffn.set_dense(on)

    def _forward(self, ids_cf):
        """The normalised output rows (rows C..T-1 of the context-first order) under the LM head."""
        B.sl_permute_rows(self.embed, ids_cf, self.x0)
        x = self.x0
        for lay in self.layers:
            x = lay.forward(x)
        self.x_top = x
        B.sl_rmsnorm_fwd(x, self.gamma_f, self.eps, self.hf, self.rstd_f)
        return self.hf[self.C:]

    def _logits(self, h_out):
        """bf16 [n_out, V] logits whose rows start on 16 bytes, as the token kernels want them."""
        V = self.lm_head.shape[0]
        logits = torch.empty(h_out.shape[0], -(-V // 8) * 8, dtype=torch.bfloat16, device=h_out.device)[:, :V]
        return torch.matmul(h_out, self.lm_head.t(), out=logits) if logits.is_contiguous() else logits.copy_(
            torch.matmul(h_out, self.lm_head.t()))

    def score(self, ids_cf, targets_out, top_k: int = 0):
        """(logp, entropy, top_ids, top_logp) of the output rows: log probabilities of targets_out (int [T - C];
        negative: none, 0), entropies, and the top_k most likely tokens (None for top_k = 0). Forward only."""
        logits = self._logits(self._forward(ids_cf))
        n, dev = logits.shape[0], logits.device
        logp, entropy = (torch.empty(n, device=dev) for _ in range(2))
        ids = torch.empty(n, top_k, dtype=torch.int32, device=dev) if top_k else None
        top = torch.empty(n, top_k, device=dev) if top_k else None
        B.sl_token_logprobs_fwd(logits, targets_out.to(torch.int32), logp, torch.empty(n, 2, device=dev), entropy, ids, top)
        return logp, entropy, ids, top

    def _head_kernels(self, h_out, targets_out):
        """Mean cross-entropy of the rows that have a target, and its gradient at the logits (in their place)."""
        logits = self._logits(h_out)
        n, dev = logits.shape[0], logits.device
        targets = targets_out.to(torch.int32)
        logp, stats = torch.empty(n, device=dev), torch.empty(n, 2, device=dev)
        B.sl_token_logprobs_fwd(logits, targets, logp, stats)
        has = ((targets >= 0) & (targets < logits.shape[1])).float()
        g = has / -has.sum().clamp(min=1.0)
        self.loss.copy_((logp * g).sum())
        B.sl_token_logprobs_bwd(logits, targets, stats, g, logits)
        return logits

    def forward_backward(self, ids_cf, targets_out):
        """ids_cf: int32 [T] token ids in context-first order; targets_out: int64 [T - C], the
        next-token targets of the output rows (rows C..T-1 of the context-first order; with
        loss="kernels" a negative one leaves its row out)."""
        h_out = self._forward(ids_cf)
        x = self.x_top
        if self.loss_kernels:
            dlogits = self._head_kernels(h_out, targets_out)
        else:
            dlogits = self._head_library(h_out, targets_out)
        self.dhf.zero_()
        self.dhf[self.C:] = torch.matmul(dlogits, self.lm_head)
        B.sl_rmsnorm_bwd(self.dhf, x, self.gamma_f, self.rstd_f, self.dx_top)
        dx = self.dx_top
        for lay in reversed(self.layers):
            dx = lay.backward(dx)
        return self.loss

    def _head_library(self, h_out, targets_out):
        logits = torch.matmul(h_out, self.lm_head.t()).float()
        n_out = logits.shape[0]
        lse = torch.logsumexp(logits, dim=1)
        self.loss.copy_((lse - logits.gather(1, targets_out[:, None])[:, 0]).mean())
        dlogits = torch.softmax(logits, dim=1)
        dlogits[torch.arange(n_out, device=logits.device), targets_out] -= 1.0
        dlogits /= n_out
        return dlogits.to(torch.bfloat16)

    def optimizer_step(self, step: int, lr: float, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0):
        for blk, master, m, v in self.opt:
            B.sl_adamw_step(master, blk.grads.flat, m, v, step, lr, betas[0], betas[1], eps, weight_decay,
                            params_bf16=blk.params.flat)

    def step(self, ids_cf, targets_out, step: int, n_steps: int, lr: float, dense_frac: float = 0.1,
             warmup_frac: float = 0.04):
        """One fine-tuning step (1-based `step` of `n_steps`): dense while step <= ceil(dense_frac *
        n_steps), then with the per-layer keep ratios; AdamW at the cosine schedule's rate for
        this step, peak `lr`."""
        self.set_dense(step <= math.ceil(dense_frac * n_steps))
        loss = self.forward_backward(ids_cf, targets_out)
        self.optimizer_step(step, cosine_lr(step, n_steps, lr, warmup_frac))
        return loss
