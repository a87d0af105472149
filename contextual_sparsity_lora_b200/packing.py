"""Packed batches: several documents in one row of tokens, each seeing its own keys.

packed_rows gives each token's interval of visible keys and its position; AttentionPlan keeps the plan that
sl_attention_masked_fwd / sl_attention_masked_bwd read, shared by every layer of a model."""
from __future__ import annotations

import torch

from . import binding as B


def packed_rows(doc_lens, seq_len: int, prefix_lens=None, window: int = 0, device="cpu"):
    """(row_lo, row_hi, positions), int32 [n_seq * seq_len], of n_seq sequences of seq_len tokens whose documents
    have the lengths doc_lens[s] (a list per sequence; what is left of a sequence is padding, which sees nothing and
    which nobody sees). A token sees its document up to itself; with prefix_lens[s][d], the first tokens of a document
    see each other whole; with window > 0, only the last `window` tokens up to itself (a prefix's tokens still see the
    prefix ahead). Positions restart at 0 in every document."""
    lo, hi, pos = [], [], []
    for s, lens in enumerate(doc_lens):
        if any(n < 0 for n in lens) or sum(lens) > seq_len or window < 0:
            raise ValueError("document lengths are not negative and fit their sequence")
        at = 0
        for d, n in enumerate(lens):
            pre = 0 if prefix_lens is None else int(prefix_lens[s][d])
            t = torch.arange(at, at + n)
            lo.append(torch.clamp(t + 1 - window, min=at) if window else torch.full((n,), at))
            hi.append(torch.clamp(t + 1, min=at + min(pre, n)))
            pos.append(t - at)
            at += n
        for part in (lo, hi, pos):
            part.append(torch.zeros(seq_len - at, dtype=torch.int64))
    return tuple(torch.cat(part).to(device=device, dtype=torch.int32) for part in (lo, hi, pos))


class AttentionPlan:
    """The plan of a batch's intervals in a buffer of its own (causal until set() is called). A captured graph
    reads what the buffer holds when it is replayed: set() before the replay changes the rows it sees."""

    def __init__(self, n_seq: int, seq_len: int, device="cuda"):
        self.n_seq, self.seq_len = int(n_seq), int(seq_len)
        self.buf = B.attention_plan_buffer(self.n_seq, self.seq_len, device)
        self.set(None, None)

    def set(self, row_lo, row_hi):
        """Each token sees keys [row_lo, row_hi) of its sequence (int32 [n_seq * seq_len]; None: 0 / position + 1)."""
        B.sl_attention_plan(row_lo, row_hi, self.n_seq, self.buf, self.seq_len)
