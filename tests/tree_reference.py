"""The draft-tree and eviction operators from their definitions, in 64 bits on
the CPU (numpy), with the error bounds that their arithmetic allows, and the
seeded inputs of their tests.

Bounds, from unit roundoffs (half a step relative to the value: bf16 2^-8, fp32
2^-24; a tensor core may truncate where it adds, so fp32 sums count 2^-23 a
term):

  x_t      a sum of d = d_c + d_r products: |dx| <= d 2^-23 sum |q_i k_i| =: ex
  weights  e^{x - lse}: relative 2 ex + 2^-20 (both logits; the exponential's
           own error is a few 2^-23 and its argument's rounding 2^-24 |x|) =: ew
  out      sum p c: (ew + (n + 32) 2^-23 + up) sum p |c| + uo |out|, up = 2^-8 where
           the weights are rounded to bf16 for their product and uo the output's
           own rounding
  lse      ex + 2^-20 (|lse| + 1)
  mass     (ew + (rows + 32) 2^-23) mass + 2^-22 |decay prev| + 2^-23 |s|
"""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -23


def words_of(parents: np.ndarray) -> np.ndarray:
    """uint64 [B, T]: node i sees itself and its ancestors (parents[b, i] < i, -1: none)."""
    B, T = parents.shape
    w = np.zeros((B, T), dtype=np.uint64)
    for b in range(B):
        for i in range(T):
            j = i
            while j >= 0:
                w[b, i] |= np.uint64(1) << np.uint64(j)
                j = int(parents[b, j])
    return w


def chain_words(B: int, T: int) -> np.ndarray:
    return words_of(np.broadcast_to(np.arange(T) - 1, (B, T)))


class Tree:
    """One batch: float64 views of the values that the device holds."""

    def __init__(self, q_c, q_r, c, k, lens, drafts, words):
        # q_c [B,T,H,d_c]; c, k: per sequence [n + d, width]; words uint64 [B,T]
        self.q_c, self.q_r, self.c, self.k = q_c, q_r, c, k
        self.lens, self.drafts, self.words = list(lens), list(drafts), words
        self.B, self.T, self.H, self.d_c = q_c.shape
        self.d_r = q_r.shape[3]

    def seen(self, b, i):
        n, d = self.lens[b], self.drafts[b]
        return np.array([t < n or bool(int(self.words[b, i]) >> (t - n) & 1) for t in range(n + d)], dtype=bool)

    def logits(self, b, i):
        """x [H, seen], the indexes seen, and sum |q k| of each."""
        use = np.nonzero(self.seen(b, i))[0]
        c, k = self.c[b][use], self.k[b][use]
        x = self.q_c[b, i] @ c.T + self.q_r[b, i] @ k.T
        mag = np.abs(self.q_c[b, i]) @ np.abs(c).T + np.abs(self.q_r[b, i]) @ np.abs(k).T
        return x, use, mag

    def attend(self, up, uo):
        """out, lse and their bounds, NaN where a row is not written."""
        B, T, H = self.B, self.T, self.H
        out = np.full((B, T, H, self.d_c), np.nan)
        lse = np.full((B, T, H), np.nan)
        eo, el = np.zeros_like(out), np.zeros_like(lse)
        for b in range(B):
            for i in range(self.drafts[b]):
                x, use, mag = self.logits(b, i)
                if len(use) == 0:
                    out[b, i], lse[b, i] = 0.0, -np.inf
                    continue
                m = x.max(1, keepdims=True)
                e = np.exp(x - m)
                z = e.sum(1, keepdims=True)
                p = e / z
                c = self.c[b][use]
                out[b, i] = p @ c
                lse[b, i] = (m + np.log(z))[:, 0]
                ex = ((self.d_c + self.d_r) * U32 * mag).max(1)
                ew = 2 * ex + 2.0 ** -20 + 2 * U32 * np.abs(x).max(1)
                eo[b, i] = (ew + (len(use) + 32) * U32 + up)[:, None] * (p @ np.abs(c)) + uo * np.abs(out[b, i])
                el[b, i] = ex + 2.0 ** -20 * (np.abs(lse[b, i]) + 1)
        return out, lse, eo, el

    def mass(self, lse, prev, decay, skip=()):
        """Per sequence: the sums and their bounds ([n + d] each); lse as given to the call."""
        res = []
        for b in range(self.B):
            n, d = self.lens[b], self.drafts[b]
            s, e = np.zeros(n + d), np.zeros(n + d)
            for i in range(d):
                x, use, mag = self.logits(b, i)
                for h in range(self.H):
                    if np.isinf(lse[b, i, h]):
                        continue
                    w = np.exp(x[h] - lse[b, i, h])
                    ex = (self.d_c + self.d_r) * U32 * mag[h]
                    s[use] += w
                    e[use] += w * (ex + 2.0 ** -20 + 2 * U32 * (np.abs(x[h]) + abs(lse[b, i, h])))
            e += s * (d * self.H + 32) * U32
            if prev is not None:
                s[:n] += decay * prev[b, :n]
                e[:n] += 2 * U32 * np.abs(decay * prev[b, :n])
            res.append((s, e + U32 * np.abs(s)))
        return res


def select(scores, n, n_sink, n_recent, budget):
    """The rows that stay, rising."""
    if n <= budget:
        return np.arange(n)
    mid = np.arange(n_sink, n - n_recent)
    x = scores[mid].astype(np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    nan = np.isnan(scores[mid])
    order = np.lexsort((mid, nan, -x))          # larger first, numbers before NaN, lower row first
    top = mid[order[:budget - n_sink - n_recent]]
    return np.sort(np.concatenate([np.arange(n_sink), top, np.arange(n - n_recent, n)])).astype(np.int64)
