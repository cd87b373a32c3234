"""64-bit and whole-number restatements of the operators around the paged attention: rotary
positions, filling a paged cache, page management, and attention over packed sequences.

Test infrastructure only; shares no code with the library.
"""
from __future__ import annotations

import math

import numpy as np
import torch


def rope(x, positions, inv_freq, axes=None, interleaved=False, inverse=False):
    """x (T, H, d) -> float64, each pair turned by positions[axis] * inv_freq."""
    y = x.detach().cpu().double().clone()
    pos = positions.cpu().reshape(-1, positions.shape[-1])
    F = inv_freq.numel()
    for f in range(F):
        a = pos[int(axes[f]) if axes is not None else 0].double() * float(inv_freq[f])
        if inverse:
            a = -a
        i, j = (2 * f, 2 * f + 1) if interleaved else (f, f + F)
        u, w = y[..., i].clone(), y[..., j].clone()
        c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
        y[..., i], y[..., j] = u * c - w * s, u * s + w * c
    return y


def token_rows(block_table, cu, seqlens, page_size, T):
    """(page, row) of each packed token, or None for padding."""
    out = [None] * T
    for b in range(len(seqlens)):
        n = int(cu[b + 1]) - int(cu[b])
        for i in range(n):
            p = int(seqlens[b]) - n + i
            out[int(cu[b]) + i] = (int(block_table[b][p // page_size]), p % page_size)
    return out


def e4m3_bytes(x32):
    """float32 values -> E4M3 bytes, nearest even, saturated (the input is already scaled)."""
    return x32.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def gather(pool, block_table, b, n):
    """First n tokens of sequence b from a pool (pages, H, page_size, d) -> (n, H, d)."""
    ps = pool.shape[2]
    t = torch.arange(n)
    pg = torch.as_tensor(block_table[b], dtype=torch.long)[t // ps]
    return pool[pg, :, t % ps]


def attention(q, k, v, scale, causal, window=0):
    """One sequence in float64: q (n, Hq, d), k and v (m, Hkv, d) -> o (n, Hq, d), lse (Hq, n).
    Row i sees keys j <= i + m - n (causal), of those the last `window`; a row that sees none
    gives zeros and -inf."""
    q, k, v = (t.detach().cpu().double() for t in (q, k, v))
    n, Hq, d = q.shape
    m, Hkv = k.shape[:2]
    o = torch.zeros(n, Hq, d, dtype=torch.float64)
    lse = torch.full((Hq, n), -math.inf, dtype=torch.float64)
    if n == 0 or m == 0:
        return o, lse
    last = torch.arange(n)[:, None] + (m - n) if causal else torch.full((n, 1), m - 1)
    j = torch.arange(m)[None, :]
    see = (j <= last) & (j > last - window if window else True)
    rows = see.any(1)
    for h in range(Hq):
        g = h // (Hq // Hkv)
        s = (q[:, h] @ k[:, g].T * scale).masked_fill(~see, -math.inf)[rows]
        z = torch.logsumexp(s, 1)
        lse[h, rows] = z
        o[rows, h] = torch.exp(s - z[:, None]) @ v[:, g]
    return o, lse


def attention_packed(q, k, v, cu_q, cu_k, scale, causal, window=0):
    """Packed sequences; rows behind the last sequence are left as NaN."""
    o = torch.full(q.shape, math.nan, dtype=torch.float64)
    lse = torch.full((q.shape[1], q.shape[0]), math.nan, dtype=torch.float64)
    for b in range(len(cu_q) - 1):
        a, e, c, f = int(cu_q[b]), int(cu_q[b + 1]), int(cu_k[b]), int(cu_k[b + 1])
        o[a:e], lse[:, a:e] = attention(q[a:e], k[c:f], v[c:f], scale, causal, window)
    return o, lse


class Pages:
    """The page state as plain lists, one slot after another."""

    def __init__(self, S, max_pages, num_pages, page_size):
        self.table = np.full((S, max_pages), -1, np.int32)
        self.lens = np.zeros(S, np.int32)
        self.ref = np.zeros(num_pages, np.int32)
        self.ps = page_size

    def held(self, n):
        return -(-int(n) // self.ps)

    def reserve(self, add):
        """-> copies (S, 2), or None when the pool or a row is too short (nothing changes)."""
        ref0, free = self.ref.copy(), [i for i in range(len(self.ref)) if self.ref[i] == 0]
        want = []
        for s, a in enumerate(add):
            old, new = self.held(self.lens[s]), self.held(self.lens[s] + a)
            if new > self.table.shape[1]:
                return None
            split = a > 0 and self.lens[s] % self.ps and ref0[self.table[s, old - 1]] > 1
            want.append((old, new if a > 0 else old, bool(split)))
        if sum(n - o + sp for o, n, sp in want) > len(free):
            return None
        copies = np.full((len(add), 2), -1, np.int32)
        free = iter(free)
        for s, (old, new, split) in enumerate(want):
            if split:
                was, now = self.table[s, old - 1], next(free)
                copies[s] = was, now
                self.ref[was] -= 1
                self.ref[now] = 1
                self.table[s, old - 1] = now
            for j in range(old, new):
                self.table[s, j] = next(free)
                self.ref[self.table[s, j]] = 1
            self.lens[s] += add[s]
        return copies

    def fork(self, src, dst, lengths=None):
        for i, (s, d) in enumerate(zip(src, dst)):
            n = int(self.lens[s]) if lengths is None else int(lengths[i])
            h = self.held(n)
            self.table[d, :h] = self.table[s, :h]
            for p in self.table[s, :h]:
                self.ref[p] += 1
            self.lens[d] = n

    def free(self, slots, keep=None):
        for i, s in enumerate(slots):
            k = 0 if keep is None else int(keep[i])
            for j in range(self.held(k), self.held(self.lens[s])):
                self.ref[self.table[s, j]] -= 1
                self.table[s, j] = -1
            self.lens[s] = k

    def compact(self):
        n = int((self.ref > 0).sum())
        holes = [i for i in range(n) if self.ref[i] == 0]
        movers = [i for i in range(n, len(self.ref)) if self.ref[i] > 0]
        copies = np.full((len(self.ref) // 2, 2), -1, np.int32)
        for k, (m, h) in enumerate(zip(movers, holes)):
            copies[k] = m, h
            self.ref[h], self.ref[m] = self.ref[m], 0
            for s in range(len(self.lens)):
                row = self.table[s, :self.held(self.lens[s])]
                row[row == m] = h
        return copies
