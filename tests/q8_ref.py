"""Plain models of the 8-bit pages and of shared pages, in 64 bits and one element after the other."""
import math

import numpy as np
import torch

E4M3_MAX = 448.0


def e4m3(x):
    """x (float64 array) to the nearest e4m3 number, ties to even; sizes above 448 saturate, NaN stays."""
    x = np.asarray(x, dtype=np.float64)
    _, e = np.frexp(np.maximum(np.abs(np.nan_to_num(x)), 2.0 ** -6))
    step = np.ldexp(1.0, e - 4)
    return np.clip(np.round(x / step) * step, -E4M3_MAX, E4M3_MAX)


def scale_for(amax):
    """The smallest power of two s in [2^-120, 2^119] with amax / s <= 448."""
    if amax == 0.0:
        return 2.0 ** -120
    m, e = math.frexp(amax / E4M3_MAX)
    return math.ldexp(1.0, min(119, max(-120, e - (m == 0.5))))


def numbers(pool):
    """The numbers of a pool of bytes, float64."""
    return pool.view(torch.float8_e4m3fn).float().double().cpu().numpy()


def quantise_into(pages, scales, page, held, rows):
    """pages [H, NB, bs, D] (numbers), scales [H, NB]: rows [n, H, D] after the `held` rows of `page`."""
    n = rows.shape[0]
    for h in range(pages.shape[0]):
        x = rows[:, h]
        finite = np.where(np.isfinite(x), np.abs(x), 0.0)
        s = scale_for(finite.max())
        if held:
            was = scales[h, page]
            s = max(s, was)
            # the kernel's ratio and products are fp32
            ratio = np.float32(was) / np.float32(s)
            old = (pages[h, page, :held].astype(np.float32) * ratio).astype(np.float64)
            pages[h, page, :held] = e4m3(old)
        y = (x.astype(np.float32) / np.float32(s)).astype(np.float64)
        pages[h, page, held:held + n] = np.where(np.isfinite(x), e4m3(y), np.nan)
        scales[h, page] = s


class Pages:
    """Page tables, a free stack and counts of holders, as lists."""

    def __init__(self, table, n_blocks, lens, score, ids, top, bs, shares=None):
        self.table = [list(r) for r in table.tolist()]
        self.n_blocks, self.len = n_blocks.tolist(), lens.tolist()
        self.score = [list(r) for r in score.tolist()]
        self.ids, self.top, self.bs = ids.tolist(), int(top), bs
        self.shares = shares.tolist() if shares is not None else None

    def pop(self):
        self.top -= 1
        return self.ids[self.top]

    def append(self, counts):
        """Pages for counts[b] rows; returns [(b, page, held, first row of the sequence's, rows)]."""
        jobs = []
        for b, n in enumerate(counts):
            at = 0
            while at < n:
                pos = self.len[b]
                if pos % self.bs == 0:
                    lb = self.n_blocks[b]
                    self.table[b][lb], self.score[b][lb] = self.pop(), 0.0
                    self.n_blocks[b] += 1
                k = min(self.bs - pos % self.bs, n - at)
                jobs.append((b, self.table[b][pos // self.bs], pos % self.bs, at, k))
                self.len[b] += k
                at += k
        return jobs

    def reorder(self, parent):
        """Returns [(from page, to page, rows)]."""
        B = len(parent)
        kids = [[c for c in range(B) if parent[c] == b] for b in range(B)]
        keeper = [b if b in k else (k[0] if k else None) for b, k in enumerate(kids)]
        part = [self.len[b] % self.bs for b in range(B)]
        change = {}
        for b in range(B):
            for i in range(self.n_blocks[b]):
                x = self.table[b][i]
                if part[b] and i == self.n_blocks[b] - 1 and kids[b]:
                    continue
                change[x] = change.get(x, 0) + len(kids[b]) - 1
        freed = []
        for x in sorted(change):
            self.shares[x] += change[x]
            if self.shares[x] < 0:
                self.shares[x] = 0
                freed.append(x)
        stack = self.ids[:self.top] + freed
        old = ([list(r) for r in self.table], [list(r) for r in self.score], list(self.n_blocks), list(self.len))
        copies = []
        for b in range(B):
            p = parent[b]
            if p < 0:
                self.n_blocks[b] = self.len[b] = 0
                continue
            n = old[2][p]
            self.table[b][:n], self.score[b][:n] = old[0][p][:n], old[1][p][:n]
            self.n_blocks[b], self.len[b] = n, old[3][p]
            if part[p] and keeper[p] != b:
                to = stack.pop()
                copies.append((self.table[b][n - 1], to, part[p]))
                self.table[b][n - 1] = to
        self.ids[:len(stack)], self.top = stack, len(stack)
        return copies

    def same_as(self, table, n_blocks, lens, score, ids, top, shares=None):
        assert n_blocks.tolist() == self.n_blocks and lens.tolist() == self.len and int(top) == self.top
        assert ids.tolist()[:self.top] == self.ids[:self.top]
        for b, n in enumerate(self.n_blocks):
            assert table[b, :n].tolist() == self.table[b][:n] and score[b, :n].tolist() == self.score[b][:n]
        if shares is not None:
            assert shares.tolist() == self.shares


def attention(q, k, v, scale):
    """q [G, D], k, v [n, D] in float64 -> out [G, D], lse [G], logits [G, n], sum of p |v| [G, D]."""
    if k.shape[0] == 0:
        z = torch.zeros_like(q)
        return z, torch.full((q.shape[0],), -math.inf, dtype=q.dtype, device=q.device), q @ k.T, z
    x = q @ k.T * scale
    p = torch.softmax(x, dim=1)
    return p @ v, torch.logsumexp(x, dim=1), x, p @ v.abs()
