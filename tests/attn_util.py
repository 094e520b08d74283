"""Plain float64 versions of the attention-half operators, and the host model
of the page bookkeeping, for the GPU tests."""

from __future__ import annotations

import numpy as np
import torch

LOG_FREE = -np.inf


def norm_ref(x, block, pre, post, gate, scale, eps):
    x = x.double()
    if block is not None:
        n = block.double()
        if post is not None:
            n = n / torch.sqrt((n * n).mean(-1, keepdim=True) + eps) * post.double()
        if gate is not None:
            n = n * gate.double()
        x = x + scale * n
    y = None if pre is None else x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * pre.double()
    return x, y


def attn_ref(q, k, v, scale, window=0):
    """q [lq, heads, D], k and v [lk, kv_heads, D] -> (out, lse) in float64; masked places never enter."""
    q, k, v = q.double().cpu(), k.double().cpu(), v.double().cpu()
    lq, heads, D = q.shape
    lk, group = k.shape[0], heads // k.shape[1]
    out = torch.zeros(lq, heads, D, dtype=torch.float64)
    lse = torch.full((lq, heads), -np.inf, dtype=torch.float64)
    for r in range(lq):
        last = r + lk - lq
        first = max(0, last - window + 1) if window else 0
        if last < first:
            continue
        kk = k[first:last + 1].repeat_interleave(group, 1)
        vv = v[first:last + 1].repeat_interleave(group, 1)
        s = torch.einsum("hd,jhd->hj", q[r], kk) * scale
        z = torch.logsumexp(s, 1)
        lse[r] = z
        out[r] = torch.einsum("hj,jhd->hd", torch.exp(s - z[:, None]), vv)
    return out, lse


def attn_bounds(dtype, out_ref, v_max):
    """|out - ref| bound.  bf16: the output's rounding (2^-8 of it) and the rounding of every softmax weight
    (2^-8 of sum p |v| <= v_max), plus f32 sums; f32: f32 sums over some hundred terms and the weights' exponent,
    2e-5 of v_max."""
    if dtype == torch.bfloat16:
        return 2.0 ** -8 * out_ref.abs() + (2.0 ** -8 + 2e-5) * v_max
    return 2e-5 * v_max + 0 * out_ref


def assert_attn(out, lse, out_ref, lse_ref, v_max, what=""):
    o = out.double().cpu()
    bound = attn_bounds(out.dtype, out_ref, v_max)
    bad = ~((o - out_ref).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, worst {float((o - out_ref).abs().max()):.3e}"
    if lse is not None:
        z = lse.double().cpu()
        empty = torch.isinf(lse_ref)
        assert torch.equal(torch.isinf(z) & (z < 0), empty), what
        # a score is a dot product of head_dim terms of order one in f32: 2e-5, relative or absolute
        err = (z - lse_ref)[~empty].abs()
        assert (err <= 2e-5 * (1 + lse_ref[~empty].abs())).all(), f"{what}: lse {float(err.max()):.3e}"


class HostPages:
    """The page bookkeeping restated on the host, one step at a time."""

    def __init__(self, num_pages, max_seqs, max_pages, page):
        self.P, self.page = num_pages, page
        self.table = -np.ones((max_seqs, max_pages), np.int32)
        self.lens = np.zeros(max_seqs, np.int32)
        self.refs = np.zeros(num_pages, np.int32)

    def pages(self, n):
        return -(-int(n) // self.page)

    def reserve(self, seqs, counts):
        """Returns the (old, new, tokens) private copies; None if refused."""
        refs0 = self.refs.copy()
        want = []
        for s, c in zip(seqs, counts):
            held = self.lens[s]
            if self.pages(held + c) > self.table.shape[1]:
                return None
            cow = bool(c > 0 and held % self.page and refs0[self.table[s, held // self.page]] > 1)
            want.append((cow, self.pages(held + c) - self.pages(held)))
        free = [p for p in range(self.P) if refs0[p] == 0]
        if sum(a + b for a, b in want) > len(free):
            return None
        copies = []
        for s, c, (cow, fresh) in zip(seqs, counts, want):
            held = int(self.lens[s])
            if cow:
                p, col = free.pop(0), held // self.page
                old = self.table[s, col]
                copies.append((int(old), p, held % self.page))
                self.refs[old] -= 1
                self.refs[p] = 1
                self.table[s, col] = p
            for j in range(fresh):
                p = free.pop(0)
                self.table[s, self.pages(held) + j] = p
                self.refs[p] = 1
            self.lens[s] += c
        return copies

    def truncate(self, seqs, lens):
        for s, n in zip(seqs, lens):
            keep = min(int(n), int(self.lens[s]))
            for c in range(self.pages(keep), self.pages(self.lens[s])):
                self.refs[self.table[s, c]] -= 1
                self.table[s, c] = -1
            self.lens[s] = keep

    def fork(self, src, dst):
        rows, lens = self.table[src].copy(), self.lens[src].copy()
        for r in rows:
            for p in r[r >= 0]:
                self.refs[p] += 1
        for s in dst:
            for p in self.table[s][self.table[s] >= 0]:
                self.refs[p] -= 1
        for s, r, n in zip(dst, rows, lens):
            self.table[s], self.lens[s] = r, n

    def compact(self):
        """Returns (mapping old -> new of the moved pages, used)."""
        used = int((self.refs > 0).sum())
        movers = [p for p in range(used, self.P) if self.refs[p] > 0]
        holes = [p for p in range(used) if self.refs[p] <= 0]
        for a, b in zip(movers, holes):
            self.refs[b], self.refs[a] = self.refs[a], 0
            self.table[self.table == a] = b
        return dict(zip(movers, holes)), used


def ints(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def starts_of(lens):
    return ints([0, *np.cumsum(lens).tolist()])
