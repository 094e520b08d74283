"""Cases for timing the attention half of a decoder layer: norms around a
block, the pages of a key-value cache, attention of one new token over those
pages, and attention over packed prompts.

`run` is one pass through one operator: the plain form (elementary torch
operations in 32 bits) where `own` is false, this package's kernels where it
is true.
"""

import math
import random
from types import SimpleNamespace

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # the norm between two blocks of one decode step of one sequence
        dict(name="norm_one_token", op="norm", tokens=1, hidden=2048, dtype="bf16", gate="none", post=True),
        # a prefill chunk with an odd number of tokens, per-channel gate
        dict(name="norm_prefill", op="norm", tokens=16391, hidden=2560, dtype="bf16", gate="channel", post=True),
        # the same join in 32 bits, a gate for every element
        dict(name="norm_f32", op="norm", tokens=509, hidden=2048, dtype="f32", gate="full", post=False),
        # one step of a batch: the last step's rejected tokens are rolled back, room is
        # reserved for the new ones, and one layer's keys and values are written
        dict(name="pages_step", op="pages_step", seqs=64, counts=3, len_lo=1, len_hi=2000, lens_seed=11, kv_heads=16,
             head_dim=128, page=16, dtype="bf16", layers=1),
        # sampling several continuations of each prompt: fork, then one token each,
        # which copies the partly filled last page of all 16 layers
        dict(name="pages_fork", op="pages_fork", parents=8, children=7, len_lo=1000, len_hi=3000, lens_seed=12,
             kv_heads=16, head_dim=128, page=64, dtype="bf16", layers=16),
        # closing the holes that finished sequences left in the pool
        dict(name="pages_compact", op="pages_compact", pages=4099, fill=0.6, kv_heads=4, head_dim=128, page=32,
             dtype="bf16", layers=16, lens_seed=13),
        # decode of one short chat
        dict(name="decode_short", op="decode", seqs=1, len_lo=333, len_hi=333, lens_seed=21, heads=16, kv_heads=16,
             head_dim=128, page=16, dtype="bf16", window=0),
        # batched decode, ragged lengths, five query heads to a key head (hidden 2560)
        dict(name="decode_batch", op="decode", seqs=64, len_lo=0, len_hi=8192, lens_seed=22, heads=20, kv_heads=4,
             head_dim=128, page=64, dtype="bf16", window=0),
        # one very long context (hidden 2048 in heads of 64)
        dict(name="decode_long", op="decode", seqs=1, len_lo=131072, len_hi=131072, lens_seed=23, heads=32, kv_heads=8,
             head_dim=64, page=16, dtype="bf16", window=0),
        # a batch of ragged prompts packed together, grouped heads, some a single token
        dict(name="prompt_packed", op="prompt", seqs=24, len_lo=1, len_hi=1500, prefix_hi=0, lens_seed=31, heads=20,
             kv_heads=4, head_dim=128, dtype="bf16", window=0),
        # one long prompt (hidden 2048 in 16 heads)
        dict(name="prompt_long", op="prompt", seqs=1, len_lo=16384, len_hi=16384, prefix_hi=0, lens_seed=32, heads=16,
             kv_heads=16, head_dim=128, dtype="bf16", window=0),
        # a small model in 32 bits; each prompt's earlier part is already in the keys
        dict(name="prompt_f32", op="prompt", seqs=5, len_lo=17, len_hi=400, prefix_hi=200, lens_seed=33, heads=8,
             kv_heads=4, head_dim=64, dtype="f32", window=0),
    ]


def _log_int(rng, lo, hi):
    """A whole number of [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "pages_step", "pages_fork", "pages_compact", "decode", "decode", "prompt", "prompt"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    seed = rng.randrange(1 << 30)
    if op == "norm":
        hidden = 8 * _log_int(rng, 8, 512)
        tokens = _log_int(rng, 1, min(16384, 40_000_000 // hidden // (2 if dtype == "f32" else 1)))
        return dict(op=op, tokens=tokens, hidden=hidden, dtype=dtype, gate=rng.choice(["none", "token", "channel", "full"]),
                    post=rng.random() < 0.7)
    kv_heads, head_dim = rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 128])
    page = rng.choice([16, 32, 64])
    row = kv_heads * head_dim * (2 if dtype == "bf16" else 4)      # bytes of one token's keys
    if op == "pages_step":
        counts = _log_int(rng, 1, 512)
        return dict(op=op, seqs=_log_int(rng, 1, max(1, min(256, 8192 // counts))), counts=counts, len_lo=1,
                    len_hi=_log_int(rng, 64, 4000), lens_seed=seed, kv_heads=kv_heads, head_dim=head_dim, page=page,
                    dtype=dtype, layers=1)
    if op == "pages_fork":
        parents = _log_int(rng, 1, 8)
        return dict(op=op, parents=parents, children=_log_int(rng, 1, 7), len_lo=100, len_hi=_log_int(rng, 200, 3000),
                    lens_seed=seed, kv_heads=kv_heads, head_dim=head_dim, page=page, dtype=dtype,
                    layers=rng.choice([1, 4, 16] if row <= 4096 else [1, 4]))
    if op == "pages_compact":
        layers = rng.choice([1, 4, 16])
        return dict(op=op, pages=_log_int(rng, 61, max(61, min(9000, (1 << 31) // (2 * layers * row * page)))),
                    fill=rng.choice([0.3, 0.5, 0.7, 0.9]), kv_heads=kv_heads, head_dim=head_dim, page=page, dtype=dtype,
                    layers=layers, lens_seed=seed)
    heads = kv_heads * rng.choice([g for g in (1, 2, 4, 5, 8) if g * kv_heads <= 40])
    if op == "decode":
        seqs = _log_int(rng, 1, 128)
        len_hi = _log_int(rng, 16, max(16, min(131072, (1 << 28) // (seqs * row))))
        return dict(op=op, seqs=seqs, len_lo=rng.choice([0, 1, len_hi // 2, len_hi]), len_hi=len_hi, lens_seed=seed,
                    heads=heads, kv_heads=kv_heads, head_dim=head_dim, page=page, dtype=dtype,
                    window=rng.choice([0, 0, 0, max(1, len_hi // 3)]))
    seqs = _log_int(rng, 1, 32)
    most = int(math.sqrt((1 << 32) / (seqs * heads))) if dtype == "bf16" else int(math.sqrt((1 << 27) / (seqs * heads)))
    len_hi = _log_int(rng, 16, max(16, min(16384, most) - 100))
    return dict(op=op, seqs=seqs, len_lo=rng.choice([1, len_hi // 2, len_hi]), len_hi=len_hi,
                prefix_hi=rng.choice([0, 0, 0, 100]), lens_seed=seed, heads=heads, kv_heads=kv_heads, head_dim=head_dim,
                dtype=dtype, window=rng.choice([0, 0, 0, max(1, len_hi // 3)]))


def _lens(case, n):
    """The n sequence lengths of a case."""
    r = random.Random(case["lens_seed"])
    return [r.randint(case["len_lo"], case["len_hi"]) for _ in range(n)]


def _prompt_lens(case):
    """Query and key lengths of a case's prompts."""
    r = random.Random(case["lens_seed"] + 1)
    lq = _lens(case, case["seqs"])
    return lq, [n + r.randint(0, case["prefix_hi"]) for n in lq]


def _pages(n, page):
    return -(-n // page)


def _compact_used(case):
    """Which pages of the pool hold tokens before compaction."""
    r = random.Random(case["lens_seed"])
    return [r.random() < case["fill"] for _ in range(case["pages"])]


def _visible(lq, lk, window):
    """Query-key pairs that the causal mask (and the window) leaves."""
    total = 0
    for i in range(lq):
        seen = i + lk - lq + 1
        total += max(0, min(seen, window) if window else seen)
    return total


# ------------------------------------------------------------------ inputs

def _randn(shape, g, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype) if math.prod(shape) < 1 << 24 \
        else torch.empty(shape, device="cuda", dtype=dtype).normal_(generator=g)


def _cumulative(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def _cache(case, lens, rows, columns, spare, g):
    """Pools, page table, lengths and reference counts: the rows' pages lie in
    the pool in a random order."""
    page, dt = case["page"], DTYPES[case["dtype"]]
    held = [_pages(n, page) for n in lens]
    total = sum(held) + spare
    shape = (case["layers"] if "layers" in case else 1, total, case["kv_heads"], page, case["head_dim"])
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    # only the pages that the rows hold are permuted among all; the rest stay free
    table = torch.full((rows, columns), -1, dtype=torch.int32, device="cuda")
    col = torch.arange(columns, device="cuda")
    h = torch.zeros(rows, dtype=torch.int64, device="cuda")
    h[: len(held)] = torch.tensor(held, device="cuda")
    table[col[None] < h[:, None]] = order[: sum(held)]
    refs = torch.zeros(total, dtype=torch.int32, device="cuda")
    refs[order[: sum(held)].long()] = 1
    n = torch.zeros(rows, dtype=torch.int32, device="cuda")
    n[: len(lens)] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return _randn(shape, g, dt), _randn(shape, g, dt), table, n, refs


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = SimpleNamespace(case=dict(case), op=case["op"])
    dt = DTYPES[case["dtype"]]
    if s.op == "norm":
        T, H = case["tokens"], case["hidden"]
        s.x, s.block = _randn((T, H), g, dt), _randn((T, H), g, dt) * 0.5
        s.post = 1 + 0.1 * _randn((H,), g, dt) if case["post"] else None
        s.pre = 1 + 0.1 * _randn((H,), g, dt)
        shape = {"none": None, "token": (T, 1), "channel": (1, H), "full": (T, H)}[case["gate"]]
        s.gate = None if shape is None else torch.sigmoid(_randn(shape, g, dt))
        s.scale = 0.22
        return s
    if s.op == "prompt":
        lq, lk = _prompt_lens(case)
        s.starts_q, s.starts_k, s.max_q, s.max_k = _cumulative(lq), _cumulative(lk), max(lq), max(lk)
        D, Hq, Hkv = case["head_dim"], case["heads"], case["kv_heads"]
        s.q = _randn((sum(lq), Hq, D), g, dt)
        s.k, s.v = _randn((sum(lk), Hkv, D), g, dt), _randn((sum(lk), Hkv, D), g, dt)
        s.scale, s.window = 1 / math.sqrt(D), case["window"]
        return s
    page = case["page"]
    if s.op == "pages_step":
        lens, c = _lens(case, case["seqs"]), case["counts"]
        new = [_pages(n + c, page) - _pages(n, page) for n in lens]
        s.base = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s.counts = torch.full((len(lens),), c, dtype=torch.int32, device="cuda")
        s.seqs = torch.randperm(len(lens), generator=g, device="cuda").to(torch.int32)
        s.base = s.base[s.seqs.long()]
        s.starts = _cumulative([c] * len(lens))
        cache = _cache(case, lens, len(lens), _pages(max(lens) + c, page), sum(new) + 7, g)
        row = (c * len(lens), case["kv_heads"], case["head_dim"])
        s.new_k, s.new_v = _randn(row, g, dt), _randn(row, g, dt)
    elif s.op == "pages_fork":
        p, c = case["parents"], case["children"]
        lens = _lens(case, p)
        cache = _cache(case, lens, p * (1 + c), _pages(max(lens) + 1, page), 2 * p * c + 5, g)
        s.src = torch.arange(p, device="cuda", dtype=torch.int32).repeat_interleave(c)
        s.dst = p + torch.randperm(p * c, generator=g, device="cuda").to(torch.int32)
        s.counts = torch.ones(p * c, dtype=torch.int32, device="cuda")
    elif s.op == "pages_compact":
        used = torch.tensor(_compact_used(case), device="cuda")
        n = case["pages"]
        rows, columns = 16, _pages(n, 16) + 1
        shape = (case["layers"], n, case["kv_heads"], page, case["head_dim"])
        ids = used.nonzero()[:, 0]
        ids = ids[torch.randperm(ids.numel(), generator=g, device="cuda")].to(torch.int32)
        table = torch.full((rows, columns), -1, dtype=torch.int32, device="cuda")
        share = _pages(ids.numel(), rows)
        held = [max(0, min(share, ids.numel() - i * share)) for i in range(rows)]
        h = torch.tensor(held, device="cuda")
        table[torch.arange(columns, device="cuda")[None] < h[:, None]] = ids
        table[rows - 1, 0] = table[0, 0]            # a page that two sequences share
        refs = torch.zeros(n, dtype=torch.int32, device="cuda")
        refs.index_add_(0, table[table >= 0].long(), torch.ones_like(table[table >= 0]))
        lens = torch.tensor([x * page for x in held], dtype=torch.int32, device="cuda")
        lens[rows - 1] = max(held[rows - 1], 1) * page
        free = (table >= 0) & (torch.arange(columns, device="cuda")[None] >= _pages(lens, page)[:, None])
        table[free] = -1
        cache = (_randn(shape, g, dt), _randn(shape, g, dt), table, lens, refs)
        s.table_out, s.refs_out = torch.empty_like(table), torch.empty_like(refs)
        s.used = torch.zeros(1, dtype=torch.int32, device="cuda")
    else:
        lens = _lens(case, case["seqs"])
        cache = _cache(case, lens, len(lens), max(1, _pages(max(lens), page)), 3, g)
        s.seqs = torch.randperm(len(lens), generator=g, device="cuda").to(torch.int32)
        s.q = _randn((len(lens), case["heads"], case["head_dim"]), g, dt)
        s.scale, s.window = 1 / math.sqrt(case["head_dim"]), case["window"]
    s.k, s.v, s.table, s.lens, s.refs = cache
    if own:
        from expert_slot_cache_topk_gb300.attention import KVPages
        s.kv = KVPages(s.k, s.v, s.table, s.lens, s.refs)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    from expert_slot_cache_topk_gb300 import attention as A
    if s.op == "norm":
        x, y = torch.empty_like(s.x), torch.empty_like(s.x)
        A.norm_residual(s.x, s.block, s.pre, x, y, post_weight=s.post, gate=s.gate, res_scale=s.scale, eps=EPS)
        return {"x": x, "y": y}
    if s.op == "prompt":
        out = torch.empty_like(s.q)
        lse = torch.empty(s.q.shape[:2], dtype=torch.float32, device=s.q.device)
        A.attn_prompt(s.q, s.k, s.v, s.starts_q, s.starts_k, out, scale=s.scale, window=s.window, lse=lse)
        return {"out": out, "lse": lse}
    if s.op == "decode":
        out = torch.empty_like(s.q)
        lse = torch.empty(s.q.shape[:2], dtype=torch.float32, device=s.q.device)
        s.kv.attend(0, s.q, s.seqs, out, scale=s.scale, window=s.window, lse=lse)
        return {"out": out, "lse": lse}
    if s.op == "pages_step":
        s.kv.truncate(s.seqs, s.base)
        s.kv.reserve(s.seqs, s.counts)
        s.kv.append(0, s.seqs, s.starts, s.new_k, s.new_v)
    elif s.op == "pages_fork":
        s.kv.fork(s.src, s.dst)
        s.kv.reserve(s.dst, s.counts)
    else:
        s.kv.compact(s.table_out, s.refs_out, s.used)
        return {"k": s.k, "v": s.v, "table": s.table_out, "refs": s.refs_out, "used": s.used}
    return {"k": s.k, "v": s.v, "table": s.table, "lens": s.lens, "refs": s.refs}


def _plain(s):
    if s.op == "norm":
        return _norm_plain(s)
    if s.op == "prompt":
        return _prompt_plain(s)
    if s.op == "decode":
        return _decode_plain(s)
    if s.op == "pages_step":
        _truncate_plain(s, s.seqs, s.base)
        _reserve_plain(s, s.seqs, s.counts)
        _append_plain(s)
    elif s.op == "pages_fork":
        _fork_plain(s)
        _reserve_plain(s, s.dst, s.counts)
    else:
        return _compact_plain(s)
    return {"k": s.k, "v": s.v, "table": s.table, "lens": s.lens, "refs": s.refs}


def _norm_plain(s):
    n = s.block.float()
    if s.post is not None:
        n = n * torch.rsqrt((n * n).mean(-1, keepdim=True) + EPS) * s.post.float()
    if s.gate is not None:
        n = n * s.gate.float()
    x = s.x.float() + s.scale * n
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s.pre.float()
    return {"x": x.to(s.x.dtype), "y": y.to(s.x.dtype)}


def _softmax_parts(scores, seen):
    """Row maxima, exponentials and sums of masked scores; rows that see nothing get zeros."""
    scores.masked_fill_(~seen, -math.inf)
    m = scores.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = scores.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    return m, p, total


def _join(o, m, total):
    some = total > 0
    out = torch.where(some, o / torch.where(some, total, torch.ones_like(total)), torch.zeros_like(o))
    return out, (m + total.log()).squeeze(-1)


def _prompt_plain(s):
    T, Hq, D = s.q.shape
    Hkv = s.k.shape[1]
    G = Hq // Hkv
    rows, cols = torch.arange(s.max_q, device="cuda"), torch.arange(s.max_k, device="cuda")
    bq, bk = s.starts_q.long(), s.starts_k.long()
    lq, lk = bq[1:] - bq[:-1], bk[1:] - bk[:-1]
    iq = (bq[:-1, None] + rows).clamp(max=T - 1)
    ik = (bk[:-1, None] + cols).clamp(max=s.k.shape[0] - 1)
    q = s.q[iq].float().mul_(s.scale).view(-1, s.max_q, Hkv, G, D).permute(0, 2, 3, 1, 4)     # [n, Hkv, G, rows, D]
    k = s.k[ik].float().permute(0, 2, 3, 1).unsqueeze(2)                                      # [n, Hkv, 1, D, cols]
    v = s.v[ik].float().permute(0, 2, 1, 3).unsqueeze(2)                                      # [n, Hkv, 1, cols, D]
    n = q.shape[0]
    scores = q.reshape(n, Hkv, G * s.max_q, D) @ k.squeeze(2)
    at = rows[None] + (lk - lq)[:, None]                                                      # last key a row sees
    seen = (cols[None, None] <= at[..., None]) & (cols[None, None] < lk[:, None, None])
    if s.window:
        seen &= cols[None, None] > at[..., None] - s.window
    scores = scores.view(n, Hkv, G, s.max_q, s.max_k)
    m, p, total = _softmax_parts(scores, seen[:, None, None])
    o = (p.view(n, Hkv, G * s.max_q, s.max_k) @ v.squeeze(2)).view(n, Hkv, G, s.max_q, D)
    o, lse = _join(o, m, total)
    token = torch.arange(T, device="cuda")
    seq = torch.searchsorted(bq[1:].contiguous(), token, right=True)
    row = token - bq[seq]
    out = o.permute(0, 3, 1, 2, 4).reshape(n, s.max_q, Hq, D)[seq, row]
    lse = lse.permute(0, 3, 1, 2).reshape(n, s.max_q, Hq)[seq, row]
    return {"out": out.to(s.q.dtype), "lse": lse}


def _decode_plain(s):
    n, Hq, D = s.q.shape
    Hkv, page = s.k.shape[2], s.k.shape[3]
    at = s.table[s.seqs.long()].long().clamp(min=0)                                           # [n, columns]
    k = s.k[0][at].float().transpose(1, 2).reshape(n, Hkv, -1, D)
    v = s.v[0][at].float().transpose(1, 2).reshape(n, Hkv, -1, D)
    scores = (s.q.float() * s.scale).view(n, Hkv, Hq // Hkv, D) @ k.transpose(2, 3)
    token, held = torch.arange(k.shape[2], device="cuda"), s.lens[s.seqs.long()].long()
    seen = token[None] < held[:, None]
    if s.window:
        seen &= token[None] >= held[:, None] - s.window
    m, p, total = _softmax_parts(scores, seen[:, None, None])
    o, lse = _join(p @ v, m, total)
    return {"out": o.reshape(n, Hq, D).to(s.q.dtype), "lse": lse.reshape(n, Hq)}


def _truncate_plain(s, seqs, lens):
    i, page = seqs.long(), s.k.shape[3]
    keep = torch.minimum(s.lens[i], lens)
    rows = s.table[i]
    gone = (rows >= 0) & (torch.arange(rows.shape[1], device="cuda")[None] >= _pages(keep, page)[:, None])
    s.refs.index_add_(0, rows.clamp(min=0).long().flatten(), -gone.to(torch.int32).flatten())
    s.table[i] = torch.where(gone, torch.full_like(rows, -1), rows)
    s.lens[i] = keep


def _reserve_plain(s, seqs, counts):
    i, page = seqs.long(), s.k.shape[3]
    held = s.lens[i]
    rows = s.table[i]
    col = torch.arange(rows.shape[1], device="cuda")[None]
    have, need = _pages(held, page)[:, None], _pages(held + counts, page)[:, None]
    tail = rows.gather(1, (have - 1).clamp(min=0).long())[:, 0].clamp(min=0).long()
    copy = (held % page != 0) & (counts > 0) & (s.refs[tail] > 1)
    fresh = ((col >= have) & (col < need)) | ((col == have - 1) & copy[:, None])
    free = torch.argsort((s.refs > 0).to(torch.int8), stable=True).to(torch.int32)
    given = free[(fresh.flatten().cumsum(0) - 1).clamp(min=0)].view_as(rows)
    # the tokens held move to the private copy of a shared last page
    to = torch.where(copy, given.gather(1, (have - 1).clamp(min=0).long())[:, 0].long(), tail)
    token = torch.arange(page, device="cuda")[None] < (held % page)[:, None]
    moved = token[:, None, :, None]
    s.k[:, to] = torch.where(moved, s.k[:, tail], s.k[:, to])
    s.v[:, to] = torch.where(moved, s.v[:, tail], s.v[:, to])
    s.refs.index_add_(0, tail, -copy.to(torch.int32))
    s.refs.index_add_(0, given.flatten().long(), fresh.flatten().to(torch.int32))
    s.table[i] = torch.where(fresh, given, rows)
    s.lens[i] = held + counts


def _append_plain(s):
    page = s.k.shape[3]
    token = torch.arange(s.new_k.shape[0], device="cuda")
    at = torch.searchsorted(s.starts[1:].contiguous(), token.to(torch.int32), right=True)
    i = s.seqs.long()[at]
    pos = s.lens[i].long() - s.starts[1:].long()[at] + token
    to = s.table[i, pos // page].long()
    s.k[0, to, :, pos % page] = s.new_k
    s.v[0, to, :, pos % page] = s.new_v


def _fork_plain(s):
    src, dst = s.src.long(), s.dst.long()
    rows, old = s.table[src], s.table[dst]
    s.refs.index_add_(0, rows.clamp(min=0).long().flatten(), (rows >= 0).to(torch.int32).flatten())
    s.refs.index_add_(0, old.clamp(min=0).long().flatten(), -(old >= 0).to(torch.int32).flatten())
    s.table[dst] = rows
    s.lens[dst] = s.lens[src]


def _compact_plain(s):
    used = s.refs > 0
    count = used.sum()
    page = torch.arange(used.numel(), device="cuda")
    movers, holes = (used & (page >= count)).nonzero()[:, 0], (~used & (page < count)).nonzero()[:, 0]
    s.k[:, holes] = s.k[:, movers]
    s.v[:, holes] = s.v[:, movers]
    to = page.clone()
    to[movers] = holes
    refs = torch.where(used, s.refs, torch.zeros_like(s.refs))
    refs[holes] = s.refs[movers]
    refs[movers] = 0
    s.refs_out.copy_(refs)
    s.table_out.copy_(torch.where(s.table >= 0, to[s.table.clamp(min=0).long()].to(torch.int32), s.table))
    s.used.copy_(count)
    return {"k": s.k, "v": s.v, "table": s.table_out, "refs": s.refs_out, "used": s.used}


# ----------------------------------------------------------- what it takes

def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        T, H = case["tokens"], case["hidden"]
        gate = {"none": 0, "token": T, "channel": H, "full": T * H}[case["gate"]]
        return {"bytes": size * (4 * T * H + gate + H * (1 + bool(case["post"]))), "flops": (10 + 5 * bool(case["post"])) * T * H}
    D, Hkv = case["head_dim"], case["kv_heads"]
    if case["op"] == "prompt":
        lq, lk = _prompt_lens(case)
        Hq = case["heads"]
        pairs = sum(_visible(a, b, case["window"]) for a, b in zip(lq, lk))
        return {"bytes": size * D * (2 * Hq * sum(lq) + 2 * Hkv * sum(lk)) + 4 * Hq * sum(lq), "flops": 4 * D * Hq * pairs}
    row = 2 * Hkv * D * size                               # one token's key and value in one layer
    if case["op"] == "decode":
        seen = sum(min(n, case["window"]) if case["window"] else n for n in _lens(case, case["seqs"]))
        Hq, n = case["heads"], case["seqs"]
        return {"bytes": seen * row + 2 * n * Hq * D * size + 4 * n * Hq, "flops": 4 * D * Hq * seen}
    page = case["page"]
    if case["op"] == "pages_step":
        lens, c = _lens(case, case["seqs"]), case["counts"]
        new = sum(_pages(n + c, page) - _pages(n, page) for n in lens)
        return {"bytes": 2 * c * len(lens) * row + 16 * new + 24 * len(lens), "flops": 0}
    if case["op"] == "pages_fork":
        lens, c = _lens(case, case["parents"]), case["children"]
        copied = sum(n % page for n in lens) * c * case["layers"]
        return {"bytes": 2 * copied * row + sum(_pages(n, page) for n in lens) * (8 + 8 * c), "flops": 0}
    used = _compact_used(case)
    movers = sum(used[sum(used):])
    return {"bytes": 2 * movers * page * row * case["layers"] + 16 * len(used), "flops": 0}


# --------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    if case["op"].startswith("pages"):
        return None                                        # values are moved, none is computed
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _norm_exact(s)
    out = torch.zeros(s.q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s.q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    group = s.q.shape[1] // (s.k.shape[1] if s.op == "prompt" else s.k.shape[2])
    if s.op == "prompt":
        a, b = s.starts_q.tolist(), s.starts_k.tolist()
        jobs = [(range(a[i], a[i + 1]), s.k[b[i]:b[i + 1]], s.v[b[i]:b[i + 1]]) for i in range(len(a) - 1)]
    else:
        jobs = []
        for i, row in enumerate(s.seqs.tolist()):
            n = int(s.lens[row])
            at = s.table[row][: _pages(n, s.k.shape[3])].long()
            flat = [x[0][at].permute(0, 2, 1, 3).reshape(-1, x.shape[2], x.shape[4])[:n] for x in (s.k, s.v)]
            jobs.append((range(i, i + 1), *flat))
    for rows, k, v in jobs:
        if not len(rows) or not len(k):
            continue
        i = torch.arange(len(rows), device="cuda")[:, None] + (len(k) - len(rows))
        j = torch.arange(len(k), device="cuda")[None]
        hidden = (j > i) | ((j <= i - s.window) if s.window else torch.zeros_like(j, dtype=torch.bool))
        for h in range(s.q.shape[1]):
            q = s.q[rows.start:rows.stop, h].double()
            x = (q @ k[:, h // group].double().T).mul_(s.scale).masked_fill_(hidden, -math.inf)
            z = torch.logsumexp(x, -1)
            lse[rows.start:rows.stop, h] = z
            x = x.sub_(torch.where(z == -math.inf, torch.zeros_like(z), z)[:, None]).exp_()
            out[rows.start:rows.stop, h] = x @ v[:, h // group].double()
    return {"out": out, "lse": lse}


def _norm_exact(s):
    b, x = s.block.double(), s.x.double()
    if s.post is not None:
        b = b / (b.pow(2).sum(-1, keepdim=True) / b.shape[-1] + EPS).sqrt() * s.post.double()
    gate = 1.0 if s.gate is None else s.gate.double()
    x = x + s.scale * (gate * b)
    y = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * s.pre.double()
    return {"x": x, "y": y}
