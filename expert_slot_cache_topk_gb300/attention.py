"""The attention half of a decoder layer: norms around a block, a paged
key-value cache, attention of one new token over it, and attention over packed
prompts (include/moe_attn.h).

Argument checks and marshalling; the work runs in the library's CUDA kernels on
the caller's stream (``stream=None`` is the legacy default stream, as elsewhere
in this package).  Tensors are torch tensors on one CUDA device, bf16 or f32;
nothing is allocated in a call except where its docstring says so.
"""

from __future__ import annotations

import ctypes as C
from typing import Optional

import torch

from . import _abi

_DTYPE = {torch.bfloat16: _abi.MOE_BF16, torch.float32: _abi.MOE_F32}
_byref = C.byref


# The checks run at every call, next to kernels of a few microseconds: they read
# each attribute once and build their messages only when they refuse.

def _hidden_type(t: torch.Tensor) -> int:
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise TypeError(f"expected a bfloat16 or float32 tensor, got {t.dtype}")
    return code


def _wrong_kind(t, ref, what):
    raise TypeError(f"{what} must be a {ref.dtype} tensor on {ref.device}, got {t.dtype} on {t.device}")


def _rows(t, x, dtype, device, shape, what):
    """(address, row distance) of a tensor with x's type, place and shape and contiguous rows."""
    if t.dtype is not dtype or t.get_device() != device:
        _wrong_kind(t, x, what)
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {list(shape)}, got {list(t.shape)}")
    row, col = t.stride()
    if col != 1 and shape[1] > 1:
        raise ValueError(f"{what}: rows must be contiguous")
    return t.data_ptr(), row


def _vector(t, x, dtype, device, n, what):
    """Address of a contiguous vector of n entries with x's type and place."""
    if t.dtype is not dtype or t.get_device() != device:
        _wrong_kind(t, x, what)
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride()[0] != 1):
        raise ValueError(f"{what} must be a contiguous vector of {n} entries")
    return t.data_ptr()


def _ints(t: torch.Tensor, n: Optional[int], device: int, what: str) -> int:
    """Address of a contiguous int32 vector of n entries."""
    if t.dtype is not torch.int32 or t.get_device() != device or t.dim() != 1 or (n is not None and t.shape[0] != n):
        raise TypeError(f"{what} must be an int32 vector" + ("" if n is None else f" of {n} entries")
                        + f" on device {device}")
    if t.stride()[0] != 1 and t.shape[0] > 1:
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _heads(t, ref, dtype, device, shape, what: str):
    """(address, token distance, head distance) of a [tokens, heads, head_dim] tensor of ref's type and place."""
    if t.dtype is not dtype or t.get_device() != device:
        _wrong_kind(t, ref, what)
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {list(shape)}, got {list(t.shape)}")
    token, head, dim = t.stride()
    if dim != 1 and shape[2] != 1:
        raise ValueError(f"{what}: the head dimension must be contiguous")
    return t.data_ptr(), token, head


def _lse(lse: Optional[torch.Tensor], n: int, heads: int, device: int) -> Optional[int]:
    if lse is None:
        return None
    if lse.dtype is not torch.float32 or lse.get_device() != device or lse.shape != (n, heads) or \
            not lse.is_contiguous():
        raise TypeError(f"lse must be a contiguous float32 tensor [{n}, {heads}] on device {device}")
    return lse.data_ptr()


def norm_residual(x, block=None, pre_weight=None, x_out=None, y=None, post_weight=None, gate=None, res_scale=1.0,
                  eps=1e-6, stream=None):
    """The join between a block and the next one, per token (row):

        n = norm(block) * post_weight        (n = block without post_weight)
        x_out = x + res_scale * gate * n     (x_out = x without a block)
        y = norm(x_out) * pre_weight         with norm(v) = v / sqrt(mean(v^2) + eps)

    x, block, x_out, y: [tokens, hidden] with contiguous rows; x_out or y may be
    None, and may be x or block themselves.  gate: None, [tokens, 1] (one per
    token), [1, hidden] or [hidden] (one per channel), or [tokens, hidden].
    """
    code = _hidden_type(x)
    dtype, device, shape = x.dtype, x.get_device(), x.shape
    if device < 0:
        raise TypeError("x must be a CUDA tensor")
    if len(shape) != 2:
        raise ValueError("x must have shape [tokens, hidden]")
    T, H = shape
    xp, x_row = _rows(x, x, dtype, device, shape, "x")
    b = xo = yo = pw = w = g = None
    b_row = xo_row = yo_row = g_row = g_col = 0
    if block is not None:
        b, b_row = _rows(block, x, dtype, device, shape, "block")
    if x_out is not None:
        xo, xo_row = _rows(x_out, x, dtype, device, shape, "x_out")
    if y is not None:
        yo, yo_row = _rows(y, x, dtype, device, shape, "y")
    if post_weight is not None:
        pw = _vector(post_weight, x, dtype, device, H, "post_weight")
    if pre_weight is not None:
        w = _vector(pre_weight, x, dtype, device, H, "pre_weight")
    if gate is not None:
        if gate.dtype is not dtype or gate.get_device() != device:
            _wrong_kind(gate, x, "gate")
        gs = gate.shape
        if len(gs) == 1:
            gate, gs = gate[None], (1, gs[0])
        if len(gs) != 2 or gs[0] not in (1, T) or gs[1] not in (1, H):
            raise ValueError(f"gate must broadcast to {[T, H]}")
        g_row, col = gate.stride()
        if gs[0] == 1:
            g_row = 0
        if gs[1] > 1:
            g_col = 1
            if col != 1:
                raise ValueError("gate rows must be contiguous")
        g = gate.data_ptr()
    a = _abi.moe_norm_args(code, H, T, xp, b, pw, g, w, xo, yo, x_row, b_row, g_row, xo_row, yo_row, g_col, res_scale, eps)
    _abi._check(_abi.lib().moe_norm_residual(_byref(a), _abi._stream(stream)))


def attn_prompt(q, k, v, starts_q, starts_k, out, scale=None, window=0, lse=None, stream=None):
    """Causal attention over packed prompts.

    q, out: [q_tokens, heads, head_dim]; k, v: [k_tokens, kv_heads, head_dim]
    (any distances between tokens and heads, head_dim contiguous); heads a
    multiple of kv_heads.  Sequence i has queries starts_q[i] : starts_q[i + 1]
    and keys starts_k[i] : starts_k[i + 1] (int32, on the device); its last keys
    are those of its queries, so query r of lq sees keys j <= r + lk - lq, and
    with window > 0 only the last `window` of them.  scale defaults to
    head_dim ** -0.5.  lse: float32 [q_tokens, heads] or None.  A query that sees
    nothing gives zeros and lse = -inf.
    """
    code = _hidden_type(q)
    dtype, device, qs, ks = q.dtype, q.get_device(), q.shape, k.shape
    if device < 0:
        raise TypeError("q must be a CUDA tensor")
    if len(qs) != 3 or len(ks) != 3:
        raise ValueError("q, k and v must have shape [tokens, heads, head_dim]")
    Tq, Hq, D = qs
    Tk, Hkv, _ = ks
    qp, q_token, q_head = _heads(q, q, dtype, device, qs, "q")
    kp, k_token, k_head = _heads(k, q, dtype, device, (Tk, Hkv, D), "k")
    vp, v_token, v_head = _heads(v, q, dtype, device, ks, "v")
    op, o_token, o_head = _heads(out, q, dtype, device, qs, "out")
    n = starts_q.shape[0] - 1 if starts_q.dim() else -1
    if n < 0:
        raise ValueError("starts_q and starts_k need at least one entry")
    a = _abi.moe_prompt_args(code, Hq, Hkv, D, n, Tq, Tk, _ints(starts_q, n + 1, device, "starts_q"),
                             _ints(starts_k, n + 1, device, "starts_k"), qp, kp, vp, op,
                             _lse(lse, Tq, Hq, device), q_token, q_head, k_token, k_head, v_token, v_head,
                             o_token, o_head, D ** -0.5 if scale is None else scale, window)
    _abi._check(_abi.lib().moe_attn_prompt(_byref(a), _abi._stream(stream)))


class KVPages:
    """A paged key-value cache over tensors that the caller owns.

    k, v: [layers, num_pages, kv_heads, page_tokens, head_dim], contiguous;
    table: int32 [max_seqs, max_pages], -1 where a sequence has no page; lens:
    int32 [max_seqs] tokens held; refs: int32 [num_pages] table entries that name
    each page (0 = free).  Token t of sequence s is at offset t % page_tokens of
    page table[s, t // page_tokens] in every layer.  The calls update table, lens
    and refs on the device, in stream order, without reading anything back.

    One workspace is allocated here (sized for at most `max_heads` query heads);
    calls on one cache share it and must not overlap.
    """

    def __init__(self, k, v, table, lens, refs, max_heads: Optional[int] = None):
        code = _hidden_type(k)
        if v.dtype is not k.dtype or v.device != k.device:
            _wrong_kind(v, k, "v")
        if k.dim() != 5 or v.shape != k.shape or not k.is_contiguous() or not v.is_contiguous():
            raise ValueError("k and v must be contiguous [layers, num_pages, kv_heads, page_tokens, head_dim]")
        if not k.is_cuda:
            raise TypeError("k and v must be CUDA tensors")
        if table.dtype != torch.int32 or table.device != k.device or table.dim() != 2 or not table.is_contiguous():
            raise TypeError(f"table must be a contiguous int32 tensor [max_seqs, max_pages] on {k.device}")
        layers, pages, kv_heads, page, dim = k.shape
        seqs, columns = table.shape
        self.k, self.v, self.table, self.lens, self.refs = k, v, table, lens, refs
        self.device = k.device
        self._dev, self._dtype = k.get_device(), k.dtype
        self.kv_heads, self.head_dim, self.max_seqs, self.num_pages = kv_heads, dim, seqs, pages
        self.status = torch.zeros(1, dtype=torch.int32, device=k.device)
        self._kv = _abi.moe_kv_pages(code, layers, kv_heads, dim, page, pages, seqs, columns, k.data_ptr(), v.data_ptr(),
                                     table.data_ptr(), _ints(lens, seqs, self._dev, "lens"),
                                     _ints(refs, pages, self._dev, "refs"), self.status.data_ptr(), None, 0)
        self.max_heads = 64 * kv_heads if max_heads is None else max_heads
        need = C.c_size_t()
        _abi._check(_abi.lib().moe_kv_work_bytes(_byref(self._kv), self.max_heads, _byref(need)))
        self._work = torch.zeros(need.value, dtype=torch.uint8, device=k.device)
        self._kv.work_d, self._kv.work_bytes = self._work.data_ptr(), need.value
        torch.cuda.current_stream(k.device).synchronize()     # the zeros are there for any stream
        self._ref = _byref(self._kv)

    @classmethod
    def empty(cls, layers, kv_heads, head_dim, page_tokens, num_pages, max_seqs, max_pages, dtype=torch.bfloat16,
              device="cuda", max_heads=None) -> "KVPages":
        """A cache with new, empty tensors."""
        shape = (layers, num_pages, kv_heads, page_tokens, head_dim)
        ints = dict(dtype=torch.int32, device=device)
        return cls(torch.empty(shape, dtype=dtype, device=device), torch.empty(shape, dtype=dtype, device=device),
                   torch.full((max_seqs, max_pages), -1, **ints), torch.zeros(max_seqs, **ints),
                   torch.zeros(num_pages, **ints), max_heads)

    def _list(self, t, what, n=None) -> int:
        return _ints(t, n, self._dev, what)

    def reserve(self, seqs, counts, stream=None):
        """Room for counts[i] more tokens in sequence seqs[i] (distinct rows).  New pages are the lowest free
        ones, in list order; a shared, partly filled last page becomes a private copy first."""
        n = seqs.shape[0]
        _abi._check(_abi.lib().moe_kv_reserve(self._ref, self._list(seqs, "seqs"), self._list(counts, "counts", n), n,
                                              _abi._stream(stream)))

    def append(self, layer, seqs, starts, k, v, stream=None):
        """Write one layer's keys and values of the newest tokens: rows starts[i] : starts[i + 1] of k and v
        [tokens, kv_heads, head_dim] are the last tokens of sequence seqs[i] (room was reserved for them)."""
        n, T = seqs.shape[0], k.shape[0]
        shape = (T, self.kv_heads, self.head_dim)
        kp, kt, kh = _heads(k, self.k, self._dtype, self._dev, shape, "k")
        vp, vt, vh = _heads(v, self.k, self._dtype, self._dev, shape, "v")
        _abi._check(_abi.lib().moe_kv_append(self._ref, layer, self._list(seqs, "seqs"),
                                             self._list(starts, "starts", n + 1), n, kp, kt, kh, vp, vt, vh, T,
                                             _abi._stream(stream)))

    def truncate(self, seqs, lens, stream=None):
        """Keep the first min(held, lens[i]) tokens of sequence seqs[i]; release the pages past them."""
        n = seqs.shape[0]
        _abi._check(_abi.lib().moe_kv_truncate(self._ref, self._list(seqs, "seqs"), self._list(lens, "lens", n), n,
                                               _abi._stream(stream)))

    def free(self, seqs, stream=None):
        """Release everything that the listed sequences hold."""
        _abi._check(_abi.lib().moe_kv_truncate(self._ref, self._list(seqs, "seqs"), None, seqs.shape[0],
                                               _abi._stream(stream)))

    def fork(self, src, dst, stream=None):
        """Sequence dst[i] becomes a copy of src[i] that shares its pages (dst distinct; all sources are read
        as they were before the call)."""
        n = src.shape[0]
        _abi._check(_abi.lib().moe_kv_fork(self._ref, self._list(src, "src"), self._list(dst, "dst", n), n,
                                           _abi._stream(stream)))

    def copy(self, src_pages, dst_pages, stream=None):
        """Copy whole pages dst_pages[i] <- src_pages[i] in every layer; table and counts stay."""
        n = src_pages.shape[0]
        _abi._check(_abi.lib().moe_kv_copy(self._ref, self._list(src_pages, "src_pages"),
                                           self._list(dst_pages, "dst_pages", n), n, _abi._stream(stream)))

    def compact(self, table_out=None, refs_out=None, used=None, stream=None):
        """Move the used pages to the front of the pool.  The table and counts that hold afterwards go to
        table_out and refs_out (None: in place); used (int32 [1]) receives the number of used pages."""
        table_out = self.table if table_out is None else table_out
        refs_out = self.refs if refs_out is None else refs_out
        if table_out.dtype != torch.int32 or table_out.shape != self.table.shape or \
                table_out.device != self.device or not table_out.is_contiguous():
            raise TypeError("table_out must be an int32 tensor like the cache's table")
        _abi._check(_abi.lib().moe_kv_compact(self._ref, table_out.data_ptr(),
                                              self._list(refs_out, "refs_out", self.num_pages),
                                              None if used is None else self._list(used, "used", 1),
                                              _abi._stream(stream)))

    def attend(self, layer, q, seqs, out, scale=None, window=0, lse=None, stream=None):
        """Attention of one new token per sequence: q, out [n, heads, head_dim]; row i reads sequence seqs[i]
        (rows may repeat), its last `window` tokens if window > 0.  scale defaults to head_dim ** -0.5.
        lse: float32 [n, heads] or None.  A sequence without tokens gives zeros and lse = -inf."""
        if q.dim() != 3:
            raise ValueError("q must have shape [n, heads, head_dim]")
        n, heads, _ = q.shape
        shape = (n, heads, self.head_dim)
        qp, qt, qh = _heads(q, self.k, self._dtype, self._dev, shape, "q")
        op, ot, oh = _heads(out, self.k, self._dtype, self._dev, shape, "out")
        _abi._check(_abi.lib().moe_attn_decode(self._ref, layer, qp, qt, qh, self._list(seqs, "seqs", n), n, heads,
                                               self.head_dim ** -0.5 if scale is None else scale, window, op, ot, oh,
                                               _lse(lse, n, heads, self._dev), _abi._stream(stream)))

    def check(self, stream=None):
        """Synchronise the stream; raise MoeError (MOE_ESTATE) if a call was refused on the device since the
        status was last zeroed."""
        _abi._check(_abi.lib().moe_kv_check(self._ref, _abi._stream(stream)))
