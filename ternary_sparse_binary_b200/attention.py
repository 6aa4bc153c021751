"""Rotary positions, the paged KV cache and attention on torch tensors (argument marshalling only).

Activations are 2-D tensors [tokens, heads * head_dim] whose last stride is 1
(a slice of a wider tensor keeps its row stride); index arrays are int32
tensors on the same device.  Calls go to the given stream, or to the current
one of the tensors' device, and nothing here synchronises.  A call that needs
scratch takes it from torch's allocator on its stream unless it is given `ws`
(a contiguous uint8 tensor of the size that the matching *_workspace_bytes
gives, 512 where there is none), which then also receives what `status()`
reads: whether an index value was out of range, or a device wait gave up.
Without `ws` such values are handled the same way, unrecorded; the rows that a
wait leaves without a result are NaN either way.  One `ws` serves one call at a
time.
"""
import contextlib
import math

import torch

from . import _abi
from ._abi import wal_head_norm, wal_kv_cache, wal_rope_plan

_LAYOUTS = {"half": _abi.WAL_ROPE_HALF, "interleaved": _abi.WAL_ROPE_INTERLEAVED}
_SCALINGS = {"none": _abi.WAL_SCALING_NONE, "linear": _abi.WAL_SCALING_LINEAR, "parts": _abi.WAL_SCALING_PARTS}
_KV_TYPES = {torch.bfloat16: _abi.WAL_KV_BF16, torch.int8: _abi.WAL_KV_INT8, torch.float8_e4m3fn: _abi.WAL_KV_E4M3}
_X_TYPES = {torch.float32: _abi.WAL_F32, torch.bfloat16: _abi.WAL_BF16}
_BF16 = {torch.bfloat16: _abi.WAL_BF16}
_HERE = contextlib.nullcontext()
_INT = 2 ** 31 - 1


def _fits(value, what):
    """ctypes would pass the low 32 bits of a larger number on."""
    if value > _INT:
        raise ValueError(f"{what}: {value} does not fit (strides, sizes and bounds are below 2^31)")
    return value


def _rows(x, what, dtypes=_X_TYPES):
    """(type, row stride, rows, columns) of an activation tensor."""
    kind = dtypes.get(x.dtype)
    if kind is None or x.dim() != 2:
        raise ValueError(f"{what}: a 2-D tensor of {' or '.join(str(d) for d in dtypes)}")
    rows, cols = x.shape
    ld, one = x.stride()
    if one != 1 and cols > 1:
        raise ValueError(f"{what}: the last stride must be 1")
    # a one-row (or empty) tensor's row stride is arbitrary; its width serves
    return kind, _fits(ld if rows > 1 else cols, what), rows, cols


def _index(x, what, n=None):
    if x.dtype != torch.int32 or x.dim() != 1 or not x.is_contiguous() or (n is not None and x.numel() != n):
        raise ValueError(f"{what}: a contiguous int32 vector" + (f" of {n}" if n is not None else ""))
    return x.data_ptr()


def _table(x, B, most, page_size):
    if x.dtype != torch.int32 or x.dim() != 2 or x.shape[0] != B or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError(f"table: int32 [{B}, pages] with last stride 1")
    # the library sees the row stride alone, which in a slice of a wider table says nothing of its columns
    if x.shape[1] * page_size < most:
        raise ValueError(f"table: {x.shape[1]} pages of {page_size} do not cover {most} tokens")
    return x.data_ptr(), _fits(x.stride(0) if B > 1 else x.shape[1], "table")


def _enter(stream, *tensors):
    """(guard, stream handle) of a call whose tensors must share a CUDA device."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != dev or dev < 0:
            raise ValueError("the tensors of a call must be on one CUDA device")
    guard = _HERE if torch.cuda.current_device() == dev else torch.cuda.device(dev)
    return guard, (torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)


def _ws(ws, like):
    if ws is None:
        return None, 0
    if ws.dtype != torch.uint8 or not ws.is_contiguous() or ws.get_device() != like.get_device():
        raise ValueError("ws: a contiguous uint8 tensor on the device of the others")
    return ws.data_ptr(), ws.numel()


def _scratch(n, like, stream):
    with _HERE if stream is None else torch.cuda.stream(stream):
        return torch.empty(n, dtype=torch.uint8, device=like.device)


def _window(window, sinks):
    """A windowed call's arguments; none without a window, where the first keys are seen as all others are."""
    if sinks < 0 or (window is not None and window < 1):
        raise ValueError("window must be at least 1 and sinks at least 0")
    return () if window is None else (min(window, _INT), min(sinks, _INT))  # beyond any sequence either way


def status(ws, stream=None):
    """Raise WalError if the last call that was given this workspace recorded one (synchronises the stream)."""
    if _ws(ws, ws)[1] < 512:
        raise ValueError("ws: at least 512 bytes")
    guard, s = _enter(stream, ws)
    with guard:
        _abi.wal_device_status(ws.data_ptr(), s)


class Rope:
    """Frequencies of rotary positions on a CUDA device plus their wal_rope_plan descriptor."""

    def __init__(self, head_dim, rot_dim=None, base=10000.0, layout="half", scaling="none", factor=1.0,
                 original_len=0.0, slow=1.0, fast=32.0, device="cuda"):
        self.head_dim, self.rot_dim = head_dim, head_dim if rot_dim is None else rot_dim
        freq = torch.empty(max(self.rot_dim // 2, 1), dtype=torch.int64)
        mscale = _abi.wal_rope_freqs(self.rot_dim, base, _SCALINGS[scaling], factor, original_len, slow, fast,
                                     freq.data_ptr())
        self.freq = freq.to(device)
        self.desc = wal_rope_plan(head_dim, self.rot_dim, _LAYOUTS[layout], mscale, self.freq.data_ptr())

    def apply(self, x, positions, out, stream=None):
        """out (bf16) = x (fp32 or bf16) rotated, [tokens, heads * head_dim]; out may be x itself."""
        xt, ldx, T, width = _rows(x, "x")
        _, ldo, *shape = _rows(out, "out", _BF16)
        if shape != [T, width] or width % self.head_dim:
            raise ValueError("x and out: [tokens, heads * head_dim]")
        guard, s = _enter(stream, x, positions, out, self.freq)
        with guard:
            _abi.wal_rope(self.desc, x.data_ptr(), xt, T, width // self.head_dim, ldx,
                          _index(positions, "positions", T), out.data_ptr(), ldo, s)

    def apply_qk(self, q, k, positions, q_out, k_out, norm=None, stream=None):
        """q_out and k_out (bf16) = q and k (fp32 or bf16), each head normalised by `norm` (a HeadNorm) and
        rotated, [tokens, heads * head_dim]; a bf16 input may be its own output."""
        xt, ldq, T, wq = _rows(q, "q")
        kt, ldk, Tk, wk = _rows(k, "k")
        _, ldyq, *q_shape = _rows(q_out, "q_out", _BF16)
        _, ldyk, *k_shape = _rows(k_out, "k_out", _BF16)
        if kt != xt or Tk != T or q_shape != [T, wq] or k_shape != [T, wk] or wq % self.head_dim or wk % self.head_dim:
            raise ValueError("q and k: [tokens, heads * head_dim] of one type, q_out and k_out of the same shapes")
        guard, s = _enter(stream, q, k, positions, q_out, k_out, self.freq, *_norm(norm))
        with guard:
            _abi.wal_qk_norm_rope(None if norm is None else norm.desc, self.desc, q.data_ptr(), k.data_ptr(), xt, T,
                                  wq // self.head_dim, wk // self.head_dim, ldq, ldk, _index(positions, "positions", T),
                                  q_out.data_ptr(), ldyq, k_out.data_ptr(), ldyk, s)


class HeadNorm:
    """Weights of the q and k heads' norms, [head_dim] of float32 or bfloat16, plus their wal_head_norm descriptor."""

    def __init__(self, q_weight, k_weight, eps=1e-6):
        kind = _X_TYPES.get(q_weight.dtype)
        for w in (q_weight, k_weight):
            if kind is None or w.dtype != q_weight.dtype or w.dim() != 1 or w.shape != q_weight.shape or not w.is_contiguous():
                raise ValueError("q_weight and k_weight: contiguous vectors [head_dim] of float32 or bfloat16")
        self.q_weight, self.k_weight, self.eps = q_weight, k_weight, eps
        self.desc = wal_head_norm(q_weight.numel(), kind, eps, q_weight.data_ptr(), k_weight.data_ptr())


def _norm(norm):
    return () if norm is None else (norm.q_weight, norm.k_weight)


class KvCache:
    """A paged KV cache: k and v [pages, heads, page_size, head_dim] (bf16,
    int8 or float8_e4m3fn) and, for the 8-bit types, fp32 scales [pages, heads,
    page_size], with their wal_kv_cache descriptor."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.dtype not in _KV_TYPES:
            raise ValueError("k and v: [pages, heads, page_size, head_dim] of bfloat16, int8 or float8_e4m3fn")
        scales = [] if k.dtype == torch.bfloat16 else [k_scale, v_scale]
        for s in scales:
            if s is None or s.shape != k.shape[:3] or s.dtype != torch.float32:
                raise ValueError("k_scale and v_scale: float32 [pages, heads, page_size]")
        if not all(t.is_contiguous() and t.device == k.device for t in [k, v, *scales]):
            raise ValueError("the cache's tensors must be contiguous and on one device")
        self.k, self.v = k, v
        self.k_scale, self.v_scale = scales if scales else (None, None)
        self.n_pages, self.n_heads, self.page_size, self.head_dim = k.shape
        self._scratch = {}  # workspace sizes of recent shapes
        self.desc = wal_kv_cache(self.n_pages, self.page_size, self.n_heads, self.head_dim, _KV_TYPES[k.dtype],
                                 k.data_ptr(), v.data_ptr(), *[s.data_ptr() for s in scales])

    @classmethod
    def empty(cls, n_pages, page_size, n_heads, head_dim, dtype=torch.bfloat16, device="cuda"):
        _abi.wal_kv_cache_sizes(n_pages, page_size, n_heads, head_dim, _KV_TYPES[dtype])
        shape = (n_pages, n_heads, page_size, head_dim)
        new = [torch.empty(shape, dtype=dtype, device=device) for _ in range(2)]
        if dtype != torch.bfloat16:
            new += [torch.empty(shape[:3], dtype=torch.float32, device=device) for _ in range(2)]
        return cls(*new)

    @property
    def nbytes(self):
        return sum(t.numel() * t.element_size() for t in (self.k, self.v, self.k_scale, self.v_scale) if t is not None)

    def append(self, k, v, slots, positions=None, rope=None, ws=None, stream=None):
        """Store the rows of k and v [tokens, heads * head_dim] (fp32 or bf16) in `slots`
        (page * page_size + offset; -1 skips a row), k rotated by `rope` at `positions` first."""
        kt, ldk, T, width = _rows(k, "k")
        vt, ldv, *shape = _rows(v, "v")
        if vt != kt or shape != [T, width] or width != self.n_heads * self.head_dim:
            raise ValueError("k and v: [tokens, heads * head_dim] of one type")
        if rope is not None:
            if positions is None:
                raise ValueError("positions are required with a rope")
            guard, s = _enter(stream, self.k, k, v, slots, positions, rope.freq)
        else:
            guard, s = _enter(stream, self.k, k, v, slots)
        wp, wn = _ws(ws, k)
        with guard:
            _abi.wal_kv_append(self.desc, k.data_ptr(), v.data_ptr(), kt, T, ldk, ldv, _index(slots, "slots", T),
                               None if rope is None else _index(positions, "positions", T),
                               None if rope is None else rope.desc, wp, wn, s)

    def append_qkv(self, q, k, v, slots, q_out, positions=None, rope=None, norm=None, ws=None, stream=None):
        """append() of k and v with each head of k normalised by `norm` (a HeadNorm) before its rotation, and
        q_out (bf16) = q [tokens, n_heads * head_dim] with the same done to it, in one launch."""
        xt, ldq, T, wq = _rows(q, "q")
        kt, ldk, *k_shape = _rows(k, "k")
        vt, ldv, *v_shape = _rows(v, "v")
        _, ldy, *q_shape = _rows(q_out, "q_out", _BF16)
        if kt != xt or vt != xt or k_shape != [T, self.n_heads * self.head_dim] or v_shape != k_shape:
            raise ValueError("q, k and v: [tokens, heads * head_dim] of one type")
        if q_shape != [T, wq] or wq % self.head_dim:
            raise ValueError("q and q_out: [tokens, n_heads * head_dim]")
        if rope is not None and positions is None:
            raise ValueError("positions are required with a rope")
        turned = () if rope is None else (positions, rope.freq)
        guard, s = _enter(stream, self.k, q, k, v, slots, q_out, *turned, *_norm(norm))
        wp, wn = _ws(ws, q)
        with guard:
            _abi.wal_qkv_append(self.desc, None if norm is None else norm.desc, None if rope is None else rope.desc,
                                q.data_ptr(), k.data_ptr(), v.data_ptr(), xt, T, wq // self.head_dim, ldq, ldk, ldv,
                                _index(slots, "slots", T), None if rope is None else _index(positions, "positions", T),
                                q_out.data_ptr(), ldy, wp, wn, s)

    def plan(self, n_new, kv_len, table, free, n_free, q_start, positions, slots, kv_len_out=None, n_free_out=None,
             max_kv=None, ws=None, stream=None):
        """The plan of a step in which sequence b gets n_new[b] tokens more (or loses -n_new[b]): its pages go from
        the list `free` [n_pages] of n_free[0] pages to its row of `table`, or back; q_start, and position and slot of
        every row of the step, are written, and the new lengths (in place without kv_len_out and n_free_out).  It
        gives back every page of the tokens that a sequence loses: one that shares pages, or whose pages behind a
        window were taken from it, drops its tokens only down to the last of those; the rest is the caller's."""
        B, T = n_new.numel(), slots.numel()
        most = table.shape[-1] * self.page_size if max_kv is None else _fits(max_kv, "max_kv")
        tp, ldt = _table(table, B, most, self.page_size)
        kv_len_out = kv_len if kv_len_out is None else kv_len_out
        n_free_out = n_free if n_free_out is None else n_free_out
        guard, s = _enter(stream, self.k, n_new, kv_len, table, free, n_free, q_start, positions, slots, kv_len_out, n_free_out)
        wp, wn = _ws(ws, slots)
        with guard:
            _abi.wal_kv_plan(self.desc, _index(n_new, "n_new"), _index(kv_len, "kv_len", B), B, tp, ldt, min(most, 2 ** 30),
                             _index(free, "free", self.n_pages), _index(n_free, "n_free", 1), T,
                             _index(q_start, "q_start", B + 1), _index(positions, "positions", T), _index(slots, "slots", T),
                             _index(kv_len_out, "kv_len_out", B), _index(n_free_out, "n_free_out", 1), wp, wn, s)

    def read(self, table, start, k_out, v_out, max_len, ws=None, stream=None):
        """Rows start[b] .. start[b + 1] - 1 of k_out and v_out (fp32 or bf16) = the first tokens of sequence b."""
        B = start.numel() - 1
        _fits(max_len, "max_len")
        kt, ldk, T, width = _rows(k_out, "k_out")
        vt, ldv, *shape = _rows(v_out, "v_out")
        if vt != kt or shape != [T, width] or width != self.n_heads * self.head_dim:
            raise ValueError("k_out and v_out: [rows, heads * head_dim] of one type")
        tp, ldt = _table(table, B, max_len, self.page_size)
        if T == 0 and ws is None:
            return
        guard, s = _enter(stream, self.k, table, start, k_out, v_out)
        wp, wn = _ws(ws, k_out)
        with guard:
            _abi.wal_kv_read(self.desc, tp, ldt, _index(start, "start"), B, max_len, k_out.data_ptr(),
                             v_out.data_ptr(), kt, T, ldk, ldv, wp, wn, s)

    def _bytes(self, fn, *shape):
        """Workspace size of a recent shape."""
        n = self._scratch.get((fn, *shape))
        if n is None:
            _fits(max(shape), "workspace size")
            if len(self._scratch) >= 256:
                self._scratch.clear()
            n = self._scratch[(fn, *shape)] = fn(self.desc, *shape)
        return n

    def attend_workspace_bytes(self, n_heads, T, B, max_q, max_kv, window=None, sinks=0):
        """Bytes of a `ws` for attend.  Not monotone: a smaller batch may need more (its keys are split
        further), so one `ws` for several shapes takes the largest of their sizes."""
        seen = _window(window, sinks)
        fn = _abi.wal_attn_paged_window_workspace_bytes if seen else _abi.wal_attn_paged_workspace_bytes
        return self._bytes(fn, n_heads, T, B, max_q, max_kv, *seen)

    def attend(self, q, q_start, kv_len, table, out, max_q, max_kv, scale=None, ws=None, stream=None, window=None, sinks=0):
        """out (bf16) = attention of the new tokens' q (bf16) [tokens, n_heads * head_dim] over the cache;
        rows q_start[b] .. q_start[b + 1] - 1 are the last tokens of sequence b's kv_len[b].  With a
        `window`, a token sees that many keys up to its own, and the first `sinks` of its sequence; without
        one it sees all, and `sinks` changes nothing."""
        ldq, ldo, T, n_heads = self._tokens(q, out)
        B = kv_len.numel()
        _fits(max(max_q, max_kv), "bounds")
        seen = _window(window, sinks)
        tp, ldt = _table(table, B, max_kv, self.page_size)
        guard, s = _enter(stream, self.k, q, q_start, kv_len, table, out)
        if ws is None:
            n = self.attend_workspace_bytes(n_heads, T, B, max_q, max_kv, window, sinks)  # 0: the call below says what is wrong
            ws = _scratch(n, q, stream) if n > 512 else None
        wp, wn = _ws(ws, q)
        call = _abi.wal_attn_paged if window is None else _abi.wal_attn_paged_window
        with guard:
            call(self.desc, q.data_ptr(), n_heads, T, ldq, _index(q_start, "q_start", B + 1), _index(kv_len, "kv_len"), tp, ldt,
                 B, max_q, max_kv, *seen, self.head_dim ** -0.5 if scale is None else scale, out.data_ptr(), ldo, wp, wn, s)

    def attend_shared_workspace_bytes(self, n_heads, T, B, G, max_q, max_prefix, max_own):
        """Bytes of a `ws` for attend_shared; not monotone, as attend's."""
        return self._bytes(_abi.wal_attn_paged_shared_workspace_bytes, n_heads, T, B, G, max_q, max_prefix, max_own)

    def attend_shared(self, q, q_start, kv_len, table, group_start, prefix_len, out, max_q, max_kv, max_prefix, max_own,
                      scale=None, ws=None, stream=None):
        """attend() of sequences that share their first tokens: group g is the sequences group_start[g] ..
        group_start[g + 1] - 1, whose first prefix_len[g] tokens (at most max_prefix, which is at most max_kv) are
        read once, from the pages of the first of them; max_own bounds the tokens behind."""
        ldq, ldo, T, n_heads = self._tokens(q, out)
        B, G = kv_len.numel(), prefix_len.numel()
        _fits(max(max_q, max_kv, max_prefix, max_own), "bounds")
        tp, ldt = _table(table, B, max_kv, self.page_size)
        guard, s = _enter(stream, self.k, q, q_start, kv_len, table, group_start, prefix_len, out)
        if ws is None:
            n = self.attend_shared_workspace_bytes(n_heads, T, B, G, max_q, max_prefix, max_own)
            ws = _scratch(n, q, stream) if n > 512 else None
        wp, wn = _ws(ws, q)
        with guard:
            _abi.wal_attn_paged_shared(self.desc, q.data_ptr(), n_heads, T, ldq, _index(q_start, "q_start", B + 1),
                                       _index(kv_len, "kv_len"), tp, ldt, B, _index(group_start, "group_start", G + 1),
                                       _index(prefix_len, "prefix_len"), G, max_q, max_kv, max_prefix, max_own,
                                       self.head_dim ** -0.5 if scale is None else scale, out.data_ptr(), ldo, wp, wn, s)

    def _tokens(self, q, out):
        """(row strides of q and out, tokens, q heads)"""
        _, ldq, T, width = _rows(q, "q", _BF16)
        _, ldo, *shape = _rows(out, "out", _BF16)
        if shape != [T, width] or width % self.head_dim:
            raise ValueError("q and out: [tokens, n_heads * head_dim]")
        return ldq, ldo, T, width // self.head_dim


def attn_prompt(q, k, v, start, out, head_dim, max_len, scale=None, ws=None, stream=None, window=None, sinks=0):
    """out (bf16) = causal attention over packed prompts; q and out [tokens, n_heads * head_dim],
    k and v [tokens, n_kv_heads * head_dim], sequence b in rows start[b] .. start[b + 1] - 1.  With a
    `window`, a token sees that many keys up to its own, and the first `sinks` of its sequence; without one
    it sees all, and `sinks` changes nothing."""
    _, ldq, T, width = _rows(q, "q", _BF16)
    _, ldk, *k_shape = _rows(k, "k", _BF16)
    _, ldv, *v_shape = _rows(v, "v", _BF16)
    _, ldo, *shape = _rows(out, "out", _BF16)
    if shape != [T, width] or k_shape != v_shape or k_shape[0] != T or width % head_dim or k_shape[1] % head_dim:
        raise ValueError("q and out: [tokens, n_heads * head_dim]; k and v: [tokens, n_kv_heads * head_dim]")
    _fits(max_len, "max_len")
    seen = _window(window, sinks)
    guard, s = _enter(stream, q, k, v, start, out)
    wp, wn = _ws(ws, q)
    call = _abi.wal_attn_prompt if window is None else _abi.wal_attn_prompt_window
    with guard:
        call(q.data_ptr(), k.data_ptr(), v.data_ptr(), width // head_dim, k_shape[1] // head_dim, head_dim, T, ldq, ldk, ldv,
             _index(start, "start"), start.numel() - 1, max_len, *seen, 1.0 / math.sqrt(head_dim) if scale is None else scale,
             out.data_ptr(), ldo, wp, wn, s)
