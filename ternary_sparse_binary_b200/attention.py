"""Rotary positions, the paged KV cache and attention on torch tensors (argument marshalling only).

Activations are 2-D tensors [tokens, heads * head_dim] whose last stride is 1
(a slice of a wider tensor keeps its row stride); index arrays are int32
tensors on the same device.  Calls go to the given stream, or to the current
one of the tensors' device.  Without `ws` each call takes a workspace of its
own from torch's allocator on that stream; a caller that passes one keeps it
free until the call has finished, and `status()` then reads what was recorded
in it.  Nothing here synchronises.
"""
import math

import torch

from . import _abi
from ._abi import wal_kv_cache, wal_rope_plan

_LAYOUTS = {"half": _abi.WAL_ROPE_HALF, "interleaved": _abi.WAL_ROPE_INTERLEAVED}
_SCALINGS = {"none": _abi.WAL_SCALING_NONE, "linear": _abi.WAL_SCALING_LINEAR, "parts": _abi.WAL_SCALING_PARTS}
_KV_TYPES = {torch.bfloat16: _abi.WAL_KV_BF16, torch.int8: _abi.WAL_KV_INT8, torch.float8_e4m3fn: _abi.WAL_KV_E4M3}
_X_TYPES = {torch.float32: _abi.WAL_F32, torch.bfloat16: _abi.WAL_BF16}


def _rows(x, what, dtypes=_X_TYPES):
    if x.dim() != 2 or x.dtype not in dtypes or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError(f"{what}: a 2-D tensor of {' or '.join(str(d) for d in dtypes)} with last stride 1")
    # a one-row (or empty) tensor's row stride is arbitrary; its width serves
    return x.stride(0) if x.shape[0] > 1 else x.shape[1]


def _index(x, what, n=None):
    if x.dtype != torch.int32 or x.dim() != 1 or not x.is_contiguous() or (n is not None and x.numel() != n):
        raise ValueError(f"{what}: a contiguous int32 vector" + (f" of {n}" if n is not None else ""))
    return x.data_ptr()


def _table(x, B):
    if x.dtype != torch.int32 or x.dim() != 2 or x.shape[0] != B or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError(f"table: int32 [{B}, pages] with last stride 1")
    return x.data_ptr(), (x.stride(0) if B > 1 else x.shape[1])


_BF16 = {torch.bfloat16: _abi.WAL_BF16}


class _Call:
    """Device, stream and workspace of one call; the tensors must share a CUDA device."""

    def __init__(self, tensors, stream, ws=None, nbytes=0):
        dev = tensors[0].device
        for t in tensors:
            if t is not None and (t.device != dev or not t.is_cuda):
                raise ValueError("the tensors of a call must be on one CUDA device")
        self.guard = torch.cuda.device(dev)
        s = stream if stream is not None else torch.cuda.current_stream(dev)
        self.stream = s.cuda_stream
        self.ws, self.nbytes = ws, nbytes
        if nbytes and ws is None:
            with torch.cuda.stream(s):
                self.ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        elif nbytes:
            if ws.device != dev or ws.dtype != torch.uint8 or not ws.is_contiguous():
                raise ValueError("ws: a contiguous uint8 tensor on the same device")
            self.nbytes = ws.numel()


def status(ws, stream=None):
    """Raise WalError if the last call that used the workspace recorded one (synchronises the stream)."""
    s = stream if stream is not None else torch.cuda.current_stream(ws.device)
    with torch.cuda.device(ws.device):
        _abi.wal_device_status(ws.data_ptr(), s.cuda_stream)


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
        if x.shape != out.shape or x.shape[1] % self.head_dim:
            raise ValueError("x and out: [tokens, heads * head_dim]")
        T = x.shape[0]
        ldx, ldo = _rows(x, "x"), _rows(out, "out", _BF16)
        call = _Call((x, positions, out, self.freq), stream)
        with call.guard:
            _abi.wal_rope(self.desc, x.data_ptr(), _X_TYPES[x.dtype], T, x.shape[1] // self.head_dim, ldx,
                          _index(positions, "positions", T), out.data_ptr(), ldo, call.stream)


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
        self.desc = wal_kv_cache(*k.shape[:1], self.page_size, self.n_heads, self.head_dim, _KV_TYPES[k.dtype],
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
        T = k.shape[0]
        if k.shape != v.shape or k.dtype != v.dtype or k.shape[1] != self.n_heads * self.head_dim:
            raise ValueError("k and v: [tokens, heads * head_dim] of one type")
        if rope is not None and positions is None:
            raise ValueError("positions are required with a rope")
        ldk, ldv = _rows(k, "k"), _rows(v, "v")
        call = _Call((self.k, k, v, slots, positions, rope.freq if rope is not None else None), stream, ws, 512)
        with call.guard:
            _abi.wal_kv_append(self.desc, k.data_ptr(), v.data_ptr(), _X_TYPES[k.dtype], T, ldk, ldv,
                               _index(slots, "slots", T),
                               None if positions is None else _index(positions, "positions", T),
                               None if rope is None else rope.desc, call.ws.data_ptr(), call.nbytes, call.stream)

    def read(self, table, start, k_out, v_out, max_len, ws=None, stream=None):
        """Rows start[b] .. start[b + 1] - 1 of k_out and v_out (fp32 or bf16) = the first tokens of sequence b."""
        B = start.numel() - 1
        if k_out.shape != v_out.shape or k_out.dtype != v_out.dtype or k_out.shape[1] != self.n_heads * self.head_dim:
            raise ValueError("k_out and v_out: [rows, heads * head_dim] of one type")
        ldk, ldv = _rows(k_out, "k_out"), _rows(v_out, "v_out")
        tp, ldt = _table(table, B)
        if k_out.shape[0] == 0:
            return
        call = _Call((self.k, table, start, k_out, v_out), stream, ws, 512)
        with call.guard:
            _abi.wal_kv_read(self.desc, tp, ldt, _index(start, "start"), B, max_len, k_out.data_ptr(),
                             v_out.data_ptr(), _X_TYPES[k_out.dtype], k_out.shape[0], ldk, ldv, call.ws.data_ptr(),
                             call.nbytes, call.stream)

    def attend_workspace_bytes(self, n_heads, T, B, max_q, max_kv):
        return _abi.wal_attn_paged_workspace_bytes(self.desc, n_heads, T, B, max_q, max_kv)

    def attend(self, q, q_start, kv_len, table, out, max_q, max_kv, scale=None, ws=None, stream=None):
        """out (bf16) = attention of the new tokens' q (bf16) [tokens, n_heads * head_dim] over the cache;
        rows q_start[b] .. q_start[b + 1] - 1 are the last tokens of sequence b's kv_len[b]."""
        T, B = q.shape[0], kv_len.numel()
        if q.shape != out.shape or q.shape[1] % self.head_dim:
            raise ValueError("q and out: [tokens, n_heads * head_dim]")
        n_heads = q.shape[1] // self.head_dim
        ldq, ldo = _rows(q, "q", _BF16), _rows(out, "out", _BF16)
        tp, ldt = _table(table, B)
        nbytes = self.attend_workspace_bytes(n_heads, T, B, max_q, max_kv)  # 0: the call below says what is wrong
        call = _Call((self.k, q, q_start, kv_len, table, out), stream, ws, max(nbytes, 512))
        with call.guard:
            _abi.wal_attn_paged(self.desc, q.data_ptr(), n_heads, T, ldq, _index(q_start, "q_start", B + 1),
                                _index(kv_len, "kv_len"), tp, ldt, B, max_q, max_kv,
                                1.0 / math.sqrt(self.head_dim) if scale is None else scale, out.data_ptr(), ldo,
                                call.ws.data_ptr(), call.nbytes, call.stream)


def attn_prompt(q, k, v, start, out, head_dim, max_len, scale=None, ws=None, stream=None):
    """out (bf16) = causal attention over packed prompts; q and out [tokens, n_heads * head_dim],
    k and v [tokens, n_kv_heads * head_dim], sequence b in rows start[b] .. start[b + 1] - 1."""
    T = q.shape[0]
    if q.shape != out.shape or k.shape != v.shape or k.shape[0] != T or q.shape[1] % head_dim or k.shape[1] % head_dim:
        raise ValueError("q and out: [tokens, n_heads * head_dim]; k and v: [tokens, n_kv_heads * head_dim]")
    ld = [_rows(x, name, _BF16) for x, name in ((q, "q"), (k, "k"), (v, "v"), (out, "out"))]
    call = _Call((q, k, v, start, out), stream, ws, 512)
    with call.guard:
        _abi.wal_attn_prompt(q.data_ptr(), k.data_ptr(), v.data_ptr(), q.shape[1] // head_dim, k.shape[1] // head_dim,
                             head_dim, T, ld[0], ld[1], ld[2], _index(start, "start"), start.numel() - 1, max_len,
                             1.0 / math.sqrt(head_dim) if scale is None else scale, out.data_ptr(), ld[3],
                             call.ws.data_ptr(), call.nbytes, call.stream)
