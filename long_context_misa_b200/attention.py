"""Python binding of the attention side of libmisa (include/misa_attention.h).

Argument marshalling only, as in misa.py: every step runs in the CUDA kernels
of libmisa.so on device memory of the caller, asynchronously on the current
stream (or ``stream``).  A call whose tensors are on another device than the
current one runs on the current stream of theirs.

Typical use (one decode step around MISA-dagger)::

    rope = Rope(64, base=10000.0, layout="interleaved")
    apply_rope(rope, [(index_q, q_pos, index_q), (index_k, q_pos, index_k), (q, q_pos, q)])
    append_kv(kv, new_k, new_v, q_pos, rope=rope)       # rotated, quantised, written
    top = dagger_topk(cache, qs, heads, k_prime, k)     # misa.py
    out = attend(kv, AttentionQueries(q, q_seq, q_pos), topk=top)
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
from typing import Optional, Sequence, Tuple

import torch

from . import misa as _m
from .misa import MISA_KEY_BF16, MISA_KEY_FP8_E4M3, Workspace

HEADER = os.path.join(os.path.dirname(_m.HEADER), "misa_attention.h")
MAX_DRAFT = 1024       # MISA_MAX_DRAFT
MAX_ROPE_GROUPS = 4    # MISA_MAX_ROPE_GROUPS
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_E4M3 = (torch.float8_e4m3fn, torch.uint8)

_P, _I32, _I64, _F64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double


class misa_kv(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P), ("seq_len", _P), ("status", _P),
                ("n_seq", _I32), ("L_cap", _I32), ("H_kv", _I32), ("d", _I32), ("dtype", _I32)]


class misa_rope(ctypes.Structure):
    _fields_ = [("phase", _P), ("rot", _I32), ("first", _I32), ("layout", _I32), ("amplitude", ctypes.c_float)]


class misa_rope_rows(ctypes.Structure):
    _fields_ = [("x", _P), ("y", _P), ("pos", _P), ("x_row", _I64), ("x_head", _I64), ("y_row", _I64),
                ("y_head", _I64), ("n", _I32), ("H", _I32), ("d", _I32)]


class misa_new_kv(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_seq", _I64), ("k_tok", _I64), ("k_head", _I64), ("v_seq", _I64),
                ("v_tok", _I64), ("v_head", _I64)]


class misa_attend_queries(ctypes.Structure):
    _fields_ = [("q", _P), ("q_seq", _P), ("q_pos", _P), ("n_q", _I32), ("H", _I32), ("scale", ctypes.c_float)]


class misa_draft(ctypes.Structure):
    _fields_ = [("start", _P), ("mask", _P), ("n", _I32)]


def _declare(lib):
    p = ctypes.POINTER
    sig = {
        "misa_rope_phases": (_I32, [_P, _I32, _F64, _I32, _F64, _F64, _F64, _F64]),
        "misa_apply_rope": (_I32, [p(misa_rope), p(misa_rope_rows), _I32, _P]),
        "misa_append_kv": (_I32, [p(misa_kv), p(misa_new_kv), _P, _I32, p(misa_rope), _P, _I32, _P]),
        "misa_read_kv": (_I32, [p(misa_kv), _P, _P, _I32, _I32, _P, _P, _P]),
        "misa_attend": (_I32, [p(misa_kv), p(misa_attend_queries), _P, _I32, p(misa_draft), _P, _P, _P,
                               ctypes.c_size_t, _P]),
        "misa_attend_workspace_bytes": (ctypes.c_size_t, [p(misa_kv), p(misa_attend_queries), _I32, _I32]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    return lib


_lib = _declare(_m._lib)


def _need(ok: bool, what: str, kind=ValueError) -> None:
    if not ok:
        raise kind(what)


def _ints(t: torch.Tensor, n: int, what: str, device) -> None:
    """A contiguous int32 tensor of n elements on the device.  (Messages are built only for a refusal: formatting
    them costs more than the checks.)"""
    if t.dtype is not torch.int32:
        raise TypeError(f"{what} must be int32, got {t.dtype}")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous with {n} entries, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, expected {device}")


def _on(t: torch.Tensor, device, what: str) -> None:
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, expected {device}")


def _call(fn, device, stream, *args) -> None:
    """fn(*args, stream) with `device` current; the default is the device's current stream."""
    if device.type != "cuda":
        raise ValueError(f"the tensors are on {device}: the kernels need a CUDA device")
    if device.index == torch._C._cuda_getDevice():
        st = fn(*args, torch._C._cuda_getCurrentRawStream(device.index) if stream is None else _m._stream(stream))
    else:
        with torch.cuda.device(device):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(device.index) if stream is None else _m._stream(stream))
    if st:
        _m._check(st)


_NO_CONTEXT = contextlib.nullcontext()


def _allocating(stream):
    """Where a call runs on a given stream, what it allocates belongs to that stream: its memory is not handed out
    again before the call is done with it."""
    if stream is None:
        return _NO_CONTEXT
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)))
    return torch.cuda.stream(stream)


class Rope:
    """Rotary positions of ``rot`` elements of a row from ``first`` on (see misa_rope).

    layout   "half" or "interleaved"
    scaling  "none", "linear", "ntk" or "yarn" (``factor``, ``orig_len``, ``beta_fast``, ``beta_slow``)
    amplitude of the rotated elements; default 1, with "yarn" 0.1 ln(factor) + 1
    phases   the increments as a host int64 tensor [rot/2] in 2^-64 turns per position, instead of ``base`` and
             ``scaling``
    """

    def __init__(self, rot: int, base: float = 10000.0, layout: str = "half", first: int = 0, scaling: str = "none",
                 factor: float = 1.0, orig_len: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0,
                 amplitude: Optional[float] = None, phases: Optional[torch.Tensor] = None, device="cuda"):
        _need(layout in ROPE_LAYOUTS, f"layout must be one of {sorted(ROPE_LAYOUTS)}, got {layout!r}")
        _need(scaling in ROPE_SCALINGS, f"scaling must be one of {sorted(ROPE_SCALINGS)}, got {scaling!r}")
        _need(int(rot) >= 2 and int(rot) % 2 == 0, f"rot must be even and >= 2, got {rot}")
        if phases is None:
            phases = torch.empty(int(rot) // 2, dtype=torch.int64)
            _m._check(_lib.misa_rope_phases(phases.data_ptr(), int(rot), float(base), ROPE_SCALINGS[scaling],
                                            float(factor), float(orig_len), float(beta_fast), float(beta_slow)))
        _need(phases.dtype == torch.int64 and tuple(phases.shape) == (int(rot) // 2,),
              f"phases must be int64 [{int(rot) // 2}], got {phases.dtype} {tuple(phases.shape)}")
        if amplitude is None:
            amplitude = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" and factor > 1 else 1.0
        self.rot, self.first, self.layout, self.amplitude = int(rot), int(first), layout, float(amplitude)
        self.phases = phases.to(device).contiguous()
        self._s = misa_rope(_m._ptr(self.phases), self.rot, self.first, ROPE_LAYOUTS[layout], self.amplitude)
        self._p = ctypes.byref(self._s)

    @property
    def struct(self) -> misa_rope:
        return self._s


def apply_rope(rope: Rope, rows: Sequence[Tuple[torch.Tensor, torch.Tensor, torch.Tensor]], stream=None) -> None:
    """Rotate up to four tensors in one launch.

    rows: (x, pos, out) triples; x and out are bf16 (or bf16 bits) [n][H][d] with consecutive elements along d and
    any other strides, out may be x itself; pos is int32 [n].  Other rows that meet are refused: those of one out,
    of out and x, of two triples.
    """
    if not 1 <= len(rows) <= MAX_ROPE_GROUPS:
        raise ValueError(f"apply_rope takes 1 to {MAX_ROPE_GROUPS} tensors, got {len(rows)}")
    groups = (misa_rope_rows * len(rows))()
    device = rope.phases.device
    for i, (x, pos, out) in enumerate(rows):
        if x.dtype not in _BF16 or out.dtype is not x.dtype:
            raise TypeError(f"rows must be bf16 and of one type, got {x.dtype} and {out.dtype}")
        shape = x.shape
        if len(shape) != 3 or out.shape != shape:
            raise ValueError(f"rows must be [n][H][d], got {tuple(shape)}, {tuple(out.shape)}")
        n, H, d = shape
        x_row, x_head, x_el = x.stride()
        y_row, y_head, y_el = out.stride()
        if (x_el != 1 or y_el != 1) and d > 1:
            raise ValueError("the elements of a row must be consecutive")
        if x.device != device or out.device != device:
            raise ValueError(f"rows are on {x.device} and {out.device}, the phases on {device}")
        _ints(pos, n, "pos", device)
        groups[i] = (x.data_ptr(), out.data_ptr(), pos.data_ptr(), x_row, x_head, y_row, y_head, n, H, d)
    _call(_lib.misa_apply_rope, device, stream, rope._p, groups, len(rows))


class KVCache:
    """Attention cache of n_seq sequences (device tensors owned by the caller).

    k, v             : bf16 (torch.bfloat16 or its bits) or e4m3 (torch.float8_e4m3fn or uint8 codes),
                       [n_seq][L_cap][H_kv][d], contiguous, d = 64 or 128
    k_scale, v_scale : float32 [n_seq][L_cap][H_kv] for e4m3, else None
    seq_len          : int32 [n_seq]
    status           : int32 [1] device error bits (allocated if None)
    """

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: Optional[torch.Tensor],
                 v_scale: Optional[torch.Tensor], seq_len: torch.Tensor, status: Optional[torch.Tensor] = None):
        _need(k.dim() == 4 and k.shape == v.shape and k.is_contiguous() and v.is_contiguous(),
              f"k and v must be contiguous [n_seq][L_cap][H_kv][d] tensors, got {tuple(k.shape)}, {tuple(v.shape)}")
        if k.dtype not in _BF16 + _E4M3 or v.dtype != k.dtype:
            raise TypeError(f"k and v must both hold bf16 or e4m3, got {k.dtype} and {v.dtype}")
        fp8 = k.dtype in _E4M3
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            _need((s is not None) == fp8, f"{name} must be given exactly for e4m3 caches")
            if s is not None:
                if s.dtype != torch.float32:
                    raise TypeError(f"{name} must be float32, got {s.dtype}")
                _need(s.shape == k.shape[:3] and s.is_contiguous(),
                      f"{name} must be contiguous {tuple(k.shape[:3])}, got {tuple(s.shape)}")
                _on(s, k.device, name)
        _on(v, k.device, "v")
        self.n_seq, self.L_cap, self.H_kv, self.d = (int(x) for x in k.shape)
        _ints(seq_len, self.n_seq, "seq_len", k.device)
        self.k, self.v, self.k_scale, self.v_scale, self.seq_len = k, v, k_scale, v_scale, seq_len
        self.dtype = MISA_KEY_FP8_E4M3 if fp8 else MISA_KEY_BF16
        self.device = k.device
        self._shape = (self.n_seq, self.L_cap, self.H_kv, self.d, self.dtype)
        self.status = status if status is not None else torch.zeros(1, dtype=torch.int32, device=k.device)
        _ints(self.status, 1, "status", k.device)
        self._s = misa_kv(_m._ptr(k), _m._ptr(v), _m._ptr(k_scale), _m._ptr(v_scale), _m._ptr(seq_len),
                          _m._ptr(self.status), self.n_seq, self.L_cap, self.H_kv, self.d, self.dtype)
        self._p = ctypes.byref(self._s)

    @classmethod
    def empty(cls, n_seq: int, L_cap: int, H_kv: int, d: int = 128, e4m3: bool = True, device="cuda") -> "KVCache":
        """An empty cache with its own zeroed tensors."""
        shape = (n_seq, L_cap, H_kv, d)
        kv = [torch.zeros(shape, dtype=torch.uint8 if e4m3 else torch.bfloat16, device=device) for _ in range(2)]
        sc = [torch.zeros(shape[:3], dtype=torch.float32, device=device) if e4m3 else None for _ in range(2)]
        return cls(*kv, *sc, torch.zeros(n_seq, dtype=torch.int32, device=device))

    @property
    def struct(self) -> misa_kv:
        return self._s

    def device_status(self) -> int:
        """MISA_DEV_* bits recorded so far (synchronises)."""
        return int(self.status.item()) & 0xFFFFFFFF


def append_kv(kv: KVCache, new_k: torch.Tensor, new_v: torch.Tensor, new_pos: torch.Tensor,
              rope: Optional[Rope] = None, rope_pos: Optional[torch.Tensor] = None, commit: bool = True,
              stream=None) -> None:
    """Write new_k, new_v (bf16 [n_seq][count][H_kv][d], consecutive along d) at new_pos [n_seq], the keys rotated
    by rope at rope_pos [n_seq][count] (default: the positions written) and quantised to the cache's type.
    new_pos may be kv.seq_len itself: the tokens go behind what is there.
    commit=False leaves seq_len (drafted tokens)."""
    shape = new_k.shape
    if new_k.dtype not in _BF16 or new_v.dtype not in _BF16:
        raise TypeError(f"new_k and new_v must be bf16, got {new_k.dtype} and {new_v.dtype}")
    if len(shape) != 4 or new_v.shape != shape or (shape[0], shape[2], shape[3]) != (kv.n_seq, kv.H_kv, kv.d):
        raise ValueError(f"new_k and new_v must be [{kv.n_seq}][count][{kv.H_kv}][{kv.d}], got {tuple(shape)} and "
                         f"{tuple(new_v.shape)}")
    count, device = shape[1], kv.device
    ks, vs = new_k.stride(), new_v.stride()
    if ks[3] != 1 or vs[3] != 1:
        raise ValueError(f"the elements of a row must be consecutive, got strides {ks} and {vs}")
    if new_k.device != device or new_v.device != device:
        raise ValueError(f"new_k and new_v are on {new_k.device} and {new_v.device}, expected {device}")
    _ints(new_pos, kv.n_seq, "new_pos", device)
    if rope_pos is not None:
        _ints(rope_pos, kv.n_seq * count, "rope_pos", device)
    if rope is not None:
        _on(rope.phases, device, "rope")
    n = misa_new_kv(new_k.data_ptr(), new_v.data_ptr(), ks[0], ks[1], ks[2], vs[0], vs[1], vs[2])
    _call(_lib.misa_append_kv, device, stream, kv._p, ctypes.byref(n), new_pos.data_ptr(), count,
          None if rope is None else rope._p, None if rope_pos is None else rope_pos.data_ptr(), 1 if commit else 0)


def read_kv(kv: KVCache, seq: torch.Tensor, tok: torch.Tensor, k_out: Optional[torch.Tensor] = None,
            v_out: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The dequantised bf16 rows of tokens tok [n][k] (-1: zeros) of sequences seq [n]: two [n][k][H_kv][d] tensors."""
    if tok.dim() != 2:
        raise ValueError(f"tok must be [n][k], got {tuple(tok.shape)}")
    n, k = tok.shape
    device, shape = kv.device, (n, k, kv.H_kv, kv.d)
    _ints(seq, n, "seq", device), _ints(tok, n * k, "tok", device)
    for t in (k_out, v_out):
        if t is not None:
            if t.dtype not in _BF16:
                raise TypeError(f"outputs must be bf16, got {t.dtype}")
            if t.shape != shape or not t.is_contiguous():
                raise ValueError(f"outputs must be contiguous {shape}, got {tuple(t.shape)}")
            _on(t, device, "output")
    if k_out is None or v_out is None:
        with _allocating(stream):
            if k_out is None:
                k_out = torch.empty(shape, dtype=torch.bfloat16, device=device)
            if v_out is None:
                v_out = torch.empty_like(k_out)
    _call(_lib.misa_read_kv, device, stream, kv._p, seq.data_ptr(), tok.data_ptr(), n, k, k_out.data_ptr(),
          v_out.data_ptr())
    return k_out, v_out


class AttentionQueries:
    """Attention queries: q bf16 (or its bits) [n_q][H][d], q_seq/q_pos int32 [n_q], scale (default 1/sqrt(d))."""

    def __init__(self, q: torch.Tensor, q_seq: torch.Tensor, q_pos: torch.Tensor, scale: Optional[float] = None):
        _need(q.dim() == 3 and q.is_contiguous(), f"q must be a contiguous [n_q][H][d] tensor, got {tuple(q.shape)}")
        if q.dtype not in _BF16:
            raise TypeError(f"q must be bf16, got {q.dtype}")
        self.n_q, self.H, self.d = (int(x) for x in q.shape)
        _ints(q_seq, self.n_q, "q_seq", q.device), _ints(q_pos, self.n_q, "q_pos", q.device)
        self.q, self.q_seq, self.q_pos = q, q_seq, q_pos
        self.scale = float(scale) if scale is not None else 1.0 / math.sqrt(self.d)
        # one element in the shape of an lse: torch allocates like a tensor in half the time of a new one
        self._lse = torch.empty((1, 1), dtype=torch.float32, device=q.device).expand(self.n_q, self.H)
        self._need = {}  # workspace bytes by the shapes that decide them
        self._s = misa_attend_queries(_m._ptr(q), _m._ptr(q_seq), _m._ptr(q_pos), self.n_q, self.H, self.scale)
        self._p = ctypes.byref(self._s)

    @property
    def struct(self) -> misa_attend_queries:
        return self._s


class Draft:
    """Drafted tokens in the cache: slot j of sequence s at position start[s] + j (int32 [n_seq]); mask int32 words
    [n_q][ceil(n/32)], bit j of a query's row set where it sees slot j (see ``tree_mask``)."""

    def __init__(self, start: torch.Tensor, mask: torch.Tensor, n: int):
        _need(1 <= int(n) <= MAX_DRAFT, f"a draft holds 1 to {MAX_DRAFT} tokens, got {n}")
        if mask.dtype not in (torch.int32, torch.uint32):
            raise TypeError(f"mask must be int32 words, got {mask.dtype}")
        _need(mask.dim() == 2 and mask.shape[1] == -(-int(n) // 32) and mask.is_contiguous(),
              f"mask must be contiguous [n_q][{-(-int(n) // 32)}], got {tuple(mask.shape)}")
        _ints(start, start.numel(), "start", mask.device)
        self.start, self.mask, self.n = start, mask, int(n)
        self._s = misa_draft(_m._ptr(start), _m._ptr(mask), self.n)
        self._p = ctypes.byref(self._s)

    @property
    def struct(self) -> misa_draft:
        return self._s


def tree_mask(parents: Sequence[int], n: Optional[int] = None) -> torch.Tensor:
    """Host mask words [len(parents)][ceil(n/32)] of a drafted tree: node j sees itself and its ancestors.

    parents[j] is the parent of node j (before it), -1 for a child of the committed prefix; n the draft's slots."""
    t = len(parents)
    n = t if n is None else int(n)
    _need(t <= n <= MAX_DRAFT, f"{t} nodes in a draft of {n} slots (at most {MAX_DRAFT})")
    seen = torch.zeros(t, -(-n // 32) * 32, dtype=torch.int64)
    for j, p in enumerate(int(x) for x in parents):
        _need(-1 <= p < j, f"the parent of node {j} must come before it, got {p}")
        if p >= 0:
            seen[j] = seen[p]
        seen[j, j] = 1
    words = (seen.view(t, seen.shape[1] // 32, 32) << torch.arange(32)).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


def attend_workspace_bytes(kv: KVCache, qs: AttentionQueries, k: int = 0, n_draft: int = 0) -> int:
    return int(_lib.misa_attend_workspace_bytes(ctypes.byref(kv.struct), ctypes.byref(qs.struct), k, n_draft))


def attend(kv: KVCache, qs: AttentionQueries, topk: Optional[torch.Tensor] = None, draft: Optional[Draft] = None,
           out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, ws: Optional[Workspace] = None,
           with_lse: bool = False, stream=None):
    """Attention over the tokens of topk [n_q][k] (-1 padded, as the top-k calls write it; k may be 0: no tokens), or
    over whole prefixes (topk None), and the drafted slots that each query's mask shows.

    Returns out [n_q][H][d] (q's type), with ``with_lse`` or a given ``lse`` the pair (out, lse fp32 [n_q][H])."""
    dev = kv.device
    if qs.d != kv.d:
        raise ValueError(f"queries of {qs.d} elements, cache of {kv.d}")
    q = qs.q
    _on(q, dev, "q")
    k = n_draft = 0
    if topk is not None:
        if topk.dim() != 2 or topk.shape[0] != qs.n_q:
            raise ValueError(f"topk must be [{qs.n_q}][k], got {tuple(topk.shape)}")
        k = topk.shape[1]
        _ints(topk, qs.n_q * k, "topk", dev)
    if draft is not None:
        if draft.mask.shape[0] != qs.n_q or draft.start.numel() != kv.n_seq:
            raise ValueError(f"draft of {draft.mask.shape[0]} mask rows and {draft.start.numel()} sequences for {qs.n_q} "
                             f"queries and {kv.n_seq} sequences")
        _on(draft.mask, dev, "draft")
        n_draft = draft.n
    if out is not None:
        if out.dtype not in _BF16:
            raise TypeError(f"out must be bf16, got {out.dtype}")
        if out.shape != q.shape or not out.is_contiguous():
            raise ValueError(f"out must be contiguous {tuple(q.shape)}, got {tuple(out.shape)}")
        _on(out, dev, "out")
    if lse is not None:
        if lse.dtype is not torch.float32:
            raise TypeError(f"lse must be float32, got {lse.dtype}")
        if lse.shape != (qs.n_q, qs.H) or not lse.is_contiguous():
            raise ValueError(f"lse must be contiguous [{qs.n_q}][{qs.H}], got {tuple(lse.shape)}")
        _on(lse, dev, "lse")
    if topk is not None and k == 0:
        # a list of nothing: one entry of nothing per query (without a list the whole prefix would be seen)
        k = 1
        with _allocating(stream):
            topk = torch.full((qs.n_q, 1), -1, dtype=torch.int32, device=dev)
    key = (k, n_draft, kv._shape)
    need = qs._need.get(key)
    if need is None:
        need = qs._need[key] = attend_workspace_bytes(kv, qs, k, n_draft)
    buf = None
    with _allocating(stream):
        if out is None:
            out = torch.empty_like(q)
        if lse is None and with_lse:
            lse = torch.empty_like(qs._lse, memory_format=torch.contiguous_format)
        if need:
            buf = (ws or Workspace(dev)).get(need)
    _call(_lib.misa_attend, dev, stream, kv._p, qs._p, None if topk is None else topk.data_ptr(), k,
          None if draft is None else draft._p, out.data_ptr(), None if lse is None else lse.data_ptr(),
          None if buf is None else buf.data_ptr(), need)
    return out if lse is None else (out, lse)


class SparseAttention:
    """The attention of a decode step around MISA-dagger (see misa.MisaDaggerDecode).

    ``before`` rotates the rows of ``rotate`` with ``rope`` (up to four (x, pos, out) triples in one launch: the
    step's index queries, its attention queries, the new keys of a bf16 index cache) and writes new_k, new_v
    [n_seq][1][H_kv][d] at new_pos, the keys rotated by ``kv_rope``; ``after`` attends over the step's top-k.
    The new keys of an e4m3 index cache reach the step as codes.  Where they come as bf16 rows, rotate them
    (apply_rope), write them with misa.append_keys_e4m3 before the step runs, and give the step itself positions of
    -1, which append nothing; all of it can be captured together.  The step has no drafted tokens.
    All buffers are the caller's or allocated here once; out [n_q][H][d] and lse [n_q][H] hold the step's result.
    """

    def __init__(self, kv: KVCache, queries: AttentionQueries, new_k: torch.Tensor, new_v: torch.Tensor,
                 new_pos: torch.Tensor, k: int, rope: Optional[Rope] = None, rotate: Sequence = (),
                 kv_rope: Optional[Rope] = None):
        if rotate and rope is None:
            raise ValueError("rotate needs a rope")
        self.kv, self.queries, self.new_k, self.new_v, self.new_pos = kv, queries, new_k, new_v, new_pos
        self.rope, self.rotate, self.kv_rope = rope, list(rotate), kv_rope
        dev = kv.device
        self.out = torch.empty_like(queries.q)
        self.lse = torch.empty((queries.n_q, queries.H), dtype=torch.float32, device=dev)
        self.ws = Workspace(dev)
        self.ws.get(attend_workspace_bytes(kv, queries, int(k)))

    def before(self, stream=None) -> None:
        if self.rotate:
            apply_rope(self.rope, self.rotate, stream=stream)
        append_kv(self.kv, self.new_k, self.new_v, self.new_pos, rope=self.kv_rope, stream=stream)

    def after(self, topk: torch.Tensor, stream=None) -> torch.Tensor:
        return attend(self.kv, self.queries, topk=topk, out=self.out, lse=self.lse, ws=self.ws, stream=stream)[0]
