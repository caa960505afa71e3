"""Rotary positions and a paged key / value cache over the C entry points of
include/fakv.h: argument checks and marshalling only, every step runs in the library's
CUDA kernels.

    rope = kv.Rope(128, base=500000.0, scaling=dict(kind="bands", factor=8.0, low=1.0, high=4.0, original=8192))
    cache = kv.PagedCache.create(layers, pages=4096, page_size=16, kv_heads=8, head_dim=128, slots=64, max_pages=1024)
    cache.grow(slots, counts)                               # pages for each slot's new tokens
    for layer in range(layers):
        q = cache.append(q, k, v, cu, slots, rope=rope, layer=layer)   # K, V written, q and k rotated
        o, lse = cache.attend(q, cu, slots, layer=layer)
    cache.check()                                           # raises if the device refused an entry, or gave up a wait

Tokens of a step are the rows of ``q`` [T, H, D], ``k`` and ``v`` [T, HKV, D]; sequence b has rows
cu[b] .. cu[b + 1] - 1 and is slot slots[b] (None: slot b). Everything that changes from step to step is
read on the device, so a step can be captured into a CUDA graph and replayed.

A training step rotates with ``rope.apply`` and its gradient with ``rope.backward``.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import fa

NO_PAGES, BAD_SLOT, REPEATED, ROW_FULL, BAD_PAGE, BAD_LENGTH = 1, 2, 4, 8, 16, 32
STATUS_BITS = {NO_PAGES: "too few free pages", BAD_SLOT: "slot out of range", REPEATED: "slot named twice",
               ROW_FULL: "row of the table too short", BAD_PAGE: "page number out of range",
               BAD_LENGTH: "length out of range"}
KINDS = {"none": 0, "linear": 1, "ntk": 2, "bands": 3, "yarn": 4}
EXPORTS = ("fakv_rope_freqs", "fakv_rope_apply", "fakv_append", "fakv_attend", "fakv_grow", "fakv_fork",
           "fakv_free", "fakv_compact")
_DT = {torch.float32: fa.FA_F32, torch.bfloat16: fa.FA_BF16}
_i, _ll, _vp = ctypes.c_int, ctypes.c_longlong, ctypes.c_void_p


class CacheError(RuntimeError):
    """What the device refused (see the FAKV_ bits of include/fakv.h)."""

    def __init__(self, bits: int):
        self.bits = bits
        super().__init__("; ".join(s for b, s in STATUS_BITS.items() if bits & b) or f"status {bits}")


class fakv_cache(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("K", "V", "table", "lens", "refs", "status")]
                + [(n, _ll) for n in ("plane_stride", "page_stride", "token_stride", "head_stride", "table_stride")]
                + [(n, _i) for n in ("planes", "num_pages", "page_size", "HKV", "D", "max_slots", "max_pages",
                                     "dtype")])


class fakv_scaling(ctypes.Structure):
    _fields_ = [("kind", _i)] + [(n, ctypes.c_double) for n in ("factor", "low", "high", "original", "beta_fast",
                                                                "beta_slow")]


class fakv_rope(ctypes.Structure):
    _fields_ = [("freqs", _vp), ("rotary_dim", _i), ("interleaved", _i), ("mscale", ctypes.c_float)]


class fakv_rope_params(ctypes.Structure):
    _fields_ = ([(n, _i) for n in ("T", "H", "HKV", "D", "dtype", "positions_64", "inverse")]
                + [(n, _ll) for n in ("q_token", "q_head", "k_token", "k_head", "qo_token", "qo_head", "ko_token",
                                      "ko_head")])


class fakv_tokens(ctypes.Structure):
    _fields_ = ([(n, _i) for n in ("B", "T", "H", "plane")]
                + [(n, _ll) for n in ("q_token", "q_head", "k_token", "k_head", "v_token", "v_head")]
                + [("scale", ctypes.c_float), ("causal", _i), ("window", _i), ("out_dtype", _i)])


# A call of a few microseconds is not to spend as many on asking for its device and stream.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)

# fakv_tokens and fakv_rope_params packed in one step (the C side takes a pointer to the bytes)
_pack_tokens = struct.Struct("@4i6qf3i").pack
_pack_rope = struct.Struct("@7i4x8q").pack

_bound = None


def _lib():
    """libfa.so with the argument types of include/fakv.h."""
    global _bound
    if _bound is None:
        lib = fa.lib()
        P = ctypes.POINTER
        for name, args in (
                ("fakv_rope_freqs", [_i, ctypes.c_double, P(fakv_scaling), _vp, P(ctypes.c_float)]),
                ("fakv_rope_apply", [_vp, _vp, _vp, _vp, _vp, P(fakv_rope), _vp, _vp]),
                ("fakv_append", [_vp] * 6 + [P(fakv_rope), P(fakv_cache), _vp, _vp]),
                ("fakv_attend", [_vp] * 5 + [P(fakv_cache), _vp, _vp]),
                ("fakv_grow", [P(fakv_cache), _vp, _vp, _i, _vp]),
                ("fakv_fork", [P(fakv_cache), _vp, _vp, _i, _vp]),
                ("fakv_free", [P(fakv_cache), _vp, _vp, _i, _vp]),
                ("fakv_compact", [P(fakv_cache), _vp])):
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = _i
        _bound = lib
    return _bound


def _check(rc: int, where: str) -> None:
    if rc:
        raise fa.FAError(rc, where)


class _on:
    """The device of a call's tensors made current for as long as the call, and the handle of its stream: ``stream``,
    or that device's current one. The memory of ``tensors`` is not handed out again before a ``stream`` of the call's
    own has passed it (the work that makes them ready is the caller's to order)."""

    __slots__ = ("back", "stream", "handle")

    def __init__(self, index, stream, *tensors):
        self.back, self.stream = -1, stream
        current = _current_device()
        if stream is not None:
            if stream.device_index != index:
                raise ValueError("the stream belongs to another device than the tensors")
            self.handle = stream.cuda_stream
            for t in tensors:
                if t is not None and t.is_cuda:
                    t.record_stream(stream)
        else:
            self.handle = _raw_stream(index)
        if current != index:
            self.back = current
            torch.cuda.set_device(index)

    def empty(self, like, shape, dtype):
        """An output, allocated in the order of the stream that the call runs on."""
        if self.stream is None:
            return torch.empty(shape, dtype=dtype, device=like.device)
        with torch.cuda.stream(self.stream):
            t = torch.empty(shape, dtype=dtype, device=like.device)
        t.record_stream(torch.cuda.current_stream())
        return t

    def leave(self):
        if self.back >= 0:
            torch.cuda.set_device(self.back)
            self.back = -1


def _rows(t, name, dtype, device, heads=None, dim=None, T=None):
    """Shape and strides of a [T, heads, D] tensor whose columns run without gaps."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must be [T, heads, D], {dtype}, on {device}")
    if (heads is not None and shape[1] != heads) or (dim is not None and shape[2] != dim) \
            or (T is not None and shape[0] != T):
        raise ValueError(f"{name} has shape {tuple(shape)}: [{T}, {heads}, {dim}] is wanted")
    if stride[2] != 1 and t.numel():
        raise ValueError(f"the columns of {name} must be contiguous")
    return shape, stride


def _out(t, name, shape, dtype, device):
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, {tuple(shape)}, {dtype}, on {device}")
    return t


def _ints(t, name, n, device):
    """Length of a contiguous int32 vector."""
    shape = t.shape
    if t.dtype != torch.int32 or len(shape) != 1 or t.device != device or not t.is_contiguous() \
            or (n is not None and shape[0] != n):
        raise ValueError(f"{name} must be a contiguous int32 vector{'' if n is None else f' of {n}'} on {device}")
    return shape[0]


class Rope:
    """Rotary positions of the first ``rotary_dim`` (None: all) of ``head_dim`` columns. ``layout``: "half" (columns
    i and i + rotary_dim / 2 are a pair) or "interleaved" (2 i and 2 i + 1). ``scaling``: None, or a dict with
    ``kind`` "linear" (factor), "ntk" (factor), "bands" (factor, low, high, original) or "yarn" (factor, beta_fast,
    beta_slow, original), and with any of them ``mscale`` to replace 1 (yarn: 0.1 ln(factor) + 1 above a factor of
    1): see include/fakv.h. The frequencies are computed once and kept on ``device``."""

    def __init__(self, head_dim, rotary_dim=None, base=10000.0, layout="half", scaling=None, device="cuda"):
        rotary_dim = head_dim if rotary_dim is None else rotary_dim
        if layout not in ("half", "interleaved"):
            raise ValueError('layout must be "half" or "interleaved"')
        if not 0 < rotary_dim <= head_dim:
            raise ValueError("rotary_dim must be in 1 .. head_dim")
        s = dict(scaling or {"kind": "none"})
        kind, mscale = s.pop("kind", None), s.pop("mscale", None)
        if kind not in KINDS:
            raise ValueError(f"scaling kind must be one of {sorted(KINDS)}")
        if kind == "yarn":
            s = {"beta_fast": 32.0, "beta_slow": 1.0, **s}
        unknown = set(s) - {n for n, _ in fakv_scaling._fields_}
        if unknown:
            raise ValueError(f"unknown scaling arguments {sorted(unknown)}")
        freqs = (ctypes.c_ulonglong * max(1, rotary_dim // 2))()
        factor = ctypes.c_float()
        sc = fakv_scaling(kind=KINDS[kind], **s)
        _check(_lib().fakv_rope_freqs(rotary_dim, base, ctypes.byref(sc), freqs, ctypes.byref(factor)),
               "fakv_rope_freqs")
        self.head_dim, self.rotary_dim, self.layout = head_dim, rotary_dim, layout
        self.mscale = float(factor.value if mscale is None else mscale)
        self.freqs = torch.frombuffer(freqs, dtype=torch.int64).clone().to(device)
        self._c = fakv_rope(self.freqs.data_ptr(), rotary_dim, int(layout == "interleaved"), self.mscale)
        self._ref = ctypes.byref(self._c)

    def apply(self, q, k, positions, inverse=False, out=None, stream=None):
        """q [T, H, D] and k [T, HKV, D] (or None) rotated by ``positions`` [T] (int32 or int64). ``out``: a pair of
        tensors to write, which may be (q, k) themselves. Returns (q, k) rotated."""
        dev, dt = q.device, q.dtype
        (T, H, _), sq = _rows(q, "q", dt, dev, None, self.head_dim)
        if dt not in _DT:
            raise TypeError(f"unsupported dtype {dt}")
        if not q.is_cuda or self.freqs.device != dev:
            raise ValueError(f"q must be on {self.freqs.device}, the device of the frequencies")
        hk, sk, so, sko, kp, kop = 0, (0, 0), None, (0, 0), None, None
        if k is not None:
            (_, hk, _), sk = _rows(k, "k", dt, dev, None, self.head_dim, T)
            kp = k.data_ptr()
        wide = positions.dtype == torch.int64
        if not (wide or positions.dtype == torch.int32) or positions.shape != (T,) or positions.device != dev \
                or not positions.is_contiguous():
            raise ValueError(f"positions must be a contiguous int32 or int64 vector of {T} on {dev}")
        on = _on(dev.index, stream, q, k, positions, self.freqs, *(out or ()))
        try:
            if out is None:
                qo, ko = on.empty(q, q.shape, dt), None if k is None else on.empty(q, k.shape, dt)
            else:
                qo, ko = out
            _, so = _rows(qo, "out[0]", dt, dev, H, self.head_dim, T)
            if k is not None:
                _, sko = _rows(ko, "out[1]", dt, dev, hk, self.head_dim, T)
                kop = ko.data_ptr()
            _check(_lib().fakv_rope_apply(
                q.data_ptr(), kp, qo.data_ptr(), kop, positions.data_ptr(), self._ref,
                _pack_rope(T, H, hk, self.head_dim, _DT[dt], wide, bool(inverse), sq[0], sq[1], sk[0], sk[1], so[0],
                           so[1], sko[0], sko[1]), on.handle), "fakv_rope_apply")
        finally:
            on.leave()
        return qo, None if k is None else ko

    def backward(self, dq, dk, positions, out=None, stream=None):
        """Gradients of ``apply``'s inputs from those of its outputs: the inverse rotation (times mscale)."""
        return self.apply(dq, dk, positions, True, out, stream)


class PagedCache:
    """Key / value pages of sequences in slots. ``k``, ``v``: [planes, pages, page_size, kv heads, D] (or without the
    planes; ``layout`` "heads": [planes, pages, kv heads, page_size, D]), bf16 or fp32, alike in shape and strides;
    ``table`` [slots, max_pages] int32 page numbers (-1: none), ``lens`` [slots] int32, ``refs`` [pages] int32: how
    many rows hold a page. The tensors stay the caller's; the methods change them in place (a length is lowered with
    ``free``, which releases the pages). ``status`` [1] int32 collects what the device refused (``check``)."""

    def __init__(self, k, v, table, lens, refs, layout="tokens", status=None):
        if layout not in ("tokens", "heads"):
            raise ValueError('layout must be "tokens" or "heads"')
        if k.dim() == 4 and v.dim() == 4:
            k, v = k[None], v[None]
        if k.dim() != 5 or k.shape != v.shape or k.dtype != v.dtype or k.device != v.device or k.dtype not in _DT:
            raise ValueError("k and v must be alike, bf16 or fp32, [planes, pages, page_size, kv heads, D]")
        if k.stride() != v.stride() or k.stride(4) != 1:
            raise ValueError("k and v must have the same strides and contiguous columns")
        dev = k.device
        if not k.is_cuda:
            raise ValueError("the cache must be on a CUDA device")
        t, h = (2, 3) if layout == "tokens" else (3, 2)
        if table.dim() != 2 or table.dtype != torch.int32 or table.device != dev or table.stride(1) != 1:
            raise ValueError("table must be an int32 matrix with contiguous rows, on the cache's device")
        _ints(lens, "lens", table.shape[0], dev)
        _ints(refs, "refs", k.shape[1], dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev) if status is None \
            else _ints(status, "status", 1, dev)
        self.k, self.v, self.table, self.lens, self.refs, self.device = k, v, table, lens, refs, dev
        self.planes, self.page_size, self.kv_heads, self.head_dim = k.shape[0], k.shape[t], k.shape[h], k.shape[4]
        self.slots, self.dtype, self._index = table.shape[0], k.dtype, dev.index
        self._tensors = (k, v, table, lens, refs, self.status)
        self._c = fakv_cache(k.data_ptr(), v.data_ptr(), table.data_ptr(), lens.data_ptr(), refs.data_ptr(),
                             self.status.data_ptr(), k.stride(0), k.stride(1), k.stride(t), k.stride(h),
                             table.stride(0), k.shape[0], k.shape[1], k.shape[t], k.shape[h], k.shape[4],
                             table.shape[0], table.shape[1], _DT[k.dtype])
        self._ref = ctypes.byref(self._c)

    @classmethod
    def create(cls, planes, pages, page_size, kv_heads, head_dim, slots, max_pages, dtype=torch.bfloat16,
               layout="tokens", device="cuda"):
        """An empty cache (its page memory zeroed)."""
        inner = (page_size, kv_heads) if layout == "tokens" else (kv_heads, page_size)
        k = torch.zeros(planes, pages, *inner, head_dim, dtype=dtype, device=device)
        return cls(k, torch.zeros_like(k), torch.full((slots, max_pages), -1, dtype=torch.int32, device=device),
                   torch.zeros(slots, dtype=torch.int32, device=device),
                   torch.zeros(pages, dtype=torch.int32, device=device), layout)

    def _batch(self, cu, slots, layer):
        """Sequences of a call and the address of its slots."""
        B = _ints(cu, "cu", None, self.device) - 1
        if B < 0:
            raise ValueError("cu must have an entry more than there are sequences")
        if not 0 <= layer < self.planes:
            raise ValueError(f"layer must be in 0 .. {self.planes - 1}")
        if slots is None:
            if B > self.slots:
                raise ValueError("more sequences than slots")
            return B, None
        _ints(slots, "slots", B, self.device)
        return B, slots.data_ptr()

    def append(self, q, k, v, cu, slots=None, rope=None, layer=0, out=None, stream=None):
        """Writes the new tokens' k and v [T, HKV, D] into the cache, k rotated by ``rope`` (None: as it is), and
        returns q [T, H, D] rotated likewise (into ``out``, contiguous, where given; q may be None). The slots'
        lengths already count the new tokens (``grow``). Rows of q past cu[-1] are not written. A slot named twice in
        one call would have two tokens for one place: which of them it keeps is not defined."""
        dev, dt, D = self.device, self.dtype, self.head_dim
        (T, _, _), sk = _rows(k, "k", dt, dev, self.kv_heads, D)
        _, sv = _rows(v, "v", dt, dev, self.kv_heads, D, T)
        B, sp = self._batch(cu, slots, layer)
        H, sq, qp, op, o = 0, (0, 0), None, None, None
        if q is not None:
            (_, H, _), sq = _rows(q, "q", dt, dev, None, D, T)
            qp = q.data_ptr()
        if rope is not None and (rope.head_dim != D or rope.freqs.device != dev):
            raise ValueError("rope is for another head_dim or device")
        on = _on(self._index, stream, q, k, v, cu, slots, out, None if rope is None else rope.freqs, *self._tensors)
        try:
            if q is not None:
                o = on.empty(q, q.shape, dt) if out is None else _out(out, "out", q.shape, dt, dev)
                op = o.data_ptr()
            _check(_lib().fakv_append(
                qp, k.data_ptr(), v.data_ptr(), op, cu.data_ptr(), sp, None if rope is None else rope._ref, self._ref,
                _pack_tokens(B, T, H, layer, sq[0], sq[1], sk[0], sk[1], sv[0], sv[1], 1.0, 1, 0, 0), on.handle),
                "fakv_append")
        finally:
            on.leave()
        return o

    def attend(self, q, cu, slots=None, scale=None, causal=True, window=0, layer=0, out_dtype=None, out=None,
               lse=None, stream=None):
        """O [T, H, D] and LSE [T, H] of the new tokens' queries over their sequences' tokens: key j is visible to
        position p iff j <= p (``causal``) and j > p - window (window 0: all). Rows past cu[-1] are not written."""
        dev, dt, D = self.device, self.dtype, self.head_dim
        shape, sq = _rows(q, "q", dt, dev, None, D)
        B, sp = self._batch(cu, slots, layer)
        odt = out_dtype if out_dtype is not None else dt if out is None else out.dtype
        if odt not in _DT:
            raise TypeError(f"unsupported output dtype {odt}")
        on = _on(self._index, stream, q, cu, slots, out, lse, *self._tensors)
        try:
            out = on.empty(q, shape, odt) if out is None else _out(out, "out", shape, odt, dev)
            lse = on.empty(q, shape[:2], torch.float32) if lse is None \
                else _out(lse, "lse", shape[:2], torch.float32, dev)
            _check(_lib().fakv_attend(
                q.data_ptr(), out.data_ptr(), lse.data_ptr(), cu.data_ptr(), sp, self._ref,
                _pack_tokens(B, shape[0], shape[1], layer, sq[0], sq[1], 0, 0, 0, 0,
                             D ** -0.5 if scale is None else scale, bool(causal), window, _DT[odt]), on.handle),
                "fakv_attend")
        finally:
            on.leave()
        return out, lse

    def _list(self, call, where, a, names, b, stream):
        n = _ints(a, names[0], None, self.device)
        bp = None
        if b is not None:
            _ints(b, names[1], n, self.device)
            bp = b.data_ptr()
        on = _on(self._index, stream, a, b, *self._tensors)
        try:
            _check(call(self._ref, a.data_ptr(), bp, n, on.handle), where)
        finally:
            on.leave()

    def grow(self, slots, add, stream=None):
        """Room for add[i] more tokens in slots[i] (the lengths grow by it): new pages, and a copy of a shared last
        page that has room. An entry that cannot be served (``check`` tells) keeps its length; an append that counts
        on it would write over the slot's last tokens."""
        self._list(_lib().fakv_grow, "fakv_grow", slots, ("slots", "add"), add, stream)

    def fork(self, src, dst, stream=None):
        """Slots dst[i] become copies of slots src[i] that share their pages; sources are read as they were before
        the call."""
        self._list(_lib().fakv_fork, "fakv_fork", src, ("src", "dst"), dst, stream)

    def free(self, slots, keep=None, stream=None):
        """Slots cut to their first keep[i] tokens (None: emptied); pages that no slot holds any more are free."""
        self._list(_lib().fakv_free, "fakv_free", slots, ("slots", "keep"), keep, stream)

    def compact(self, stream=None):
        """Moves pages so that those in use are the lowest-numbered ones, and renumbers the table."""
        on = _on(self._index, stream, *self._tensors)
        try:
            _check(_lib().fakv_compact(self._ref, on.handle), "fakv_compact")
        finally:
            on.leave()

    def check(self) -> None:
        """Waits for the device (all its streams). Raises CacheError if a call on this cache refused an entry since the
        last check, and fa.FAError if a wait in one of the library's kernels ran out: outputs may then be unwritten."""
        torch.cuda.synchronize(self.device)
        bits = int(self.status.item())
        if bits:
            self.status.zero_()
            torch.cuda.synchronize(self.device)
            raise CacheError(bits)
        on = _on(self._index, None)
        try:
            _check(fa.fa_device_status(on.handle), "fa_device_status")
        finally:
            on.leave()
