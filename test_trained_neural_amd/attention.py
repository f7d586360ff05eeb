"""The attention window's operators: Python binding of ``include/tm_attention.h``.

Rotary positions, a paged key/value cache held in 8 bits, the attention that
reads it and its pages' housekeeping.  As in the package's other calls, this
is argument marshalling only: the functions carry the C names and check
types, shapes and devices before a pointer is passed on.  ``Rotary`` and
``PagedCache`` keep a frequency table and a cache's blob and allocate
outputs; ``WindowAttention`` puts them together as the attention of
``mac_segment``, with torch's plain products for its two projections.
Nothing here records gradients (``Rotary``'s is a call of its own).

Calls run on the current stream of the tensors' device (or on ``stream``).
"""
from __future__ import annotations

import ctypes
import math

import torch

import test_trained_neural_amd as T

TM_ROPE_HALF, TM_ROPE_INTERLEAVED = 0, 1
TM_ROPE_NONE, TM_ROPE_LINEAR, TM_ROPE_BASE, TM_ROPE_PARTS = 0, 1, 2, 3
TM_CACHE_NONFINITE, TM_CACHE_NO_PAGES, TM_CACHE_FULL, TM_CACHE_BAD_ENTRY = 1, 2, 4, 8
TM_CACHE_PAGE, TM_CACHE_BLOCK = 64, 16

EXPORTED = ("tm_rotary_frequencies", "tm_rotary", "tm_cache_create", "tm_cache_destroy", "tm_cache_bytes",
            "tm_cache_layout", "tm_cache_init", "tm_cache_workspace_bytes", "tm_cache_append", "tm_cache_attend",
            "tm_cache_read", "tm_cache_fork", "tm_cache_free", "tm_cache_compact", "tm_cache_check")

# kernel class of tm_timing_enable / tm_timing_read
K_ATTENTION = 10

_vp, _i, _l, _d, _f, _z = (ctypes.c_void_p, ctypes.c_int, ctypes.c_long, ctypes.c_double, ctypes.c_float,
                           ctypes.c_size_t)
_declared = None


def _lib():
    global _declared
    if _declared is None:
        L = T.lib()
        for name, args in (
                ("tm_rotary_frequencies", [_i, _d, _i, _d, _d, _d, _d, ctypes.POINTER(_d), ctypes.POINTER(_d)]),
                ("tm_rotary", [_vp, _l, _l, _vp, _l, _l, _vp, _i, _vp, _d, _i, _i, _i, _i, _i, _i, _i, _i, _vp]),
                ("tm_cache_create", [_i, _i, _i, _i, _i, ctypes.POINTER(_vp)]),
                ("tm_cache_layout", [_vp, ctypes.POINTER(_z)]),
                ("tm_cache_init", [_vp, _vp, _vp]),
                ("tm_cache_append", [_vp, _vp, _vp, _vp, _vp, _l, _l, _vp, _l, _l, _i, _i, _i, _vp, _vp]),
                ("tm_cache_attend", [_vp, _vp, _vp, _vp, _vp, _l, _l, _vp, _i, _i, _i, _f, _i, _i, _i, _i, _vp, _vp]),
                ("tm_cache_read", [_vp, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _vp]),
                ("tm_cache_fork", [_vp, _vp, _vp, _vp, _i, _vp]),
                ("tm_cache_free", [_vp, _vp, _vp, _vp, _i, _vp]),
                ("tm_cache_compact", [_vp, _vp, _vp, _vp]),
                ("tm_cache_check", [_vp, _vp, ctypes.POINTER(_i), ctypes.POINTER(_i), _vp])):
            fn = getattr(L, name)
            fn.restype, fn.argtypes = _i, args
        L.tm_cache_destroy.restype, L.tm_cache_destroy.argtypes = None, [_vp]
        L.tm_cache_bytes.restype, L.tm_cache_bytes.argtypes = _z, [_vp]
        L.tm_cache_workspace_bytes.restype, L.tm_cache_workspace_bytes.argtypes = _z, [_vp, _i, _i, _i]
        _declared = L
    return _declared


# ---------------------------------------------------------------------------
# argument checks
#
# What a call checks of its tensors' types, shapes, distances and devices
# follows from those alone, so each call keeps, per combination that has
# passed, what it read off them (a step of a few microseconds would otherwise
# spend most of them here).  Addresses are checked on every call.

_passed = {}


def _once(key, check):
    """check()'s result, remembered under ``key``."""
    v = _passed.get(key)
    if v is None:
        if len(_passed) > 4096:
            _passed.clear()
        v = _passed[key] = check()
    return v


def _look(t):
    """What a check sees of a tensor."""
    return None if t is None else (t.shape, t.stride(), t.dtype, t.device)


def _on(device, *named):
    """Every given tensor is on ``device``, a GPU."""
    if device.type != "cuda":
        raise ValueError("tensors must be device tensors")
    for name, t in named:
        if t is not None and t.device != device:
            raise ValueError("%s is on %s, the call is on %s" % (name, t.device, device))


def _heads_of(name, t, aligned=True):
    """(batch distance, token distance) in elements of a [batch][tokens]
    [heads][dim] tensor whose last two axes are contiguous."""
    if t.dim() != 4:
        raise ValueError("%s must be [batch][tokens][heads][dim], got %d axes" % (name, t.dim()))
    B, N, H, d = t.shape
    sb, st, sh, sd = t.stride()
    if (sd != 1 and d > 1) or (sh != d and H > 1):
        raise ValueError("the last two axes of %s must be contiguous" % name)
    st, sb = (H * d if N <= 1 else st), (N * H * d if B <= 1 else sb)
    if aligned and (sb % 8 or st % 8):
        raise ValueError("%s must be 16-byte aligned, its distances multiples of 8 elements" % name)
    return sb, st


def _aligned(name, ptr):
    if ptr % 16:
        raise ValueError("%s must be 16-byte aligned" % name)
    return ptr


def _list(name, t, n):
    if t is not None:
        if t.dtype != torch.int32:
            raise TypeError("%s must be torch.int32, got %s" % (name, t.dtype))
        if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
            raise ValueError("%s must be contiguous and hold %d values, got %s" % (name, n, tuple(t.shape)))


_INT_MAX = (1 << 31) - 1


def _int(v):
    """A number as the C calls take it: one beyond 32 bits (which would lose
    its upper ones) as the largest, or as -1, which they refuse or treat as it."""
    return v if -1 <= v <= _INT_MAX else max(-1, min(v, _INT_MAX))


def _at(t):
    return None if t is None else t.data_ptr()


def _elsewhere(index, stream):
    """Whether a call on device ``index`` has to change the current device or
    stream first."""
    return stream is not None or torch._C._cuda_getDevice() != index


def _there(device, stream):
    """The device of a call as the current one, or ``stream`` as the current
    stream (then also the one that the call's own buffers are allocated
    for)."""
    if stream is None:
        return torch.cuda.device(device)
    if stream.device != device:
        raise ValueError("stream is on %s, the call is on %s" % (stream.device, device))
    return torch.cuda.stream(stream)


_raw_stream = torch._C._cuda_getCurrentRawStream


# ---------------------------------------------------------------------------
# the C calls, one to one

def tm_rotary_frequencies(rot_dim, base=10000.0, scaling=TM_ROPE_NONE, factor=1.0, original_len=0.0, beta_fast=32.0,
                          beta_slow=1.0):
    """(list of rot_dim / 2 frequencies, factor of the result)."""
    rot_dim = _int(rot_dim)
    f, s = (_d * max(1, min(rot_dim, 1024) // 2))(), _d(1.0)
    T._check("tm_rotary_frequencies", _lib().tm_rotary_frequencies(rot_dim, base, scaling, factor, original_len,
                                                                  beta_fast, beta_slow, f, ctypes.byref(s)))
    return list(f), s.value


def _rotary_geometry(x, y, positions, freq):
    dt = T._dtype_code(x)
    T._same(x.dtype, ("y", y))
    T._same(torch.int32, ("positions", positions))
    T._same(torch.float64, ("freq", freq))
    T._shape("y", y, x.shape)
    _on(x.device, ("x", x), ("y", y), ("positions", positions), ("freq", freq))
    (xb, xt), (yb, yt) = _heads_of("x", x, False), _heads_of("y", y, False)
    B, N, H, d = x.shape
    per_token = positions.dim() == 2
    T._shape("positions", positions, (B, N) if per_token else (B,))
    if not positions.is_contiguous() or not freq.is_contiguous() or freq.dim() != 1:
        raise ValueError("positions and freq must be contiguous")
    return (xb, xt), (yb, yt), 1 if per_token else 0, (B, N, H, d, 2 * freq.shape[0]), dt, x.device.index


def tm_rotary(x, y, positions, freq, result_scale=1.0, layout=TM_ROPE_HALF, inverse=False, stream=None):
    """x, y [B][T][H][d] (any distances between tokens and entries; y may be
    x); positions int32 [B][T], or [B] (the first token's); freq [rot_dim / 2]
    fp64."""
    d_x, d_y, per_token, sizes, dt, index = _once(
        ("rotary", _look(x), _look(y), _look(positions), _look(freq)), lambda: _rotary_geometry(x, y, positions, freq))
    if _elsewhere(index, stream):
        with _there(x.device, stream):
            return tm_rotary(x, y, positions, freq, result_scale, layout, inverse)
    rc = _lib().tm_rotary(x.data_ptr(), *d_x, y.data_ptr(), *d_y, positions.data_ptr(), per_token, freq.data_ptr(),
                          result_scale, *sizes, layout, 1 if inverse else 0, dt, _raw_stream(index))
    if rc:
        T._check("tm_rotary", rc)


def tm_cache_create(kv_heads, head_dim, n_pages, n_seqs, seq_pages):
    h = _vp()
    T._check("tm_cache_create", _lib().tm_cache_create(*map(_int, (kv_heads, head_dim, n_pages, n_seqs, seq_pages)),
                                                       ctypes.byref(h)))
    return h


def tm_cache_destroy(cache):
    _lib().tm_cache_destroy(cache)


def tm_cache_bytes(cache):
    return _lib().tm_cache_bytes(cache)


def tm_cache_layout(cache):
    """Offsets of meta, scales, keys and values in the blob."""
    o = (_z * 4)()
    T._check("tm_cache_layout", _lib().tm_cache_layout(cache, o))
    return tuple(int(x) for x in o)


def tm_cache_workspace_bytes(cache, batch, n_tokens, heads=0):
    return _lib().tm_cache_workspace_bytes(cache, _int(batch), _int(n_tokens), _int(heads))


# ---------------------------------------------------------------------------

class Rotary:
    """Rotary positions of one table of frequencies: ``y = rotary(x,
    positions)``; ``inverse=True`` gives the gradient with respect to x."""

    def __init__(self, rot_dim, base=10000.0, layout=TM_ROPE_HALF, scaling=TM_ROPE_NONE, factor=1.0, original_len=0.0,
                 beta_fast=32.0, beta_slow=1.0, device="cuda"):
        f, self.result_scale = tm_rotary_frequencies(rot_dim, base, scaling, factor, original_len, beta_fast,
                                                     beta_slow)
        self.rot_dim, self.layout = rot_dim, layout
        self.freq = torch.tensor(f, dtype=torch.float64, device=device)

    def __call__(self, x, positions, inverse=False, out=None, stream=None):
        if stream is not None:
            _on(x.device, ("x", x))
            with _there(x.device, stream):
                return self(x, positions, inverse, out)
        if out is None:
            out = torch.empty_like(x, memory_format=torch.contiguous_format)
        tm_rotary(x, out, positions, self.freq, self.result_scale, self.layout, inverse)
        return out


class PagedCache:
    """A paged cache in 8 bits: the handle and its blob (``blob``: a uint8
    tensor of ``tm_cache_bytes`` bytes that already holds a cache, whose count
    of an append in progress is cleared in the order of the current stream; by
    default a new, empty one).  The views ``meta``, ``lengths``, ``refs``, ``table``,
    ``scales``, ``k``, ``v`` and ``status`` show its regions."""

    def __init__(self, kv_heads, head_dim, n_pages, n_seqs, seq_pages, device="cuda", blob=None):
        self.handle = None
        self.handle = tm_cache_create(kv_heads, head_dim, n_pages, n_seqs, seq_pages)
        self.kv_heads, self.head_dim, self.n_pages = kv_heads, head_dim, n_pages
        self.n_seqs, self.seq_pages = n_seqs, seq_pages
        need = tm_cache_bytes(self.handle)
        fresh = blob is None
        if fresh:
            blob = torch.empty(need, dtype=torch.uint8, device=device)
        T._same(torch.uint8, ("blob", blob))
        T._blob("blob", blob, need)
        if blob.data_ptr() % 256:
            raise ValueError("blob must be 256-byte aligned")
        self.blob, self.device = blob, blob.device
        self._h, self._b, self._index = self.handle.value, blob.data_ptr(), blob.device.index
        o, cells = tm_cache_layout(self.handle), n_pages * kv_heads * TM_CACHE_PAGE * head_dim
        ints = 64 + n_seqs + n_pages + n_seqs * seq_pages
        self.meta = blob[:4 * ints].view(torch.int32)
        self.status, self.lengths = self.meta[:64], self.meta[64:64 + n_seqs]
        self.refs = self.meta[64 + n_seqs:64 + n_seqs + n_pages]
        self.table = self.meta[64 + n_seqs + n_pages:].view(n_seqs, seq_pages)
        self.scales = blob[o[1]:o[1] + n_pages * kv_heads * 8].view(n_pages, kv_heads, 2, 4)
        self.k = blob[o[2]:o[2] + cells].view(torch.float8_e4m3fn).view(n_pages, kv_heads, TM_CACHE_PAGE, head_dim)
        self.v = blob[o[3]:o[3] + cells].view(torch.float8_e4m3fn).view(n_pages, kv_heads, head_dim, TM_CACHE_PAGE)
        self._need, self._kind = {}, (kv_heads, head_dim, blob.device)   # what a call's checks go by
        self._scale = 1.0 / math.sqrt(head_dim)
        if fresh:
            self.init()
        else:
            self.status[2:3].zero_()

    def __del__(self):
        try:
            if self.handle is not None and _declared is not None:
                tm_cache_destroy(self.handle)
        except Exception:
            pass

    def _call(self, name, *args):
        rc = getattr(_declared, name)(self._h, self._b, *args, _raw_stream(self._index))
        if rc:
            T._check(name, rc)

    def _workspace(self, batch, n_tokens, heads):
        """Workspace of one call: from torch's allocator, in the stream's
        order, so that calls on several streams and captured graphs have their
        own."""
        key = (batch, n_tokens, heads)
        need = self._need.get(key)
        if need is None:
            if len(self._need) > 4096:
                self._need.clear()
            need = self._need[key] = tm_cache_workspace_bytes(self.handle, batch, n_tokens, heads)
        return self.blob.new_empty(need)

    def init(self, stream=None):
        if _elsewhere(self._index, stream):
            with _there(self.device, stream):
                return self.init()
        self._call("tm_cache_init")

    def append(self, seqs, k, v, counts=None, stream=None):
        """Writes k, v [B][T][kv_heads][d] behind the sequences ``seqs``
        (int32 [B]; None: 0 ..); counts int32 [B]: tokens of each entry."""
        if _elsewhere(self._index, stream):
            with _there(self.device, stream):
                return self.append(seqs, k, v, counts)

        def check():
            dt = T._dtype_code(k)
            T._same(k.dtype, ("v", v))
            T._shape("v", v, k.shape)
            d_k, d_v = _heads_of("k", k), _heads_of("v", v)
            B, N = k.shape[:2]
            T._shape("k", k, (B, N, self.kv_heads, self.head_dim))
            _list("seqs", seqs, B)
            _list("counts", counts, B)
            _on(self.device, ("k", k), ("v", v), ("seqs", seqs), ("counts", counts))
            return d_k, d_v, (B, N, dt)

        d_k, d_v, sizes = _once((self._kind, "append", _look(k), _look(v), _look(seqs), _look(counts)), check)
        ws = self._workspace(sizes[0], sizes[1], 0)
        self._call("tm_cache_append", _at(seqs), _at(counts), _aligned("k", k.data_ptr()), *d_k,
                   _aligned("v", v.data_ptr()), *d_v, *sizes, ws.data_ptr())

    def attend(self, seqs, q, counts=None, scale=None, window=0, sink=0, max_len=0, out=None, stream=None):
        """Attention of q [B][T][heads][d], each sequence's last tokens
        (``counts`` of them), over the cache; scale: 1 / sqrt(d) by default.
        Returns [B][T][heads][d] of q's type (``out`` may be a contiguous q).
        Rows behind an entry's count are left as they were: zeros in a new
        output."""
        if _elsewhere(self._index, stream):
            with _there(self.device, stream):
                return self.attend(seqs, q, counts, scale, window, sink, max_len, out)

        def check():
            dt = T._dtype_code(q)
            d_q = _heads_of("q", q)
            B, N, H, d = q.shape
            T._shape("q", q, (B, N, H, self.head_dim))
            _list("seqs", seqs, B)
            _list("counts", counts, B)
            _on(self.device, ("q", q), ("out", out), ("seqs", seqs), ("counts", counts))
            if out is not None:
                T._same(q.dtype, ("out", out))
                T._shape("out", out, q.shape)
                if not out.is_contiguous():
                    raise ValueError("out must be contiguous")
            return d_q, (B, N, H), dt

        d_q, sizes, dt = _once((self._kind, "attend", _look(q), _look(seqs), _look(counts), _look(out)), check)
        pq = _aligned("q", q.data_ptr())
        if out is None:
            out = (torch.empty_like if counts is None else torch.zeros_like)(q, memory_format=torch.contiguous_format)
        ws = self._workspace(*sizes)
        self._call("tm_cache_attend", _at(seqs), _at(counts), pq, *d_q, out.data_ptr(), *sizes,
                   self._scale if scale is None else scale, _int(window), _int(sink), _int(max_len), dt, ws.data_ptr())
        return out

    def read(self, seqs, start, n_tokens, dtype=torch.float32, k=None, v=None, stream=None):
        """(k, v) [B][n_tokens][kv_heads][d]: the values that the tokens
        start .. of each sequence are held as; rows behind a sequence's end
        are left as they were (zeros in new outputs)."""
        if _elsewhere(self._index, stream):
            with _there(self.device, stream):
                return self.read(seqs, start, n_tokens, dtype, k, v)
        B = self.n_seqs if seqs is None else seqs.shape[0]
        shape = (B, n_tokens, self.kv_heads, self.head_dim)
        _list("seqs", seqs, B)
        k = torch.zeros(shape, dtype=dtype, device=self.device) if k is None else k
        v = torch.zeros(shape, dtype=dtype, device=self.device) if v is None else v
        dt = T._dtype_code(k)
        T._same(k.dtype, ("v", v))
        T._shape("k", k, shape)
        T._shape("v", v, shape)
        if not k.is_contiguous() or not v.is_contiguous():
            raise ValueError("k and v must be contiguous")
        _on(self.device, ("k", k), ("v", v), ("seqs", seqs))
        self._call("tm_cache_read", _at(seqs), _int(start), k.data_ptr(), v.data_ptr(), B, n_tokens, dt)
        return k, v

    def fork(self, src, dst, stream=None):
        """Sequence dst[i] (empty) becomes a copy of src[i] that shares its
        pages (int32 [n] each)."""
        if _elsewhere(self._index, stream):
            with _there(self.device, stream):
                return self.fork(src, dst)
        n = src.shape[0]

        def check():
            _list("src", src, n)
            _list("dst", dst, n)
            _on(self.device, ("src", src), ("dst", dst))
            return True

        _once((self._kind, "fork", _look(src), _look(dst)), check)
        self._call("tm_cache_fork", src.data_ptr(), dst.data_ptr(), n)

    def free(self, seqs, keep=None, stream=None):
        """Drops all tokens of the sequences, or those behind the first
        keep[i] (int32 [n] each; seqs None: 0 .. n_seqs - 1)."""
        if _elsewhere(self._index, stream):
            with _there(self.device, stream):
                return self.free(seqs, keep)
        n = self.n_seqs if seqs is None else seqs.shape[0]

        def check():
            _list("seqs", seqs, n)
            _list("keep", keep, n)
            _on(self.device, ("seqs", seqs), ("keep", keep))
            return True

        _once((self._kind, "free", n, _look(seqs), _look(keep)), check)
        self._call("tm_cache_free", _at(seqs), _at(keep), n)

    def compact(self, stream=None):
        """Moves the pages in use to the lowest numbers."""
        if _elsewhere(self._index, stream):
            with _there(self.device, stream):
                return self.compact()
        ws = self._workspace(0, 0, 0)
        self._call("tm_cache_compact", ws.data_ptr())

    def check(self, stream=None):
        """(sticky flags, pages in use); waits for the stream."""
        if _elsewhere(self._index, stream):
            with _there(self.device, stream):
                return self.check()
        f, n = _i(0), _i(0)
        self._call("tm_cache_check", ctypes.byref(f), ctypes.byref(n))
        return int(f.value), int(n.value)


def _product(x, w):
    """x times a weight of PyTorch's Linear layout, or an ``Int8Linear``.  The
    rows are one matrix (copied where a view of more axes does not allow it):
    of a view whose rows do not follow each other torch makes a batched product
    with the weight as a transposed operand of batch distance 0, and in bf16
    that has ended in a memory fault (an output's half of 2 x 1024 rows times
    1024 x 1024)."""
    if not isinstance(w, torch.Tensor):
        return w(x)
    return torch.nn.functional.linear(x.reshape(-1, x.shape[-1]), w).view(x.shape[:-1] + (w.shape[0],))


def _layer_weights(w_qkv, w_out, heads, kv_heads, norm, dtype):
    """(D, d, the vectors' type) of a layer's two projections, and their checks."""
    D, d = w_out.shape[0], w_out.shape[1] // heads
    for name, w, shape in (("w_out", w_out, (D, heads * d)), ("w_qkv", w_qkv, ((heads + 2 * kv_heads) * d, D))):
        if tuple(w.shape) != shape:
            raise ValueError("%s must have shape %s, got %s" % (name, shape, tuple(w.shape)))
    plain = [w for w in (w_qkv, w_out) if isinstance(w, torch.Tensor)]
    dtype = dtype or (plain[0].dtype if plain else torch.bfloat16)
    for w in plain:
        T._same(dtype, ("the weights", w))
    if norm is not None and (norm.heads, norm.kv_heads) != (heads, kv_heads):
        raise ValueError("the norm is for %d and %d heads, the layer has %d and %d"
                         % (norm.heads, norm.kv_heads, heads, kv_heads))
    return D, d, dtype


class WindowAttention:
    """The attention of ``mac_segment``'s window, for whole segments and for
    the single tokens that follow: grouped-query attention with rotary
    positions over a paged 8-bit cache.

    w_qkv [(heads + 2 kv_heads) d][D] and w_out [D][heads d] (PyTorch's Linear
    layout, bf16 or fp32) project the window's vectors and the result; the
    projections are plain products, or 8-bit ones where a weight is an
    ``Int8Linear`` (the vectors are then of ``dtype``, bf16 by default).
    ``norm`` (a ``HeadNorm`` of these heads) norms queries and keys, with the
    rotary positions it has in the same pass.  ``persistent`` [P][D] are the window's
    first rows, the same for every sequence and segment: their keys and
    values are written once, into a sequence of their own that each segment's
    sequences fork, so they share its pages.  ``batch`` sequences of up to
    ``max_tokens`` window tokens behind the persistent ones; ``rotary``
    rotates queries and keys by their place in the window (None: no
    positions).

    ``attention(window)`` takes [B][P + 2 S][D] (its first P rows are
    ``persistent``) and returns the attention output [B][S][D] for the
    segment's S rows; the window stays in the cache.  ``attention.token(x)``
    then takes the next tokens' vectors [B][n][D], behind what the cache
    holds, and returns theirs.  Nothing is recorded for gradients.  The tokens
    held are counted on the host, so these calls are not for capture into a
    graph (the cache's own are)."""

    def __init__(self, w_qkv, w_out, heads, kv_heads, batch, max_tokens, persistent=None, rotary=None, norm=None,
                 dtype=None):
        D, d, self.dtype = _layer_weights(w_qkv, w_out, heads, kv_heads, norm, dtype)
        T._same(self.dtype, ("persistent", persistent))
        if norm is not None and rotary is not None:
            raise ValueError("with a norm, the rotary positions are the norm's")
        self.P = 0 if persistent is None else persistent.shape[0]
        T._shape("persistent", persistent, (self.P, D))
        if max_tokens < 1 or batch < 1:
            raise ValueError("batch and max_tokens must be positive")
        self.w_qkv, self.w_out, self.heads, self.kv_heads, self.head_dim = w_qkv, w_out, heads, kv_heads, d
        self.batch, self.max_tokens, self.rotary, self.persistent = batch, max_tokens, rotary, persistent
        self.norm = norm
        dev = w_qkv.device
        up = lambda n: -(-n // TM_CACHE_PAGE)  # noqa: E731
        pages = up(self.P + max_tokens)
        self.cache = PagedCache(kv_heads, d, up(self.P) + batch * (pages - self.P // TM_CACHE_PAGE), batch + 1, pages,
                                device=dev)
        self._slots = torch.arange(batch, dtype=torch.int32, device=dev)
        self._root = torch.full((batch,), batch, dtype=torch.int32, device=dev)
        self._held = self.P   # tokens of each sequence
        self.refresh()

    @torch.no_grad()
    def refresh(self):
        """Starts over with the weights and persistent rows as they are now:
        the windows are dropped, the persistent tokens written again."""
        if self.P:
            k, v = self._project(self.persistent[None], 0)[1:]
        self.cache.free(None)
        self._held = self.P
        if self.P:
            self.cache.append(self._root[:1], k, v)
            self.cache.fork(self._root, self._slots)

    def _project(self, x, start):
        """Queries, keys (both rotated) and values of vectors that stand at
        ``start`` .. of their windows: views of one projection."""
        B, n, _ = x.shape
        qkv = _product(x, self.w_qkv).view(B, n, self.heads + 2 * self.kv_heads, self.head_dim)
        q_k = qkv[:, :, :self.heads + self.kv_heads]
        turn = self.rotary if self.norm is None else self.norm.rotary
        first = None if turn is None else torch.full((B,), start, dtype=torch.int32, device=x.device)
        if self.norm is not None:
            self.norm(q_k, first, out=q_k)
        elif turn is not None:
            turn(q_k, first, out=q_k)
        return qkv[:, :, :self.heads], qkv[:, :, self.heads:self.heads + self.kv_heads], \
            qkv[:, :, self.heads + self.kv_heads:]

    def _read(self, q):
        y = self.cache.attend(self._slots, q, max_len=self._held)
        return _product(y.flatten(2), self.w_out)

    def _room(self, x, n, held):
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("WindowAttention counts its tokens on the host: it cannot be captured into a graph")
        T._same(self.dtype, ("the window", x))
        _on(self.cache.device, ("the window", x))
        if x.dim() != 3 or x.shape[0] != self.batch or x.shape[2] != self.w_qkv.shape[1]:
            raise ValueError("expected [%d][tokens][%d], got %s" % (self.batch, self.w_qkv.shape[1], tuple(x.shape)))
        if n < 1 or held + n > self.P + self.max_tokens:
            raise ValueError("%d tokens behind %d: the window holds %d" % (n, held, self.P + self.max_tokens))

    @torch.no_grad()
    def __call__(self, window):
        n = window.shape[1] - self.P
        self._room(window, n, self.P)
        if n % 2:
            raise ValueError("a window holds %d persistent rows and as many recalled as segment rows, got %d rows"
                             % (self.P, window.shape[1]))
        q, k, v = self._project(window[:, self.P:], self.P)   # before anything is dropped, should it fail
        self.cache.free(self._slots)
        if self.P:
            self.cache.fork(self._root, self._slots)
        self._held = self.P
        self.cache.append(self._slots, k, v)
        self._held = self.P + n
        return self._read(q[:, n // 2:])

    @torch.no_grad()
    def token(self, x):
        n = x.shape[1]
        self._room(x, n, self._held)
        q, k, v = self._project(x, self._held)
        self.cache.append(self._slots, k, v)
        self._held += n
        return self._read(q)
