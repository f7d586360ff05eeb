"""A layer's operators beside the memory: Python binding of
``include/tm_layer.h``.

Norms of queries and keys for each head with their rotary positions, linear
attention with a decay (a memory of one matrix: prompts, single tokens and
the gradients), and products with weights held in 8-bit integers.  Argument
marshalling only, as in the package's other calls: the functions carry the C
names and check types, shapes and devices before a pointer is passed on.
``HeadNorm``, ``LinearAttention`` and ``Int8Linear`` keep weights and sizes
and allocate outputs and workspaces; ``LinearWindow`` puts them together as
an attention of ``mac_segment``.  Nothing here records gradients (a
``backward`` is a call of its own).

Calls run on the current stream of the tensors' device (or on ``stream``).
"""
from __future__ import annotations

import ctypes
import math

import torch

import test_trained_neural_amd as T
from .attention import (TM_ROPE_HALF, _aligned, _at, _elsewhere, _heads_of, _int, _layer_weights, _list, _look, _on, _once,
                        _product, _raw_stream, _there)

EXPORTED = ("tm_head_norm", "tm_head_norm_workspace_bytes", "tm_head_norm_backward", "tm_linear_attention",
            "tm_linear_workspace_bytes", "tm_linear_attention_backward", "tm_int8_quantize", "tm_int8_matmul",
            "tm_int8_workspace_bytes", "tm_int8_linear")

# kernel class of tm_timing_enable / tm_timing_read
K_LAYER = 11

_vp, _i, _l, _d, _z = ctypes.c_void_p, ctypes.c_int, ctypes.c_long, ctypes.c_double, ctypes.c_size_t
_declared = None


def _lib():
    global _declared
    if _declared is None:
        L = T.lib()
        token = [_vp, _l, _l]
        for name, res, args in (
                ("tm_head_norm", _i, token * 2 + [_vp, _vp, _d, _vp, _i, _vp, _d] + [_i] * 8 + [_vp]),
                ("tm_head_norm_workspace_bytes", _z, [_i] * 5),
                ("tm_head_norm_backward", _i,
                 token * 3 + [_vp] * 4 + [_d, _vp, _i, _vp, _d] + [_i] * 8 + [_vp, _vp]),
                ("tm_linear_attention", _i, token * 3 + [_vp, _i, _vp, _vp, _vp, _vp, _d] + [_i] * 7 + [_vp, _vp]),
                ("tm_linear_workspace_bytes", _z, [_i] * 7),
                ("tm_linear_attention_backward", _i,
                 token * 3 + [_vp, _i, _vp, _vp] + token + [_vp] * 6 + [_d] + [_i] * 7 + [_vp, _vp]),
                ("tm_int8_quantize", _i, [_vp, _l, _vp, _l, _vp, _l, _i, _i, _vp]),
                ("tm_int8_matmul", _i, [_vp, _vp, _vp, _vp, _l, _vp, _l, _l, _i, _i, _i, _vp]),
                ("tm_int8_workspace_bytes", _z, [_l, _i]),
                ("tm_int8_linear", _i, [_vp, _l, _vp, _vp, _l, _vp, _l, _l, _i, _i, _i, _vp, _vp])):
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _declared = L
    return _declared


def _f32(device, *named):
    """Contiguous fp32 tensors of a shape each (None tensors are skipped)."""
    for name, t, shape in named:
        T._same(torch.float32, (name, t))
        T._shape(name, t, shape)
        if t is not None and not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
        _on(device, (name, t))


# ---------------------------------------------------------------------------
# the C calls, one to one

def _norm_geometry(x, y, w_q, w_k, positions, freq, heads, kv_heads, dy=None):
    dt = T._dtype_code(x)
    T._same(x.dtype, ("y" if dy is None else "dx", y), ("dy", dy))
    T._shape("y" if dy is None else "dx", y, x.shape)
    T._shape("dy", dy, x.shape)
    _on(x.device, ("x", x), ("y", y), ("dy", dy), ("positions", positions), ("freq", freq))
    dist = [_heads_of("x", x, False), _heads_of("y", y, False)] + ([] if dy is None else [_heads_of("dy", dy, False)])
    B, N, H, d = x.shape
    if heads < 1 or kv_heads < 0 or heads + kv_heads != H:
        raise ValueError("x has %d heads, the call %d and %d" % (H, heads, kv_heads))
    _f32(x.device, ("w_q", w_q, (d,)), ("w_k", w_k, (d,)))
    per_token = 0
    if (freq is None) != (positions is None):
        raise ValueError("positions and freq are given together")
    if freq is not None:
        T._same(torch.int32, ("positions", positions))
        T._same(torch.float64, ("freq", freq))
        per_token = 1 if positions.dim() == 2 else 0
        T._shape("positions", positions, (B, N) if per_token else (B,))
        if not positions.is_contiguous() or not freq.is_contiguous() or freq.dim() != 1:
            raise ValueError("positions and freq must be contiguous")
    rot = 0 if freq is None else 2 * freq.shape[0]
    return dist, per_token, (B, N, heads, kv_heads, d, rot), dt, x.device.index


def tm_head_norm(x, y, w_q, w_k, heads, kv_heads, eps, positions=None, freq=None, result_scale=1.0,
                 layout=TM_ROPE_HALF, stream=None):
    """x, y [B][T][heads + kv_heads][d] (any distances between tokens and
    entries; y may be x); w_q, w_k fp32 [d] or None; positions int32 [B][T],
    or [B] (the first token's); freq [rot_dim / 2] fp64."""
    dist, per_token, sizes, dt, index = _once(
        ("head_norm", _look(x), _look(y), _look(w_q), _look(w_k), _look(positions), _look(freq), heads, kv_heads),
        lambda: _norm_geometry(x, y, w_q, w_k, positions, freq, heads, kv_heads))
    if _elsewhere(index, stream):
        with _there(x.device, stream):
            return tm_head_norm(x, y, w_q, w_k, heads, kv_heads, eps, positions, freq, result_scale, layout)
    rc = _lib().tm_head_norm(x.data_ptr(), *dist[0], y.data_ptr(), *dist[1], _at(w_q), _at(w_k), eps, _at(positions),
                             per_token, _at(freq), result_scale, *sizes, layout, dt, _raw_stream(index))
    if rc:
        T._check("tm_head_norm", rc)


def tm_head_norm_workspace_bytes(batch, n_tokens, heads, kv_heads, head_dim):
    return _lib().tm_head_norm_workspace_bytes(*map(_int, (batch, n_tokens, heads, kv_heads, head_dim)))


def tm_head_norm_backward(x, dy, dx, w_q, w_k, dw_q, dw_k, heads, kv_heads, eps, workspace, positions=None, freq=None,
                          result_scale=1.0, layout=TM_ROPE_HALF, stream=None):
    """dx (x's shape; may be dy or x), dw_q and dw_k (fp32 [d] or None) are
    written."""
    dist, per_token, sizes, dt, index = _once(
        ("head_norm_backward", _look(x), _look(dy), _look(dx), _look(w_q), _look(w_k), _look(positions), _look(freq),
         heads, kv_heads), lambda: _norm_geometry(x, dx, w_q, w_k, positions, freq, heads, kv_heads, dy))
    d = x.shape[3]
    _f32(x.device, ("dw_q", dw_q, (d,)), ("dw_k", dw_k, (d,)))
    if _elsewhere(index, stream):
        with _there(x.device, stream):
            return tm_head_norm_backward(x, dy, dx, w_q, w_k, dw_q, dw_k, heads, kv_heads, eps, workspace, positions,
                                         freq, result_scale, layout)
    T._blob("workspace", workspace, tm_head_norm_workspace_bytes(*sizes[:5]))
    _on(x.device, ("workspace", workspace))
    rc = _lib().tm_head_norm_backward(x.data_ptr(), *dist[0], dy.data_ptr(), *dist[2], dx.data_ptr(), *dist[1],
                                      _at(w_q), _at(w_k), _at(dw_q), _at(dw_k), eps, _at(positions), per_token,
                                      _at(freq), result_scale, *sizes, layout, dt, workspace.data_ptr(),
                                      _raw_stream(index))
    if rc:
        T._check("tm_head_norm_backward", rc)


def _linear_geometry(q, k, v, log_decay, counts, state_in, state_out, dout, dstate_out, outs):
    dt = T._dtype_code(q)
    T._same(q.dtype, ("k", k), ("v", v), ("dout", dout))
    named = [("q", q), ("k", k), ("v", v)] + ([] if dout is None else [("dout", dout)])
    dist = [_heads_of(*p) for p in named]
    B, N, H, dk = q.shape
    K, dv = v.shape[2:]
    T._shape("k", k, (B, N, K, dk))
    T._shape("v", v, (B, N, K, dv))
    T._shape("dout", dout, (B, N, H, dv))
    if H % K if K else True:
        raise ValueError("%d query heads do not share %d key heads" % (H, K))
    per_token = 1 if log_decay.dim() == 3 else 0
    _f32(q.device, ("log_decay", log_decay, (B, N, K) if per_token else (K,)),
         ("state_in", state_in, (B, K, dk, dv)), ("state_out", state_out, (B, K, dk, dv)),
         ("dstate_out", dstate_out, (B, K, dk, dv)))
    _list("counts", counts, B)
    _on(q.device, ("counts", counts), *named)
    for name, t, shape, dtype in outs((B, N, H, K, dk, dv)):
        T._same(dtype, (name, t))
        T._shape(name, t, shape)
        if t is not None and not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
        _on(q.device, (name, t))
    return dist, per_token, (B, N, H, K, dk, dv), dt, q.device.index


def tm_linear_workspace_bytes(batch, n_tokens, heads, kv_heads, key_dim, value_dim, backward=False):
    return _lib().tm_linear_workspace_bytes(*map(_int, (batch, n_tokens, heads, kv_heads, key_dim, value_dim)),
                                            1 if backward else 0)


def _tokens(named, dist):
    return [x for (name, t), d in zip(named, dist) for x in (_aligned(name, t.data_ptr()), *d)]


def tm_linear_attention(q, k, v, log_decay, out, scale, workspace, state_in=None, state_out=None, counts=None,
                        stream=None):
    """q [B][T][heads][key_dim], k [B][T][kv_heads][key_dim], v
    [B][T][kv_heads][value_dim] (any distances between tokens and entries that
    are multiples of 8), log_decay fp32 [B][T][kv_heads] or [kv_heads], out
    [B][T][heads][value_dim], states fp32 [B][kv_heads][key_dim][value_dim]
    (state_out may be state_in)."""
    def check():
        return _linear_geometry(q, k, v, log_decay, counts, state_in, state_out, None, None, lambda z: (
            ("out", out, (z[0], z[1], z[2], z[5]), q.dtype),))

    dist, per_token, sizes, dt, index = _once(
        ("linear", _look(q), _look(k), _look(v), _look(log_decay), _look(counts), _look(state_in), _look(state_out),
         _look(out)), check)
    if _elsewhere(index, stream):
        with _there(q.device, stream):
            return tm_linear_attention(q, k, v, log_decay, out, scale, workspace, state_in, state_out, counts)
    _room(workspace, tm_linear_workspace_bytes(*sizes), q.device)
    rc = _lib().tm_linear_attention(*_tokens((("q", q), ("k", k), ("v", v)), dist), log_decay.data_ptr(), per_token,
                                    _at(counts), _at(state_in), _at(state_out), out.data_ptr(), scale, *sizes, dt,
                                    _at(workspace), _raw_stream(index))
    if rc:
        T._check("tm_linear_attention", rc)


def _room(workspace, need, device):
    """A workspace holds what the call needs (None: where it needs nothing)."""
    if need or workspace is not None:
        T._blob("workspace", workspace, max(need, 1))
        _on(device, ("workspace", workspace))


def tm_linear_attention_backward(q, k, v, log_decay, dout, dq, dk, dv, scale, workspace, state_in=None,
                                 dstate_out=None, dlog_decay=None, dstate_in=None, counts=None, stream=None):
    """dq, dk, dv (contiguous, of q's type), dlog_decay (fp32, log_decay's
    shape, or None) and dstate_in (fp32 or None; may be dstate_out) are
    written."""
    def check():
        return _linear_geometry(q, k, v, log_decay, counts, state_in, None, dout, dstate_out, lambda z: (
            ("dq", dq, q.shape, q.dtype), ("dk", dk, k.shape, q.dtype), ("dv", dv, v.shape, q.dtype),
            ("dlog_decay", dlog_decay, log_decay.shape, torch.float32),
            ("dstate_in", dstate_in, (z[0], z[3], z[4], z[5]), torch.float32)))

    dist, per_token, sizes, dt, index = _once(
        ("linear_backward", _look(q), _look(k), _look(v), _look(log_decay), _look(counts), _look(state_in),
         _look(dout), _look(dstate_out), _look(dq), _look(dk), _look(dv), _look(dlog_decay), _look(dstate_in)), check)
    if _elsewhere(index, stream):
        with _there(q.device, stream):
            return tm_linear_attention_backward(q, k, v, log_decay, dout, dq, dk, dv, scale, workspace, state_in,
                                                dstate_out, dlog_decay, dstate_in, counts)
    _room(workspace, tm_linear_workspace_bytes(*sizes, True), q.device)
    a = _tokens((("q", q), ("k", k), ("v", v), ("dout", dout)), dist)
    rc = _lib().tm_linear_attention_backward(*a[:9], log_decay.data_ptr(), per_token, _at(counts), _at(state_in),
                                             *a[9:], _at(dstate_out), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                             _at(dlog_decay), _at(dstate_in), scale, *sizes, dt, _at(workspace),
                                             _raw_stream(index))
    if rc:
        T._check("tm_linear_attention_backward", rc)


def _rows_of(name, t):
    """(rows, columns, distance) of a 2-d tensor with contiguous rows."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("%s must be [rows][columns] with contiguous rows" % name)
    return t.shape[0], t.shape[1], t.shape[1] if t.shape[0] <= 1 else t.stride(0)


def _codes_of(name, codes, scales, rows, cols=None):
    T._same(torch.int8, (name, codes))
    T._same(torch.float32, ("%s's scales" % name, scales))
    if codes.dim() != 2 or not codes.is_contiguous() or not scales.is_contiguous():
        raise ValueError("%s must be contiguous [rows][columns], its scales contiguous" % name)
    T._shape(name, codes, (rows, codes.shape[1]))
    T._shape("%s's scales" % name, scales, (rows,))
    if codes.shape[1] % 16 or (cols is not None and codes.shape[1] < cols):
        raise ValueError("the rows of %s must be a multiple of 16 and hold the %s columns" % (name, cols))
    return codes.shape[1]


def tm_int8_quantize(x, codes, scales, stream=None):
    """x [rows][cols] (any distance between rows), codes int8
    [rows][code_row] (cols up to a multiple of 16), scales fp32 [rows]."""
    M, K, row = _rows_of("x", x)
    dt = T._dtype_code(x)
    wide = _codes_of("codes", codes, scales, M, K)
    _on(x.device, ("x", x), ("codes", codes), ("scales", scales))
    if _elsewhere(x.device.index, stream):
        with _there(x.device, stream):
            return tm_int8_quantize(x, codes, scales)
    T._check("tm_int8_quantize", _lib().tm_int8_quantize(x.data_ptr(), row, codes.data_ptr(), wide, scales.data_ptr(),
                                                         M, _int(K), dt, _raw_stream(x.device.index)))


def tm_int8_matmul(a, a_scales, w, w_scales, y, cols, stream=None):
    """y [rows][outs] (bf16 or fp32) from codes a [rows][code_row] and w
    [outs][code_row] with their scales; what stands behind ``cols`` in them
    must be zero."""
    M, N, row = _rows_of("y", y)
    dt = T._dtype_code(y)
    wide = _codes_of("a", a, a_scales, M, cols)
    if _codes_of("w", w, w_scales, N, cols) != wide:
        raise ValueError("the rows of a and w must be of one length")
    _on(y.device, ("y", y), ("a", a), ("a's scales", a_scales), ("w", w), ("w's scales", w_scales))
    if _elsewhere(y.device.index, stream):
        with _there(y.device, stream):
            return tm_int8_matmul(a, a_scales, w, w_scales, y, cols)
    T._check("tm_int8_matmul", _lib().tm_int8_matmul(a.data_ptr(), a_scales.data_ptr(), w.data_ptr(),
                                                     w_scales.data_ptr(), wide, y.data_ptr(), row, M, _int(N),
                                                     _int(cols), dt, _raw_stream(y.device.index)))


def tm_int8_workspace_bytes(rows, cols):
    return _lib().tm_int8_workspace_bytes(max(-1, min(rows, (1 << 62))), _int(cols))


def _int8_geometry(x, w, w_scales, y):
    M, K, x_row = _rows_of("x", x)
    dt = T._dtype_code(x)
    T._same(x.dtype, ("y", y))
    N = w.shape[0]
    T._shape("y", y, (M, N))
    y_row = _rows_of("y", y)[2]
    wide = _codes_of("w", w, w_scales, N, K)
    _on(x.device, ("x", x), ("y", y), ("w", w), ("w's scales", w_scales))
    return x_row, wide, y_row, (M, _int(N), _int(K)), dt, x.device.index


def tm_int8_linear(x, w, w_scales, y, workspace, stream=None):
    """y [rows][outs] = x [rows][cols] times w's rows: x's rows as codes
    (tm_int8_quantize), then tm_int8_matmul."""
    x_row, wide, y_row, sizes, dt, index = _once(("int8", _look(x), _look(w), _look(w_scales), _look(y)),
                                                 lambda: _int8_geometry(x, w, w_scales, y))
    if _elsewhere(index, stream):
        with _there(x.device, stream):
            return tm_int8_linear(x, w, w_scales, y, workspace)
    T._blob("workspace", workspace, tm_int8_workspace_bytes(sizes[0], sizes[2]) or 1)
    _on(x.device, ("workspace", workspace))
    rc = _lib().tm_int8_linear(x.data_ptr(), x_row, w.data_ptr(), w_scales.data_ptr(), wide, y.data_ptr(), y_row,
                               *sizes, dt, workspace.data_ptr(), _raw_stream(index))
    if rc:
        T._check("tm_int8_linear", rc)


def _zeros_like(*ts):
    """Contiguous tensors of zeros of the given ones' shapes and types, in one
    piece of memory (one fill), each 16-byte aligned."""
    at, places = 0, []
    for t in ts:
        places.append((at, at + T._nbytes(t)))
        at = -(-places[-1][1] // 16) * 16
    whole = ts[0].new_zeros(at, dtype=torch.uint8)
    return [whole[a:b].view(t.dtype).view(t.shape) for t, (a, b) in zip(ts, places)]


# ---------------------------------------------------------------------------

class HeadNorm:
    """Norms of queries and keys for each head, with their rotary positions in
    the same pass: ``y = norm(x, positions)`` takes x
    [B][T][heads + kv_heads][d], a view of a projection's output for instance.
    w_q, w_k: fp32 [d] (None: ones; w_k is not read without key heads); rotary:
    a ``Rotary`` (None: no rotation, positions are not read).
    ``backward(x, dy, positions)`` gives (dx, dw_q, dw_k) of the same call.
    The weights are read where they are at every call; other tensors in their
    place need another ``HeadNorm``."""

    def __init__(self, heads, kv_heads=0, w_q=None, w_k=None, eps=1e-6, rotary=None):
        if heads < 1 or kv_heads < 0:
            raise ValueError("heads must be positive, kv_heads not negative")
        w_k = w_k if kv_heads else None
        d = next((w.shape[0] for w in (w_q, w_k) if w is not None), None)
        for name, w in (("w_q", w_q), ("w_k", w_k)):
            if w is not None:
                _f32(w.device, (name, w, (d,)))
        self.heads, self.kv_heads, self.w_q, self.w_k, self.eps, self.rotary = heads, kv_heads, w_q, w_k, eps, rotary
        # what a call's checks go by, beside its own tensors
        self._kind = ("head_norm", heads, kv_heads, d, w_q is not None, w_k is not None,
                      *(w.device for w in (w_q, w_k) if w is not None),
                      None if rotary is None else (rotary.rot_dim, rotary.freq.device))

    def _rotation(self, positions):
        """The rotation's part of a call: positions, freq, result_scale, layout."""
        r = self.rotary
        if r is None:   # positions are not read
            return None, None, 1.0, TM_ROPE_HALF
        if positions is None:
            raise ValueError("positions are needed")
        return positions, r.freq, r.result_scale, r.layout

    def __call__(self, x, positions=None, out=None, stream=None):
        if stream is not None:
            _on(x.device, ("x", x))
            with _there(x.device, stream):
                return self(x, positions, out)
        positions, freq, result_scale, layout = self._rotation(positions)

        def check():
            y = x if out is None else out   # a new output is contiguous
            dist, per_token, sizes, dt, index = _norm_geometry(x, y, self.w_q, self.w_k, positions, freq, self.heads,
                                                               self.kv_heads)
            B, N, H, d = x.shape
            return dist[0], (N * H * d, H * d) if out is None else dist[1], per_token, sizes, dt, index

        d_x, d_y, per_token, sizes, dt, index = _once((self._kind, _look(x), _look(positions), _look(out)), check)
        if _elsewhere(index, None):
            with _there(x.device, None):
                return self(x, positions, out)
        if out is None:
            out = x.new_empty(x.shape)
        rc = _lib().tm_head_norm(x.data_ptr(), *d_x, out.data_ptr(), *d_y, _at(self.w_q), _at(self.w_k), self.eps,
                                 _at(positions), per_token, _at(freq), result_scale, *sizes, layout, dt,
                                 _raw_stream(index))
        if rc:
            T._check("tm_head_norm", rc)
        return out

    def backward(self, x, dy, positions=None, dx=None, stream=None):
        """(dx, dw_q, dw_k [d] fp32; dw_k None without key heads); dx may be
        dy or x."""
        if stream is not None:
            _on(x.device, ("x", x))
            with _there(x.device, stream):
                return self.backward(x, dy, positions, dx)
        if dx is None:
            dx = x.new_empty(x.shape)
        new = lambda: x.new_empty(x.shape[3], dtype=torch.float32)  # noqa: E731
        dw_q, dw_k = new(), new() if self.kv_heads else None
        ws = x.new_empty(tm_head_norm_workspace_bytes(*x.shape[:2], self.heads, self.kv_heads, x.shape[3]),
                         dtype=torch.uint8)
        tm_head_norm_backward(x, dy, dx, self.w_q, self.w_k, dw_q, dw_k, self.heads, self.kv_heads, self.eps, ws,
                              *self._rotation(positions))
        return dx, dw_q, dw_k


class LinearAttention:
    """Linear attention with a decay, a memory of one matrix for each key
    head: S_t = exp(log_decay_t) S_{t-1} + k_t v_t', y_t = scale S_t' q_t.

    ``y, state = memory(q, k, v, log_decay, state)`` takes prompts, drafts and
    single tokens; log_decay fp32 [B][T][kv_heads] (a gate for each token) or
    [kv_heads]; state fp32 [B][kv_heads][key_dim][value_dim] (None: zeros).
    scale: 1 / sqrt(key_dim) by default.  ``backward`` gives the gradients of
    the same call."""

    def __init__(self, kv_heads, key_dim, value_dim=None):
        value_dim = key_dim if value_dim is None else value_dim
        if kv_heads < 1 or not all(8 <= n <= 256 and n % 8 == 0 for n in (key_dim, value_dim)):
            raise ValueError("kv_heads must be positive, key_dim and value_dim multiples of 8 up to 256")
        self.kv_heads, self.key_dim, self.value_dim = kv_heads, key_dim, value_dim
        self._scale, self._kind = 1.0 / math.sqrt(key_dim), ("linear", kv_heads, key_dim, value_dim)

    def init_state(self, batch, device="cuda"):
        return torch.zeros((batch, self.kv_heads, self.key_dim, self.value_dim), dtype=torch.float32, device=device)

    def _sizes(self, q, k, v):
        for name, t, d in (("q", q, self.key_dim), ("k", k, self.key_dim), ("v", v, self.value_dim)):
            if t.dim() != 4 or t.shape[3] != d or (t is not q and t.shape[2] != self.kv_heads):
                raise ValueError("%s must be [batch][tokens][%s][%d], got %s"
                                 % (name, "heads" if t is q else self.kv_heads, d, tuple(t.shape)))
        B, N, H = q.shape[:3]
        return B, N, H, self.kv_heads, self.key_dim, self.value_dim

    def __call__(self, q, k, v, log_decay, state=None, counts=None, scale=None, out=None, state_out=None, stream=None):
        """(y [B][T][heads][value_dim], state behind the tokens).  counts
        int32 [B]: tokens of each entry; rows behind them are left as they
        were in ``out`` (zeros in a new output).  ``state_out`` may be
        ``state`` (the state is then updated in place)."""
        if stream is not None:
            _on(q.device, ("q", q))
            with _there(q.device, stream):
                return self(q, k, v, log_decay, state, counts, scale, out, state_out)
        def check():
            sizes = self._sizes(q, k, v)
            B, N, H, K, dk, dv = sizes
            dist, per_token, _, dt, index = _linear_geometry(
                q, k, v, log_decay, counts, state, state_out, None, None, lambda z: (("out", out, (B, N, H, dv), q.dtype),))
            return (dist[0], dist[1], dist[2], per_token, sizes, dt, index, (B, N, H, dv), (B, K, dk, dv),
                    tm_linear_workspace_bytes(*sizes))

        d_q, d_k, d_v, per_token, sizes, dt, index, shape, cells, need = _once(
            (self._kind, _look(q), _look(k), _look(v), _look(log_decay), _look(state), _look(counts), _look(out),
             _look(state_out)), check)
        if _elsewhere(index, None):
            with _there(q.device, None):
                return self(q, k, v, log_decay, state, counts, scale, out, state_out)
        if out is None:
            out = (q.new_empty if counts is None else q.new_zeros)(shape)
        if state_out is None:
            state_out = log_decay.new_empty(cells)
        ws = q.new_empty(need, dtype=torch.uint8) if need else None
        rc = _lib().tm_linear_attention(
            _aligned("q", q.data_ptr()), *d_q, _aligned("k", k.data_ptr()), *d_k, _aligned("v", v.data_ptr()), *d_v,
            log_decay.data_ptr(), per_token, _at(counts), _at(state), state_out.data_ptr(), out.data_ptr(),
            self._scale if scale is None else scale, *sizes, dt,
            _at(ws), _raw_stream(index))
        if rc:
            T._check("tm_linear_attention", rc)
        return out, state_out

    def backward(self, q, k, v, log_decay, dout, state=None, dstate=None, counts=None, scale=None, stream=None):
        """(dq, dk, dv, dlog_decay, dstate_in) of a call with these arguments:
        dout is the gradient of its y, dstate of the state that it returned
        (None: zeros).  Rows behind an entry's count are zero."""
        if stream is not None:
            _on(q.device, ("q", q))
            with _there(q.device, stream):
                return self.backward(q, k, v, log_decay, dout, state, dstate, counts, scale)
        def check():
            sizes = self._sizes(q, k, v)
            dist, per_token, _, dt, index = _linear_geometry(q, k, v, log_decay, counts, state, None, dout, dstate,
                                                             lambda z: ())
            return dist, per_token, sizes, dt, index, tm_linear_workspace_bytes(*sizes, True)

        (d_q, d_k, d_v, d_o), per_token, sizes, dt, index, need = _once(
            (self._kind, "backward", _look(q), _look(k), _look(v), _look(log_decay), _look(dout), _look(state),
             _look(dstate), _look(counts)), check)
        if _elsewhere(index, None):
            with _there(q.device, None):
                return self.backward(q, k, v, log_decay, dout, state, dstate, counts, scale)
        if counts is None:
            dq, dk, dv, dld = (t.new_empty(t.shape) for t in (q, k, v, log_decay))
        else:
            dq, dk, dv, dld = _zeros_like(q, k, v, log_decay)
        dstate_in = log_decay.new_empty((sizes[0],) + sizes[3:])
        ws = q.new_empty(need, dtype=torch.uint8) if need else None
        rc = _lib().tm_linear_attention_backward(
            _aligned("q", q.data_ptr()), *d_q, _aligned("k", k.data_ptr()), *d_k, _aligned("v", v.data_ptr()), *d_v,
            log_decay.data_ptr(), per_token, _at(counts), _at(state), _aligned("dout", dout.data_ptr()), *d_o, _at(dstate),
            dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dld.data_ptr(), dstate_in.data_ptr(),
            self._scale if scale is None else scale, *sizes, dt, _at(ws), _raw_stream(index))
        if rc:
            T._check("tm_linear_attention_backward", rc)
        return dq, dk, dv, dld, dstate_in


class Int8Linear:
    """A product with a weight held in 8-bit integers with a scale for each
    output: ``y = linear(x)``, x [..][cols] of bf16 or fp32, each of its rows
    taken as 8-bit integers with a scale too.

    ``Int8Linear(weight)`` lays out weight [outs][cols] (PyTorch's Linear
    layout); or codes int8 [outs][cols up to a multiple of 16] (zeros behind
    cols), scales fp32 [outs] and cols are given."""

    def __init__(self, weight=None, codes=None, scales=None, cols=None):
        if weight is not None:
            if codes is not None or scales is not None:
                raise ValueError("either weight or codes and scales")
            N, cols = weight.shape
            codes = torch.empty((N, -(-cols // 16) * 16), dtype=torch.int8, device=weight.device)
            scales = torch.empty(N, dtype=torch.float32, device=weight.device)
            tm_int8_quantize(weight, codes, scales)
        cols = codes.shape[1] if cols is None else cols
        wide = _codes_of("codes", codes, scales, codes.shape[0], cols)
        if wide - cols >= 16:
            raise ValueError("codes of %d columns for cols %d" % (wide, cols))
        _on(codes.device, ("scales", scales))
        self.codes, self.scales, self.cols, self.outs = codes, scales, cols, codes.shape[0]
        self._kind = ("int8_linear", codes.shape, cols, codes.device)   # what a call's checks go by, beside x and out

    @property
    def shape(self):
        return self.outs, self.cols

    @property
    def device(self):
        return self.codes.device

    def __call__(self, x, out=None, stream=None):
        """x [..][cols], any strides (copied where its rows are not contiguous,
        or of more than two axes and not contiguous); out: [..][outs],
        contiguous, or 2-d with contiguous rows (x being 2-d then)."""
        if stream is not None:
            _on(x.device, ("x", x))
            with _there(x.device, stream):
                return self(x, out)

        def check():
            _on(self.codes.device, ("x", x), ("out", out))
            dt = T._dtype_code(x)
            if x.dim() < 1 or x.shape[-1] != self.cols:
                raise ValueError("x is %s, the weight has %d columns" % (tuple(x.shape), self.cols))
            shape = x.shape[:-1] + (self.outs,)
            rows = math.prod(x.shape[:-1])
            rowwise = x.dim() == 2 and (self.cols <= 1 or x.stride(1) == 1)
            x_row = _rows_of("x", x)[2] if rowwise else self.cols
            y_row = self.outs
            if out is not None:
                T._same(x.dtype, ("out", out))
                T._shape("out", out, shape)
                if out.dim() == 2:
                    y_row = _rows_of("out", out)[2]
                elif not out.is_contiguous():
                    raise ValueError("out must be contiguous")
            return (not rowwise and not x.is_contiguous(), shape, x_row, y_row, (rows, _int(self.outs), self.cols), dt,
                    x.device.index, tm_int8_workspace_bytes(rows, self.cols))

        copy, shape, x_row, y_row, sizes, dt, index, need = _once((self._kind, _look(x), _look(out)), check)
        if _elsewhere(index, None):
            with _there(x.device, None):
                return self(x, out)
        if copy:
            x = x.contiguous()
        if out is None:
            out = x.new_empty(shape)
        ws = x.new_empty(need, dtype=torch.uint8)
        codes = self.codes
        rc = _lib().tm_int8_linear(x.data_ptr(), x_row, codes.data_ptr(), self.scales.data_ptr(), codes.shape[1],
                                   out.data_ptr(), y_row, *sizes, dt, ws.data_ptr(), _raw_stream(index))
        if rc:
            T._check("tm_int8_linear", rc)
        return out


def _logits(x, w):
    """x [..][D] times w [heads][D], in fp32 from the product on: a logit
    rounded to 8 bits is off by up to 2^-6 at 4, which the decays, summed over
    thousands of tokens, keep.  bf16 rows are read as they are (a copy of them
    in fp32 costs a window of 4 x 4096 rows of 4096 90 us of 960); for a single
    head they are copied, since the library takes 16 ms for one column of such
    a product."""
    if x.dtype == torch.float32 or w.shape[0] == 1:
        return _product(x.float(), w.float())
    return torch.mm(x.reshape(-1, x.shape[-1]), w.t(), out_dtype=torch.float32).view(x.shape[:-1] + (w.shape[0],))


class LinearWindow:
    """Linear attention as the attention of ``mac_segment``'s window and of
    the single tokens that follow, with a state in the place of
    ``WindowAttention``'s cache: it does not grow with what was read.

    w_qkv [(heads + 2 kv_heads) d][D], w_out [D][heads d], ``persistent``
    [P][D], ``norm`` and ``dtype`` as ``WindowAttention``'s (the norm's rotary
    positions count on from the window's first row).  What a token keeps of the
    past: ``log_decay`` fp32 [kv_heads], or a gate, the logarithm of
    sigmoid(x w_gate' + gate_bias), with w_gate [kv_heads][D] of the vectors'
    type and gate_bias fp32 [kv_heads] (None: zeros); the logits are formed in
    fp32.

    ``attention(window)`` takes [B][P + 2 S][D] (its first P rows are
    ``persistent``, whose state is kept) and returns the output [B][S][D] for
    the segment's S rows; ``attention.token(x)`` takes the next vectors
    [B][n][D] and returns theirs.  Nothing is recorded for gradients.  The
    tokens are counted on the host: not for capture into a graph
    (``LinearAttention`` itself is)."""

    def __init__(self, w_qkv, w_out, heads, kv_heads, batch, log_decay=None, w_gate=None, gate_bias=None,
                 persistent=None, norm=None, dtype=None):
        D, d, self.dtype = _layer_weights(w_qkv, w_out, heads, kv_heads, norm, dtype)
        T._same(self.dtype, ("persistent", persistent), ("w_gate", w_gate))
        if (log_decay is None) == (w_gate is None):
            raise ValueError("either log_decay or w_gate")
        if batch < 1:
            raise ValueError("batch must be positive")
        dev = w_qkv.device
        self.P = 0 if persistent is None else persistent.shape[0]
        T._shape("persistent", persistent, (self.P, D))
        T._shape("w_gate", w_gate, (kv_heads, D))
        _f32(dev, ("log_decay", log_decay, (kv_heads,)), ("gate_bias", gate_bias, (kv_heads,)))
        self.w_qkv, self.w_out, self.heads, self.kv_heads, self.head_dim, self.D = w_qkv, w_out, heads, kv_heads, d, D
        self.log_decay, self.w_gate, self.gate_bias = log_decay, w_gate, gate_bias
        self.batch, self.persistent, self.norm, self.device = batch, persistent, norm, dev
        self.memory = LinearAttention(kv_heads, d)
        self.refresh()

    @torch.no_grad()
    def refresh(self):
        """Starts over with the weights and persistent rows as they are now."""
        self.state = self._root = self.memory.init_state(self.batch, self.device)
        self._held = 0
        if self.P:
            rows = self.persistent[None].expand(self.batch, -1, -1)
            self._root = self._read(rows)[1]
        self.state, self._held = self._root.clone(), self.P

    def _read(self, x, out_state=None):
        """(outputs before w_out, state) of vectors behind the held ones."""
        B, n, _ = x.shape
        qkv = _product(x, self.w_qkv).view(B, n, self.heads + 2 * self.kv_heads, self.head_dim)
        q_k = qkv[:, :, :self.heads + self.kv_heads]
        if self.norm is not None:
            first = torch.full((B,), self._held, dtype=torch.int32, device=x.device)
            self.norm(q_k, first, out=q_k)
        g = self.log_decay
        if g is None:
            g = _logits(x, self.w_gate)
            g = torch.nn.functional.logsigmoid(g if self.gate_bias is None else g + self.gate_bias)
        return self.memory(qkv[:, :, :self.heads], qkv[:, :, self.heads:self.heads + self.kv_heads],
                           qkv[:, :, self.heads + self.kv_heads:], g, state=self.state, state_out=out_state)

    def _check(self, x):
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("LinearWindow counts its tokens on the host: it cannot be captured into a graph")
        T._same(self.dtype, ("the window", x))
        _on(self.device, ("the window", x))
        if x.dim() != 3 or x.shape[0] != self.batch or x.shape[2] != self.D:
            raise ValueError("expected [%d][tokens][%d], got %s" % (self.batch, self.D, tuple(x.shape)))

    @torch.no_grad()
    def __call__(self, window):
        self._check(window)
        n = window.shape[1] - self.P
        if n < 2 or n % 2:
            raise ValueError("a window holds %d persistent rows and as many recalled as segment rows, got %d rows"
                             % (self.P, window.shape[1]))
        state, held = self.state, self._held
        self.state, self._held = self._root, self.P
        try:
            y, self.state = self._read(window[:, self.P:])
        except Exception:   # what was read before is still there
            self.state, self._held = state, held
            raise
        self._held = self.P + n
        return _product(y[:, n // 2:].flatten(2), self.w_out)

    @torch.no_grad()
    def token(self, x):
        self._check(x)
        n = x.shape[1]
        if n < 1:
            raise ValueError("no tokens")
        y, _ = self._read(x, self.state)   # in place
        self._held += n
        return _product(y.flatten(2), self.w_out)
