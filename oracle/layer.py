"""fp64 model of the layer's operators (tests only): norms of head vectors
with rotary positions, linear attention with a decay, rows as 8-bit integers,
and their gradients.  Everything is taken token by token from the
definitions; nothing is shared with the library."""
import numpy as np

from oracle import attention as A


def _norm_parts(x, w_q, w_k, heads, eps):
    r = 1.0 / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    w = np.ones(x.shape[2:])
    if w_q is not None:
        w[:heads] = w_q
    if w_k is not None:
        w[heads:] = w_k
    return r, w


def head_norm(x, w_q, w_k, heads, eps, pos=None, freq=None, scale=1.0, interleaved=False):
    """x [B][T][H][d]; pos [B][T] or None."""
    r, w = _norm_parts(x, w_q, w_k, heads, eps)
    n = x * r * w
    return n if pos is None else A.rotate(n, pos, freq, scale, interleaved)


def head_norm_backward(x, dy, w_q, w_k, heads, eps, pos=None, freq=None, scale=1.0, interleaved=False):
    """(dx, dw_q, dw_k)."""
    r, w = _norm_parts(x, w_q, w_k, heads, eps)
    dn = dy if pos is None else A.rotate(dy, pos, freq, scale, interleaved, True)
    u = x * r
    dw = (dn * u).sum(axis=(0, 1))
    e = dn * w
    dx = r * (e - u * (e * u).mean(axis=-1, keepdims=True))
    return dx, dw[:heads].sum(axis=0), dw[heads:].sum(axis=0)


def _decays(g, B, T, K):
    return np.exp(np.broadcast_to(g, (B, T, K)))


def linear(q, k, v, g, scale, state, counts=None):
    """(y [B][T][H][dv], state): S = e^g S + k v', y = scale S' q."""
    B, T, H, dk = q.shape
    K, dv = v.shape[2:]
    keep = _decays(g, B, T, K)
    S, y = np.array(state, dtype=np.float64), np.zeros((B, T, H, dv))
    for b in range(B):
        for t in range(T if counts is None else counts[b]):
            S[b] = keep[b, t][:, None, None] * S[b] + k[b, t][:, :, None] * v[b, t][:, None, :]
            y[b, t] = scale * np.einsum("kgd,kde->kge", q[b, t].reshape(K, H // K, dk), S[b]).reshape(H, dv)
    return y, S


def linear_backward(q, k, v, g, scale, state, dy, dstate, counts=None):
    """(dq, dk, dv, dg [B][T][K], dstate_in)."""
    B, T, H, dk_ = q.shape
    K, dv_ = v.shape[2:]
    keep = _decays(g, B, T, K)
    dq, dk, dv, dg = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape), np.zeros((B, T, K))
    R = np.array(dstate, dtype=np.float64)
    for b in range(B):
        S = [np.array(state[b], dtype=np.float64)]
        n = T if counts is None else counts[b]
        for t in range(n):
            S.append(keep[b, t][:, None, None] * S[-1] + k[b, t][:, :, None] * v[b, t][:, None, :])
        for t in range(n - 1, -1, -1):
            yy = scale * dy[b, t].reshape(K, H // K, dv_)
            qq = q[b, t].reshape(K, H // K, dk_)
            R[b] += np.einsum("kgd,kge->kde", qq, yy)
            dq[b, t] = np.einsum("kde,kge->kgd", S[t + 1], yy).reshape(H, dk_)
            dk[b, t] = np.einsum("kde,ke->kd", R[b], v[b, t])
            dv[b, t] = np.einsum("kde,kd->ke", R[b], k[b, t])
            R[b] *= keep[b, t][:, None, None]
            dg[b, t] = (R[b] * S[t]).sum(axis=(1, 2))
    return dq, dk, dv, dg, R


def int8_rows(x):
    """(codes, scales) of rows of fp32 values, as the header defines them:
    (127 x) / m in fp32 (for bf16 values the same in 64 bits)."""
    x = x.astype(np.float32)
    m = np.abs(x).max(axis=1)
    fine = np.isfinite(m)
    with np.errstate(all="ignore"):
        down = np.where(m > 1e36, np.float32(2.0 ** -10), np.float32(1))[:, None]   # 127 x would overflow
        q = np.where((fine & (m > 0))[:, None], np.float32(127) * (x * down) / (m[:, None] * down), np.float32(0))
    scales = np.where(fine, m / np.float32(127), np.float32(np.nan)).astype(np.float32)
    return np.rint(np.where(fine[:, None], q, 0.0)).astype(np.int64), scales
