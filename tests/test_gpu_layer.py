"""The layer's operators on the GPU against the fp64 oracle: norms of queries
and keys with rotary positions, linear attention with a decay and the
gradients of both, products with 8-bit integers.

Tolerances, per element, with u = 2^-24.  Norms: a sum of d squares and its
root, the weight and the rotation (its angle as in the rotation's own test)
in fp32, one rounding to the dtype.  Linear attention: with |.| the same
formula over absolute values, a weight of a pair and a state's element carry
(T + 2 d + 256) u (sums over tokens and widths in fp32; an exponential's
argument of up to 150 rounded to fp32), bf16 calls round a pair's weight to 8
bits (r = 2^-8) and read the state with 16; the result is rounded once.
Products with integers are exact up to three fp32 roundings, in a fixed order:
they are compared bit for bit."""
import math

import numpy as np
import pytest
import torch

import test_trained_neural_amd as T
from harness import say
from oracle import layer as O

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def normal(shape, seed, dtype=BF, scale=1.0):
    x = np.random.default_rng(seed).standard_normal(shape).astype(np.float32) * scale
    t = torch.from_numpy(x).to("cuda").to(dtype)
    return t, f64(t)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def within(got, want, tol, what):
    got = f64(got)
    off = np.abs(got - want)
    worst = float((off / np.maximum(tol, 1e-300)).max()) if off.size else 0.0
    say("%s: worst %.3f of its tolerance" % (what, worst))
    assert np.all(off <= tol), (what, worst)


# ---- head norms ----

NORMS = [  # dtype, B, T, heads, kv_heads, d, r, interleaved, per token, strided
    (BF, 2, 5, 3, 1, 64, 64, False, True, False), (BF, 1, 1, 1, 0, 2, 2, False, False, False),
    (BF, 3, 70, 8, 2, 128, 128, True, True, True), (F32, 2, 33, 6, 3, 96, 64, False, False, True),
    (F32, 1, 9, 1, 1, 33, 6, True, True, False), (BF, 2, 4, 2, 2, 37, 18, False, True, False),
    (BF, 1, 700, 1, 1, 40, 20, True, False, False), (F32, 4, 1, 32, 8, 256, 256, False, False, True),
    (BF, 2, 3, 5, 1, 33, 32, True, True, True), (BF, 2, 17, 4, 4, 64, 0, False, True, True),
    (BF, 1, 3, 2, 1, 1024, 1024, False, True, False), (BF, 1, 3, 2, 1, 1023, 510, False, True, False),
    (F32, 1, 3, 2, 1, 1000, 0, True, True, False), (BF, 1, 9, 3, 2, 210, 126, False, True, True),
    (BF, 1, 2, 1, 0, 1, 0, False, True, False), (F32, 1, 5, 2, 2, 512, 512, True, True, True)]


def norm_case(case):
    dtype, B, N, H, K, d, r, inter, per_token, strided = case
    x, _ = normal((B, N, H + K + 2, d), 1, dtype, 3.0)
    x = x[:, :, 1:H + K + 1] if strided else x[:, :, :H + K].contiguous()
    rng = np.random.default_rng(2)
    pos = rng.integers(-5, 1 << 20, (B, N) if per_token else B)
    full = pos if per_token else pos[:, None] + np.arange(N)
    rot = T.Rotary(r, base=500000.0, layout=T.TM_ROPE_INTERLEAVED if inter else T.TM_ROPE_HALF, scaling=T.TM_ROPE_PARTS,
                   factor=8.0, original_len=2048) if r else None
    w_q, wq = normal(d, 3, F32)
    w_k, wk = normal(d, 4, F32) if K else (None, None)
    norm = T.HeadNorm(H, K, w_q, w_k, eps=1e-3, rotary=rot)
    positions = ints(pos.tolist()) if r else None
    args = (full, rot.freq.cpu().numpy(), rot.result_scale, inter) if r else ()
    return x, norm, positions, wq, wk, args


def turned(size, case, args):
    """Error of a rotation of elements of `size`, and the size it can give them."""
    d, r, inter = case[5], case[6], case[7]
    err, big = np.zeros(size.shape), size.copy()
    if r:
        full, f, scale = args[:3]
        n = r // 2
        a, b = (size[..., 0:r:2], size[..., 1:r:2]) if inter else (size[..., :n], size[..., n:r])
        s = scale * (a + b)
        e = s * (2.0 ** -51 * np.abs(full[..., None] * f)[:, :, None] + 2.0 ** -21)
        for to, v in ((err, e), (big, s)):
            if inter:
                to[..., 0:r:2] = to[..., 1:r:2] = v
            else:
                to[..., :n] = to[..., n:r] = v
    return err, big


@pytest.mark.parametrize("case", NORMS, ids=lambda c: "-".join(str(x) for x in c))
def test_head_norm(case):
    dtype, H, d = case[0], case[3], case[5]
    x, norm, positions, wq, wk, args = norm_case(case)
    y = norm(x, positions)
    want = O.head_norm(f64(x), wq, wk, H, 1e-3, *args)
    plain = np.abs(O.head_norm(f64(x), wq, wk, H, 1e-3))
    err, big = turned(plain, case, args)
    within(y, want, err + big * (d + 16) * U + np.abs(want) * torch.finfo(dtype).eps / 2, "y")
    z = x.clone() if x.is_contiguous() else x
    norm(z, positions, out=z)   # in place
    assert torch.equal(z, y)


@pytest.mark.parametrize("case", NORMS, ids=lambda c: "-".join(str(x) for x in c))
def test_head_norm_backward(case):
    dtype, B, N, H, K, d = case[:6]
    x, norm, positions, wq, wk, args = norm_case(case)
    dy, _ = normal(x.shape, 7, dtype)
    dx, dw_q, dw_k = norm.backward(x, dy, positions)
    X, G = f64(x), f64(dy)
    want = O.head_norm_backward(X, G, wq, wk, H, 1e-3, *args)
    r = 1.0 / np.sqrt((X * X).mean(-1, keepdims=True) + 1e-3)
    w = np.concatenate([np.tile(np.abs(wq), (H, 1))] + ([np.tile(np.abs(wk), (K, 1))] if K else []))
    u = np.abs(X * r)
    err, big = turned(np.abs(G), case, args)
    small = (d + 16) * U
    tol = r * (w * err + u * (w * err * u).mean(-1, keepdims=True) + 2 * small * (w * big + u * (w * big * u).mean(-1, keepdims=True)))
    within(dx, want[0], tol + np.abs(want[0]) * torch.finfo(dtype).eps / 2, "dx")
    part = (err * u + big * u * (small + (B * N * max(H, K) + 32) * U)).sum((0, 1))
    within(dw_q, want[1], part[:H].sum(0), "dw_q")
    if K:
        within(dw_k, want[2], part[H:].sum(0), "dw_k")
    else:
        assert dw_k is None
    for over in (dy, x):   # dx in the place of either
        if over.is_contiguous() and (over is dy or x.is_contiguous()):
            a, g = x.clone(), dy.clone()
            got = norm.backward(a, g, positions, dx=g if over is dy else a)
            assert torch.equal(got[0], dx) and torch.equal(got[1], dw_q)


def test_head_norm_many_tokens_and_streams():
    """More tokens than the backward has workgroups, arrays past the caches' size, another stream."""
    norm = T.HeadNorm(4, 2, *(normal(64, s, F32)[0] for s in (1, 2)))
    x, dy = normal((3, 9001, 6, 64), 3)[0], normal((3, 9001, 6, 64), 4)[0]
    y, (dx, dq, dk) = norm(x), norm.backward(x, dy)
    want = O.head_norm_backward(f64(x), f64(dy), f64(norm.w_q), f64(norm.w_k), 4, 1e-6)
    for g, w in ((dq, want[1]), (dk, want[2])):
        assert np.linalg.norm(f64(g) - w) <= 1e-6 * np.linalg.norm(w) * math.sqrt(64)
    assert np.abs(f64(dx) - want[0]).max() <= 2.0 ** -8 * np.abs(want[0]).max()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y2, (dx2, dq2, dk2) = norm(x, stream=s), norm.backward(x, dy, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(dq, dq2) and torch.equal(dk, dk2)
    big = torch.randn(2, 16384, 40, 128, device="cuda").to(BF)   # 2 x 335 MB
    n = T.HeadNorm(32, 8)
    got = n(big)
    part = n(big[:, 5000:5003].contiguous())
    assert torch.equal(got[:, 5000:5003], part)


def test_head_norm_edges():
    n = T.HeadNorm(2, 1, eps=0.0)
    x = torch.zeros(1, 2, 3, 8, device="cuda")
    x[0, 0, 1], x[0, 1, 2, 3] = 2.0, math.inf
    y = n(x)
    assert torch.isnan(y[0, 0, 0]).all() and torch.equal(y[0, 0, 1], torch.ones(8, device="cuda"))
    assert torch.isnan(y[0, 1, 2, 3]) and not y[0, 1, 2, :3].any()
    assert n(x[:0]).shape == (0, 2, 3, 8)
    dx, dq, dk = n.backward(x[:, :0], x[:, :0])
    assert dx.shape == (1, 0, 3, 8) and not dq.any() and not dk.any()


# ---- linear attention ----

LINEAR = [  # dtype, B, T, heads, kv_heads, dk, dv, per token, ragged, with a state
    (BF, 2, 1, 3, 3, 64, 64, True, False, True), (F32, 2, 5, 6, 2, 64, 64, False, False, True),
    (BF, 3, 16, 2, 1, 8, 16, True, True, False), (BF, 1, 17, 2, 2, 128, 128, True, False, True),
    (BF, 2, 64, 4, 4, 128, 128, True, False, True), (BF, 2, 65, 4, 2, 128, 128, False, True, True),
    (F32, 2, 130, 3, 1, 64, 96, True, True, True), (F32, 1, 100, 2, 2, 256, 40, True, False, True),
    (BF, 1, 200, 2, 1, 256, 256, True, True, True), (F32, 1, 90, 2, 1, 40, 256, False, False, False),
    (BF, 1, 600, 2, 1, 24, 72, True, False, True), (F32, 2, 700, 1, 1, 32, 8, True, True, True),
    (BF, 1, 1100, 1, 1, 128, 64, False, False, True), (BF, 5, 9, 8, 2, 136, 200, False, True, True),
    (F32, 1, 33, 1, 1, 104, 104, True, False, True), (BF, 1, 300, 6, 1, 16, 32, True, False, True)]


def linear_case(case, wipes=True):
    dtype, B, N, H, K, dk, dv, per_token, ragged, state = case
    (q, Q), (k, KK), (v, V) = (normal((B, N, h, d), s, dtype) for h, d, s in ((H, dk, 1), (K, dk, 2), (K, dv, 3)))
    rng = np.random.default_rng(5)
    g = -np.abs(rng.standard_normal((B, N, K) if per_token else K)) * np.exp(rng.uniform(-6, 1.5, (B, N, K) if per_token else K))
    if per_token and wipes:
        g.flat[:: 37] = -math.inf
        g.flat[5 :: 41] = 0.0
        g.flat[7 :: 53] = -3000.0
    g = torch.from_numpy(g.astype(np.float32)).to("cuda")
    counts = [(N * (b + 1)) // B if b else (0 if B > 2 else N // 2) for b in range(B)] if ragged else None
    s, S = normal((B, K, dk, dv), 4, F32) if state else (None, np.zeros((B, K, dk, dv)))
    return q, k, v, g, counts, s, (Q, KK, V, f64(g), S)


def linear_error(case):
    dtype, N, dk, dv = case[0], case[2], case[5], case[6]
    return (N + 2 * max(dk, dv) + 256) * U, (2.0 ** -8 if dtype == BF else 0.0), torch.finfo(dtype).eps / 2


@pytest.mark.parametrize("case", LINEAR, ids=lambda c: "-".join(str(x) for x in c))
def test_linear_attention(case):
    dtype, B, N, H, K, dk, dv = case[:7]
    q, k, v, g, counts, s, (Q, KK, V, G, S) = linear_case(case)
    m = T.LinearAttention(K, dk, dv)
    c = None if counts is None else ints(counts)
    y, end = m(q, k, v, g, state=s, counts=c)
    scale = 1 / math.sqrt(dk)
    want, want_s = O.linear(Q, KK, V, G, scale, S, counts)
    size, size_s = O.linear(*map(np.abs, (Q, KK, V)), G, scale, np.abs(S), counts)
    e, r, half = linear_error(case)
    within(y, want, size * (e + r) + np.abs(want) * half, "y")
    within(end, want_s, size_s * e, "state")
    # strided inputs, an output that keeps its rows behind the counts, the state in place
    cat = torch.cat((q, torch.zeros_like(q[:, :, :1])), 2)
    out = torch.full((B, N, H, dv), 7.0, dtype=dtype, device="cuda")
    own = m.init_state(B) if s is None else s.clone()
    y2, s2 = m(cat[:, :, :H], k, v, g, state=own, counts=c, out=out, state_out=own)
    assert s2.data_ptr() == own.data_ptr() and torch.equal(s2, end)
    for b in range(B):
        n = N if counts is None else counts[b]
        assert torch.equal(y2[b, :n], y[b, :n]) and (y2[b, n:] == 7.0).all() and not y[b, n:].any()


@pytest.mark.parametrize("case", LINEAR, ids=lambda c: "-".join(str(x) for x in c))
def test_linear_attention_backward(case):
    dtype, B, N, H, K, dk, dv, per_token = case[:8]
    q, k, v, g, counts, s, (Q, KK, V, G, S) = linear_case(case)
    dy, DY = normal((B, N, H, dv), 8, dtype)
    ds, DS = normal((B, K, dk, dv), 9, F32)
    m = T.LinearAttention(K, dk, dv)
    c = None if counts is None else ints(counts)
    got = m.backward(q, k, v, g, dy, state=s, dstate=ds, counts=c)
    scale = 1 / math.sqrt(dk)
    want = O.linear_backward(Q, KK, V, G, scale, S, DY, DS, counts)
    size = O.linear_backward(*map(np.abs, (Q, KK, V)), G, scale, np.abs(S), np.abs(DY), np.abs(DS), counts)
    e, r, half = linear_error(case)
    e *= H // K
    for n, name in enumerate(("dq", "dk", "dv")):
        within(got[n], want[n], size[n] * (e + r) + np.abs(want[n]) * half, name)
    within(got[4], want[4], size[4] * e, "dstate")
    # a decay's gradient is a difference of what flows into and out of the tokens behind it, within its segment
    flow = (np.abs(Q) * size[0]).reshape(B, N, K, -1).sum(-1) + (np.abs(KK) * size[1]).sum(-1)
    flow = np.stack([flow[:, a:a + 256].sum(1) for a in range(0, N, 256)], 1).repeat(256, 1)[:, :N]
    last = (size[4] * np.abs(S)).sum((2, 3))[:, None]
    ends = np.abs(size[3]) + flow + last
    tol = ends * e
    if not per_token:
        within(got[3], want[3].sum((0, 1)), tol.sum((0, 1)), "dlog_decay")
    else:
        if counts is not None:
            for b in range(B):
                assert not got[3][b, counts[b]:].any()
        within(got[3], want[3], tol, "dlog_decay")
    # and altogether, a token's to 1e-5 of their mean size; a head's is the sum of n = B N of them, whose errors may
    # have one sign (what passes a chunk is in all its tokens): n 1e-5 rms = sqrt(n) 1e-5 norm
    off = np.linalg.norm(f64(got[3]) - (want[3] if per_token else want[3].sum((0, 1))))
    assert off <= 1e-5 * np.linalg.norm(want[3]) * (1.0 if per_token else math.sqrt(B * N))


def test_linear_attention_stepwise():
    """A prompt in one call, in pieces, and token by token: the same within the tolerances of both."""
    B, N, H, K, d = 2, 150, 4, 2, 64
    case = (BF, B, N, H, K, d, d, True, False, True)
    q, k, v, g, _, s, (Q, KK, V, G, S) = linear_case(case)
    m = T.LinearAttention(K, d)
    want, want_s = O.linear(Q, KK, V, G, d ** -0.5, S)
    size, size_s = O.linear(*map(np.abs, (Q, KK, V)), G, d ** -0.5, np.abs(S))
    e, r, half = linear_error(case)
    for cuts in ([0, 150], [0, 64, 150], [0, 1, 2, 19, 20, 100, 149, 150], list(range(151))):
        st, ys = s, []
        for a, b in zip(cuts, cuts[1:]):
            y, st = m(q[:, a:b], k[:, a:b], v[:, a:b], g[:, a:b].contiguous(), state=st)
            ys.append(y)
        within(torch.cat(ys, 1), want, size * (e + r) + np.abs(want) * half, "y of %d pieces" % (len(cuts) - 1))
        within(st, want_s, size_s * e, "state of %d pieces" % (len(cuts) - 1))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513, 1025])
def test_linear_attention_at_every_border(N, dtype):
    """Lengths around the chunks', segments' and token path's borders, forward and backward; tokens first in memory,
    keys and values shared by the batch, the same call twice bit for bit."""
    B, H, K, dk, dv = 2, 2, 1, 16, 24
    case = (dtype, B, N, H, K, dk, dv, True, False, True)
    q, k, v, g, _, s, (Q, KK, V, G, S) = linear_case(case)
    q = q.transpose(0, 1).contiguous().transpose(0, 1)       # [T][B] in memory
    k, v = k[:1].expand(B, -1, -1, -1), v[:1].expand(B, -1, -1, -1)
    KK, V = np.repeat(KK[:1], B, 0), np.repeat(V[:1], B, 0)
    m = T.LinearAttention(K, dk, dv)
    y, end = m(q, k, v, g, state=s)
    scale = dk ** -0.5
    want, want_s = O.linear(Q, KK, V, G, scale, S)
    size, size_s = O.linear(*map(np.abs, (Q, KK, V)), G, scale, np.abs(S))
    e, r, half = linear_error(case)
    within(y, want, size * (e + r) + np.abs(want) * half, "y")
    within(end, want_s, size_s * e, "state")
    again = m(q, k, v, g, state=s)
    assert torch.equal(again[0], y) and torch.equal(again[1], end)
    dy, DY = normal((B, N, H, dv), 8, dtype)
    got = m.backward(q, k, v, g, dy, state=s)
    want = O.linear_backward(Q, KK, V, G, scale, S, DY, np.zeros_like(S))
    size = O.linear_backward(*map(np.abs, (Q, KK, V)), G, scale, np.abs(S), np.abs(DY), np.zeros_like(S))
    for n, name in enumerate(("dq", "dk", "dv")):
        within(got[n], want[n], size[n] * (2 * e + r) + np.abs(want[n]) * half, name)
    within(got[4], want[4], size[4] * 2 * e, "dstate")
    assert np.linalg.norm(f64(got[3]) - want[3]) <= 1e-5 * np.linalg.norm(want[3])
    again = m.backward(q, k, v, g, dy, state=s)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk", range(8, 257, 8))
def test_linear_attention_at_every_width(dk, dtype):
    """Every width of keys, with values of 264 less it, over whole and begun chunks, forward and backward."""
    dv = 264 - dk
    case = (dtype, 2, 70, 2, 1, dk, dv, True, False, True)
    q, k, v, g, _, s, (Q, KK, V, G, S) = linear_case(case)
    m = T.LinearAttention(1, dk, dv)
    y, end = m(q, k, v, g, state=s)
    scale = dk ** -0.5
    want, want_s = O.linear(Q, KK, V, G, scale, S)
    size, size_s = O.linear(*map(np.abs, (Q, KK, V)), G, scale, np.abs(S))
    e, r, half = linear_error(case)
    within(y, want, size * (e + r) + np.abs(want) * half, "y")
    within(end, want_s, size_s * e, "state")
    dy, DY = normal((2, 70, 2, dv), 8, dtype)
    got = m.backward(q, k, v, g, dy, state=s)
    want = O.linear_backward(Q, KK, V, G, scale, S, DY, np.zeros_like(S))
    size = O.linear_backward(*map(np.abs, (Q, KK, V)), G, scale, np.abs(S), np.abs(DY), np.zeros_like(S))
    for n, name in enumerate(("dq", "dk", "dv")):
        within(got[n], want[n], size[n] * (2 * e + r) + np.abs(want[n]) * half, name)
    within(got[4], want[4], size[4] * 2 * e, "dstate")
    assert np.linalg.norm(f64(got[3]) - want[3]) <= 1e-5 * np.linalg.norm(want[3])


def test_linear_attention_wide_groups_and_far_rows():
    """64 query heads on one key head, rows a megabyte apart, a state of its own for none."""
    m = T.LinearAttention(1, 8)
    big = torch.zeros(1, 40, (1 << 19) + 512, dtype=BF, device="cuda")
    q = big[:, :, :512].unflatten(2, (64, 8))
    x, Q = normal((1, 40, 64, 8), 1)
    q.copy_(x)
    (k, KK), (v, V) = normal((1, 40, 1, 8), 2), normal((1, 40, 1, 8), 3)
    g = torch.full((1,), -0.1, device="cuda")
    for n in (40, 7):
        y, end = m(q[:, :n], k[:, :n], v[:, :n], g)
        want, ws = O.linear(Q[:, :n], KK[:, :n], V[:, :n], f64(g), 8 ** -0.5, np.zeros((1, 1, 8, 8)))
        size, _ = O.linear(*(np.abs(t[:, :n]) for t in (Q, KK, V)), f64(g), 8 ** -0.5, np.zeros((1, 1, 8, 8)))
        within(y, want, size * 2.0 ** -7 + np.abs(want) * 2.0 ** -8, "y")
        assert np.linalg.norm(f64(end) - ws) <= 1e-6 * np.linalg.norm(ws)
    z = torch.zeros(0, 5, 1, 8, dtype=BF, device="cuda")
    y, end = m(z, z, z, g)
    assert y.shape == (0, 5, 1, 8) and end.shape == (0, 1, 8, 8)
    assert not m.backward(z, z, z, g, z)[3].any()


@pytest.mark.parametrize("T_", [9, 100, 600])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_linear_attention_non_finite(T_, dtype):
    """A non-finite value or key touches no earlier output, one behind the count nothing."""
    m = T.LinearAttention(1, 64)
    q, k, v, g, _, s, _ = linear_case((dtype, 1, T_, 1, 1, 64, 64, True, False, True), wipes=False)
    y, _ = m(q, k, v, g, state=s)
    for name, what in (("v", v), ("k", k)):
        for value in (math.nan, math.inf):
            at = T_ - 4
            bad = what.clone()
            bad[0, at, 0, 3] = value
            z, end = m(q, bad if name == "k" else k, bad if name == "v" else v, g, state=s)
            assert torch.equal(z[0, :at], y[0, :at]) and not torch.isfinite(z[0, at:, 0, 3]).any()
            assert not torch.isfinite(end[0, 0, :, 3]).all()
            z, end = m(q, bad if name == "k" else k, bad if name == "v" else v, g, state=s, counts=ints([at]))
            assert torch.equal(z[0, :at], y[0, :at]) and torch.isfinite(end).all()


def test_linear_attention_empty():
    m = T.LinearAttention(2, 16, 8)
    s = normal((3, 2, 16, 8), 1, F32)[0]
    e = lambda n, h, d: torch.zeros(3, n, h, d, dtype=BF, device="cuda")  # noqa: E731
    y, end = m(e(0, 4, 16), e(0, 2, 16), e(0, 2, 8), torch.zeros(2, device="cuda"), state=s)
    assert y.shape == (3, 0, 4, 8) and torch.equal(end, s)
    got = m.backward(e(0, 4, 16), e(0, 2, 16), e(0, 2, 8), torch.zeros(2, device="cuda"), e(0, 4, 8), dstate=s)
    assert torch.equal(got[4], s) and not got[3].any()
    y, end = m(e(3, 4, 16), e(3, 2, 16), e(3, 2, 8), torch.zeros(3, 3, 2, device="cuda"), state=s, counts=ints([0, 0, 0]))
    assert torch.equal(end, s)
    y, end = m(e(700, 4, 16), e(700, 2, 16), e(700, 2, 8), torch.zeros(2, device="cuda"), state=s, counts=ints([-5, 0, 9000]))
    assert torch.equal(end, s) and not y.any()


# ---- products with 8-bit integers ----

INT8 = [  # dtype, rows, cols, outs
    (BF, 1, 1, 1), (BF, 1, 64, 128), (F32, 3, 100, 7), (BF, 8, 1024, 300), (BF, 16, 4096, 128), (F32, 17, 33, 129),
    (BF, 33, 257, 64), (F32, 129, 384, 131), (BF, 130, 1000, 257), (BF, 300, 384, 1152), (F32, 5, 131072, 3),
    (BF, 600, 64, 5), (BF, 2, 16, 4097), (F32, 257, 2047, 385), (BF, 1024, 512, 768)]


def rounded(x, dtype):
    """fp64 values rounded once: an fp32 value halfway between two of bf16 goes to the side of what it came from."""
    f = x.astype(np.float32)
    if dtype == BF:
        half = (f.view(np.uint32) & 0xFFFF) == 0x8000
        f = np.where(half & (f != x), np.nextafter(f, np.where(x > f, np.float32(np.inf), np.float32(-np.inf))), f)
    return torch.from_numpy(f).to(dtype)


def int8_case(dtype, M, K, N):
    x, X = normal((M, K), 1, dtype, 2.0)
    w, W = normal((N, K), 2, F32)
    return x, w, O.int8_rows(X), O.int8_rows(W)


@pytest.mark.parametrize("case", INT8, ids=lambda c: "-".join(str(x) for x in c))
def test_int8_linear(case):
    dtype, M, K, N = case
    x, w, (cx, sx), (cw, sw) = int8_case(*case)
    lin = T.Int8Linear(w)
    assert np.array_equal(lin.codes[:, :K].cpu().numpy(), cw) and not lin.codes[:, K:].any()
    assert np.array_equal(lin.scales.cpu().numpy(), sw)
    wide = lin.codes.shape[1]
    codes, scales = torch.full((M, wide), 9, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    T.tm_int8_quantize(x, codes, scales)
    assert np.array_equal(codes[:, :K].cpu().numpy(), cx) and not codes[:, K:].any()
    assert np.array_equal(scales.cpu().numpy(), sx)
    sums = (cx.astype(np.float64) @ cw.T.astype(np.float64))   # whole numbers, exact
    want = rounded(sums * sx[:, None].astype(np.float64) * sw[None].astype(np.float64), dtype)
    y = lin(x)
    assert torch.equal(y.cpu(), want)
    z = torch.full((M, N + 3), 5.0, dtype=dtype, device="cuda")   # rows that are further apart
    T.tm_int8_matmul(codes, scales, lin.codes, lin.scales, z[:, 1:N + 1], K)
    assert torch.equal(z[:, 1:N + 1], y) and (z[:, 0] == 5).all() and (z[:, N + 1:] == 5).all()
    wide_x = torch.zeros(M, K + 5, dtype=dtype, device="cuda")
    wide_x[:, 2:K + 2] = x
    assert torch.equal(lin(wide_x[:, 2:K + 2]), y)
    assert torch.equal(lin(x.view(1, M, K))[0], y)


def test_int8_edges():
    x = torch.zeros(7, 40, dtype=F32, device="cuda")
    x[1, 3], x[2, 5], x[3, 7] = math.nan, -math.inf, 1e-42
    x[4] = 3.4e38 * torch.linspace(-1, 1, 40)
    x[5, 0], x[5, 1] = 127.0, 2.5     # halfway between two codes: to the even one
    x[6, 0], x[6, 1] = -127.0, 3.5
    codes, scales = torch.empty(7, 48, dtype=torch.int8, device="cuda"), torch.empty(7, device="cuda")
    T.tm_int8_quantize(x, codes, scales)
    want, ws = O.int8_rows(x.cpu().numpy())
    assert np.array_equal(codes[:, :40].cpu().numpy(), want) and np.array_equal(scales.cpu().numpy(), ws, equal_nan=True)
    assert codes[5, 1] == 2 and codes[6, 1] == 4 and codes[3, 7] == 127 and not codes[:, 40:].any()
    lin = T.Int8Linear(torch.ones(3, 40, device="cuda"))
    y = lin(x)
    assert not y[0].any() and torch.isnan(y[1:3]).all() and torch.isfinite(y[3:]).all()
    assert lin(x[:0]).shape == (0, 3)
    # the largest sums
    full = T.Int8Linear(torch.ones(2, 131072, device="cuda"))
    y = full(torch.ones(1, 131072, dtype=BF, device="cuda"))
    assert abs(float(y[0, 0]) / 131072 - 1) <= 2.0 ** -8
    d = torch.randn(300, 512, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    lin = T.Int8Linear(torch.randn(300, 512, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda"))
    whole = lin(d)
    for n in (1, 2, 5, 16, 17, 40, 64, 100, 129):   # a row does not depend on how many there are
        assert torch.equal(lin(d[:n]), whole[:n])
