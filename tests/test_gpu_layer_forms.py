"""Every way in which the layer's operators are launched: the sizes here are
the ones at which a call takes another tile, division or loop than its
neighbours (the rules are beside the kernels), with remainders in each."""
import math

import numpy as np
import pytest
import torch

import test_gpu_layer as L
import test_trained_neural_amd as T
from oracle import layer as O
from test_gpu_layer import BF, F32, U, f64, ints, normal, within

pytestmark = pytest.mark.gpu


def seeded(shape, seed, dtype):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


# ---- products with 8-bit integers ----

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", [
    (777, 1000, 1537), (1000, 130, 1100),      # tiles of 64: begun steps of columns, begun tiles on both sides
    (2500, 200, 2700), (3300, 1040, 2048),     # of 128
    (3700, 150, 3700), (8200, 640, 1700),      # of 256: bands of eight tiles and begun ones
    (8, 8208, 4100), (3, 4112, 5001),          # rows coded by each workgroup, 32 rows of the weight each, many steps
    (16, 9000, 4100), (30, 5000, 700), (64, 3001, 200), (100, 8192, 300)],   # few rows, their codes made beforehand
    ids=lambda s: "x".join(map(str, s)))
def test_int8_launch_forms(size, dtype):
    """Bit for bit, with rows of the output that are an odd number of elements apart, and codes and product by themselves."""
    L.test_int8_linear((dtype, *size))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_int8_rows_are_the_same_in_every_form(dtype):
    """A row's result in tiles of 256, 128 and 64 and among few rows."""
    w, x = seeded((3700, 150), 1, F32), seeded((3700, 150), 2, dtype)
    lin = T.Int8Linear(w)
    whole = lin(x)
    for n in (1, 7, 16, 17, 33, 64, 65, 100, 700, 2500, 3699):
        assert torch.equal(lin(x[:n]), whole[:n]), n
        assert torch.equal(lin(x[-n:]), whole[-n:]), n


@pytest.mark.parametrize("dtype", [BF, F32])
def test_int8_takes_any_strides(dtype):
    """Rows whose elements are apart, of two axes as of three; one row, one column, rows shared by all."""
    lin = T.Int8Linear(seeded((40, 48), 1, F32))
    x = seeded((48, 30), 2, dtype)
    want = lin(x.t().contiguous())
    assert torch.equal(lin(x.t()), want) and torch.equal(lin(x.t()[None])[0], want)
    assert torch.equal(lin(x.t()[4:5]), want[4:5]) and torch.equal(lin(x[:, 4]), want[4])
    out = torch.zeros(30, 41, dtype=dtype, device="cuda")
    assert torch.equal(lin(x.t(), out=out[:, 1:]), want) and not out[:, 0].any()
    assert torch.equal(lin(x.t()[:1].expand(5, -1)), want[:1].expand(5, -1))
    one = T.Int8Linear(seeded((3, 1), 3, F32))
    assert torch.equal(one(x[:, 5:6]), one(x[:, 5:6].contiguous()))


# ---- linear attention: divided sequences of every width, long walks ----

DIVIDED = [  # dtype, B, T, heads, kv_heads, dk, dv, per token, ragged, with a state
    (BF, 1, 460, 4, 2, 128, 128, True, False, True), (BF, 2, 460, 2, 2, 160, 96, True, True, True),
    (BF, 1, 333, 2, 1, 192, 192, False, False, True), (F32, 1, 460, 3, 1, 64, 96, True, True, True),
    (F32, 2, 333, 2, 2, 128, 64, True, True, True), (F32, 1, 460, 2, 2, 96, 128, False, False, True),
    (F32, 1, 333, 2, 1, 184, 72, True, False, True), (F32, 1, 333, 1, 1, 256, 136, True, False, True),
    (BF, 1, 333, 1, 1, 232, 256, True, False, False),
    (BF, 1, 2100, 8, 8, 128, 128, True, False, True), (F32, 1, 2100, 9, 9, 64, 128, True, False, True)]   # 128 tokens at least


def linear_near(case, q, k, v, g, counts, s, host, entries, got):
    """Outputs and states of some of the entries against the oracle."""
    dtype, B, N, H, K, dk, dv = case[:7]
    Q, KK, V, G, S = host
    y, end = got
    at = lambda x: x[entries] if x.ndim > 1 else x  # noqa: E731
    n = None if counts is None else [counts[b] for b in entries]
    scale = 1 / math.sqrt(dk)
    want, want_s = O.linear(Q[entries], KK[entries], V[entries], at(G), scale, S[entries], n)
    size, size_s = O.linear(*(np.abs(x[entries]) for x in (Q, KK, V)), at(G), scale, np.abs(S[entries]), n)
    e, _, half = L.linear_error(case)
    r = 2.0 ** -16 if dtype == BF else 0.0   # a pair's weight and the state in two parts
    within(y[entries], want, size * (e + r) + np.abs(want) * half, "y")
    within(end[entries], want_s, size_s * e, "state")


@pytest.mark.parametrize("case", DIVIDED, ids=lambda c: "-".join(str(x) for x in c))
def test_linear_attention_divided(case):
    q, k, v, g, counts, s, host = L.linear_case(case)
    m = T.LinearAttention(case[4], case[5], case[6])
    got = m(q, k, v, g, state=s, counts=None if counts is None else ints(counts))
    linear_near(case, q, k, v, g, counts, s, host, list(range(case[1])), got)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,N,H,K,d", [(16, 513, 16, 16, 16), (16, 1100, 32, 16, 16), (16, 1025, 16, 16, 8),   # undivided
                                       (8, 2300, 32, 16, 8)])                                                  # four of 576
def test_linear_attention_long_walks(B, N, H, K, d, dtype):
    """A workgroup's walk over more than the 512 tokens whose decays are summed at a time, whole and ragged, with tokens
    that drop the past around each such border."""
    case = (dtype, B, N, H, K, d, d, True, False, True)
    q, k, v, g, _, s, host = L.linear_case(case)
    for t in (510, 511, 512, 513, 576, 1023, 1024, 1088):
        if t < N:
            g[t % B, t] = -math.inf
            g[(t + 1) % B, t] = 0.0
    host = (*host[:3], f64(g), host[4])
    m = T.LinearAttention(K, d)
    counts = [N - 37 * b if b % 3 else N for b in range(B)]
    counts[1] = 512
    entries = [0, 1, B // 2 + 1, B - 1]
    for c in (None, counts):
        got = m(q, k, v, g, state=s, counts=None if c is None else ints(c))
        linear_near(case, q, k, v, g, c, s, host, entries, got)
        if c is not None:
            for b in range(B):
                assert not got[0][b, c[b]:].any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(128, 128), (192, 64), (64, 192), (256, 256)])
def test_linear_attention_backward_of_several_segments(dk, dv, dtype):
    """Gradients through several segments, their length halved or not, at the widths whose kernels differ."""
    case = (dtype, 2, 300, 2, 1, dk, dv, True, True, True)
    L.test_linear_attention_backward(case)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [4, 7, 90, 500])
def test_linear_attention_grows_and_turns(N, dtype):
    """Decays above 0 (the state grows), a negative scale, views of one projection and of a wider gradient, without a state."""
    B, H, K, d = 2, 4, 2, 32
    case = (dtype, B, N, H, K, d, d, True, False, False)
    wide, _ = normal((B, N, H + 2 * K + 1, d), 21, dtype)
    q, k, v = wide[:, :, :H], wide[:, :, H:H + K], wide[:, :, H + K:H + 2 * K]
    Q, KK, V = f64(q), f64(k), f64(v)
    g = seeded((B, N, K), 22, F32) * 0.3
    dwide, _ = normal((B, N, H + 3, d), 23, dtype)
    dy = dwide[:, :, 2:H + 2]
    m, zero = T.LinearAttention(K, d), np.zeros((B, K, d, d))
    y, end = m(q, k, v, g, scale=-0.3)
    e, _, half = L.linear_error(case)
    r = 2.0 ** -16 if dtype == BF else 0.0
    want, want_s = O.linear(Q, KK, V, f64(g), -0.3, zero)
    size, size_s = O.linear(*map(np.abs, (Q, KK, V)), f64(g), 0.3, zero)
    within(y, want, size * (e + r) + np.abs(want) * half, "y")
    within(end, want_s, size_s * e, "state")
    got = m.backward(q, k, v, g, dy, scale=-0.3)
    want = O.linear_backward(Q, KK, V, f64(g), -0.3, zero, f64(dy), zero)
    size = O.linear_backward(*map(np.abs, (Q, KK, V)), f64(g), 0.3, zero, np.abs(f64(dy)), zero)
    for n, name in enumerate(("dq", "dk", "dv")):
        within(got[n], want[n], size[n] * (2 * e + r) + np.abs(want[n]) * half, name)
    within(got[4], want[4], size[4] * 2 * e, "dstate")
    assert np.linalg.norm(f64(got[3]) - want[3]) <= 1e-5 * np.linalg.norm(want[3])
    same = m.backward(q.contiguous(), k.contiguous(), v.contiguous(), g, dy.contiguous(), scale=-0.3)
    assert all(torch.equal(a, b) for a, b in zip(got, same))


# ---- head norms: several tokens a group of lanes, arrays past the caches ----

@pytest.mark.parametrize("dtype,inter", [(F32, False), (F32, True), (BF, False)])
def test_head_norm_backward_of_several_tokens(dtype, inter):
    """More groups of tokens than partial sums: a group of lanes walks over two and three tokens, from one entry into the
    next, with angles and sums of its own; the last group is a begun one."""
    B, N, d = 3, (5501 if dtype == F32 else 22003), 128
    case = (dtype, B, N, 2, 1, d, d, inter, True, False)
    L.test_head_norm_backward(case)


@pytest.mark.parametrize("dtype,layout", [(BF, T.TM_ROPE_HALF), (BF, T.TM_ROPE_INTERLEAVED), (F32, T.TM_ROPE_HALF)])
def test_head_norm_past_the_caches(dtype, layout):
    """Calls whose arrays exceed the caches read and write past them: token by token the same bits as smaller calls, and
    the sums of the weights' gradients those of the parts."""
    B, N, H, K, d = 2, (8192 if dtype == BF else 4096), 16, 8, 128
    norm = T.HeadNorm(H, K, normal(d, 1, F32)[0], normal(d, 2, F32)[0], rotary=T.Rotary(d, layout=layout))
    x, dy = seeded((B, N, H + K, d), 3, dtype), seeded((B, N, H + K, d), 4, dtype)
    assert 2 * x.numel() * x.element_size() <= 256 << 20 < 3 * x.numel() * x.element_size()
    x2 = seeded((B, 2 * N, H + K, d), 5, dtype)
    pos = ints(np.random.default_rng(6).integers(0, 1 << 18, (B, N)).tolist())
    pos2 = torch.cat((pos, pos + 1), 1)
    y, (dx, dq, dk) = norm(x2, pos2), norm.backward(x, dy, pos)
    parts, n = [], N // 8
    for a in range(0, N, n):
        cut = lambda t: t[:, a:a + n].contiguous()  # noqa: E731
        for b in (a, N + a):
            assert torch.equal(norm(x2[:, b:b + n].contiguous(), pos2[:, b:b + n].contiguous()), y[:, b:b + n])
        parts.append(norm.backward(cut(x), cut(dy), cut(pos)))
        assert torch.equal(parts[-1][0], dx[:, a:a + n])
    # a sum of n = B N H random terms of about 1 passes through partial sums of up to sqrt n, and the errors of n
    # roundings of those add up like sqrt n of them: n 2^-24, with a factor of 8
    for got, i, heads in ((dq, 1, H), (dk, 2, K)):
        want = sum(p[i].double() for p in parts)
        bound = 8 * U * math.sqrt(B * N * heads) * math.sqrt(B * N * heads)
        assert float((got.double() - want).abs().max()) <= bound


@pytest.mark.parametrize("dtype", [BF, F32])
def test_head_norm_backward_into_views(dtype):
    """dx as part of a projection's gradient, in the place of such a dy, and of such an x; what stands beside is left."""
    H, K, d = 4, 2, 64
    norm = T.HeadNorm(H, K, normal(d, 1, F32)[0], normal(d, 2, F32)[0], rotary=T.Rotary(d))
    x, dy, pos = seeded((2, 9, H + 2 * K, d), 3, dtype), seeded((2, 9, H + 2 * K, d), 4, dtype), ints([5, 900])
    cut = lambda t: t[:, :, :H + K]  # noqa: E731
    want = norm.backward(cut(x).contiguous(), cut(dy).contiguous(), pos)
    for place in ("own", "dy", "x"):
        a, g, own = x.clone(), dy.clone(), torch.full_like(x, 7.0)
        to = {"own": own, "dy": g, "x": a}[place]
        beside = to[:, :, H + K:].clone()
        got = norm.backward(cut(a), cut(g), pos, dx=cut(to))
        assert all(torch.equal(p, q) for p, q in zip(got, want)), place
        assert torch.equal(to[:, :, H + K:], beside) and torch.equal(cut(to), want[0])
