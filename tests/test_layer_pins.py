"""The layer's operators without a GPU: the oracle against closed forms and
differences, the library's exports, and what its calls refuse on the host
before anything is launched."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import test_trained_neural_amd as T
from oracle import layer as O
from test_trained_neural_amd import layer as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = lambda n: ctypes.c_void_p((1 << 20) + n)  # noqa: E731   never read: every call here is refused


def rand(*shape, seed=0):
    return np.random.default_rng(seed).standard_normal(shape)


# ---- the oracle ----

def test_norm_by_hand():
    x = np.array([[[[3.0, 4.0]]]])
    assert np.allclose(O.head_norm(x, None, None, 1, 0.0), x / math.sqrt(12.5))
    assert np.allclose(O.head_norm(x, [2.0, -1.0], None, 1, 0.0), x / math.sqrt(12.5) * [2, -1])
    turned = O.head_norm(x, None, None, 1, 0.0, np.array([[1]]), np.array([math.pi / 2]))
    assert np.allclose(turned, np.array([-4.0, 3.0]) / math.sqrt(12.5))


def test_norm_gradients_are_differences():
    x, dy, wq, wk = rand(2, 3, 4, 6), rand(2, 3, 4, 6, seed=1), rand(6, seed=2), rand(6, seed=3)
    args = (np.arange(6).reshape(2, 3), np.array([1.0, 0.3]), 1.1, True)
    f = lambda x, wq, wk: (O.head_norm(x, wq, wk, 3, 0.1, *args) * dy).sum()  # noqa: E731
    got = O.head_norm_backward(x, dy, wq, wk, 3, 0.1, *args)
    for n, at in enumerate(([x, wq, wk])):
        for i in np.random.default_rng(4).choice(at.size, 5, replace=False):
            at.flat[i] += 1e-6
            hi = f(x, wq, wk)
            at.flat[i] -= 2e-6
            lo = f(x, wq, wk)
            at.flat[i] += 1e-6
            assert abs((hi - lo) / 2e-6 - got[n].flat[i]) < 1e-6


def test_linear_by_hand():
    q, k, v = rand(1, 5, 2, 3), rand(1, 5, 1, 3, seed=1), rand(1, 5, 1, 2, seed=2)
    zero = np.zeros((1, 1, 3, 2))
    y, S = O.linear(q, k, v, np.array([0.0]), 1.0, zero)       # nothing is dropped: causal sums
    scores = np.tril(q[0, :, 1] @ k[0, :, 0].T)
    assert np.allclose(y[0, :, 1], scores @ v[0, :, 0]) and np.allclose(S[0, 0], k[0, :, 0].T @ v[0, :, 0])
    y, S = O.linear(q, k, v, np.array([-np.inf]), 2.0, rand(1, 1, 3, 2))   # all is: a token sees itself
    assert np.allclose(y[0, 3, 0], 2 * (q[0, 3, 0] @ k[0, 3, 0]) * v[0, 3, 0])
    y, S = O.linear(q, k, v, np.array([-0.5]), 1.0, zero, [3])
    assert not y[0, 3:].any() and np.allclose(S[0, 0], sum(math.exp(-0.5 * (2 - j)) * np.outer(k[0, j, 0], v[0, j, 0]) for j in range(3)))


def test_linear_gradients_are_differences():
    B, N, H, K, dk, dv = 2, 6, 4, 2, 3, 2
    a = [rand(B, N, H, dk), rand(B, N, K, dk, seed=1), rand(B, N, K, dv, seed=2), -np.abs(rand(B, N, K, seed=3)),
         rand(B, K, dk, dv, seed=4)]
    dy, dS, counts = rand(B, N, H, dv, seed=5), rand(B, K, dk, dv, seed=6), [6, 4]

    def f(q, k, v, g, S):
        y, S = O.linear(q, k, v, g, 0.7, S, counts)
        return (y * dy).sum() + (S * dS).sum()

    got = O.linear_backward(*a[:4], 0.7, a[4], dy, dS, counts)
    for n, at in enumerate(a):
        for i in np.random.default_rng(7).choice(at.size, 6, replace=False):
            at.flat[i] += 1e-6
            hi = f(*a)
            at.flat[i] -= 2e-6
            lo = f(*a)
            at.flat[i] += 1e-6
            assert abs((hi - lo) / 2e-6 - got[n].flat[i]) < 1e-6 * max(1, abs(got[n].flat[i]))


def test_int8_by_hand():
    codes, scales = O.int8_rows(np.array([[127.0, 2.5, -3.5, 0.4], [0, 0, 0, 0], [1, np.inf, 0, 0]], dtype=np.float32))
    x = torch.from_numpy(rand(50, 300, seed=8)).to(torch.bfloat16).double().numpy()
    m = np.abs(x).max(axis=1, keepdims=True)
    assert np.array_equal(O.int8_rows(x)[0], np.rint(127 * x / m))   # bf16: what 64 bits give
    assert codes.tolist() == [[127, 2, -4, 0], [0] * 4, [0] * 4] and scales[:2].tolist() == [1.0, 0.0] and np.isnan(scales[2])


# ---- the library, on the host ----

def declared():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "tm_layer.h")).read(), flags=re.S)
    return set(re.findall(r"\b(tm_[a-z0-9_]+)\s*\(", src))


def test_library_exports_every_declared_symbol():
    assert declared() == set(L.EXPORTED)
    lib = ctypes.CDLL(T.LIB_PATH)
    for s in L.EXPORTED:
        assert hasattr(lib, s) and hasattr(L, s), s


NORM = dict(x=P(0), xb=512, xt=512, y=P(1 << 16), yb=512, yt=512, wq=P(64), wk=P(64), eps=1e-6, pos=P(0), per=1, freq=P(0),
            scale=1.0, B=2, N=4, H=6, K=2, d=64, r=64, layout=0, dtype=T.TM_BF16)


def head_norm(**kw):
    a = dict(NORM, yb=4 * 512, **kw) if "yb" not in kw else dict(NORM, **kw)
    return L._lib().tm_head_norm(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), T.TM_ERR_DTYPE), (dict(layout=2), T.TM_ERR_INVALID), (dict(B=-1), T.TM_ERR_INVALID),
    (dict(H=0), T.TM_ERR_INVALID), (dict(K=-1), T.TM_ERR_INVALID), (dict(H=65535), T.TM_ERR_INVALID),
    (dict(d=1025, r=0), T.TM_ERR_INVALID), (dict(d=0, r=0), T.TM_ERR_INVALID), (dict(r=63), T.TM_ERR_INVALID),
    (dict(r=66), T.TM_ERR_INVALID), (dict(r=-2), T.TM_ERR_INVALID), (dict(eps=-1.0), T.TM_ERR_INVALID),
    (dict(eps=math.nan), T.TM_ERR_INVALID), (dict(scale=math.inf), T.TM_ERR_INVALID), (dict(x=None), T.TM_ERR_INVALID),
    (dict(y=None), T.TM_ERR_INVALID), (dict(y=P(1)), T.TM_ERR_INVALID), (dict(wq=P(2)), T.TM_ERR_INVALID),
    (dict(pos=None), T.TM_ERR_INVALID), (dict(freq=None), T.TM_ERR_INVALID), (dict(freq=P(4)), T.TM_ERR_INVALID),
    (dict(yt=511), T.TM_ERR_INVALID), (dict(yb=500), T.TM_ERR_INVALID), (dict(xt=-8), T.TM_ERR_INVALID),
    (dict(y=P(0)), T.TM_ERR_INVALID), (dict(N=1 << 30, B=1 << 10), T.TM_ERR_INVALID), (dict(B=0), T.TM_OK),
    (dict(N=0), T.TM_OK)])
def test_head_norm_refuses(kw, code):
    assert head_norm(**kw) == code


def test_head_norm_backward_refuses():
    f = L._lib().tm_head_norm_backward
    ok = [P(0), 2048, 512, P(0), 2048, 512, P(1 << 16), 2048, 512, P(0), P(0), P(0), P(0), 1e-6, P(0), 1, P(0), 1.0, 2, 4, 6, 2,
          64, 64, 0, T.TM_BF16, P(0), None]
    for at, value in ((3, None), (6, None), (11, P(2)), (26, None), (26, P(16)), (25, 5), (4, -1), (7, 100)):
        a = list(ok)
        a[at] = value
        assert f(*a) in (T.TM_ERR_INVALID, T.TM_ERR_DTYPE), at
    a = list(ok)
    a[6], a[7] = a[3], 4096   # in dy's place with other distances
    assert f(*a) == T.TM_ERR_INVALID


LIN = [P(0), 512, 128, P(0), 512, 128, P(0), 512, 128, P(0), 1, None, P(0), P(0), P(0), 1.0, 2, 4000, 2, 2, 64, 64, T.TM_BF16, P(0), None]


@pytest.mark.parametrize("at,value", [
    (22, 3), (0, None), (0, P(8)), (1, 4), (2, -8), (3, None), (6, P(2)), (9, None), (9, P(2)), (11, P(2)), (12, P(4)),
    (13, P(8)), (14, None), (14, P(8)), (15, math.inf), (16, -1), (17, -1), (18, 3), (18, 0), (18, 130), (19, 0), (20, 60),
    (20, 264), (20, 0), (21, 4), (21, 512), (23, None), (23, P(16)), (17, (1 << 30) + 1),
    (2, 1 << 23), (18, 32770), (16, 1 << 23)])
def test_linear_attention_refuses(at, value):
    a = list(LIN)
    a[at] = value
    assert L._lib().tm_linear_attention(*a) in (T.TM_ERR_INVALID, T.TM_ERR_DTYPE)


@pytest.mark.parametrize("at,value", [(13, None), (13, P(2)), (14, 4), (16, P(4)), (17, None), (18, P(8)), (19, None),
                                      (20, P(2)), (21, P(4)), (22, math.nan), (30, None), (29, 9), (27, 12)])
def test_linear_attention_backward_refuses(at, value):
    a = LIN[:13] + [P(0), 512, 128, P(0), P(0), P(0), P(0), P(0), P(0)] + LIN[15:]
    a[at] = value
    assert L._lib().tm_linear_attention_backward(*a) in (T.TM_ERR_INVALID, T.TM_ERR_DTYPE)


def test_linear_empty_calls_and_sizes():
    a = list(LIN)
    a[16] = 0
    assert L._lib().tm_linear_attention(*a) == T.TM_OK
    a = list(LIN)
    a[17], a[13] = 0, None
    assert L._lib().tm_linear_attention(*a) == T.TM_OK
    for b, n in ((0, 0), (0, 5), (3, 0), (1, 1), (5, 16)):
        assert T.tm_linear_workspace_bytes(b, n, 2, 2, 64, 64) == 0
        assert (T.tm_linear_workspace_bytes(b, n, 2, 2, 64, 64, True) > 0) == (b * n > 0)
    assert T.tm_linear_workspace_bytes(2, 4000, 2, 2, 64, 60) == 0 and T.tm_linear_workspace_bytes(2, 4000, 3, 2, 64, 64) == 0
    assert 0 < T.tm_linear_workspace_bytes(2, 4096, 2, 2, 64, 64) < T.tm_linear_workspace_bytes(2, 4096, 2, 2, 64, 64, True)


def test_int8_refuses():
    f, g, h = L._lib().tm_int8_quantize, L._lib().tm_int8_matmul, L._lib().tm_int8_linear
    quant = [P(0), 100, P(0), 112, P(0), 4, 100, T.TM_BF16, None]
    for at, value in ((0, None), (0, P(1)), (1, -1), (2, None), (2, P(8)), (3, 96), (3, 113), (4, None), (5, -1), (6, 0),
                      (6, 131073), (7, 4), (5, 1 << 31)):
        a = list(quant)
        a[at] = value
        assert f(*a) in (T.TM_ERR_INVALID, T.TM_ERR_DTYPE), at
    mat = [P(0), P(0), P(0), P(0), 112, P(0), 64, 4, 64, 100, T.TM_BF16, None]
    for at, value in ((0, None), (1, P(2)), (2, P(4)), (3, None), (4, 96), (5, None), (5, P(1)), (6, 63), (7, -1), (8, -1),
                      (9, 0), (9, 113), (10, 2)):
        a = list(mat)
        a[at] = value
        assert g(*a) in (T.TM_ERR_INVALID, T.TM_ERR_DTYPE), at
    lin = [P(0), 100, P(0), P(0), 112, P(0), 64, 4, 64, 100, T.TM_BF16, P(0), None]
    for at, value in ((0, None), (1, -1), (2, P(4)), (3, None), (4, 128), (5, None), (6, 63), (7, 1 << 31), (9, 96), (11, None),
                      (11, P(16))):
        a = list(lin)
        a[at] = value
        assert h(*a) in (T.TM_ERR_INVALID, T.TM_ERR_DTYPE), at
    for a, n, fn in ((quant, 5, f), (mat, 7, g), (mat, 8, g), (lin, 7, h), (lin, 8, h)):
        a = list(a)
        a[n] = 0
        assert fn(*a) == T.TM_OK
    assert T.tm_int8_workspace_bytes(4, 0) == 0 and T.tm_int8_workspace_bytes(-1, 4) == 0


# ---- the binding's own checks ----

def test_binding_refuses():
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    norm = T.HeadNorm(2, 1)
    with pytest.raises(ValueError):
        norm(z(1, 2, 3, 8))                     # not on a GPU
    with pytest.raises(TypeError):
        norm(z(1, 2, 3, 8, dtype=torch.float16))
    with pytest.raises(ValueError):
        T.HeadNorm(0)
    with pytest.raises(ValueError):
        T.LinearAttention(2, 60)
    m = T.LinearAttention(2, 64)
    with pytest.raises(ValueError):
        m(z(1, 2, 2, 64), z(1, 2, 2, 64), z(1, 2, 2, 64), torch.zeros(2))
    with pytest.raises(ValueError):
        m(z(1, 2, 2, 32), z(1, 2, 2, 64), z(1, 2, 2, 64), torch.zeros(2))
    with pytest.raises(ValueError):
        T.Int8Linear(codes=torch.zeros(4, 20, dtype=torch.int8), scales=torch.zeros(4))
    with pytest.raises(ValueError):
        T.Int8Linear(codes=torch.zeros(4, 32, dtype=torch.int8), scales=torch.zeros(4), cols=16)
    with pytest.raises(TypeError):
        T.Int8Linear(codes=torch.zeros(4, 32), scales=torch.zeros(4))
