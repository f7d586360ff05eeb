"""How exact the layer's operators are, closer than their types' rounding.

Linear attention of bf16 calls: a weight of a pair of tokens and the state
before a chunk each enter their products as two bf16 parts, the second what
the first leaves.  A part is off by at most 2^-8 of what it stands for
(torch.finfo(bfloat16).eps / 2), so both together by 2^-16; the sums are fp32
as in the other tests, and the result is rounded once, by at most 2^-8."""
import math

import numpy as np
import pytest
import torch

import test_gpu_layer as L
import test_trained_neural_amd as T
from oracle import layer as O
from test_gpu_layer import BF, F32, f64, ints, normal, within

pytestmark = pytest.mark.gpu
PARTS = 2.0 ** -16


@pytest.mark.parametrize("case", [c for c in L.LINEAR if c[0] == BF] + [
    (BF, 2, 6, 4, 2, 64, 64, True, False, True), (BF, 1, 16, 2, 2, 128, 128, True, False, True),
    (BF, 1, 330, 4, 4, 192, 160, True, False, True), (BF, 2, 500, 2, 1, 64, 128, False, True, True)],
    ids=lambda c: "-".join(str(x) for x in c))
def test_linear_attention_in_parts(case):
    """Outputs and gradients of token arrays: nothing but their own rounding is coarser than 16 bits."""
    dtype, B, N, H, K, dk, dv = case[:7]
    q, k, v, g, counts, s, (Q, KK, V, G, S) = L.linear_case(case)
    m = T.LinearAttention(K, dk, dv)
    c = None if counts is None else ints(counts)
    scale = 1 / math.sqrt(dk)
    e, _, half = L.linear_error(case)
    want, _ = O.linear(Q, KK, V, G, scale, S, counts)
    size, _ = O.linear(*map(np.abs, (Q, KK, V)), G, scale, np.abs(S), counts)
    within(m(q, k, v, g, state=s, counts=c)[0], want, size * (e + PARTS) + np.abs(want) * half, "y")
    (dy, DY), (ds, DS) = normal((B, N, H, dv), 8, dtype), normal((B, K, dk, dv), 9, F32)
    got = m.backward(q, k, v, g, dy, state=s, dstate=ds, counts=c)
    want = O.linear_backward(Q, KK, V, G, scale, S, DY, DS, counts)
    size = O.linear_backward(*map(np.abs, (Q, KK, V)), G, scale, np.abs(S), np.abs(DY), np.abs(DS), counts)
    for n, name in enumerate(("dq", "dk", "dv")):
        within(got[n], want[n], size[n] * (e * (H // K) + PARTS) + np.abs(want[n]) * half, name)


@pytest.mark.parametrize("n", [6, 7, 16, 64, 65, 400])
def test_linear_attention_of_single_pairs(n):
    """With everything before a token dropped its output is its own pair alone, scale (q . k) v: a weight of too few bits
    has nothing to hide behind.  The same for the three gradients."""
    case = (BF, 2, n, 4, 2, 64, 64, True, False, True)
    q, k, v, _, _, s, (Q, KK, V, _, S) = L.linear_case(case)
    g = torch.full((2, n, 2), -math.inf, device="cuda")
    m = T.LinearAttention(2, 64)
    y, end = m(q, k, v, g, state=s)
    e, _, half = L.linear_error(case)
    want, _ = O.linear(Q, KK, V, f64(g), 0.125, S)
    size, _ = O.linear(*map(np.abs, (Q, KK, V)), f64(g), 0.125, np.abs(S))
    within(y, want, size * (e + PARTS) + np.abs(want) * half, "y")
    dy, DY = normal(q.shape, 8, BF)
    got = m.backward(q, k, v, g, dy, state=s)
    want = O.linear_backward(Q, KK, V, f64(g), 0.125, S, DY, np.zeros_like(S))
    size = O.linear_backward(*map(np.abs, (Q, KK, V)), f64(g), 0.125, np.abs(S), np.abs(DY), np.zeros_like(S))
    for i, name in enumerate(("dq", "dk", "dv")):
        within(got[i], want[i], size[i] * (2 * e + PARTS) + np.abs(want[i]) * half, name)


# ---- the gradient of a decay that drops everything ----

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [1, 40, 65, 700])
def test_gradient_of_a_dropping_decay_is_zero(n, dtype):
    """What a token keeps is exp(-inf) = 0 or, from -1000 on, counts as it: the derivative by its logarithm is 0, exactly,
    for each token and summed for each head; the tokens beside it keep theirs."""
    B, H, K, d = 2, 4, 2, 64
    case = (dtype, B, n, H, K, d, d, True, False, True)
    q, k, v, g, _, s, (Q, KK, V, _, S) = L.linear_case(case, wipes=False)
    rng = np.random.default_rng(11)
    drop = torch.from_numpy(rng.random((B, n, K)) < 0.05).to("cuda")
    drop[:, n // 2] = True
    g = g.clamp(min=-0.05)
    g[drop] = -math.inf
    g[:, n // 2, 1] = -1000.0
    (dy, DY), (ds, DS) = normal(q.shape, 8, dtype), normal((B, K, d, d), 9, F32)
    m = T.LinearAttention(K, d)
    counts = [n, max(1, n - 9)]
    got = m.backward(q, k, v, g, dy, state=s, dstate=ds, counts=ints(counts))[3]
    assert not got[drop].any()
    want = O.linear_backward(Q, KK, V, f64(g), d ** -0.5, S, DY, DS, counts)[3]
    assert not want[f64(drop) > 0].any()
    assert np.linalg.norm(f64(got) - want) <= 1e-5 * np.linalg.norm(want)
    head = torch.tensor([-math.inf, -0.01], device="cuda")
    got = m.backward(q, k, v, head, dy, state=s, dstate=ds, counts=ints(counts))[3]
    want = O.linear_backward(Q, KK, V, f64(head), d ** -0.5, S, DY, DS, counts)[3]
    assert got[0] == 0
    # a sum over tokens whose errors may have one sign: sqrt(B n) times a token's 1e-5
    assert abs(float(got[1]) - want[..., 1].sum()) <= 1e-5 * np.linalg.norm(want) * math.sqrt(B * n)
