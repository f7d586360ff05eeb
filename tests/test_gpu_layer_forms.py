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
