"""The layer's operators together, as a layer uses them: LinearWindow and
WindowAttention with 8-bit projections and head norms, stage by stage and as
mac_segment's attention; a training step through norm and linear attention;
calls captured into graphs and on other streams."""
import math

import numpy as np
import pytest
import torch

import test_trained_neural_amd as T
from oracle import layer as O
from test_gpu_layer import U, f64, ints, normal
from test_gpu_parity import small
from test_gpu_window import weights
from test_trained_neural_amd import inputs as I

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def a_norm(heads, kv, d, rotary=True):
    return T.HeadNorm(heads, kv, *(1 + 0.1 * normal(d, s, F32)[0] for s in (91, 92)),
                      rotary=T.Rotary(d) if rotary else None)


# ---- WindowAttention with a norm and 8-bit weights ----

@pytest.mark.parametrize("dtype,heads,kv,d,P,S,codes", [(BF, 6, 2, 64, 20, 40, "both"), (F32, 4, 4, 32, 64, 33, "qkv"),
                                                        (BF, 8, 1, 128, 0, 70, "out"), (BF, 2, 2, 96, 3, 50, "none")])
def test_window_attention_with_norm_and_codes(dtype, heads, kv, d, P, S, codes):
    B, D = 2, 64
    w, w_out, pers = weights(heads, kv, d, D, P, dtype, d)
    norm = a_norm(heads, kv, d)
    wq = T.Int8Linear(w) if codes in ("both", "qkv") else w
    wo = T.Int8Linear(w_out) if codes in ("both", "out") else w_out
    at = T.WindowAttention(wq, wo, heads, kv, B, 2 * S + 5, pers, norm=norm, dtype=dtype)
    pool = T.PagedCache(kv, d, at.cache.n_pages, B + 1, at.cache.seq_pages)
    product = lambda x, m: m(x) if isinstance(m, T.Int8Linear) else torch.nn.functional.linear(x, m)  # noqa: E731

    def project(x, start):   # each step by a call of its own
        Bx, n, _ = x.shape
        qkv = product(x, wq).view(Bx, n, heads + 2 * kv, d)
        qk = norm(qkv[:, :, :heads + kv].contiguous(), ints([start] * Bx))
        return qk[:, :, :heads].contiguous(), qk[:, :, heads:].contiguous(), qkv[:, :, heads + kv:].contiguous()

    if P:
        pool.append(ints([B]), *project(pers[None], 0)[1:])
        pool.fork(ints([B] * B), ints(list(range(B))))
    g = torch.Generator(device="cuda").manual_seed(S)
    x = torch.randn((B, 2 * S, D), generator=g, device="cuda").to(dtype)
    window = x if pers is None else torch.cat([pers[None].expand(B, P, D), x], dim=1)
    y = at(window)
    q, k, v = project(window[:, P:], P)
    pool.append(ints([0, 1]), k, v)
    assert torch.equal(y, product(pool.attend(ints([0, 1]), q[:, S:].contiguous(), max_len=P + 2 * S).flatten(2), wo))
    t = torch.randn((B, 3, D), generator=g, device="cuda").to(dtype)
    y = at.token(t)
    q, k, v = project(t, P + 2 * S)
    pool.append(ints([0, 1]), k, v)
    assert torch.equal(y, product(pool.attend(ints([0, 1]), q, max_len=P + 2 * S + 3).flatten(2), wo))
    assert at.cache.check()[0] == 0


def test_window_attention_refuses_what_does_not_fit():
    w, w_out, pers = weights(4, 2, 32, 48, 5, BF, 1)
    with pytest.raises(ValueError, match="norm"):
        T.WindowAttention(w, w_out, 4, 2, 2, 20, pers, T.Rotary(32), norm=a_norm(4, 2, 32))
    with pytest.raises(ValueError, match="heads"):
        T.WindowAttention(w, w_out, 4, 2, 2, 20, pers, norm=a_norm(2, 2, 32))
    with pytest.raises(ValueError, match="shape"):
        T.WindowAttention(T.Int8Linear(w), w_out[:, :-32], 4, 2, 2, 20, pers)
    with pytest.raises(TypeError):
        T.WindowAttention(T.Int8Linear(w), T.Int8Linear(w_out), 4, 2, 2, 20, pers, dtype=F32)
    for kw in ({}, {"log_decay": torch.zeros(2, device="cuda"), "w_gate": w[:2]}):
        with pytest.raises(ValueError, match="either"):
            T.LinearWindow(w, w_out, 4, 2, 2, **kw)


# ---- LinearWindow ----

@pytest.mark.parametrize("heads,kv,d,P,S,gate", [(6, 2, 64, 20, 40, True), (4, 4, 32, 1, 3, False), (2, 1, 128, 0, 90, True)])
def test_linear_window(heads, kv, d, P, S, gate):
    """fp32, against the oracle step by step: projections as torch makes them (checked by norm), then norm and attention
    within the error of fp32 sums of (tokens + widths) terms each."""
    B, D = 2, 64
    w, w_out, pers = weights(heads, kv, d, D, P, F32, d)
    norm = a_norm(heads, kv, d)
    wg, bias = (normal((kv, D), 93, F32)[0] / 8, normal(kv, 94, F32)[0] + 2) if gate else (None, None)
    ld = None if gate else torch.tensor([-0.5 / (h + 1) for h in range(kv)], device="cuda")
    at = T.LinearWindow(w, w_out, heads, kv, B, log_decay=ld, w_gate=wg, gate_bias=bias, persistent=pers, norm=norm)
    W, WO = f64(w), f64(w_out)
    freq = norm.rotary.freq.cpu().numpy()
    S0 = np.zeros((B, kv, d, d))

    def step(x, held, state):
        X = f64(x)
        qkv = (X @ W.T).reshape(B, -1, heads + 2 * kv, d)
        pos = held + np.tile(np.arange(X.shape[1]), (B, 1))
        qk = O.head_norm(qkv[:, :, :heads + kv], f64(norm.w_q), f64(norm.w_k), heads, 1e-6, pos, freq)
        g = -np.log1p(np.exp(-(X @ f64(wg).T + f64(bias)))) if gate else f64(ld)
        y, s = O.linear(qk[:, :, :heads], qk[:, :, heads:], qkv[:, :, heads + kv:], g, d ** -0.5, state)
        return y.reshape(B, -1, heads * d) @ WO.T, s

    # relative to a result's norm: sums of up to D + d + tokens terms, each off by 2^-24 of its size (random signs: the
    # square root), and the chain of five of them
    bound = 5 * math.sqrt(D + 2 * d + 2 * S + P) * U * 8
    near = lambda got, want: np.linalg.norm(f64(got) - want) <= bound * np.linalg.norm(want)  # noqa: E731
    root = step(pers[None].expand(B, -1, -1), 0, S0)[1] if P else S0
    g = torch.Generator(device="cuda").manual_seed(S)
    rows = lambda n: torch.randn((B, n, D), generator=g, device="cuda")  # noqa: E731
    for _ in range(2):
        x = rows(2 * S)
        y = at(x if pers is None else torch.cat([pers[None].expand(B, P, D), x], dim=1))
        want, state = step(x, P, root)
        assert y.shape == (B, S, D) and near(y, want[:, S:]) and near(at.state, state)
        held = P + 2 * S
        for n in (1, 5, 20):
            x = rows(n)
            want, state = step(x, held, state)
            assert near(at.token(x), want) and near(at.state, state)
            held += n
    window = torch.cat(([pers[None].expand(B, P, D)] if P else []) + [rows(2 * S)], dim=1)
    y = at(window)
    at.refresh()
    assert torch.equal(at(window), y)
    with pytest.raises(ValueError, match="rows"):
        at(window[:, :-1])
    with pytest.raises(ValueError, match="expected"):
        at.token(rows(1)[:1])
    with pytest.raises(TypeError):
        at.token(rows(1).to(BF))
    assert torch.equal(at(window), y)


def test_as_the_attention_of_a_segment():
    """mac_segment with either layer, 8-bit projections and head norms in both."""
    wl = small("layers", 64, 2, 2, 16, 2, 1, 64, "bf16")
    p = I.make_params(wl)
    mem = T.NeuralMemory(wl.dim, wl.depth, wl.expansion, wl.chunk)
    D, B, S, P = wl.dim, 2, 32, 7
    w, w_out, pers = weights(4, 2, 32, D, P, BF, 3)
    gen = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    kvq, conv = (rnd(3, D, D) / 8).to(BF), rnd(3, D, 1)
    wg, gb = rnd(3, 1, D) / 8, torch.tensor([-3.0, 1.0, -3.0], device="cuda")
    x = rnd(B, S, D).to(BF)
    linear = T.LinearWindow(T.Int8Linear(w), T.Int8Linear(w_out), 4, 2, B, w_gate=(rnd(2, D) / 8).to(BF), persistent=pers,
                            norm=a_norm(4, 2, 32))
    window = T.WindowAttention(T.Int8Linear(w), T.Int8Linear(w_out), 4, 2, B, 4 * S, pers, norm=a_norm(4, 2, 32))
    for at in (linear, window):
        seen = []

        def attention(rows):
            seen.append((rows.clone(), at(rows)))
            return seen[-1][1]

        st = mem.init_state(B, 1, torch.from_numpy(p.init_weights))
        out, st = T.mac_segment(mem, st, x, pers, attention, kvq, conv, wg, gb, 1)
        assert torch.isfinite(out).all() and out.abs().max() > 0
        rows, y = seen[0]
        assert torch.equal(rows[:, :P], pers[None].expand(B, P, D)) and torch.equal(rows[:, P + S:], x)
        assert torch.equal(at(rows), y)   # a segment starts from the persistent rows
        st2 = mem.init_state(B, 1, torch.from_numpy(p.init_weights))
        assert torch.equal(T.mac_segment(mem, st2, x, pers, at, kvq, conv, wg, gb, 1)[0], out)


# ---- gradients through both operators ----

@pytest.mark.parametrize("dtype", [F32, BF])
def test_training_step(dtype):
    """d loss / d (projections, norm weights, decays, state) through norm and linear attention, against the oracle's chain."""
    B, N, H, K, d = 2, 90, 4, 2, 32
    norm = a_norm(H, K, d)
    m = T.LinearAttention(K, d)
    qkv, QKV = normal((B, N, H + 2 * K, d), 1, dtype)
    g = -torch.rand(B, N, K, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    (s, S), (dy, DY), (ds, DS) = normal((B, K, d, d), 4, F32), normal((B, N, H, d), 5, dtype), normal((B, K, d, d), 6, F32)
    pos = ints(np.tile(np.arange(N), (B, 1)).tolist())
    qk = norm(qkv[:, :, :H + K], pos)
    q, k, v = qk[:, :, :H], qk[:, :, H:], qkv[:, :, H + K:]
    y, end = m(q, k, v, g, state=s)
    dqk = torch.empty_like(qk)
    dq, dk, dv, dg, ds0 = m.backward(q, k, v, g, dy, state=s, dstate=ds)
    dqk[:, :, :H], dqk[:, :, H:] = dq, dk
    dx, dwq, dwk = norm.backward(qkv[:, :, :H + K], dqk, pos)

    args = (np.tile(np.arange(N), (B, 1)), norm.rotary.freq.cpu().numpy())
    ws = f64(norm.w_q), f64(norm.w_k)
    X = QKV[:, :, :H + K]
    n = O.head_norm(X, *ws, H, 1e-6, *args)
    V = QKV[:, :, H + K:]
    G = f64(g)
    wy, wend = O.linear(n[:, :, :H], n[:, :, H:], V, G, d ** -0.5, S)
    wq, wk, wv, wg, ws0 = O.linear_backward(n[:, :, :H], n[:, :, H:], V, G, d ** -0.5, S, DY, DS)
    wx, wdq, wdk = O.head_norm_backward(X, np.concatenate([wq, wk], 2), *ws, H, 1e-6, *args)
    # bf16: a chain of four roundings to 8 bits (qk, the pairs' weights, dq and dk, the result), each off by at most
    # 2^-8; fp32: the sums of up to N + d terms
    bound = 4 * 2.0 ** -8 if dtype == BF else 8 * (N + d) * U
    for name, a, b in (("y", y, wy), ("end", end, wend), ("dv", dv, wv), ("dx", dx, wx), ("dw_q", dwq, wdq), ("dw_k", dwk, wdk),
                       ("dg", dg, wg), ("ds", ds0, ws0)):
        assert np.linalg.norm(f64(a) - b) <= bound * np.linalg.norm(b), name


# ---- graphs and streams ----

def test_captured_and_replayed():
    """Every call in one graph, replayed on new inputs with eager work of the same calls between the replays."""
    B, N, H, K, d, D = 2, 200, 4, 2, 64, 96
    norm, m = a_norm(H, K, d), T.LinearAttention(K, d)
    lin = T.Int8Linear(normal(((H + 2 * K) * d, D), 1, F32)[0] / 10)
    thin = T.Int8Linear(normal((40, D), 2, F32)[0])
    x, g, s = torch.zeros(B, N, D, dtype=BF, device="cuda"), torch.zeros(B, N, K, device="cuda"), m.init_state(B)
    dy, pos = torch.zeros(B, N, H, d, dtype=BF, device="cuda"), ints(np.tile(np.arange(N), (B, 1)).tolist())

    def work():
        qkv = lin(x).view(B, N, H + 2 * K, d)
        qk = norm(qkv[:, :, :H + K], pos)
        y, end = m(qk[:, :, :H], qk[:, :, H:], qkv[:, :, H + K:], g, state=s)
        one, after = m(qk[:, :1, :H], qk[:, :1, H:], qkv[:, :1, H + K:], g[:, :1].contiguous(), state=end)
        grads = m.backward(qk[:, :, :H], qk[:, :, H:], qkv[:, :, H + K:], g, dy, state=s, dstate=end)
        back = norm.backward(qkv[:, :, :H + K], torch.cat(grads[:2], 2), pos)
        return [y, end, one, after, *grads, *back, thin(x[0, :3])]

    def fill(seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for t in (x, dy, s):
            t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
        g.copy_(-torch.rand(g.shape, generator=gen, device="cuda"))

    fill(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):   # two graphs of the same calls: each has workspaces of its own
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = work()
        graphs.append((gr, out))
    for seed in (2, 3, 4, 5):
        fill(seed)
        want = [t.clone() for t in work()]
        for gr, out in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for gr, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_calls_on_two_streams():
    m, norm = T.LinearAttention(2, 64), a_norm(4, 2, 64)
    lin = T.Int8Linear(normal((512, 256), 1, F32)[0])
    work = lambda st: [m.backward(q, k, v, g, q, stream=st), m(q, k, v, g, stream=st), norm.backward(qk, qk, pos, stream=st),  # noqa: E731
                       (lin(x, stream=st), lin(x[:5], stream=st))]
    q, k, v = (normal((2, 700, h, 64), s)[0] for h, s in ((4, 1), (2, 2), (2, 3)))
    qk, pos = torch.cat((q, k), 2), ints([0, 5])
    g, x = -torch.rand(2, device="cuda"), normal((600, 256), 4)[0]
    want = work(None)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [work(st) for _ in range(3) for st in (a, b)]
    torch.cuda.synchronize()
    for one in got:
        for x1, y1 in zip(one, want):
            assert all(torch.equal(p, r) for p, r in zip(x1, y1))
    with pytest.raises(ValueError):
        m(q, k, v, g, state=torch.zeros(2, 2, 64, 64))


def test_timing_class():
    from test_trained_neural_amd.layer import K_LAYER
    m = T.LinearAttention(1, 64)
    q = normal((1, 40, 1, 64), 1)[0]
    try:
        T.tm_timing_enable(1 << K_LAYER)
        T.tm_timing_read(K_LAYER)
        m(q, q, q, torch.zeros(1, device="cuda"))
        ms, n = T.tm_timing_read(K_LAYER)
    finally:
        T.tm_timing_enable(0)
    assert n == 1 and ms > 0


@pytest.mark.parametrize("kv", [2, 1])
@pytest.mark.parametrize("biased", [False, True])
def test_linear_window_gates_in_fp32(biased, kv):
    """A bf16 layer whose gates keep most of the state: log sigmoid of logits of 3 to 9, formed in fp32.  Queries, keys and
    values are the layer's own (a projection rounded to bf16); the state is held to the roundings of its sums and to the
    logits', a sum of D products: dz <= D 2^-24 sum |x w|, and d log sigmoid(z) <= exp(-z) dz."""
    B, D, heads, d, n = 2, 64, 4, 64, 120
    w, w_out, _ = weights(heads, kv, d, D, 0, BF, d)
    wg = normal((kv, D), 93, BF)[0] / 8
    wg[:, 0] = 4.0 if biased else 6.0
    bias = torch.full((kv,), 2.0, device="cuda") if biased else None
    at = T.LinearWindow(w, w_out, heads, kv, B, w_gate=wg, gate_bias=bias)
    x, _ = normal((B, n, D), 7, BF)
    x[:, :, 0] = 1.0
    at.token(x)
    qkv = torch.nn.functional.linear(x, w).view(B, n, heads + 2 * kv, d)
    Q, KK, V = f64(qkv[:, :, :heads]), f64(qkv[:, :, heads:heads + kv]), f64(qkv[:, :, heads + kv:])
    X, W = f64(x), f64(wg)
    z = X @ W.T + (2.0 if biased else 0.0)
    assert z.min() > 3 and z.max() < 9
    off = np.exp(-z) * D * U * (np.abs(X) @ np.abs(W).T + 2.0) + 4 * U * np.log1p(np.exp(-z))
    zero = np.zeros((B, kv, d, d))
    g = -np.log1p(np.exp(-z))
    want = O.linear(Q, KK, V, g, d ** -0.5, zero)[1]
    size = O.linear(np.abs(Q), np.abs(KK), np.abs(V), g, d ** -0.5, zero)[1]
    assert np.all(np.abs(f64(at.state) - want) <= size * ((n + 2 * d + 256) * U + off.sum(1)[:, :, None, None]))


@pytest.mark.parametrize("layer", ["linear", "window"])
def test_bf16_layers_of_plain_weights(layer):
    """Plain bf16 weights of 1024 x 1024, several sequences, persistent rows in front: windows and outputs that are views."""
    B, S, D, heads, kv, d, P = 2, 512, 1024, 16, 4, 64, 16
    w, w_out, pers = weights(heads, kv, d, D, P, BF, 3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((B, 2 * S, D), generator=gen, device="cuda").to(BF)
    window = torch.cat([pers[None].expand(B, P, D), x], dim=1)
    make = lambda n: T.LinearWindow(w, w_out, heads, kv, n, log_decay=torch.full((kv,), -0.01, device="cuda"), persistent=pers) \
        if layer == "linear" else T.WindowAttention(w, w_out, heads, kv, n, 2 * S, pers)  # noqa: E731
    y = make(B)(window)
    assert y.shape == (B, S, D) and torch.isfinite(y).all()
    for b in range(B):   # a sequence by itself: its products' sums may be split otherwise, 8-bit roundings follow
        one = make(1)(window[b:b + 1])
        assert float((one[0].double() - y[b].double()).norm() / y[b].double().norm()) <= 4 * 2.0 ** -8
