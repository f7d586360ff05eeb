"""The attention window's operators together, as memory as a context uses
them: WindowAttention (rotary positions, fork of the persistent tokens,
append, attention, single tokens) stage by stage against the oracle, and as
mac_segment's attention."""
import math

import numpy as np
import pytest
import torch

import test_trained_neural_amd as T
from harness import say
from oracle import attention as O
from test_gpu_attention import expect, ints
from test_gpu_parity import small
from test_trained_neural_amd import inputs as I

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def weights(heads, kv, d, D, P, dtype, seed):
    rng = np.random.default_rng(seed)
    t = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to("cuda").to(dtype)  # noqa: E731
    return t((heads + 2 * kv) * d, D) / math.sqrt(D), t(D, heads * d) / math.sqrt(heads * d), t(P, D) if P else None


class Staged:
    """WindowAttention's steps one by one, each checked: the rotation against
    the oracle, the cache against its model, the attention within its bounds."""

    def __init__(self, w, w_out, heads, kv, batch, P, rotary, cache):
        self.w, self.w_out, self.heads, self.kv, self.rotary, self.g = w, w_out, heads, kv, rotary, cache
        self.m = O.Cache(kv, cache.head_dim, cache.n_pages, cache.n_seqs, cache.seq_pages)
        self.batch, self.P = batch, P

    def project(self, x, start):
        B, n, _ = x.shape
        H, d = self.heads + self.kv, self.g.head_dim
        qkv = torch.nn.functional.linear(x, self.w).view(B, n, H + self.kv, d)
        y = self.rotary(qkv[:, :, :H].contiguous(), ints([start] * B))
        pos = start + np.tile(np.arange(n), (B, 1))
        f = self.rotary.freq.cpu().numpy()
        raw = qkv[:, :, :H].float().cpu().numpy()
        want = O.rotate(raw, pos, f, self.rotary.result_scale)
        size = np.abs(raw).max(axis=-1, keepdims=True)
        assert np.all(np.abs(y.float().cpu().numpy() - want) <= torch.finfo(x.dtype).eps / 2 * np.abs(want) + size * 2.0 ** -20)
        return y[:, :, :self.heads], y[:, :, self.heads:], qkv[:, :, H:].contiguous()

    def append(self, seqs, k, v):
        k, v = k.contiguous(), v.contiguous()
        self.g.append(ints(seqs), k, v)
        self.m.append(seqs, [k.shape[1]] * len(seqs), k.float().cpu().numpy(), v.float().cpu().numpy())
        n = max(self.m.lengths)
        gk, gv = (t.cpu().numpy() for t in self.g.read(None, 0, n))
        for s, held in enumerate(self.m.lengths):
            wk, wv = self.m.held(s)
            assert np.array_equal(gk[s, :held], wk) and np.array_equal(gv[s, :held], wv)
        assert self.g.check() == (0, self.m.used())

    def attend(self, q, held):
        q = q.contiguous()
        slots = list(range(self.batch))
        y = self.g.attend(ints(slots), q, max_len=held)
        expect(self.g, self.m, slots, q, None, 1 / math.sqrt(self.g.head_dim), 0, 0, y, y)
        return torch.nn.functional.linear(y.flatten(2), self.w_out)

    def segment(self, window):
        slots = list(range(self.batch))
        self.g.free(ints(slots))
        self.m.free(slots)
        if self.P:
            self.g.fork(ints([self.batch] * self.batch), ints(slots))
            self.m.fork([self.batch] * self.batch, slots)
        q, k, v = self.project(window[:, self.P:], self.P)
        self.append(slots, k, v)
        n = k.shape[1]
        return self.attend(q[:, n // 2:], self.P + n)


@pytest.mark.parametrize("dtype,heads,kv,d,P,S", [(BF, 6, 2, 64, 20, 40), (F32, 4, 4, 32, 64, 33), (BF, 8, 1, 128, 0, 70),
                                                  (BF, 2, 2, 96, 3, 150)])
def test_segments_and_tokens(dtype, heads, kv, d, P, S):
    B, D = 2, 64
    w, w_out, pers = weights(heads, kv, d, D, P, dtype, d)
    rotary = T.Rotary(d)
    at = T.WindowAttention(w, w_out, heads, kv, B, 2 * S + 5, pers, rotary)
    pool = T.PagedCache(kv, d, at.cache.n_pages, B + 1, at.cache.seq_pages)
    ref = Staged(w, w_out, heads, kv, B, P, rotary, pool)
    if P:
        ref.append([B], *ref.project(pers[None], 0)[1:])
    g = torch.Generator(device="cuda").manual_seed(S)
    rows = lambda n: torch.randn((B, n, D), generator=g, device="cuda").to(dtype)  # noqa: E731
    for _ in range(2):
        x = rows(2 * S)
        window = x if pers is None else torch.cat([pers[None].expand(B, P, D), x], dim=1)
        y = at(window)
        assert torch.equal(y, ref.segment(window))
        held = P + 2 * S
        for n in (1, 3, 1):
            x = rows(n)
            y = at.token(x)
            q, k, v = ref.project(x, held)
            ref.append([0, 1], k, v)
            held += n
            assert torch.equal(y, ref.attend(q, held))
    assert at.cache.check() == (0, ref.m.used())
    if P >= 64:   # the persistent tokens' whole pages are held once
        assert int(at.cache.refs.max()) == B + 1
    with pytest.raises(ValueError, match="holds"):
        at.token(rows(1))
    with pytest.raises(ValueError, match="rows"):
        at(torch.cat([window, window[:, :1]], dim=1)[:, :-2])
    with pytest.raises(ValueError, match="expected"):
        at.token(rows(1)[:1])
    at.refresh()
    assert torch.equal(at(window), ref.segment(window))


def test_window_records_no_gradients_and_refuses_capture(monkeypatch):
    w, w_out, pers = weights(4, 2, 32, 48, 5, BF, 1)
    at = T.WindowAttention(w.requires_grad_(), w_out.requires_grad_(), 4, 2, 2, 20, pers, T.Rotary(32))
    x = torch.cat([pers[None].expand(2, 5, 48), torch.ones((2, 8, 48), dtype=BF, device="cuda")], dim=1)
    y = at(x)
    assert not y.requires_grad and not at.token(x[:, :1]).requires_grad
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    for call in (lambda: at(x), lambda: at.token(x[:, :1])):
        with pytest.raises(RuntimeError, match="captured"):
            call()
    monkeypatch.undo()
    assert torch.equal(at(x), y)                                    # the refusals changed nothing


@pytest.mark.parametrize("P", [0, 5])
def test_window_after_a_call_that_failed(P, monkeypatch):
    """A window or tokens of another type, device or rank are refused with the
    sequences as they were; where a later step fails, what is counted is what
    the cache holds."""
    w, w_out, pers = weights(4, 2, 32, 48, P, BF, 2)
    at, ref = (T.WindowAttention(w, w_out, 4, 2, 2, 24, pers, T.Rotary(32)) for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(4)
    rows = lambda n: torch.randn((2, n, 48), generator=g, device="cuda").to(BF)  # noqa: E731
    window = rows(P + 8)
    if P:
        window[:, :P] = pers
    x, nxt = rows(1), rows(2)
    assert torch.equal(at(window), ref(window))
    for bad, error in ((window.float(), TypeError), (window.cpu(), ValueError), (window[0], (ValueError, IndexError))):
        for call in (at, at.token):
            with pytest.raises(error):
                call(bad)
        assert at.cache.lengths.tolist() == ref.cache.lengths.tolist()
    assert torch.equal(at.token(x), ref.token(x))
    append = at.cache.append

    def fails(*args):
        raise T.TMError("append", T.TM_ERR_HIP)

    monkeypatch.setattr(at.cache, "append", fails)
    with pytest.raises(T.TMError):
        at.token(x)
    monkeypatch.setattr(at.cache, "append", append)
    assert torch.equal(at.token(nxt), ref.token(nxt))               # the failed token counts nowhere
    monkeypatch.setattr(at.cache, "append", fails)
    with pytest.raises(T.TMError):
        at(window)
    monkeypatch.setattr(at.cache, "append", append)
    ref.cache.free(ints([0, 1]), ints([P, P]))                      # the persistent rows alone are held
    ref._held = P
    assert at.cache.lengths.tolist() == ref.cache.lengths.tolist()
    assert torch.equal(at.token(x), ref.token(x))
    assert torch.equal(at(window), ref(window))


def test_as_attention_of_mac_segment():
    """Two segments through mac_segment with WindowAttention equal those with
    a function that makes its calls one by one on a cache of its own."""
    wl = small("macwin", 64, 2, 2, 16, 2, 2, 64, "bf16", offsets=(-4.5, 1.0, -6.0))
    H, d, S, P, B = wl.heads, wl.dim, 32, 4, wl.batch
    D = H * d
    p = I.make_params(wl)
    pi = I.make_prologue(wl, p, conv_len=2)
    dev = "cuda"
    x = torch.from_numpy(pi.x).to(dev).to(BF)
    w_kvq = torch.from_numpy(np.ascontiguousarray(pi.w_kvq.transpose(0, 2, 1))).to(dev).to(BF)
    conv = torch.from_numpy(pi.conv).to(dev)
    wg = torch.from_numpy(np.ascontiguousarray(pi.w_gate.transpose(0, 2, 1))).to(dev)
    gb = torch.from_numpy(pi.gate_bias).to(dev)
    w, w_out, pers = weights(4, 2, 32, D, P, BF, 3)
    rotary = T.Rotary(32, layout=T.TM_ROPE_INTERLEAVED)
    at = T.WindowAttention(w, w_out, 4, 2, B, 2 * S, pers, rotary)
    seen = []

    def by_hand(window):
        cache = T.PagedCache(2, 32, 20, B, 4)
        qkv = torch.nn.functional.linear(window, w).view(B, P + 2 * S, 8, 32)
        n = ints([list(range(P + 2 * S))] * B)
        qk = rotary(qkv[:, :, :6].contiguous(), n)
        cache.append(None, qk[:, :P, 4:].contiguous(), qkv[:, :P, 6:].contiguous())
        cache.append(None, qk[:, P:, 4:].contiguous(), qkv[:, P:, 6:].contiguous())
        y = cache.attend(None, qk[:, P + S:, :4].contiguous(), max_len=P + 2 * S)
        seen.append(window.clone())
        return torch.nn.functional.linear(y.flatten(2), w_out)

    outs = []
    for attention in (at, by_hand):
        mem = T.NeuralMemory(d, wl.depth, wl.expansion, wl.chunk, device=dev)
        st = mem.init_state(B, H, torch.from_numpy(p.init_weights))
        hx = torch.zeros((B, 1, 3, D), dtype=F32, device=dev)
        hy = torch.zeros_like(hx)
        for i in range(2):
            out, st = T.mac_segment(mem, st, x[:, i * S:(i + 1) * S].contiguous(), pers, attention, w_kvq, conv, wg, gb,
                                    H, hx, hy)
            outs.append(out)
        assert mem.check(st) == (False, 2 * S)
    say("segments", [float(o.abs().mean()) for o in outs])
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
    assert torch.equal(seen[0][:, :P], pers[None].expand(B, P, D)) and torch.isfinite(outs[1]).all()
