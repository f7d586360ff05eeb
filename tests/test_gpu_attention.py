"""The attention window's operators on the GPU against the fp64 oracle:
rotary positions, the paged 8-bit cache's bookkeeping and codes (exactly),
and the attention that reads it.

Tolerances of the attention, per element: a weight p carries the error of its
score (both products and the scale in fp32) and, in bf16 calls, its rounding
to bf16; the sum over the tokens is fp32; the result is rounded once.  With
u = 2^-24, S the row's largest scale * sum |q||k| and A the weighted mean of
|v|:  |error| <= A (2 (d + 8) u S + 8 u + L u + r) + half a step of |o|,
r = 2^-8 for bf16 (a weight's rounding), 2^-23 for fp32 (three parts)."""
import math

import numpy as np
import pytest
import torch

import test_trained_neural_amd as T
from harness import say
from oracle import attention as O

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def normal(shape, seed, dtype=BF, scale=1.0):
    x = np.random.default_rng(seed).standard_normal(shape).astype(np.float32) * scale
    t = torch.from_numpy(x).to("cuda").to(dtype)
    return t, t.float().cpu().numpy().astype(np.float64)


# ---- rotary ----

ROTARY = [  # dtype, B, T, H, d, r, interleaved, per token, strided
    (BF, 2, 5, 3, 64, 64, False, True, False), (BF, 1, 1, 1, 2, 2, False, False, False),
    (BF, 3, 70, 10, 128, 128, True, True, True), (F32, 2, 33, 9, 96, 64, False, False, True),
    (F32, 1, 9, 2, 33, 6, True, True, False), (BF, 2, 4, 2, 37, 18, False, True, False),
    (BF, 1, 1000, 1, 40, 20, True, False, False), (F32, 4, 1, 40, 256, 256, False, False, True),
    (BF, 2, 3, 5, 33, 32, True, True, True), (F32, 1, 257, 6, 8, 4, False, True, False)]


@pytest.mark.parametrize("case", ROTARY, ids=lambda c: "-".join(str(x) for x in c))
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary(case, inverse):
    dtype, B, N, H, d, r, inter, per_token, strided = case
    x, _ = normal((B, N, H + 2, d), 1, dtype)
    x = x[:, :, 1:H + 1] if strided else x[:, :, :H].contiguous()
    rng = np.random.default_rng(2)
    pos = rng.integers(-5, 1 << 20, (B, N) if per_token else B)
    pos.flat[0] = (1 << 31) - 1 if per_token else (1 << 30)
    rot = T.Rotary(r, base=500000.0, layout=T.TM_ROPE_INTERLEAVED if inter else T.TM_ROPE_HALF,
                   scaling=T.TM_ROPE_PARTS, factor=8.0, original_len=2048)
    y = rot(x, ints(pos.tolist()), inverse=inverse)
    full = pos if per_token else pos[:, None] + np.arange(N)
    xr = x.float().cpu().numpy().astype(np.float64)
    f = rot.freq.cpu().numpy()
    want = O.rotate(xr, full, f, rot.result_scale, inter, inverse)
    # half a step of the result, and both elements times the angle's error:
    # fp64 product and reduction at the angle's size, fp32 sine of the rest
    n = r // 2
    a, b = (xr[..., 0:r:2], xr[..., 1:r:2]) if inter else (xr[..., :n], xr[..., n:r])
    err = rot.result_scale * (np.abs(a) + np.abs(b)) * (2.0 ** -51 * np.abs(full[..., None] * f)[:, :, None] + 2.0 ** -21)
    tol = np.zeros_like(xr)
    if inter:
        tol[..., 0:r:2] = tol[..., 1:r:2] = err
    else:
        tol[..., :n] = tol[..., n:r] = err
    tol[..., :r] += np.abs(want[..., :r]) * torch.finfo(dtype).eps / 2
    got = y.float().cpu().numpy()
    assert np.all(np.abs(got - want) <= tol)
    assert np.array_equal(got[..., r:], xr[..., r:])


def test_rotary_in_place_and_strided_output():
    x, _ = normal((2, 6, 4, 64), 3)
    pos = ints([[3 * i + j for j in range(6)] for i in range(2)])
    rot = T.Rotary(48, device="cuda")
    want = rot(x, pos)
    qkv = torch.zeros((2, 6, 8, 64), dtype=BF, device="cuda")
    rot(x, pos, out=qkv[:, :, 2:6])
    assert torch.equal(qkv[:, :, 2:6], want) and not qkv[:, :, :2].any() and not qkv[:, :, 6:].any()
    rot(x, pos, out=x)
    assert torch.equal(x, want)
    assert rot(x[:, :0], pos[:, :0].contiguous()).shape == (2, 0, 4, 64)


@pytest.mark.parametrize("layout", [T.TM_ROPE_HALF, T.TM_ROPE_INTERLEAVED])
@pytest.mark.parametrize("dtype,d,r", [(BF, 128, 128), (F32, 96, 64)])
def test_rotary_of_large_tensors(dtype, d, r, layout):
    """What is too large for the caches takes another way to memory: the same
    bits as in parts, in place too."""
    x = torch.randn((2, 9000, 40, d), device="cuda", dtype=dtype)
    assert x.numel() * x.element_size() * 2 > 256 << 20
    pos = torch.arange(18000, dtype=torch.int32, device="cuda").view(2, 9000) * 7
    rot = T.Rotary(r, layout=layout)
    y = rot(x, pos)
    for b in range(2):
        for t in range(0, 9000, 3000):
            part = x[b:b + 1, t:t + 3000]
            assert part.numel() * part.element_size() * 2 < 256 << 20
            assert torch.equal(y[b:b + 1, t:t + 3000], rot(part, pos[b:b + 1, t:t + 3000].contiguous()))
    rot(x, pos, out=x)
    assert torch.equal(x, y)


# ---- the cache against its model ----

class Pair:
    """A cache on the GPU and its model, given the same calls."""

    def __init__(self, H, d, n_pages, n_seqs, seq_pages, dtype=BF, seed=0):
        self.g = T.PagedCache(H, d, n_pages, n_seqs, seq_pages)
        # what lies in unwritten places must not matter: NaN codes, NaN scales
        for x in (self.g.k, self.g.v):
            x.view(torch.uint8).fill_(0xff)
        self.g.scales.fill_(0xff)
        self.g.table.fill_(-7)
        self.m = O.Cache(H, d, n_pages, n_seqs, seq_pages)
        self.dtype, self.rng, self.H, self.d = dtype, np.random.default_rng(seed), H, d

    def tokens(self, B, N, scale=None):
        # sizes of blocks that differ, so that scales grow and stay
        s = 2.0 ** self.rng.integers(-6, 7, (B, N, 1, 1)) if scale is None else scale
        x = (self.rng.standard_normal((B, N, 2 * self.H, self.d)) * s).astype(np.float32)
        return torch.from_numpy(x).to("cuda").to(self.dtype)

    def append(self, seqs, N, counts=None, x=None):
        x = self.tokens(len(seqs), N) if x is None else x
        k, v = x[:, :, :self.H], x[:, :, self.H:]
        self.g.append(ints(seqs), k, v, None if counts is None else ints(counts))
        self.m.append(seqs, [N] * len(seqs) if counts is None else counts, k.float().cpu().numpy(),
                      v.float().cpu().numpy())

    def fork(self, src, dst):
        self.g.fork(ints(src), ints(dst))
        self.m.fork(src, dst)

    def free(self, seqs, keep=None):
        self.g.free(ints(seqs), None if keep is None else ints(keep))
        self.m.free(seqs, keep)

    def compact(self):
        self.g.compact()
        self.m.compact()

    def check(self):
        assert self.g.lengths.tolist() == self.m.lengths
        assert self.g.refs.tolist() == self.m.refs
        table = self.g.table.cpu().numpy()
        for s, pages in enumerate(self.m.pages):
            assert table[s, :len(pages)].tolist() == pages, s
        assert self.g.check() == (self.m.flags, self.m.used())
        n = max(self.m.lengths)
        if n:
            k, v = (x.cpu().numpy() for x in self.g.read(None, 0, n))
            for s, held in enumerate(self.m.lengths):
                wk, wv = self.m.held(s)
                assert np.array_equal(k[s, :held], wk) and np.array_equal(v[s, :held], wv), s
                assert not k[s, held:].any() and not v[s, held:].any()


@pytest.mark.parametrize("H,d,dtype", [(1, 32, BF), (2, 64, F32), (3, 96, BF), (2, 128, BF), (1, 160, F32), (2, 192, BF),
                                       (1, 224, BF), (1, 256, F32)])
def test_append_against_model(H, d, dtype):
    p = Pair(H, d, 20, 5, 6, dtype, seed=d)
    p.append([0, 3], 1)
    p.check()
    p.append([0, 1, 3], 15, [15, 7, 0])
    p.append([3, 0, 4], 70, [70, 1, 64])
    p.check()
    for _ in range(5):
        p.append([4, 1, 0, 3], 3, [3, 2, 1, 3])
    p.check()
    p.append([1, 0], 130, [-4, 500])                     # counts are clamped to 0 .. n_tokens
    p.check()
    say("held", p.m.lengths, "used", p.m.used())


def test_fork_copy_on_write_free_and_compact():
    p = Pair(2, 64, 40, 10, 5, BF, seed=9)
    p.append([0, 1], 150, [150, 64])
    p.fork([0, 0, 1, 2], [3, 4, 5, 6])                   # 2 is empty: so is 6
    p.check()
    p.append([3, 4, 0, 5], 5)                            # all who share a last page copy it
    p.check()
    p.free([0])
    p.append([2, 6], 70)
    p.check()
    p.free([3, 5, 4], [130, 64, 1])                      # into a shared page, at its end, into the first
    p.check()
    p.append([3, 4], 3)
    p.check()
    p.compact()
    p.check()
    p.free([1, 2])
    p.compact()
    p.append([0, 1], 66)
    p.check()
    p.compact()
    p.check()
    p.free(list(range(10)))
    p.check()
    p.compact()
    p.check()


def test_random_calls_against_model():
    p = Pair(1, 32, 30, 12, 4, BF, seed=4)
    rng = np.random.default_rng(4)
    for i in range(60):
        op = rng.integers(0, 6)
        seqs = rng.permutation(14)[:rng.integers(1, 7)] - 1   # -1 and 12 are out of range
        if op <= 2:
            n = int(rng.integers(1, 90))
            p.append(seqs.tolist(), n, rng.integers(0, n + 1, len(seqs)).tolist())
        elif op == 3:
            p.fork(seqs.tolist(), rng.permutation(14)[:len(seqs)].tolist())
        elif op == 4:
            p.free(seqs.tolist(), rng.integers(-1, 200, len(seqs)).tolist() if rng.integers(2) else None)
        else:
            p.compact()
        if i % 5 == 4:
            p.check()
    say("flags", p.m.flags, "used", p.m.used())


@pytest.mark.parametrize("H,d,dtype,n_seqs,n_pages", [(1, 32, BF, 300, 420), (3, 64, F32, 40, 60), (2, 256, BF, 9, 14)])
def test_single_tokens_against_model(H, d, dtype, n_seqs, n_pages):
    """Calls of one token an entry: new pages, copies of shared ones, scales
    that grow, entries left out, until the pool is used up."""
    p = Pair(H, d, n_pages, n_seqs, 3, dtype, seed=d)
    rng = np.random.default_rng(d)
    p.append(list(range(n_seqs)), 62, rng.integers(0, 63, n_seqs).tolist())
    p.fork([0, 1, 0], [n_seqs - 1, n_seqs - 2, n_seqs - 3])        # (not empty: left out)
    p.free([2, 3, 4])
    p.fork([5, 5, 6], [2, 3, 4])
    p.check()
    for i in range(12):
        seqs = rng.permutation(n_seqs + 2)[:rng.integers(1, n_seqs + 1)] - 1   # -1 and n_seqs are out of range
        seqs[rng.integers(len(seqs))] = seqs[0]                     # and one is listed twice
        p.append(seqs.tolist(), 1, rng.integers(-1, 3, len(seqs)).tolist() if i % 3 == 2 else None)
        if i % 4 == 3:
            p.check()
    for i in range(100 if n_seqs < 100 else 30):                    # everyone, over page ends, out of pages
        p.append(list(range(n_seqs)), 1)
        if i % 25 == 24:
            p.check()
    p.check()
    assert p.m.flags & O.NO_PAGES
    p.free([0])
    p.append([1, 2, 3], 1)
    p.check()
    say("flags", p.m.flags, "used", p.m.used(), "longest", max(p.m.lengths))


@pytest.mark.parametrize("H,d,dtype,n_seqs,n_pages", [(1, 32, BF, 120, 230), (3, 96, F32, 40, 75), (2, 256, BF, 9, 14),
                                                      (5, 128, BF, 60, 130)])
def test_few_tokens_against_model(H, d, dtype, n_seqs, n_pages):
    """Calls of 2 to 16 tokens an entry: over page ends, into copies of shared
    pages (two pages at once), entries left out, until the pool is used up."""
    p = Pair(H, d, n_pages, n_seqs, 3, dtype, seed=d + 1)
    rng = np.random.default_rng(d)
    p.append(list(range(n_seqs)), 63, rng.integers(40, 64, n_seqs).tolist())
    p.free([2, 3, 4])
    p.fork([5, 5, 6], [2, 3, 4])
    for i in range(10):
        N = int(rng.integers(2, 17))
        seqs = rng.permutation(n_seqs + 2)[:rng.integers(1, n_seqs + 1)] - 1   # -1 and n_seqs are out of range
        seqs[rng.integers(len(seqs))] = seqs[0]                     # and one is listed twice
        p.append(seqs.tolist(), N, rng.integers(-1, N + 2, len(seqs)).tolist() if i % 3 else None)
        if i == 4:
            a, b = int(seqs[-1] % n_seqs), int((seqs[-1] + 1) % n_seqs)
            p.free([b])
            p.fork([a], [b])
        p.check()
    for i in range(12):                                             # everyone, out of pages
        p.append(list(range(n_seqs)), 16)
        if i % 4 == 3:
            p.check()
    p.check()
    assert p.m.flags & O.NO_PAGES
    p.free([0])
    p.append([1, 2, 3], 9)
    p.check()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", range(32, 257, 32))
def test_append_and_read_every_width(d, dtype):
    """Each way that an append is launched (single tokens of few and of many
    entries, a few tokens, many), into copies too, at every head width and
    type; what is held reads back exactly in both types."""
    p = Pair(1, d, 330, 140, 3, dtype, seed=d + 3)
    p.append(list(range(130)), 20, [1 + i % 20 for i in range(130)])
    p.fork([3, 4, 15, 20], [130, 131, 132, 133])
    p.append(list(range(4, 134)), 1)
    p.append([5, 3, 20], 1)
    p.fork([7, 7], [134, 135])
    p.append([134, 7, 8], 9)
    p.append([135, 9, 10], 50)
    p.check()
    k, v = p.g.read(None, 5, 40)
    for x, y in zip((k, v), p.g.read(None, 5, 40, dtype=BF)):
        assert torch.equal(x.to(BF), y) and torch.equal(x, y.float())


@pytest.mark.parametrize("N", [1, 9, 40])
def test_append_into_a_scattered_pool(N):
    """Free pages far apart and in bunches of more than a call wants: each
    entry gets the lowest ones, whatever lies between, until there are none."""
    p = Pair(1, 32, 3300, 40, 6, BF, seed=N)
    rng = np.random.default_rng(N)
    holes = {0, 3, 255, 256, 1023, 1024, 1500, 2047, 2048, 2600, 3290, 3299}
    holes |= set(range(2700, 3240, 7)) | {3 + int(x) for x in rng.integers(0, 900, 12)}
    for page in range(3300):
        if page not in holes:
            p.m.refs[page] = 1
    p.g.refs.copy_(ints(p.m.refs))
    seqs = list(range(30))
    p.append(seqs, 63 if N < 40 else 30, [60 + i % 4 if N < 40 else 30 for i in range(30)])
    p.fork([0, 1, 2], [30, 31, 32])
    for i in range(14):
        p.append([int(x) for x in rng.permutation(33)], N)
        if i % 3 == 2:
            p.free([int(x) for x in rng.permutation(33)[:2]])        # low pages go free again: the bound follows
        p.check()
    assert p.m.flags & ~(O.NO_PAGES | O.FULL) == 0


def test_few_tokens_take_the_last_pages():
    """An entry that needs two pages (a copy and the next) and finds one takes
    none; the page goes to the next call."""
    p = Pair(1, 64, 4, 5, 3, BF, seed=9)
    p.append([0, 1], 60)
    p.fork([0], [2])
    p.append([3], 60)                                               # one page is left
    p.append([2, 1], 8)                                             # 2 needs two, 1 one: none
    assert p.m.flags == O.NO_PAGES and p.m.lengths[:3] == [60, 60, 60]
    p.check()
    p.append([2], 4)                                                # a copy alone fits
    p.check()
    assert p.m.lengths[2] == 64 and p.m.used() == 4
    p.free([3])
    p.append([0, 2, 1], 2)                                          # 0 and 1 stay in their pages, 2 begins one
    p.check()


def test_entries_left_out():
    p = Pair(1, 64, 4, 6, 3, BF, seed=5)
    p.append([0, 0, 9, -1, 1], 10)                       # the second 0, 9 and -1 are left out
    assert p.m.flags == O.BAD_ENTRY
    p.check()
    p.append([0], 190)                                   # beyond seq_pages * 64
    assert p.m.flags & O.FULL and p.m.lengths[0] == 10
    p.check()
    p.append([2, 3, 1, 4], 130, [64, 130, 1, 64])        # 2 has a page, 3's three are too many; 1 needs none
    assert p.m.flags & O.NO_PAGES and p.m.lengths[:5] == [10, 11, 64, 0, 0]
    p.check()
    p.append([4], 1)                                     # one page is left
    p.check()
    p.fork([0, 0, 0], [3, 3, 9])                         # 3 twice; out of range
    p.fork([2, 1, 4], [0, 5, 1])                         # not empty; its source is a destination; not empty
    p.check()
    p.append([0], 1)                                     # a copy of its shared page finds no page
    assert p.m.lengths[0] == 10
    p.check()
    p.free([0, 0, 40], [5, 2, 0])
    p.check()


def test_nonfinite_and_extreme_tokens():
    p = Pair(1, 32, 4, 2, 2, F32, seed=6)
    x = p.tokens(1, 40, scale=1.0)
    x[0, 3, 0, 5], x[0, 3, 1, 6], x[0, 20, 0, 7] = math.nan, math.inf, -math.inf
    x[0, 34] = 0
    x[0, 35:] *= 1e38 / 4
    p.append([0], 40, x=x)
    assert p.m.flags == O.NONFINITE
    p.check()
    y = p.tokens(1, 20, scale=1e-37)                     # below the least scale: held as zeros
    p.append([1], 20, x=y)
    p.check()


def test_snapshot_and_bad_tables():
    """A copy of meta is a snapshot; table entries out of range are left out
    by every call."""
    p = Pair(1, 64, 8, 3, 4, BF, seed=7)
    p.append([0, 1], 100)
    snap = p.g.meta.clone()
    k0, v0 = p.g.read(ints([0]), 0, 100)
    p.g.free(ints([0]))
    p.g.meta.copy_(snap)
    p.check()
    p.g.table[0, 1] = 99
    p.g.table[1, 0] = -3
    k, _ = p.g.read(ints([0]), 0, 100)
    assert torch.equal(k[:, :64], k0[:, :64]) and not k[:, 64:].any()
    x = p.tokens(2, 1)
    p.g.append(ints([0, 1]), x[:, :, :1], x[:, :, 1:])   # 0's last page is out of range
    assert p.g.lengths.tolist() == [100, 101, 0] and p.g.check()[0] == O.BAD_ENTRY
    p.g.fork(ints([0]), ints([2]))
    p.g.compact()
    p.g.free(None)
    assert p.g.lengths.tolist() == [0, 0, 0]


def unwritten_first_page(pair):
    """Takes page 0 out of the pool as it lies there (NaN codes, NaN scales)."""
    pair.g.refs[0], pair.m.refs[0] = 1, 1


@pytest.mark.parametrize("H,d,dtype,N,L", [(2, 64, BF, 1, 300), (1, 64, F32, 3, 300), (1, 32, BF, 17, 300), (1, 128, BF, 40, 300),
                                           (1, 256, BF, 20, 300), (1, 160, F32, 1, 300), (1, 64, BF, 2, 5000),
                                           (1, 96, F32, 1, 5000), (1, 64, BF, 70, 300), (2, 128, F32, 100, 300),
                                           (1, 192, BF, 90, 2000), (1, 64, BF, 130, 5000)])
def test_attend_bad_tables(H, d, dtype, N, L):
    """Pages whose table entries are out of range are not visible, whatever
    lies in the others: few and many rows, one range and several."""
    p = Pair(H, d, 90, 3, 80, dtype, seed=d + N)
    unwritten_first_page(p)
    p.append([2, 1], L, [L, 150], x=p.tokens(2, L, scale=1.0))
    bad, scale = {0: 99, 2: -3, (L - 1) // 64: 1 << 30}, 1 / math.sqrt(d)
    for page, entry in bad.items():
        p.g.table[2, page] = entry
    q, qn = normal((2, N, 2 * H, d), 3, dtype, 0.5)
    out = p.g.attend(ints([2, 1]), q, max_len=L)
    k, v = p.m.held(2)
    see = np.ones(L, bool)
    for page in bad:
        see[page * 64:page * 64 + 64] = False
    u, half = 2.0 ** -24, torch.finfo(dtype).eps / 2
    for i in range(N):
        at = see & (np.arange(L) <= L - N + i)
        want, spread, size = O.attend(k[at], v[at], qn[0, i:i + 1], scale)
        tol = spread * (2 * (d + 8) * u * size + 8 * u + L * u + (2.0 ** -8 if dtype == BF else 2.0 ** -23)) + half * np.abs(want)
        assert np.all(np.abs(out[0, i].float().cpu().numpy() - want[0]) <= tol[0]), i
    expect(p.g, p.m, [1], q[1:], None, scale, 0, 0, out[1:], out[1:])


@pytest.mark.parametrize("N", [1, 5])
@pytest.mark.parametrize("left", [7, 100000, -3])
def test_append_count_left_behind(N, left):
    """A blob whose append count is not 0 (a copy taken in the middle of a
    call): cleared where a handle adopts it, otherwise an append says so."""
    p = Pair(1, 64, 6, 2, 3, BF, seed=N)
    p.append([0], 30)
    p.g.status[2] = left
    old = p.g
    p.g = T.PagedCache(1, 64, 6, 2, 3, blob=old.blob)
    p.append([0], N)
    p.check()
    old.status[2] = left
    x = p.tokens(1, N)
    old.append(ints([0]), x[:, :, :1], x[:, :, 1:])                  # one workgroup: it is not the last by this count
    assert old.lengths.tolist() == [30 + N, 0] and old.check()[0] == O.BAD_ENTRY
    old.status.zero_()
    p.append([0, 1], N)
    p.check()


# ---- attention ----

def expect(cache, model, seqs, q, counts, scale, window, sink, got, before):
    """Every row of `got` against the oracle; rows behind the counts equal
    `before`."""
    B, N, H, d = q.shape
    bf = got.dtype == BF
    u, half = 2.0 ** -24, torch.finfo(got.dtype).eps / 2
    qn, y, was = (t.float().cpu().numpy().astype(np.float64) for t in (q, got, before))
    for b, s in enumerate(seqs):
        n = N if counts is None else min(max(counts[b], 0), N)
        assert np.array_equal(y[b, n:], was[b, n:]), "rows behind the count"
        if n == 0:
            continue
        L = model.lengths[s] if 0 <= s < len(model.lengths) else 0
        k, v = model.held(s) if L else (np.zeros((0, model.H, d)), np.zeros((0, model.H, d)))
        want, spread, size = O.attend(k, v, qn[b, :n], scale, window, sink)
        tol = spread * (2 * (d + 8) * u * size + 8 * u + L * u + (2.0 ** -8 if bf else 2.0 ** -23)) + half * np.abs(want)
        off = np.abs(y[b, :n] - want)
        assert np.all(off <= tol), (b, s, float((off - tol).max()), np.argwhere(off > tol)[:4].tolist())


ATTEND = [  # dtype, kv heads, heads, d, lengths, query tokens, counts, window, sink
    (BF, 1, 1, 64, [1], 1, None, 0, 0),
    (BF, 2, 8, 128, [0, 1, 63, 64, 65, 200], 1, None, 0, 0),
    (F32, 2, 8, 128, [0, 1, 63, 64, 65, 200], 1, None, 0, 0),
    (BF, 3, 9, 96, [40, 130, 5], 7, [7, 3, 7], 0, 0),
    (F32, 3, 9, 96, [40, 130, 5], 7, [0, 9, 7], 0, 0),
    (BF, 1, 16, 32, [333, 70], 3, None, 50, 0),
    (BF, 1, 17, 32, [333, 70], 2, None, 1, 5),
    (F32, 2, 2, 160, [500], 40, None, 100, 70),
    (BF, 2, 6, 192, [150, 260], 20, [20, 1], 64, 64),
    (BF, 1, 5, 224, [90, 91], 90, None, 0, 0),
    (F32, 1, 4, 256, [300], 33, None, 0, 0),
    (BF, 2, 128, 64, [77], 1, None, 0, 0),
    (BF, 2, 4, 64, [700, 64, 0], 130, [130, 65, 10], 0, 0),
    (F32, 1, 3, 64, [260], 257, None, 90, 3)]


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
@pytest.mark.parametrize("max_len", [0, 1])
def test_attend(case, max_len):
    dtype, H, heads, d, lengths, N, counts, window, sink = case
    seqs = [len(lengths) - i for i in range(len(lengths))]         # not in order, sequence 0 unused
    p = Pair(H, d, 60, len(lengths) + 1, 40, dtype, seed=d + N)
    for at in range(0, max(lengths), 61):                          # pages of different sequences alternate
        p.append(seqs, 61, [min(max(n - at, 0), 61) for n in lengths])
    q, _ = normal((len(seqs), N, heads + 3, d), 5, dtype, 0.5)
    q = q[:, :, 1:heads + 1] if d % 8 == 0 else q[:, :, :heads].contiguous()
    out = torch.full((len(seqs), N, heads, d), 3.0, dtype=dtype, device="cuda")
    before = out.clone()
    scale = 0.3 / math.sqrt(d)
    p.g.attend(ints(seqs), q, None if counts is None else ints(counts), scale, window, sink, max_len, out)
    expect(p.g, p.m, seqs, q, counts, scale, window, sink, out, before)


SHAPES = {  # how a call is launched: entries, kv heads, heads of each, query tokens, lengths (entries take them in turn), pages
    "few rows, waves share the sequence": (2, 2, 3, 4, [300, 70], 5),
    "few rows of many heads, waves share the sequence": (2, 40, 3, 4, [700, 70], 11),
    "few rows, ranges": (2, 2, 3, 4, [1500, 700], 30),
    "few rows, many ranges": (2, 1, 2, 1, [9300, 1000], 150),
    "two row groups": (2, 1, 5, 5, [1500, 70], 30),
    "four row groups": (2, 1, 12, 5, [1500, 70], 30),
    "four row groups, many ranges": (1, 1, 60, 1, [9000], 150),
    "many rows, waves share the sequence": (2, 1, 2, 70, [200, 130], 4),
    "many rows of many heads, waves share the sequence": (4, 64, 1, 70, [500, 460], 8),
    "many rows, ranges": (2, 1, 2, 70, [2600, 900], 41),
    "many rows, many ranges": (1, 1, 5, 33, [5000], 80),
    "many rows, many tiles": (8, 64, 1, 70, [150, 71, 20], 3)}


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", range(32, 257, 32))
@pytest.mark.parametrize("shape", SHAPES)
def test_attend_every_width(shape, d, dtype):
    """Each way that a call is launched, at every head width and type: ragged
    counts, without a mask and with a window and a sink."""
    B, H, G, N, lengths, pages = SHAPES[shape]
    lengths = [lengths[b % len(lengths)] for b in range(B)]
    seqs = list(range(B))[::-1]
    p = Pair(H, d, sum(-(-n // 64) for n in lengths) + 2, B, pages, dtype, seed=d + N)
    p.append(seqs, max(lengths), lengths, x=p.tokens(B, max(lengths), scale=1.0))
    q, _ = normal((B, N, H * G, d), 5, dtype, 0.5)
    counts = [N - 2 * b % N for b in range(B)] if N > 1 else None
    for window, sink in ((0, 0), (100, 70)):
        out = torch.full((B, N, H * G, d), 3.0, dtype=dtype, device="cuda")
        before = out.clone()
        p.g.attend(ints(seqs), q, None if counts is None else ints(counts), window=window, sink=sink, out=out)
        expect(p.g, p.m, seqs, q, counts, 1 / math.sqrt(d), window, sink, out, before)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-30, -1e-42])
@pytest.mark.parametrize("dtype,N", [(BF, 3), (F32, 2), (BF, 40), (F32, 40)])
def test_attend_scales(dtype, N, scale):
    """No scale (the mean of what is seen), a negative and a tiny one; masked
    tokens stay out of it."""
    p = Pair(1, 64, 10, 2, 4, dtype, seed=12)
    p.append([0, 1], 150, [150, 70])
    q, _ = normal((2, N, 3, 64), 6, dtype)
    out = p.g.attend(ints([0, 1]), q, scale=scale, window=60, sink=4)
    expect(p.g, p.m, [0, 1], q, None, scale, 60, 4, out, out)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_long_and_divided(dtype):
    """A sequence over many ranges, and the same sequence listed twice."""
    p = Pair(1, 64, 140, 2, 140, dtype, seed=3)
    x = p.tokens(1, 8900, scale=1.0)
    p.append([1], 8900, x=x)
    for N in (1, 6, 20):
        q, _ = normal((2, N, 4, 64), N, dtype)
        out = p.g.attend(ints([1, 1]), q)
        expect(p.g, p.m, [1, 1], q, None, 0.125, 0, 0, out, out)
        out = p.g.attend(ints([1, 1]), q, window=3000, sink=200)
        expect(p.g, p.m, [1, 1], q, None, 0.125, 3000, 200, out, out)


@pytest.mark.parametrize("d,heads,N,L", [(64, 6, 1, 1000), (128, 8, 1, 4000), (96, 4, 3, 300), (32, 2, 20, 700), (256, 4, 12, 900),
                                         (192, 3, 16, 500), (64, 64, 1, 3000)])
def test_attend_weights_of_few_rows(d, heads, N, L):
    """bf16 calls of up to 64 rows a key head keep 16 bits of the softmax
    weights (two parts, each off by 2^-8 at most): r = 2^-16 in the bound."""
    p = Pair(1, d, 70, 1, 70, BF, seed=d)
    p.append([0], L, x=p.tokens(1, L, scale=1.0))
    q, qn = normal((1, N, heads, d), 21, BF)
    scale, u = 1 / math.sqrt(d), 2.0 ** -24
    for max_len in (0, L):
        got = p.g.attend(ints([0]), q, max_len=max_len).float().cpu().numpy()[0]
        want, spread, size = O.attend(*p.m.held(0), qn[0], scale)
        tol = spread * (2 * (d + 8) * u * size + 8 * u + L * u + 2.0 ** -16) + 2.0 ** -8 * np.abs(want)
        off = np.abs(got - want)
        assert np.all(off <= tol), float((off - tol).max())


@pytest.mark.parametrize("N", [1, 5, 14, 33])
def test_attend_stays_in_its_workspace(N):
    """Whatever max_len a call names, it writes its partial results within
    the workspace that tm_cache_workspace_bytes gives (here inside a larger
    buffer), and the result holds."""
    A = T.attention
    c = T.PagedCache(4, 32, 700, 5, 600)
    x = normal((1, 1500, 8, 32), 3)[0]
    c.append(ints([4]), x[:, :, :4], x[:, :, 4:])
    for s in range(4):
        c.fork(ints([4]), ints([s]))
    q = normal((4, N, 8, 32), 4)[0]
    need = A.tm_cache_workspace_bytes(c.handle, 4, N, 8)
    want = c.attend(None, q)
    room = torch.full((need + (64 << 20),), 0x5a, dtype=torch.uint8, device="cuda")
    for pages in (1, 7, 24, 25, 64, 128, 256, 511, 512, 513, 600):
        out = torch.empty_like(q)
        rc = A._lib().tm_cache_attend(c.handle, c.blob.data_ptr(), None, None, q.data_ptr(), q.stride(0), q.stride(1),
                                      out.data_ptr(), 4, N, 8, 1 / math.sqrt(32), 0, 0, 64 * pages, T.TM_BF16,
                                      room.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert rc == T.TM_OK
        assert bool((room[need:] == 0x5a).all()), pages
        # each of the two is off by a weight's and the result's rounding: the weighted mean of |v| is at most the largest
        assert float((out.float() - want.float()).abs().max()) <= 2 * 2.0 ** -8 * float(x.abs().max() + want.abs().max()) * 1.01


def test_attend_window_beyond_any_sequence():
    """A window wider than any sequence is none, also for rows that stand
    before the sequence's start."""
    p = Pair(1, 64, 10, 2, 4, BF, seed=13)
    p.append([0, 1], 150, [150, 5])
    for N in (3, 40, 100):
        q = normal((2, N, 2, 64), N)[0]
        out = p.g.attend(ints([0, 1]), q, window=(1 << 31) - 1, sink=(1 << 31) - 1)
        expect(p.g, p.m, [0, 1], q, None, 0.125, 0, 0, out, out)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N,heads,L,max_len", [(1, 8, 200, 200), (4, 8, 700, 700), (4, 8, 2000, 0), (14, 8, 700, 0), (40, 8, 300, 300),
                                               (50, 8, 2000, 0)])
def test_attend_into_its_queries(dtype, N, heads, L, max_len):
    """The output may take the queries' place, however the call is launched."""
    p = Pair(2, 64, 70, 2, 32, dtype, seed=N)
    p.append([0, 1], L, [L, 150], x=p.tokens(2, L, scale=1.0))
    q = normal((2, N, heads, 64), 3, dtype)[0]
    counts = ints([N, max(1, N // 2)])
    want = p.g.attend(None, q, counts, max_len=max_len, out=q.clone())
    assert torch.equal(p.g.attend(None, q, counts, max_len=max_len, out=q), want)


def test_values_beyond_the_largest_scale():
    """Finite elements beyond 448 * 2^119 are held as that, in the order of a
    block's other elements, and set no flag."""
    c = T.PagedCache(1, 32, 4, 2, 2)
    top = 448.0 * 2.0 ** 119
    x = torch.full((1, 20, 1, 32), 1.0, device="cuda")
    x[0, 3, 0, 4], x[0, 3, 0, 5], x[0, 3, 0, 6] = 3.4e38, -3.3e38, top
    c.append(ints([0]), x, x)
    c.append(ints([1]), x[:, 3:4].contiguous(), x[:, 3:4].contiguous())
    for s, t in ((0, 3), (1, 0)):
        for y in c.read(ints([s]), t, 1):
            assert y[0, 0, 0, 4:7].tolist() == [top, -top, top] and not y[0, 0, 0, 7:].any()
    assert c.check()[0] == 0


def test_numbers_past_32_bits():
    """Windows, sinks, lengths and starts past 32 bits are what they say."""
    p = Pair(1, 64, 10, 2, 4, BF, seed=16)
    p.append([0, 1], 150, [150, 70])
    q, big = normal((2, 3, 2, 64), 3)[0], 1 << 32
    want = p.g.attend(None, q)
    for kw in (dict(window=big + 5), dict(window=20, sink=big + 1), dict(max_len=big + 64), dict(window=big, sink=big)):
        assert torch.equal(p.g.attend(None, q, **kw), want)
    k, v = p.g.read(None, big + 3, 10)
    assert not k.any() and not v.any()
    for kw in (dict(window=-big), dict(sink=-big + 2), dict(max_len=-big)):
        with pytest.raises(T.TMError):
            p.g.attend(None, q, **kw)
    with pytest.raises(T.TMError):
        p.g.read(None, -big, 10)


def test_pools_past_32_bit_offsets():
    """Pages whose keys and values lie beyond 4 GiB of the pool's start: the
    same calls as on a small pool give the same codes and results."""
    H, d, far = 8, 256, 36000
    small, big = T.PagedCache(H, d, 12, 3, 4), T.PagedCache(H, d, far + 12, 3, 4)
    assert big.k.numel() > 1 << 32
    big.refs[:far] = 1                                              # all but the last pages are taken
    x, q = normal((2, 130, 2 * H, d), 1)[0], normal((2, 3, 2 * H, d), 2)[0]
    outs = []
    for c in (small, big):
        c.append(ints([0, 2]), x[:, :, :H], x[:, :, H:])
        c.fork(ints([2]), ints([1]))
        c.append(ints([1]), x[:1, :1, :H], x[:1, :1, H:])           # a copy of the shared last page
        outs.append([c.attend(None, torch.cat([q, q[:1]])), c.attend(ints([1]), x[:1, :, :H])] + list(c.read(None, 0, 131)))
        c.free(ints([0]))
    big.compact()                                                   # the last pages move down by one sequence's
    outs.append([outs[1][0]] + [big.attend(ints([1]), x[:1, :, :H])] + list(big.read(None, 0, 131)))
    assert all(torch.equal(a, b) for a, b in zip(outs[0], outs[1]))
    assert torch.equal(outs[2][1], outs[1][1]) and torch.equal(outs[2][2][1:], outs[1][2][1:])
    assert int(big.table[1, 0]) >= far and big.check() == (0, far + 4)


def test_attend_sharp_scores_and_masked_rows():
    """Scores of hundreds (one token takes all the weight), a sequence out of
    range, a non-finite query row beside finite ones."""
    p = Pair(1, 64, 10, 3, 4, BF, seed=8)
    p.append([0, 2], 200)
    q, _ = normal((4, 2, 2, 64), 1, BF, 8.0)
    q[1, 0, 1] = math.nan
    out = p.g.attend(ints([0, 2, 7, -1]), q, scale=1.0)
    assert torch.isnan(out[1, 0, 1]).all()
    out[1, 0, 1] = 0
    q0 = q.clone()
    q0[1, 0, 1] = 0
    keep = out.clone()
    w = p.g.attend(ints([0, 2, 7, -1]), q0, scale=1.0)
    keep[1, 0, 1] = w[1, 0, 1]
    assert torch.equal(keep, w)                                     # the NaN row touched no other
    assert not out[2:].any()
    expect(p.g, p.m, [0, 2, 7, -1], q0, None, 1.0, 0, 0, w, w)


@pytest.mark.parametrize("dtype,N", [(BF, 2), (F32, 3), (BF, 11), (BF, 50), (F32, 50)])
def test_attend_rows_do_not_depend_on_each_other(dtype, N):
    """A row's bits are the same whatever the rows beside it are (small
    queries among large ones, whose maxima grow at other pages)."""
    p = Pair(1, 64, 20, 2, 12, dtype, seed=14)
    p.append([0, 1], 700, [700, 333])
    q, _ = normal((2, N, 4, 64), 15, dtype)
    small, big = q * 1.5, q * 12
    mixed, others = small.clone(), small.clone()
    mixed[:, ::2, 1::2] = big[:, ::2, 1::2]
    others[:, ::2, 1::2] = 0
    a, b = (p.g.attend(ints([0, 1]), x) for x in (mixed, others))
    a[:, ::2, 1::2] = 0
    b[:, ::2, 1::2] = 0
    assert torch.equal(a, b)


def test_streams_and_graphs():
    """Append, attend and free in a captured graph, replayed between eager
    calls; two graphs of one cache's reads on two streams."""
    p = Pair(2, 64, 30, 4, 8, BF, seed=11)
    p.append([0, 1, 2, 3], 100)
    x, q = p.tokens(4, 1), normal((4, 1, 4, 64), 2)[0]
    seqs, keep = ints([0, 1, 2, 3]), ints([100] * 4)
    xs, qs = torch.empty_like(x), torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            p.g.append(seqs, x[:, :, :2], x[:, :, 2:])
            p.g.attend(seqs, q)
            p.g.free(seqs, keep)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.g.append(seqs, xs[:, :, :2], xs[:, :, 2:])
        out = p.g.attend(seqs, qs)
        p.g.free(seqs, keep)
    for i in range(4):
        x, q = p.tokens(4, 1), normal((4, 1, 4, 64), 20 + i)[0]
        xs.copy_(x)
        qs.copy_(q)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        p.g.append(seqs, x[:, :, :2], x[:, :, 2:])
        want = p.g.attend(seqs, q)
        p.g.free(seqs, keep)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and p.g.lengths.tolist() == [100] * 4
    # reads on two streams at once, each with its own workspace
    q2 = normal((4, 3, 4, 64), 31)[0]
    want, want2 = p.g.attend(seqs, q), p.g.attend(seqs, q2)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    outs = []
    for _ in range(10):
        outs.append((p.g.attend(seqs, q, stream=side), p.g.attend(seqs, q2, stream=other)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want) and torch.equal(b, want2) for a, b in outs)


@pytest.mark.parametrize("N", [1, 5, 40])
def test_append_replayed(N):
    """A captured append, replayed over page ends and into a copy, between
    eager appends of other entries: each as its model says."""
    p = Pair(3, 64, 40, 5, 8, BF, seed=N)
    p.append([0, 1, 2], 62)
    p.fork([1], [3])
    seqs, x = [0, 3, 1], p.tokens(3, N)
    xs, ids = torch.empty_like(x), ints(seqs)
    p.g.append(ids[:0], xs[:0, :, :3], xs[:0, :, 3:])               # (loads the kernels; appends nothing)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.g.append(ids, xs[:, :, :3], xs[:, :, 3:])
    for i in range(6):
        x = p.tokens(3, N)
        xs.copy_(x)
        graph.replay()
        p.m.append(seqs, [N] * 3, x[:, :, :3].float().cpu().numpy(), x[:, :, 3:].float().cpu().numpy())
        p.append([2, 4], 3)
        p.check()
    assert p.m.flags == 0


def test_refusals_on_device():
    c = T.PagedCache(2, 64, 4, 2, 2)
    x = torch.zeros((1, 3, 2, 64), dtype=BF, device="cuda")
    for bad, match in ((x[:, :, :1], "shape"), (x[..., :32], "contiguous"), (x.cpu(), "on")):
        with pytest.raises(ValueError, match=match):
            c.append(ints([0]), bad, bad)
    with pytest.raises(TypeError, match="v"):
        c.append(ints([0]), x, x.float())
    with pytest.raises(ValueError, match="seqs"):
        c.append(ints([0, 1]), x, x)
    with pytest.raises(TypeError, match="int32"):
        c.attend(torch.zeros(1, dtype=torch.int64, device="cuda"), x)
    with pytest.raises(ValueError, match="16-byte"):
        y = torch.zeros(1 * 3 * 2 * 64 + 4, dtype=BF, device="cuda")[4:].view(1, 3, 2, 64)
        c.attend(ints([0]), y)
    with pytest.raises(T.TMError):
        c.attend(ints([0]), torch.zeros((1, 1, 3, 64), dtype=BF, device="cuda"))
    with pytest.raises(T.TMError):
        c.append(None, x.expand(3, 3, 2, 64), x.expand(3, 3, 2, 64))   # more entries than sequences
    assert c.check() == (0, 0)


def test_timing_class():
    c = T.PagedCache(1, 64, 4, 2, 2)
    x = torch.ones((1, 3, 1, 64), dtype=BF, device="cuda")
    T.tm_timing_enable(1 << T.attention.K_ATTENTION)
    T.tm_timing_read(T.attention.K_ATTENTION)
    c.append(ints([0]), x, x)
    y = c.attend(ints([0]), x)
    torch.cuda.synchronize()
    ms, n = T.tm_timing_read(T.attention.K_ATTENTION)
    T.tm_timing_enable(0)
    assert n == 2 and ms > 0 and bool((y == 1).all())
