"""The attention window's operators: what is measured, and their plain forms.

Three kinds of calls stand here, those that a server of memory-as-context
layers makes around the memory's own: rotary positions (``Rotary``), a paged
cache held in 8 bits with the attention that reads it (``PagedCache.append``,
``PagedCache.attend``), and the pages' own housekeeping (``fork``, ``free``,
``compact``).  The plain forms are elementary torch operations on the same
buffers.

The cache's buffers, as the framework documents them (one blob of bytes, each
region 256-byte aligned):

    meta    int32: status [64], lengths [n_seqs], refs [n_pages] (how many
            table entries hold the page, 0: free), table [n_seqs][seq_pages]
    scales  uint8 [n_pages][kv_heads][2 (k, v)][4]: exponent + 127 of the
            power of two that a block of 16 tokens is scaled by
    k       e4m3 [n_pages][kv_heads][64 tokens][dim]
    v       e4m3 [n_pages][kv_heads][dim][64 tokens]
"""
import math

import numpy as np
import torch

own = False

PAGE, BLOCK = 64, 16          # tokens of a page, and of a block with one scale
E_MIN, E_MAX = -110, 119      # range of a block's exponent
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# the cases

def rotary(name, batch, tokens, heads, dim, rot, layout, scaling, back, dtype, far):
    return {"name": name, "op": "rotary", "batch": batch, "tokens": tokens, "heads": heads, "dim": dim, "rot": rot,
            "layout": layout, "scaling": scaling, "back": back, "dtype": dtype, "far": far}


def append(name, batch, tokens, held, most, kv_heads, dim, dtype):
    return {"name": name, "op": "append", "batch": batch, "tokens": tokens, "held": held, "most": most,
            "kv_heads": kv_heads, "dim": dim, "dtype": dtype}


def attend(name, batch, queries, ragged, heads, kv_heads, dim, least, most, window, sink, dtype):
    return {"name": name, "op": "attend", "batch": batch, "queries": queries, "ragged": ragged, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "least": least, "most": most, "window": window, "sink": sink,
            "dtype": dtype}


def fork(name, parents, children, least, most, kv_heads, dim, dtype):
    return {"name": name, "op": "fork", "parents": parents, "children": children, "least": least, "most": most,
            "kv_heads": kv_heads, "dim": dim, "dtype": dtype}


def compact(name, seqs, least, most, every, kv_heads, dim):
    return {"name": name, "op": "compact", "seqs": seqs, "least": least, "most": most, "every": every,
            "kv_heads": kv_heads, "dim": dim}


def listed():
    return [
        # one new token of each of 4 sequences, queries and keys together: a step's latency
        rotary("rotary_step", 4, 1, 8, 64, 64, "half", "none", False, "bf16", 4000),
        # two long prompts, 32 query and 8 key heads, positions scaled for a long context
        rotary("rotary_prompt", 2, 16384, 40, 128, 128, "interleaved", "parts", False, "bf16", 1000000),
        # the gradient of a training step through rotary positions on part of the head
        rotary("rotary_gradient", 3, 1023, 9, 96, 64, "half", "linear", True, "f32", 60000),
        # a decode step that drops a rejected draft token and writes the accepted one, 64 sequences
        append("append_step", 64, 1, 500, 4000, 8, 128, "bf16"),
        # eight prompts of ragged lengths admitted to slots that were just released
        append("append_prompts", 8, 4096, 0, 0, 8, 128, "bf16"),
        # the smallest decode step: one token against a window of persistent, recalled and segment tokens
        attend("attend_step", 2, 1, False, 6, 6, 64, 1500, 2064, 0, 0, "bf16"),
        # a serving batch's decode step, lengths as they come
        attend("attend_batch", 48, 1, False, 32, 8, 128, 2000, 30000, 0, 0, "bf16"),
        # four tokens of one very long stream, in 32 bits, wide heads
        attend("attend_far", 1, 4, False, 16, 2, 256, 1000003, 1000003, 0, 0, "f32"),
        # a whole segment over its window, as memory as a context runs it
        attend("attend_window", 2, 1024, False, 6, 6, 64, 2064, 2064, 0, 0, "bf16"),
        # a prompt's chunk behind a longer context: a sliding window and the persistent tokens
        attend("attend_prompt", 2, 2048, True, 32, 8, 128, 5000, 7001, 4096, 16, "bf16"),
        # sampling 16 continuations of each of 8 prompts: fork, then each writes its first token
        fork("fork_samples", 8, 16, 100, 1000, 8, 128, "bf16"),
        # a pool with a third of its sequences gone, brought together at its low end
        compact("compact_pool", 256, 500, 4000, 3, 8, 128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "append", "append", "attend", "attend", "attend", "attend", "fork", "compact"])
    dim = 32 * rng.randint(1, 8)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    kv = rng.choice([1, 2, 3, 4, 6, 8])
    if op == "rotary":
        batch, heads = _log(rng, 1, 32), rng.randint(1, 48)
        most = max(1, min(16384, (2 * 16384 * 40 * 128) // (2 * batch * heads * dim)))
        return rotary("", batch, _log(rng, 1, most), heads, dim, rng.choice([dim, dim // 2, 2 * rng.randint(1, dim // 2)]),
                      rng.choice(["half", "interleaved"]), rng.choice(["none", "linear", "parts"]), rng.random() < 0.4,
                      dtype, _log(rng, 1000, 2000000))
    if op == "append":
        if rng.random() < 0.5:   # a few tokens of many sequences
            held = _log(rng, 1, 500)
            return append("", _log(rng, 1, 128), rng.randint(1, 8), held, held + _log(rng, 1, 2000), kv, dim, dtype)
        batch = _log(rng, 1, 16)
        return append("", batch, _log(rng, 2, 16384 // batch), 0, 0, kv, dim, dtype)
    if op == "attend":
        group = rng.randint(1, 8)
        window = rng.choice([0, 0, 0, _log(rng, 16, 4096)])
        sink = rng.choice([0, rng.randint(1, 100)]) if window else 0
        if rng.random() < 0.6:   # single tokens and short drafts
            batch = _log(rng, 1, 64)
            most = _log(rng, 1, min(400000, 48 * 16000 * 8 * 128 // (batch * kv * dim)))
            return attend("", batch, rng.randint(1, 5), rng.random() < 0.3, kv * group, kv, dim, max(1, most // rng.choice([1, 2, 10])), most,
                          window, sink, dtype)
        batch = _log(rng, 1, 8)
        queries = _log(rng, 6, 2048)
        most = min(12000, queries + _log(rng, 1, 8000))
        while batch * queries * most * kv * group * dim > 50 * 10 ** 9 // (2 if dtype == "f32" else 1):
            queries, most, batch = max(6, queries // 2), max(6, most // 2), max(1, batch // 2)
        return attend("", batch, queries, rng.random() < 0.5, kv * group, kv, dim, max(1, most // rng.choice([1, 2])), most,
                      window, sink, dtype)
    if op == "fork":
        least = _log(rng, 1, 500)
        return fork("", _log(rng, 1, 16), _log(rng, 1, 16), least, least + _log(rng, 1, 2000), kv, dim, dtype)
    least = _log(rng, 1, 1000)
    return compact("", _log(rng, 2, 256), least, least + _log(rng, 1, 3000), rng.randint(2, 5), kv, dim)


# ---------------------------------------------------------------------------
# a case's inputs

def _spread(least, most, n):
    return [least + (most - least) * i // max(1, n - 1) for i in range(n)]


def _ceil(a, b):
    return -(-a // b)


def _pool(kv_heads, dim, n_pages, n_seqs, seq_pages):
    """An empty pool's blob and its views."""
    up = lambda n: _ceil(n, 256) * 256  # noqa: E731
    ints, cells = 64 + n_seqs + n_pages + n_seqs * seq_pages, n_pages * kv_heads * PAGE * dim
    o_s = up(4 * ints)
    o_k = o_s + up(n_pages * kv_heads * 8)
    o_v = o_k + up(cells)
    blob = torch.zeros(o_v + up(cells), dtype=torch.uint8, device="cuda")
    meta = blob[:4 * ints].view(torch.int32)
    c = {"blob": blob, "meta": meta, "status": meta[:64], "lengths": meta[64:64 + n_seqs],
         "refs": meta[64 + n_seqs:64 + n_seqs + n_pages], "table": meta[64 + n_seqs + n_pages:].view(n_seqs, seq_pages),
         "scales": blob[o_s:o_s + n_pages * kv_heads * 8].view(n_pages, kv_heads, 2, 4),
         "k": blob[o_k:o_k + cells].view(n_pages, kv_heads, PAGE, dim),
         "v": blob[o_v:o_v + cells].view(n_pages, kv_heads, dim, PAGE)}
    if own:   # the handle that a program makes once for its pool
        import test_trained_neural_amd as T
        c["cache"] = T.PagedCache(kv_heads, dim, n_pages, n_seqs, seq_pages, device="cuda", blob=blob)
    return c


def _fill(c, lengths, order, g):
    """Sequences of `lengths` tokens on the pages of `order`: values of about unit size, as a cache of normalised keys and
    values holds them (a block's largest value near the top of the type's range)."""
    n_seqs, seq_pages = c["table"].shape
    held = np.array([_ceil(n, PAGE) for n in lengths], np.int64)
    total = int(held.sum())
    table = np.zeros((n_seqs, seq_pages), np.int32)
    rows = np.repeat(np.arange(len(lengths)), held)
    cols = np.arange(total) - np.repeat(np.cumsum(held) - held, held)
    table[rows, cols] = order[:total]
    refs = np.zeros(c["refs"].numel(), np.int32)
    refs[order[:total]] = 1
    c["table"].copy_(torch.from_numpy(table))
    c["refs"].copy_(torch.from_numpy(refs))
    c["lengths"][:len(lengths)] = torch.tensor(lengths, dtype=torch.int32)
    for x in (c["k"], c["v"]):
        flat = x.view(-1)
        for at in range(0, flat.numel(), 1 << 28):
            part = flat[at:at + (1 << 28)]
            part.copy_(torch.randn(part.numel(), generator=g, device="cuda").mul_(100).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    c["scales"].copy_(torch.randint(119, 122, c["scales"].shape, generator=g, device="cuda", dtype=torch.uint8))


def _counts(case):
    n = case["queries"] if case["op"] == "attend" else case["tokens"]
    ragged = case.get("ragged", case["op"] == "append" and case["held"] == 0)
    return _spread(_ceil(n, 2), n, case["batch"]) if ragged else [n] * case["batch"]


def _lengths(case, r):
    n = _spread(case["least"], case["most"], case["batch"] if case["op"] == "attend" else case.get("parents") or case["seqs"])
    r.shuffle(n)
    return n


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 31))
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    s = {"case": dict(case)}
    dt = TYPES.get(case.get("dtype"))
    if case["op"] == "rotary":
        b, t, h, d = case["batch"], case["tokens"], case["heads"], case["dim"]
        if case["back"]:
            s["x"] = normal(b, t, h, d).to(dt)
        else:   # queries and keys beside the values in one projection's output
            s["x"] = normal(b, t, h + max(1, h // 4), d).to(dt)[:, :, :h]
        start = r.randint(0, case["far"], b)
        if t == 1:
            s["positions"] = ints(start.tolist())
        else:
            s["positions"] = torch.from_numpy((start[:, None] + np.arange(t)[None]).astype(np.int32)).to("cuda")
        s["freq"], s["scale"] = _frequencies(case)
        if own:
            import test_trained_neural_amd as T
            s["rotary"] = T.Rotary(case["rot"], base=10000.0, device="cuda", **_scaling(case, T),
                                   layout=T.TM_ROPE_HALF if case["layout"] == "half" else T.TM_ROPE_INTERLEAVED)
        return s
    kv, d = case["kv_heads"], case["dim"]
    if case["op"] == "append":
        b, t = case["batch"], case["tokens"]
        n = _counts(case)
        r.shuffle(n)
        held = _spread(case["held"], case["most"], b)
        r.shuffle(held)
        pages = [_ceil(a + c, PAGE) for a, c in zip(held, n)]
        n_pages = sum(pages) + 8
        c = s["c"] = _pool(kv, d, n_pages, b + 3, max(pages) + 1)
        # the slots hold what the call will drop: last step's tokens, or earlier prompts
        _fill(c, [a + t for a in held] if case["held"] else n, r.permutation(n_pages), g)
        s["seqs"] = ints(list(range(b)))
        s["keep"] = ints(held)
        s["counts"] = ints(n) if case["held"] == 0 else None
        s["kv"] = normal(b, t, 2 * kv, d)
        s["kv"][..., :: max(1, d // 4)] *= 4.0   # a few wide channels, as keys have
        s["kv"] = s["kv"].to(dt)
        return s
    if case["op"] == "attend":
        b, t = case["batch"], case["queries"]
        lengths = _lengths(case, r)
        n_pages = sum(_ceil(n, PAGE) for n in lengths) + 5
        s["c"] = _pool(kv, d, n_pages, b + 2, _ceil(case["most"], PAGE) + 1)
        _fill(s["c"], lengths, r.permutation(n_pages), g)
        s["seqs"] = ints(list(range(b)))
        s["q"] = normal(b, t, case["heads"], d).to(dt)
        s["counts"] = ints(_counts(case)) if case["ragged"] else None
        s["out"] = torch.zeros(b, t, case["heads"], d, dtype=dt, device="cuda")
        return s
    if case["op"] == "fork":
        p, n = case["parents"], case["parents"] * case["children"]
        lengths = _lengths(case, r)
        held = sum(_ceil(x, PAGE) for x in lengths)
        n_pages = held + 2 * n + 7
        s["c"] = _pool(kv, d, n_pages, p + n, _ceil(case["most"], PAGE) + 2)
        _fill(s["c"], lengths, r.permutation(n_pages), g)
        s["src"] = ints([i % p for i in range(n)])
        s["dst"] = ints([p + i for i in range(n)])
        s["kv"] = normal(n, 1, 2 * kv, d).to(dt)
        return s
    lengths = _lengths(case, r)
    n_pages = sum(_ceil(x, PAGE) for x in lengths) + 3
    c = s["c"] = _pool(kv, d, n_pages, case["seqs"], _ceil(case["most"], PAGE) + 1)
    _fill(c, lengths, np.arange(n_pages), g)
    gone = torch.arange(r.randint(case["every"]), case["seqs"], case["every"], dtype=torch.int32, device="cuda")
    _free(c, gone, None)
    s["meta"] = c["meta"].clone()
    return s


def _scaling(case, T):
    if case["scaling"] == "linear":
        return {"scaling": T.TM_ROPE_LINEAR, "factor": 8.0}
    if case["scaling"] == "parts":
        return {"scaling": T.TM_ROPE_PARTS, "factor": 16.0, "original_len": 4096}
    return {}


def _frequencies(case):
    """The angle that each pair turns by per token (64 bits, on the GPU), and the factor of the result."""
    r = case["rot"]
    f = 10000.0 ** (-2.0 * torch.arange(r // 2, dtype=torch.float64) / r)
    if case["scaling"] == "linear":
        return (f / 8.0).cuda(), 1.0
    if case["scaling"] != "parts":
        return f.cuda(), 1.0
    # pairs that turn over 32 times within the original length stay, those that turn less than once are
    # stretched by the factor, and between them the share goes linearly with the pair's index
    at = lambda turns: r * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
    lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), r // 2 - 1)
    share = ((torch.arange(r // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return (f * (1 - share) + f / 16.0 * share).cuda(), 0.1 * math.log(16.0) + 1.0


# ---------------------------------------------------------------------------
# one pass

def run(s):
    return _OPS[s["case"]["op"]](s)


def _pool_outputs(c):
    return {"k": c["k"].view(torch.float8_e4m3fn), "v": c["v"].view(torch.float8_e4m3fn), "scales": c["scales"],
            "lengths": c["lengths"], "refs": c["refs"], "table": c["table"]}


def _run_rotary(s):
    if own:
        return s["rotary"](s["x"], s["positions"], inverse=s["case"]["back"])
    return _rotary(s["x"], s["positions"], s["freq"], s["scale"], s["case"])


def _run_append(s):
    c, kv = s["c"], s["case"]["kv_heads"]
    k, v = s["kv"][:, :, :kv], s["kv"][:, :, kv:]
    if own:
        c["cache"].free(s["seqs"], s["keep"])
        c["cache"].append(s["seqs"], k, v, s["counts"])
    else:
        _free(c, s["seqs"], s["keep"])
        _append(c, s["seqs"], k, v, s["counts"])
    return _pool_outputs(c)


def _run_attend(s):
    case = s["case"]
    if own:
        return s["c"]["cache"].attend(s["seqs"], s["q"], s["counts"], window=case["window"], sink=case["sink"], out=s["out"])
    return _attend(s["c"], s["seqs"], s["q"], s["counts"], case["window"], case["sink"], s["out"])


def _run_fork(s):
    c, kv = s["c"], s["case"]["kv_heads"]
    k, v = s["kv"][:, :, :kv], s["kv"][:, :, kv:]
    if own:
        c["cache"].free(s["dst"])
        c["cache"].fork(s["src"], s["dst"])
        c["cache"].append(s["dst"], k, v)
    else:
        _free(c, s["dst"], None)
        _fork(c, s["src"], s["dst"])
        _append(c, s["dst"], k, v, None)
    return _pool_outputs(c)


def _run_compact(s):
    s["c"]["meta"].copy_(s["meta"])   # the pool as the snapshot has it
    if own:
        s["c"]["cache"].compact()
    else:
        _compact(s["c"])
    return _pool_outputs(s["c"])


_OPS = {"rotary": _run_rotary, "append": _run_append, "attend": _run_attend, "fork": _run_fork, "compact": _run_compact}


# ---------------------------------------------------------------------------
# the plain forms

def _rotary(x, positions, freq, scale, case):
    pos = positions if positions.dim() == 2 else positions[:, None]
    angle = pos.double()[:, :, None] * freq                       # far positions: 64 bits
    if case["back"]:
        angle = -angle                                            # the transpose of a rotation
    cos, sin = (torch.cos(angle) * scale).float()[:, :, None], (torch.sin(angle) * scale).float()[:, :, None]
    r = case["rot"]
    turned, rest = x[..., :r].float(), x[..., r:]
    if case["layout"] == "half":
        a, b = turned[..., :r // 2], turned[..., r // 2:]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    else:
        a, b = turned[..., 0::2], turned[..., 1::2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    return torch.cat([y.to(x.dtype), rest], dim=-1)


def _free(c, seqs, keep):
    at = seqs.long()
    n = c["lengths"][at]
    keep = torch.zeros_like(n) if keep is None else torch.minimum(keep, n)
    col = torch.arange(c["table"].shape[1], device=n.device)[None]
    gone = (col >= ((keep + PAGE - 1) // PAGE)[:, None]) & (col < ((n + PAGE - 1) // PAGE)[:, None])
    c["refs"].index_add_(0, c["table"][at].flatten().long() * gone.flatten(), -gone.flatten().int())
    c["lengths"][at] = keep


def _fork(c, src, dst):
    src, dst = src.long(), dst.long()
    n = c["lengths"][src]
    col = torch.arange(c["table"].shape[1], device=n.device)[None]
    held = col < ((n + PAGE - 1) // PAGE)[:, None]
    pages = c["table"][src]
    c["refs"].index_add_(0, pages.flatten().long() * held.flatten(), held.flatten().int())
    c["table"][dst] = torch.where(held, pages, c["table"][dst])
    c["lengths"][dst] = n


def _exponent(amax):
    """The least e with amax <= 448 2^e."""
    m, e = torch.frexp(amax)                      # amax = m 2^e, m in [1/2, 1): 448 2^k is 0.875 2^(k + 9)
    e = e - 9 + (m > 0.875).int()
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)


def _codes(x, e):
    return torch.ldexp(x, -e).clamp(-448, 448).to(torch.float8_e4m3fn)


def _append(c, seqs, k, v, counts):
    B, T, H, d = k.shape
    dev, at = k.device, seqs.long()
    old = c["lengths"][at].long()
    n = torch.full_like(old, T) if counts is None else counts.long()
    # pages: those that the new tokens begin, and a copy of a last page that others hold too
    first = (old + PAGE - 1) // PAGE
    tail = c["table"][at, (old // PAGE).clamp(max=c["table"].shape[1] - 1)].long()
    copied = (old % PAGE > 0) & (n > 0) & (c["refs"][tail] > 1)
    need = (old + n + PAGE - 1) // PAGE - first + copied
    lowest = torch.argsort(c["refs"] > 0, stable=True)            # free pages, the lowest first
    begin = torch.cumsum(need, 0) - need
    j = torch.arange(int(_ceil(T, PAGE)) + 2, device=dev)[None]
    new = j < need[:, None]
    row = torch.arange(B, device=dev)[:, None].expand_as(new)[new]
    page = lowest[(begin[:, None] + j)[new]]
    c["table"][at[row], ((old // PAGE)[:, None] + (first - old // PAGE - copied.long())[:, None] + j)[new]] = page.int()
    c["refs"][page] = 1
    c["refs"].index_add_(0, tail, -copied.int())
    own_tail = c["table"][at, (old // PAGE).clamp(max=c["table"].shape[1] - 1)].long()
    who = copied.nonzero()[:, 0]
    for name in ("k", "v", "scales"):
        c[name][own_tail[who]] = c[name][tail[who]]
    # the tokens in blocks of 16, from the block that holds the first one
    t = torch.arange(T, device=dev)[None]
    p = old[:, None] + t
    live = t < n[:, None]
    row = torch.arange(B, device=dev)[:, None].expand_as(p)[live]
    p, slot = p[live], (p - (old // BLOCK * BLOCK)[:, None])[live]
    nb = _ceil(T + BLOCK - 1, BLOCK)
    page = c["table"][at[row], p // PAGE].long()
    for which, (name, x) in enumerate((("k", k), ("v", v))):
        x = x.float()
        blocks = torch.zeros(B, nb * BLOCK, H, d, device=dev)
        blocks[row, slot] = x[live]
        e = _exponent(blocks.abs().view(B, nb, BLOCK, H, d).amax(dim=(2, 4)))              # [B][nb][H]
        # the block that was begun before: its scale only grows, and what it held is rounded to the new one
        started = (old % BLOCK > 0) & (n > 0)
        ob, who = (old // BLOCK % (PAGE // BLOCK)), started.nonzero()[:, 0]
        op = own_tail[who]
        had = c["scales"][op, :, which, ob[who]].int() - 127                                # [started][H]
        grown = torch.maximum(e[who, 0], had)
        e[who, 0] = grown
        at16 = ob[who][:, None] * BLOCK + torch.arange(BLOCK, device=dev)[None]
        seen = torch.arange(BLOCK, device=dev)[None] < (old % BLOCK)[who][:, None]
        r, q = seen.nonzero(as_tuple=True)
        if name == "k":
            held = c["k"][op[r], :, at16[r, q], :].view(torch.float8_e4m3fn).float()       # [tokens][H][d]
        else:
            held = c["v"][op[r], :, :, at16[r, q]].view(torch.float8_e4m3fn).float()
        held = _codes(held, (grown - had)[r][:, :, None]).view(torch.uint8)
        codes = _codes(x[live], e[row, slot // BLOCK][:, :, None]).view(torch.uint8)
        if name == "k":
            c["k"][op[r], :, at16[r, q], :] = held
            c["k"][page, :, p % PAGE, :] = codes
        else:
            c["v"][op[r], :, :, at16[r, q]] = held
            c["v"][page, :, :, p % PAGE] = codes
        c["scales"][page, :, which, p % PAGE // BLOCK] = (e[row, slot // BLOCK] + 127).to(torch.uint8)
    c["lengths"][at] = (old + n).int()


def _scaled(c, name, pages):
    """Codes of `pages` [..] times their blocks' scales, 32 bits: [..][H][64][d], or [..][H][d][64] for v."""
    x = c[name][pages].view(torch.float8_e4m3fn).float()
    e = c["scales"][pages][..., 0 if name == "k" else 1, :].int() - 127
    s = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e).repeat_interleave(BLOCK, dim=-1)
    return x * (s[..., :, None] if name == "k" else s[..., None, :])


def _visible(length, count, queries, keys, window, sink):
    """[B][queries][keys]: which key each query sees; query i of `count` stands at length - count + i."""
    dev = length.device
    pos = (length - count)[:, None] + torch.arange(queries, device=dev)[None]
    j = torch.arange(keys, device=dev)
    see = j <= pos[..., None]
    if window:
        see &= (j > pos[..., None] - window) | (j < sink)
    return see


def _attend(c, seqs, q, counts, window, sink, out):
    B, T, Hq, d = q.shape
    H = c["k"].shape[1]
    at = seqs.long()
    length = c["lengths"][at].long()
    count = torch.full_like(length, T) if counts is None else counts.long()
    pages = c["table"][at].long()                                 # [B][P], the longest sequence's
    L = pages.shape[1] * PAGE
    k = _scaled(c, "k", pages).transpose(1, 2).reshape(B, H, L, d)
    x = q.float().view(B, T, H, Hq // H, d).permute(0, 2, 3, 1, 4).reshape(B, H, -1, d) / math.sqrt(d)
    score = torch.matmul(x, k.transpose(-1, -2)).view(B, H, Hq // H, T, L)
    del k
    see = _visible(length, count, T, L, window, sink)[:, None, None]
    score = torch.where(see, score, torch.full_like(score[:1, :1, :1, :1, :1], -math.inf))
    top = score.amax(dim=-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    del score
    total = p.sum(dim=-1, keepdim=True)
    v = _scaled(c, "v", pages).permute(0, 2, 1, 4, 3).reshape(B, H, L, d)
    v = torch.where(torch.arange(L, device=v.device)[None, None, :, None] < length[:, None, None, None], v, torch.zeros_like(v[:1, :1, :1, :1]))
    y = torch.matmul(p.view(B, H, -1, L), v).view(B, H, Hq // H, T, d) / torch.where(total > 0, total, torch.ones_like(total))
    y = y.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, d).to(q.dtype)
    live = (torch.arange(T, device=q.device)[None] < count[:, None])[:, :, None, None]
    out.copy_(torch.where(live, y, out))                          # rows behind a sequence's count stay
    return out


def _compact(c):
    used = c["refs"] > 0
    page = torch.arange(used.numel(), device=used.device)
    n = used.sum()
    src, dst = (used & (page >= n)).nonzero()[:, 0], (~used & (page < n)).nonzero()[:, 0]
    for name in ("k", "v", "scales", "refs"):
        c[name][dst] = c[name][src]
    c["refs"][src] = 0
    page[src] = dst
    col = torch.arange(c["table"].shape[1], device=used.device)[None]
    held = col < ((c["lengths"] + PAGE - 1) // PAGE)[:, None]
    c["table"].copy_(torch.where(held, page[c["table"].long() * held].int(), c["table"]))


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    op, d = case["op"], case["dim"]
    size = 2 if case.get("dtype") == "bf16" else 4
    if op == "rotary":
        n = case["batch"] * case["tokens"] * case["heads"]
        return {"bytes": 2.0 * n * d * size + 4 * case["batch"] * case["tokens"], "flops": 3.0 * n * case["rot"]}
    kv = case["kv_heads"]
    token = kv * d * 2                                            # bytes of a token's codes
    if op == "append":
        n = sum(_counts(case))
        return {"bytes": float(n * token * (size + 1) + n * kv * 2 / 16 + 8 * case["batch"]), "flops": 3.0 * n * token}
    if op == "attend":
        pairs = held = 0
        for n, t in zip(_spread(case["least"], case["most"], case["batch"]), _counts(case)):
            pos = np.arange(max(0, n - t), n, dtype=np.int64)
            lo = np.maximum(0, pos - case["window"] + 1) if case["window"] else np.zeros_like(pos)
            pairs += int((pos - lo + 1).sum() + np.minimum(lo, case["sink"]).sum())
            if pos.size:
                held += int(n - lo[0] + min(int(lo[0]), case["sink"]))
        rows = sum(_counts(case)) * case["heads"]
        return {"bytes": float(held * token * (1 + 1 / (16 * d)) + 2 * rows * d * size), "flops": 4.0 * pairs * case["heads"] * d}
    if op == "fork":
        n = case["children"] * case["parents"]
        lengths = _spread(case["least"], case["most"], case["parents"])
        tails = sum(x % PAGE for x in lengths) * case["children"]
        shared = sum(_ceil(x, PAGE) for x in lengths) * case["children"]
        return {"bytes": float(tails * token * 2 + n * token * (size + 1) + shared * 8), "flops": 3.0 * n * token}
    pages = [_ceil(x, PAGE) for x in _spread(case["least"], case["most"], case["seqs"])]
    total, gone = sum(pages), sum(pages) / case["every"]
    moved = gone * (total - gone) / total                         # holes among the pages that stay low, on average
    return {"bytes": float(2 * moved * PAGE * token + 8 * total), "flops": 0.0}


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))


def _exact_rotary(s):
    case = s["case"]
    x = s["x"].double()
    pos = s["positions"].double()
    pos = pos[:, None] if pos.dim() == 1 else pos
    r, h = case["rot"], case["rot"] // 2
    turn = torch.polar(torch.full((), s["scale"], dtype=torch.float64, device="cuda").expand(*pos.shape, h),
                       pos[..., None] * s["freq"])[:, :, None]
    if case["back"]:
        turn = turn.conj()
    y = x.clone()
    i = torch.arange(h, device="cuda")
    a, b = (i, i + h) if case["layout"] == "half" else (2 * i, 2 * i + 1)
    z = torch.complex(x[..., a], x[..., b]) * turn
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_attend(s):
    case, c = s["case"], s["c"]
    B, T, Hq, d = s["q"].shape
    H = case["kv_heads"]
    if B * case["most"] * H * d > 1 << 31 or B * T * case["most"] * Hq * d > 1 << 42:
        return None
    y = torch.zeros(B, T, Hq, d, dtype=torch.float64, device="cuda")
    for b, (n, t) in enumerate(zip(c["lengths"][:B].tolist(), _counts(case))):
        t0 = max(0, t - n)                                        # rows before the sequence's start see nothing
        j = torch.arange(n, device="cuda")
        page = c["table"][b].long()[j // PAGE]
        i = torch.arange(t0, t, device="cuda")[:, None] + n - t
        see = j <= i
        if case["window"]:
            see = see & ((i - j < case["window"]) | (j < case["sink"]))
        for h in range(H):
            two = lambda w: 2.0 ** (c["scales"][page, h, w, j % PAGE // BLOCK].double() - 127)[:, None]  # noqa: E731
            k = c["k"][page, h, j % PAGE].view(torch.float8_e4m3fn).double() * two(0)
            v = c["v"][page, h, :, j % PAGE].view(torch.float8_e4m3fn).double() * two(1)
            for g in range(h * (Hq // H), (h + 1) * (Hq // H)):
                p = torch.softmax((s["q"][b, t0:t, g].double() @ k.T / math.sqrt(d)).masked_fill(~see, -math.inf), dim=-1)
                y[b, t0:t, g] = p @ v
    return y


def _exact_append(s):
    """The pool after the call, unrounded: values over their blocks' scales.  Pages go out the lowest first; a begun block's
    scale only grows, and what it held counts in the new one."""
    case, c = s["case"], s["c"]
    B, kv = case["batch"], case["kv_heads"]
    counts = s["counts"].tolist() if s["counts"] is not None else [case["tokens"]] * B
    if sum(counts) * kv > 1 << 20:
        return None
    keep = s["keep"].tolist()
    table, lengths, refs = (c[n].cpu().numpy() for n in ("table", "lengths", "refs"))
    for b in range(B):
        refs[table[b, _ceil(keep[b], PAGE):_ceil(int(lengths[b]), PAGE)]] -= 1
    free = iter(np.flatnonzero(refs == 0).tolist())
    for b in range(B):
        for i in range(_ceil(keep[b], PAGE), _ceil(keep[b] + counts[b], PAGE)):
            table[b, i] = next(free)
    x, scales, out = s["kv"].double().cpu().numpy(), c["scales"].cpu().numpy().astype(np.int64) - 127, {}
    for w, name in enumerate(("k", "v")):
        y = c[name].view(torch.float8_e4m3fn).double().cpu().numpy()
        y = y if name == "k" else y.swapaxes(2, 3)
        for b in range(B):
            t = 0
            while t < counts[b]:
                at = keep[b] + t
                page, o, i = table[b, at // PAGE], at % PAGE, at % BLOCK
                block = x[b, t:min(t + BLOCK - i, counts[b]), w * kv:(w + 1) * kv]
                e = np.clip(np.ceil(np.log2(np.maximum(np.abs(block).max(axis=(0, 2)), 1e-300) / 448)), E_MIN, E_MAX)
                if i:
                    had = scales[page, :, w, o // BLOCK]
                    e = np.maximum(e, had)
                    y[page, :, o - i:o] *= 2.0 ** (had - e)[:, None, None]
                y[page, :, o:o + len(block)] = (block / 2.0 ** e[None, :, None]).swapaxes(0, 1)
                scales[page, :, w, o // BLOCK] = e
                t += len(block)
        out[name] = torch.from_numpy(np.ascontiguousarray(y if name == "k" else y.swapaxes(2, 3)))
    return out | {"scales": None, "lengths": None, "refs": None, "table": None}


# forks and moved pages hold copies of codes: whole values, compared as they are
_EXACT = {"rotary": _exact_rotary, "append": _exact_append, "attend": _exact_attend, "fork": lambda s: None, "compact": lambda s: None}
