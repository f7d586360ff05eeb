"""The operators of a layer beside the memory: what is measured, and their plain forms.

Three kinds of calls stand here, those that a layer makes between its input and its mixing of tokens: the norms of
queries and keys for each head with the rotary positions in the same pass (``HeadNorm``), linear attention with a decay
(``LinearAttention``: prompts, single tokens and the gradients of both), and products with weights held in 8-bit
integers (``Int8Linear``).  The plain forms are elementary torch operations.
"""
import math

import torch

own = False

CHUNK = 64                    # tokens of a chunk of the plain form of linear attention
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------------------
# the cases

def norm(name, batch, tokens, heads, kv_heads, dim, rot, layout, back, dtype, far):
    return {"name": name, "op": "norm", "batch": batch, "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "rot": rot, "layout": layout, "back": back, "dtype": dtype, "far": far}


def linear(name, batch, tokens, ragged, heads, kv_heads, key, value, gates, back, dtype):
    return {"name": name, "op": "linear", "batch": batch, "tokens": tokens, "ragged": ragged, "heads": heads,
            "kv_heads": kv_heads, "key": key, "value": value, "gates": gates, "back": back, "dtype": dtype}


def int8(name, rows, cols, outs, dtype):
    return {"name": name, "op": "int8", "rows": rows, "cols": cols, "outs": outs, "dtype": dtype}


def listed():
    return [
        # one new token of each of 4 sequences, its queries and keys together: a step's latency
        norm("norm_step", 4, 1, 6, 2, 64, 64, "half", False, "bf16", 4000),
        # two long prompts, 32 query and 8 key heads
        norm("norm_prompt", 2, 8192, 32, 8, 128, 128, "interleaved", False, "bf16", 1000000),
        # a training step's gradients of the projections and of both norms' weights, rotary on part of the head
        norm("norm_gradient", 4, 2047, 16, 4, 96, 64, "half", True, "bf16", 60000),
        # the smallest call: a draft of five tokens of two sequences, in 32 bits, a fixed decay for each head
        linear("linear_draft", 2, 5, False, 6, 2, 64, 64, False, False, "f32"),
        # a serving batch's single tokens, with the decay that each token's gate gives
        linear("linear_step", 48, 1, False, 16, 16, 128, 128, True, False, "bf16"),
        # one long prompt of few heads: the sequence itself has to fill the card
        linear("linear_prompt", 1, 32768, False, 8, 8, 128, 128, True, False, "bf16"),
        # prompts of ragged lengths, queries in groups, keys and values of other widths, in 32 bits
        linear("linear_ragged", 8, 2001, True, 12, 4, 64, 96, False, False, "f32"),
        # a training step's gradients, those of the gates and of the state that came in among them
        linear("linear_gradient", 2, 4096, False, 16, 16, 128, 128, True, True, "bf16"),
        # the same for a small layer in 32 bits with a learnt decay for each head, a ragged batch
        linear("linear_gradient_small", 3, 333, True, 4, 2, 64, 32, False, True, "f32"),
        # a decode step's projection of 8 tokens: the weights have to be read
        int8("int8_step", 8, 4096, 6144, "bf16"),
        # the projection of prompts' tokens
        int8("int8_prompt", 8192, 4096, 6144, "bf16"),
        # sizes that no tile divides, in 32 bits
        int8("int8_odd", 777, 1000, 1537, "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "linear", "linear", "linear", "int8", "int8"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        dim, kv = 2 * rng.randint(16, 128), rng.randint(0, 8)
        heads, batch = rng.randint(1, 40), _log(rng, 1, 32)
        rot = rng.choice([dim, dim, 0, 2 * rng.randint(1, dim // 2)])
        most = max(1, 2 * 8192 * 40 * 128 // (2 * batch * (heads + kv) * dim))
        return norm("", batch, _log(rng, 1, min(8192, most)), heads, kv, dim, rot, rng.choice(["half", "interleaved"]),
                    rng.random() < 0.4, dtype, _log(rng, 1000, 2000000))
    if op == "linear":
        kv, group = rng.randint(1, 16), rng.choice([1, 1, 2, 3, 4])
        key, value = 8 * rng.randint(2, 32), 8 * rng.randint(2, 32)
        gates, back = rng.random() < 0.5, rng.random() < 0.4
        room = 2 * 4096 * 16 * 128 * 128 // (group * kv * key * value * (2 if dtype == "f32" else 1) * (2 if back else 1))
        if not back and rng.random() < 0.4:   # single tokens and short drafts
            return linear("", min(_log(rng, 1, 128), max(1, room // 8)), rng.randint(1, 8), rng.random() < 0.3, kv * group, kv,
                          key, value, gates, False, dtype)
        batch = min(_log(rng, 1, 16), max(1, room // 16))
        return linear("", batch, _log(rng, 2, max(2, min(16384, room // batch))), rng.random() < 0.5, kv * group, kv, key, value,
                      gates, back, dtype)
    cols, outs = _log(rng, 16, 8192), _log(rng, 1, 8192)
    most = 8192 * 4096 * 6144 // (2 * cols * outs)
    return int8("", _log(rng, 1, max(1, min(16384, most, 2 ** 27 // cols, 2 ** 27 // outs))), cols, outs, dtype)


# ---------------------------------------------------------------------------
# a case's inputs

def _counts(case):
    n, b = case["tokens"], case["batch"]
    return [n - n * i // (2 * b) for i in range(b)] if case["ragged"] else [n] * b


def _frequencies(rot):
    return 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / max(1, rot))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = TYPES[case["dtype"]]
    rand = lambda *n: torch.randn(*n, generator=g, device="cuda")  # noqa: E731
    s = dict(case)
    if own:
        import test_trained_neural_amd as T
    if case["op"] == "norm":
        B, N, H, d = case["batch"], case["tokens"], case["heads"] + case["kv_heads"], case["dim"]
        # the projections' output: queries, keys and as many values in one tensor, channels of unequal size
        qkv = (rand(B, N, H + case["kv_heads"], d) * (0.5 + rand(H + case["kv_heads"], d).abs())).to(dt)
        s["x"] = qkv[:, :, :H]
        s["w_q"] = 1 + 0.1 * rand(d)
        s["w_k"] = 1 + 0.1 * rand(d) if case["kv_heads"] else None
        s["positions"] = torch.randint(0, case["far"], (B, N), generator=g, device="cuda", dtype=torch.int32)
        s["freq"] = _frequencies(case["rot"])
        if case["back"]:
            s["dy"] = rand(B, N, H, d).to(dt)
        if own:
            rotary = T.Rotary(case["rot"], layout=T.TM_ROPE_HALF if case["layout"] == "half" else T.TM_ROPE_INTERLEAVED) \
                if case["rot"] else None
            s["norm"] = T.HeadNorm(case["heads"], case["kv_heads"], s["w_q"], s["w_k"], eps=EPS, rotary=rotary)
        return s
    if case["op"] == "linear":
        B, N, H, K, dk, dv = (case[n] for n in ("batch", "tokens", "heads", "kv_heads", "key", "value"))
        s["q"], s["k"] = (torch.nn.functional.normalize(rand(B, N, h, dk), dim=-1).mul_(dk ** 0.25).to(dt) for h in (H, K))
        s["v"], s["state"] = rand(B, N, K, dv).to(dt), rand(B, K, dk, dv)
        if case["gates"]:   # a forgetting gate for each token; a document that begins drops what came before
            alpha = torch.sigmoid(rand(B, N, K) - 3 * torch.rand(K, generator=g, device="cuda"))
            begins = torch.rand(B, N, 1, generator=g, device="cuda") < 1 / 1500
            s["log_decay"] = torch.where(begins, -math.inf, torch.log1p(-alpha))
        else:               # what a head keeps of a token's past: from 1 - 2^-3 to 1 - 2^-9
            s["log_decay"] = torch.log1p(-torch.exp2(-3 - 6 * torch.rand(K, generator=g, device="cuda")))
        s["counts"] = torch.tensor(_counts(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
        s["scale"] = dk ** -0.5
        if case["back"]:
            s["dy"], s["dstate"] = rand(B, N, H, dv).to(dt), rand(B, K, dk, dv)
        if own:
            s["attention"] = T.LinearAttention(K, dk, dv)
        return s
    M, K, N = case["rows"], case["cols"], case["outs"]
    # model vectors with a few channels larger than the others; weights as an initialised layer has them
    s["x"] = (rand(M, K) * torch.exp(0.5 * rand(K))).to(dt)
    w = rand(N, K) / math.sqrt(K)
    top = w.abs().amax(1, keepdim=True)
    wide = -(-K // 16) * 16
    s["codes"] = torch.zeros(N, wide, dtype=torch.int8, device="cuda")
    s["codes"][:, :K] = torch.round(127 * w / top).to(torch.int8)
    s["scales"] = top[:, 0] / 127
    if own:
        s["product"] = T.Int8Linear(codes=s["codes"], scales=s["scales"], cols=K)
    return s


# ---------------------------------------------------------------------------
# the operators, plainly

def _turn(s, x, back):
    """x rotated by its tokens' angles (back: by the negative ones)."""
    r, half = s["rot"], s["layout"] == "half"
    if not r:
        return x
    angle = s["positions"].double()[:, :, None, None] * s["freq"]
    c, n = torch.cos(angle).float(), torch.sin(angle).float()
    n = -n if back else n
    a, b = (x[..., :r // 2], x[..., r // 2:r]) if half else (x[..., 0:r:2], x[..., 1:r:2])
    u, w = a * c - b * n, a * n + b * c
    turned = torch.cat((u, w), -1) if half else torch.stack((u, w), -1).flatten(-2)
    return torch.cat((turned, x[..., r:]), -1)


def _weights(s):
    H, K = s["heads"], s["kv_heads"]
    return s["w_q"].expand(H, -1) if not K else torch.cat((s["w_q"].expand(H, -1), s["w_k"].expand(K, -1)))


def _norm(s):
    x = s["x"].float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * _weights(s)
    return _turn(s, y, False).to(s["x"].dtype)


def _norm_back(s):
    x, w, H = s["x"].float(), _weights(s), s["heads"]
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    dn, unit = _turn(s, s["dy"].float(), True), x * r
    dw = (dn * unit).sum((0, 1))
    dn = dn * w
    dx = r * (dn - unit * (dn * unit).mean(-1, keepdim=True))
    return [dx.to(s["x"].dtype), dw[:H].sum(0), dw[H:].sum(0) if s["kv_heads"] else None]


def _chunks(x, kv_heads):
    """[B][T][heads][d] as [B][kv_heads][heads of the group][chunk][CHUNK][d] in 32 bits, zeros behind the last token."""
    B, N, H, d = x.shape
    x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, -N % CHUNK))
    return x.view(B, -1, CHUNK, kv_heads, H // kv_heads, d).permute(0, 3, 4, 1, 2, 5)


def _tokens(x, n):
    """Back to [B][n][heads][d]."""
    B, K, G, C, _, d = x.shape
    return x.permute(0, 3, 4, 1, 2, 5).reshape(B, C * CHUNK, K * G, d)[:, :n]


def _linear_parts(s):
    """What forward and backward share: the chunks, with nothing in them behind an entry's count, and their decays.  The
    logarithms are summed in 64 bits; -inf as -1000, whose exponential is zero too."""
    B, N, K = s["batch"], s["tokens"], s["kv_heads"]
    on = torch.arange(N, device="cuda") < s["counts"][:, None] if s["ragged"] else torch.ones(B, N, dtype=torch.bool, device="cuda")
    there = on[:, :, None, None]
    q, k, v = (_chunks(torch.where(there, s[n], 0), K) for n in "qkv")
    g = s["log_decay"].expand(B, N, K).double().clamp(min=-1000.0)
    g = _chunks64(torch.where(on[:, :, None], g, 0.0))                                # [B][K][C][CHUNK]
    inner = g.cumsum(-1)
    ends = inner[..., -1].cumsum(-1)                                                  # over all tokens up to a chunk's end
    causal = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device="cuda").tril()
    decay = torch.where(causal, (inner[..., :, None] - inner[..., None, :]).clamp(max=0.0).exp(), 0.0).float()[:, :, None]
    head = inner.exp().float()[:, :, None, :, :, None]                                # of what stood before the chunk
    tail = (inner[..., -1:] - inner).exp().float()[:, :, None, :, :, None]            # of a token by the chunk's end
    border = torch.nn.functional.pad(ends, (1, 0))                                    # [B][K][C + 1]
    below = torch.ones(border.shape[-1], border.shape[-1], dtype=torch.bool, device="cuda").tril()
    carry = torch.where(below, (border[..., :, None] - border[..., None, :]).clamp(max=0.0).exp(), 0.0).float()  # from border c' to c
    return q, k, v, there, decay, head, tail, carry


def _chunks64(g):
    B, N, K = g.shape
    return torch.nn.functional.pad(g, (0, 0, 0, -N % CHUNK)).view(B, -1, CHUNK, K).permute(0, 3, 1, 2)


def _states(s, k, v, tail, carry):
    """The state at every border between chunks: [B][K][C + 1][key][value]."""
    own_part = ((k * tail).transpose(-1, -2) @ v)[:, :, 0]
    parts = torch.cat((s["state"][:, :, None], own_part), 2)
    return (carry @ parts.flatten(3)).view(parts.shape)


def _linear(s):
    q, k, v, there, decay, head, tail, carry = _linear_parts(s)
    S = _states(s, k, v, tail, carry)
    y = (q @ k.transpose(-1, -2) * decay) @ v + head * (q @ S[:, :, None, :-1])
    y = torch.where(there, _tokens(y * s["scale"], s["tokens"]), 0.0)
    return [y.to(s["q"].dtype), S[:, :, -1]]


def _linear_back(s):
    q, k, v, there, decay, head, tail, carry = _linear_parts(s)
    K, n, dt = s["kv_heads"], s["tokens"], s["q"].dtype
    S = _states(s, k, v, tail, carry)
    dy = _chunks(torch.where(there, s["dy"], 0), K) * s["scale"]
    part = ((q * head).transpose(-1, -2) @ dy).sum(2)
    parts = torch.cat((part, s["dstate"][:, :, None]), 2)
    R = (carry.transpose(-1, -2) @ parts.flatten(3)).view(parts.shape)   # gradient of the state at every border
    scores, pull = q @ k.transpose(-1, -2), dy @ v.transpose(-1, -2) * decay
    far_q = head * (dy @ S[:, :, None, :-1].transpose(-1, -2))
    far_k = tail * (v @ R[:, :, None, 1:].transpose(-1, -2))
    dq = pull @ k + far_q
    dk = (pull.transpose(-1, -2) @ q).sum(2, keepdim=True) + far_k
    dv = ((scores * decay).transpose(-1, -2) @ dy).sum(2, keepdim=True) + tail * (k @ R[:, :, None, 1:])
    # of the decays: every pair of tokens on either side of one, and the states' own part at a chunk's end
    pairs = (scores * pull).tril(-1)
    here = (pairs.sum(-1) - pairs.sum(-2) + (q * far_q).sum(-1)).sum(2) - (k * far_k).sum(-1)[:, :, 0]
    flow = (S[:, :, 1:] * R[:, :, 1:]).sum((-1, -2))
    dg = here.flip(-1).cumsum(-1).flip(-1) + flow[..., None]             # [B][K][C][CHUNK]
    dg = torch.where(there[..., 0], dg.flatten(2).transpose(1, 2)[:, :n], 0.0)
    if not s["gates"]:
        dg = dg.sum((0, 1))
    dq, dk, dv = (torch.where(there, _tokens(x, n), 0.0).to(dt) for x in (dq, dk, dv))
    return [dq, dk, dv, dg, R[:, :, 0]]


def _int8(s):
    x, K = s["x"].float(), s["cols"]
    top = x.abs().amax(1, keepdim=True)
    codes = torch.where(top > 0, torch.round(127 * x / top), 0.0)
    return ((codes @ s["codes"][:, :K].float().t()) * (top / 127) * s["scales"]).to(s["x"].dtype)


# ---------------------------------------------------------------------------

def run(s):
    if own:
        if s["op"] == "norm":
            if s["back"]:
                return list(s["norm"].backward(s["x"], s["dy"], s["positions"]))
            return s["norm"](s["x"], s["positions"])
        if s["op"] == "linear":
            if s["back"]:
                return list(s["attention"].backward(s["q"], s["k"], s["v"], s["log_decay"], s["dy"], state=s["state"],
                                                    dstate=s["dstate"], counts=s["counts"], scale=s["scale"]))
            return list(s["attention"](s["q"], s["k"], s["v"], s["log_decay"], state=s["state"], counts=s["counts"],
                                       scale=s["scale"]))
        return s["product"](s["x"])
    if s["op"] == "norm":
        return _norm_back(s) if s["back"] else _norm(s)
    if s["op"] == "linear":
        return _linear_back(s) if s["back"] else _linear(s)
    return _int8(s)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        n = case["batch"] * case["tokens"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": (3 if case["back"] else 2) * n * e + 4 * case["batch"] * case["tokens"], "flops": (16 if case["back"] else 8) * n}
    if case["op"] == "linear":
        H, K, dk, dv = (case[n] for n in ("heads", "kv_heads", "key", "value"))
        n, back = sum(_counts(case)), case["back"]
        tokens = (H * dk + K * dk + K * dv) * (2 if back else 1) + H * dv
        gates = n * K * 4 * (2 if back else 1) if case["gates"] else 0
        # a token's own part: one product with the state for each query head, one into it for each key head
        return {"bytes": n * tokens * e + gates + (3 if back else 2) * 4 * case["batch"] * K * dk * dv,
                "flops": n * (H + K) * 2 * dk * dv * (3 if back else 1)}
    M, K, N = case["rows"], case["cols"], case["outs"]
    return {"bytes": M * K * e + N * K + 4 * N + M * N * e, "flops": 2 * M * N * K}


# ---------------------------------------------------------------------------
# what the definitions give in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _norm_exact(s)
    if case["op"] == "linear":
        return _linear_exact(s)
    x, K = s["x"].double(), s["cols"]
    step = x.abs().max(1, keepdim=True).values / 127
    levels = torch.round(x * 127 / (step * 127).clamp(min=1e-300))
    return (levels * step) @ (s["codes"][:, :K].double() * s["scales"].double()[:, None]).t()


def _norm_exact(s):
    """The norm and the rotation as a function of x, and its gradients by the chain rule of torch's own record in 64 bits."""
    x = s["x"].double().requires_grad_(s["back"])
    w_q = s["w_q"].double().requires_grad_(s["back"])
    w_k = s["w_k"].double().requires_grad_(s["back"]) if s["kv_heads"] else None
    H, r = s["heads"], s["rot"]
    z = x / (x.pow(2).sum(-1, keepdim=True) / s["dim"] + EPS).sqrt()
    z = z * w_q if w_k is None else torch.cat((z[:, :, :H] * w_q, z[:, :, H:] * w_k), 2)
    if r:
        lo = torch.arange(r // 2, device="cuda") if s["layout"] == "half" else torch.arange(0, r, 2, device="cuda")
        hi = lo + (r // 2 if s["layout"] == "half" else 1)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["positions"].double()[..., None] * s["freq"])[:, :, None]
        t = torch.complex(z[..., lo], z[..., hi]) * turn
        y = z.clone()
        y[..., lo], y[..., hi] = t.real, t.imag
        z = y
    if not s["back"]:
        return z
    got = torch.autograd.grad(z, [x, w_q] + ([w_k] if w_k is not None else []), s["dy"].double())
    return [got[0], got[1], got[2] if w_k is not None else None]


def _linear_exact(s):
    """Token by token: S = decay S + k v', y = scale q S; backwards the same way with every state kept."""
    B, N, H, K, dk, dv = (s[n] for n in ("batch", "tokens", "heads", "kv_heads", "key", "value"))
    G = H // K
    q, k, v = s["q"].double().view(B, N, K, G, dk), s["k"].double(), s["v"].double()
    keep = torch.exp(s["log_decay"].double()).expand(B, N, K)
    n = _counts(case=s)
    live = [torch.tensor([float(t < c) for c in n], dtype=torch.float64, device="cuda")[:, None, None, None] if t >= min(n) else None
            for t in range(N)]
    S = s["state"].double()
    kept = torch.empty(N + 1, B, K, dk, dv, dtype=torch.float64, device="cuda") if s["back"] else None
    if s["back"]:
        kept[0] = S
    y = torch.zeros(B, N, K, G, dv, dtype=torch.float64, device="cuda")
    for t in range(N):
        new = keep[:, t, :, None, None] * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        S = new if live[t] is None else torch.where(live[t] > 0, new, S)
        if s["back"]:
            kept[t + 1] = S
        else:
            row = s["scale"] * (q[:, t] @ S)
            y[:, t] = row if live[t] is None else row * live[t]
    if not s["back"]:
        return [y.view(B, N, H, dv), S]
    dy = s["dy"].double().view(B, N, K, G, dv) * s["scale"]
    dq, dk_, dv_ = (torch.zeros_like(x) for x in (q, k, v))
    dg = torch.zeros(B, N, K, dtype=torch.float64, device="cuda")
    R = s["dstate"].double()
    for t in range(N - 1, -1, -1):
        more = R + q[:, t].transpose(-1, -2) @ dy[:, t]
        before = keep[:, t, :, None, None] * more
        parts = (dy[:, t] @ kept[t + 1].transpose(-1, -2), (more * v[:, t, :, None, :]).sum(-1), (more * k[:, t, :, :, None]).sum(-2),
                 (before * kept[t]).sum((-1, -2)))
        if live[t] is not None:
            before = torch.where(live[t] > 0, before, R)
            parts = (parts[0] * live[t], parts[1] * live[t][..., 0], parts[2] * live[t][..., 0], parts[3] * live[t][..., 0, 0])
        dq[:, t], dk_[:, t], dv_[:, t], dg[:, t] = parts
        R = before
    return [dq.view(B, N, H, dk), dk_, dv_, dg if s["gates"] else dg.sum((0, 1)), R]
