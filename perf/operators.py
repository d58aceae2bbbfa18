"""The gated delta rule's operators, as measured cases: inputs, plain forms, float64 definitions.

Four operators of one mixer:

  scan   the gated delta rule over prompts, dense [b, L, ..] or packed
  step   one decode token per sequence against a cache of states
  norm   the RMS norm of every head's output, then the gate
  conv   the causal depthwise convolution in front, over packed sequences

The recurrence, per sequence and value head (key head = head // (heads / key_heads)):

  a_t = exp(softplus(dt_t + dt_bias) A),  b_t = sigmoid(beta_t),  q, k L2-normalised per head
  u_t = b_t (v_t - a_t S_{t-1}^T k_t),  S_t = a_t S_{t-1} + k_t u_t^T,  y_t = scale S_t^T q_t
"""
import math

import torch

own = False

CHUNK = 64
L2_EPS = 1e-6
NORM_EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases

def _scan(name, n, length, key_heads, heads, k, v, io="bf16", packed=False, h0=False):
    return {"name": name, "op": "scan", "n": n, "length": length, "key_heads": key_heads,
            "heads": heads, "k": k, "v": v, "io": io, "packed": packed, "h0": h0}


def _step(name, n, key_heads, heads, k, v, io="bf16", pad=0):
    return {"name": name, "op": "step", "n": n, "key_heads": key_heads, "heads": heads,
            "k": k, "v": v, "io": io, "pad": pad}


def listed():
    return [
        # a batch of equal prompts from the start of the sequence: the throughput case
        _scan("scan b8 L2048", 8, 2048, 16, 32, 128, 128),
        # one long prompt, its state carried in from an earlier part of it
        _scan("scan b1 L8192", 1, 8192, 16, 32, 128, 128, h0=True),
        # a server's prompts of different lengths in one buffer, into a cache of states
        _scan("scan packed 24", 24, 1301, 8, 16, 128, 128, packed=True, h0=True),
        # a small model's odd-length prompts: 64-wide values, three value heads to a key head
        _scan("scan b2 L777 h6", 2, 777, 2, 6, 128, 64, h0=True),
        # float32 tensors, as a numerics check of a model runs them
        _scan("scan f32 L500", 2, 500, 4, 8, 64, 64, io="f32"),
        # one sequence decoding: latency
        _step("step b1", 1, 16, 32, 128, 128),
        # a serving batch, padded to a captured size, states anywhere in the cache
        _step("step b250+6", 256, 16, 32, 128, 128, pad=6),
        _step("step f32 b33", 33, 8, 8, 64, 96, io="f32"),
        # the norm of a decode batch and of a prompt batch
        {"name": "norm decode", "op": "norm", "tokens": 256, "heads": 32, "width": 128, "io": "bf16"},
        {"name": "norm prompt", "op": "norm", "tokens": 16384, "heads": 32, "width": 128, "io": "bf16"},
        # the convolution of a decode batch (sequences of one token) and of packed prompts
        {"name": "conv decode", "op": "conv", "n": 256, "length": 1, "channels": 8192, "width": 4,
         "io": "bf16", "pad": 6},
        {"name": "conv packed 24", "op": "conv", "n": 24, "length": 1301, "channels": 4096, "width": 4,
         "io": "bf16", "pad": 5},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan", "step", "step", "norm", "conv"])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("scan", "step"):
        key_heads = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
        heads = key_heads * rng.choice([1, 1, 2, 2, 3])
        k = rng.choice([64, 128, 128, 128])
        v = rng.choice([64, 128, 128, 128, 96, 256])
    if op == "scan":
        length = _log(rng, 1, 8192) if io == "bf16" else _log(rng, 1, 2048)
        most = max(1, min(48, 8 * 2048 * 32 * 128 // (length * heads * v)))
        n = _log(rng, 1, most)
        return {"op": op, "n": n, "length": length, "key_heads": key_heads, "heads": heads, "k": k,
                "v": v, "io": io, "packed": n > 1 and rng.random() < 0.5, "h0": rng.random() < 0.6}
    if op == "step":
        n = _log(rng, 1, max(1, min(384, 256 * 32 * 128 * 128 // (heads * k * v))))
        return {"op": op, "n": n, "key_heads": key_heads, "heads": heads, "k": k, "v": v, "io": io,
                "pad": rng.randrange(0, 1 + n // 8)}
    if op == "norm":
        heads, width = rng.choice([1, 3, 8, 16, 24, 32, 80]), rng.choice([64, 64, 128, 128, 128, 96, 256, 77])
        tokens = _log(rng, 1, 16384 * 32 * 128 // (heads * width * (2 if io == "f32" else 1)))
        return {"op": op, "tokens": min(tokens, 65536), "heads": heads, "width": width, "io": io}
    channels = rng.choice([96, 512, 1536, 1792, 4096, 5376, 8192, 331])
    length = _log(rng, 1, 4096)
    n = _log(rng, 1, max(1, min(256, 24 * 1301 * 4096 // (length * channels * (2 if io == "f32" else 1)))))
    return {"op": op, "n": n, "length": length, "channels": channels, "width": rng.choice([4, 4, 4, 3, 2]),
            "io": io, "pad": rng.choice([0, 0, 5, 64])}


def _lengths(case):
    """The sequences' lengths of a packed case: between a token and twice `length`, the mean near it."""
    n, length = case["n"], case["length"]
    return [1 + (2 * length - 2) * ((7 * i + 3) % n) // max(1, n - 1) if length > 1 else 1 for i in range(n)]


def _tokens(case):
    packed = case.get("packed", True)
    return sum(_lengths(case)) if packed else case["n"] * case["length"]


# ------------------------------------------------------------------ the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _rand(gen, *shape):
    return torch.rand(shape, generator=gen, device="cuda")


def _silu(x):
    return x / (1 + torch.exp(-x))


def _gates(gen, heads):
    """Decay rates and step biases as a mixer is initialised: A in [-16, -1], steps in [1e-3, 0.1]."""
    A = -torch.exp(_rand(gen, heads) * math.log(16.0))
    step = torch.exp(_rand(gen, heads) * math.log(100.0) + math.log(1e-3))
    return A, step + torch.log(-torch.expm1(-step))


def prepare(case, seed):
    gen = _gen(seed)
    s = {"op": case["op"]}
    dtype = DTYPES[case["io"]]
    if case["op"] in ("scan", "step"):
        hk, h, K, V = case["key_heads"], case["heads"], case["k"], case["v"]
        s["A"], s["dt_bias"] = _gates(gen, h)
        s["scale"] = K ** -0.5
    if case["op"] == "scan":
        # q, k and v lie side by side in the convolution's output, dt and beta in a projection's
        packed = case["packed"]
        rows = (1, _tokens(case)) if packed else (case["n"], case["length"])
        qkv = _silu(_randn(gen, *rows, 2 * hk * K + h * V)).to(dtype)
        q, k, v = qkv.split([hk * K, hk * K, h * V], -1)
        s["q"], s["k"], s["v"] = q.unflatten(-1, (hk, K)), k.unflatten(-1, (hk, K)), v.unflatten(-1, (h, V))
        s["beta"], s["dt"] = _randn(gen, *rows, 2 * h).to(dtype).split([h, h], -1)
        s["cu_seqlens"] = s["slots"] = s["lengths"] = None
        n = case["n"]
        if packed:
            s["lengths"] = _lengths(case)
            s["cu_seqlens"] = torch.tensor([0] + s["lengths"], device="cuda").cumsum(0).to(torch.int32)
            s["slots"] = torch.randperm(n + 3, generator=gen, device="cuda")[:n].to(torch.int32)
            n += 3
        s["h0"] = 0.3 * _randn(gen, n, h, K, V) if case["h0"] else None
        # packed prompts update their cache in place
        s["h_last"] = (s["h0"] if case["h0"] else torch.zeros(n, h, K, V, device="cuda")) if packed else None
    elif case["op"] == "step":
        n = case["n"]
        qkv = _silu(_randn(gen, n, 2 * hk * K + h * V)).to(dtype)
        q, k, v = qkv.split([hk * K, hk * K, h * V], -1)
        s["q"], s["k"], s["v"] = q.unflatten(-1, (hk, K)), k.unflatten(-1, (hk, K)), v.unflatten(-1, (h, V))
        s["beta"], s["dt"] = _randn(gen, n, 2 * h).to(dtype).split([h, h], -1)
        s["state"] = 0.3 * _randn(gen, n + 2, h, K, V)
        s["slots"] = torch.randperm(n + 2, generator=gen, device="cuda")[:n].to(torch.int32)
        s["slots"][n - case["pad"]:] = -1  # the padded rows of a captured batch
        s["y"] = torch.zeros(n, h, V, dtype=dtype, device="cuda")
    elif case["op"] == "norm":
        t, h, w = case["tokens"], case["heads"], case["width"]
        s["x"] = (0.2 * _randn(gen, t, h, w)).to(dtype)
        s["z"] = _randn(gen, t, h, w).to(dtype)
        s["weight"] = 1 + 0.1 * _randn(gen, w)
    else:
        C, W, n = case["channels"], case["width"], case["n"]
        s["lengths"] = _lengths(case)
        s["cu_seqlens"] = torch.tensor([0] + s["lengths"], device="cuda").cumsum(0).to(torch.int32)
        rows = sum(s["lengths"]) + case["pad"]  # the buffer's rows behind the last sequence
        s["x"] = _randn(gen, rows, C).to(dtype)
        s["w"] = (_rand(gen, C, W) * 2 - 1) * W ** -0.5
        s["bias"] = (_rand(gen, C) * 2 - 1) * W ** -0.5
        s["state"] = _randn(gen, n + 2, C, W - 1)
        s["slots"] = torch.randperm(n + 2, generator=gen, device="cuda")[:n].to(torch.int32)
        s["u"] = torch.zeros(rows, C, dtype=dtype, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        from selective_state_space_28_b200 import ops
        if s["op"] == "scan":
            return ops.gdr_chunk_scan_fwd(s["q"], s["k"], s["v"], s["dt"], s["A"], s["beta"], dt_bias=s["dt_bias"],
                                          h0=s["h0"], scale=s["scale"], l2_eps=L2_EPS, cu_seqlens=s["cu_seqlens"],
                                          slots=s["slots"], h_last=s["h_last"])
        if s["op"] == "step":
            return ops.gdr_scan_step(s["state"], s["q"], s["k"], s["v"], s["dt"], s["A"], s["beta"],
                                     dt_bias=s["dt_bias"], scale=s["scale"], l2_eps=L2_EPS, slots=s["slots"],
                                     y=s["y"]), s["state"]
        if s["op"] == "norm":
            return ops.gdr_gated_rmsnorm_fwd(s["x"], s["z"], s["weight"], eps=NORM_EPS)
        return ops.ssm_conv1d_packed_fwd(s["x"], s["w"], s["bias"], s["state"], cu_seqlens=s["cu_seqlens"],
                                         slots=s["slots"], u=s["u"])
    if s["op"] == "scan":
        return _scan_plain(s)
    if s["op"] == "step":
        return _step_plain(s)
    if s["op"] == "norm":
        x, z = s["x"].float(), s["z"].float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + NORM_EPS) * s["weight"]
        return (x * _silu(z)).to(s["x"].dtype)
    return _conv_plain(s)


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-torch.abs(x)))


def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _l2norm(x):
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + L2_EPS)


def _pad_rows(s):
    """For a packed case, the row of the packed buffer of every (sequence, token), and which exist."""
    lengths = torch.tensor(s["lengths"], device="cuda")
    at = torch.arange(max(s["lengths"]), device="cuda")
    live = at < lengths[:, None]
    return torch.where(live, s["cu_seqlens"][:-1, None].long() + at, 0), live


def _unit_lower_inverse(m):
    """The inverse of I + m for strictly lower triangular m [.., 64, 64], blocks of twice the size each time:
    [[P, 0], [R, Q]]^-1 = [[P^-1, 0], [-Q^-1 R P^-1, Q^-1]]."""
    size = m.shape[-1]
    inv = torch.eye(size, device=m.device).expand(m.shape).contiguous()
    half = 1
    while half < size:
        blocks = inv.unflatten(-1, (-1, 2, half)).unflatten(-4, (-1, 2, half))  # [.., I, 2, half, J, 2, half]
        below = m.unflatten(-1, (-1, 2, half)).unflatten(-4, (-1, 2, half))
        on = range(size // (2 * half))
        P = torch.stack([blocks[..., i, 0, :, i, 0, :] for i in on], -3)
        Q = torch.stack([blocks[..., i, 1, :, i, 1, :] for i in on], -3)
        R = torch.stack([below[..., i, 1, :, i, 0, :] for i in on], -3)
        X = -(Q @ (R @ P))
        for i in on:
            blocks[..., i, 1, :, i, 0, :] = X[..., i, :, :]
        half *= 2
    return inv


def _scan_plain(s):
    q, k, v, dt, beta = (s[x].float() for x in ("q", "k", "v", "dt", "beta"))
    h, dtype = v.shape[2], s["v"].dtype
    packed = s["cu_seqlens"] is not None
    live = None
    if packed:
        rows, live = _pad_rows(s)
        q, k, v, dt, beta = (x[0][rows] for x in (q, k, v, dt, beta))
    n, length, hk, K = k.shape
    V = v.shape[3]
    q, k = (_l2norm(x).repeat_interleave(h // hk, 2) for x in (q, k))
    q = q * s["scale"]
    # logarithms of the decays: their running sums are subtracted, so 64 bits
    g = (_softplus(dt + s["dt_bias"]) * s["A"]).double()
    b = _sigmoid(beta)
    if packed:  # rows behind a sequence neither decay nor write
        g, b = (torch.where(live[..., None], x, 0) for x in (g, b))
    chunks = -(-length // CHUNK)

    def cut(x):  # [n, L, h, ..] -> [n, h, chunks, 64, ..], zeros behind the end
        x = torch.nn.functional.pad(x, [0, 0] * (x.dim() - 2) + [0, chunks * CHUNK - length])
        return x.unflatten(1, (chunks, CHUNK)).movedim(3, 1)

    q, k, v = cut(q), cut(k), cut(v)
    g, b = cut(g).cumsum(-1), cut(b)[..., None]
    below = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device="cuda").tril(-1)
    upto = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device="cuda").tril()
    span = torch.exp(torch.where(upto, g[..., :, None] - g[..., None, :], 0)).float()
    T = _unit_lower_inverse(torch.where(below, (k @ k.mT) * span * b, 0))
    P = torch.where(upto, (q @ k.mT) * span, 0)
    del span
    into = torch.exp(g).float()[..., None]               # decay from the chunk's start
    rest = torch.exp(g[..., -1:] - g).float()[..., None]  # decay to the chunk's end
    U = T @ (b * v)
    W = T @ (b * into * k)
    Q, R = q * into, k * rest
    S = torch.zeros(n, h, K, V, device="cuda")
    if s["h0"] is not None:
        S = s["h0"][s["slots"].long()] if packed else s["h0"]
    y = torch.empty_like(v)
    for c in range(chunks):  # the recurrence itself: a chunk needs the state before it
        u = U[:, :, c] - W[:, :, c] @ S
        y[:, :, c] = Q[:, :, c] @ S + P[:, :, c] @ u
        S = S * into[:, :, c, -1:] + R[:, :, c].mT @ u
    y = y.movedim(1, 3).flatten(1, 2)[:, :length].to(dtype)
    if not packed:
        return y, S
    s["h_last"][s["slots"].long()] = S
    return y[live][None], s["h_last"]


def _step_plain(s):
    on = s["slots"] >= 0
    slots = s["slots"][on].long()
    q, k, v, dt, beta = (s[x][on].float() for x in ("q", "k", "v", "dt", "beta"))
    r = v.shape[1] // k.shape[1]
    q, k = (_l2norm(x).repeat_interleave(r, 1) for x in (q, k))
    a = torch.exp(_softplus(dt + s["dt_bias"]) * s["A"])
    S = s["state"][slots] * a[..., None, None]
    u = _sigmoid(beta)[..., None] * (v - (S * k[..., None]).sum(2))
    S = S + k[..., None] * u[..., None, :]
    s["y"][on] = (s["scale"] * (S * q[..., None]).sum(2)).to(s["y"].dtype)
    s["state"][slots] = S
    return s["y"], s["state"]


def _conv_plain(s):
    x, w = s["x"].float(), s["w"]
    W, slots = w.shape[1], s["slots"].long()
    start, end = s["cu_seqlens"][:-1].long(), s["cu_seqlens"][1:].long()
    old = s["state"][slots]  # [n, C, W - 1], oldest first
    total = sum(s["lengths"])
    row = torch.arange(total, device="cuda")
    seq = (row[:, None] >= end).sum(1)
    at = row - start[seq]
    acc = s["bias"].expand(total, -1)
    new = []
    for j in range(W):  # the taps, oldest first
        back = W - 1 - j
        before = old[seq, :, torch.clamp(W - 1 + at - back, 0, W - 2)]
        acc = acc + w[:, j] * torch.where((at >= back)[:, None], x[torch.clamp(row - back, min=0)], before)
        if back:  # the state: the last W - 1 inputs, the old ones where the sequence is shorter
            t = end - start - back
            kept = old.gather(2, torch.clamp(W - 1 + t, 0, W - 2)[:, None, None].expand(-1, old.shape[1], 1))[..., 0]
            new.append(torch.where((t >= 0)[:, None], x[torch.clamp(start + t, min=0)], kept))
    s["u"][:total] = _silu(acc).to(s["u"].dtype)
    s["state"][slots] = torch.stack(new, -1)
    return s["u"], s["state"]


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    es = 2 if case["io"] == "bf16" else 4
    if case["op"] in ("scan", "step"):
        hk, h, K, V = case["key_heads"], case["heads"], case["k"], case["v"]
        if case["op"] == "scan":
            t, states = _tokens(case), case["n"] * (2 if case["h0"] else 1)
        else:
            t = case["n"] - case["pad"]
            states = 2 * t
        # S^T k, the decay with the outer product, S^T q
        return {"bytes": t * es * (2 * hk * K + 2 * h * V + 2 * h) + 4 * states * h * K * V,
                "flops": 7 * t * h * K * V}
    if case["op"] == "norm":
        size = case["tokens"] * case["heads"] * case["width"]
        return {"bytes": 3 * es * size, "flops": 9 * size}
    t, C, W = _tokens(case), case["channels"], case["width"]
    return {"bytes": 2 * es * t * C + 8 * case["n"] * C * (W - 1) + 4 * C * (W + 1), "flops": (2 * W + 5) * t * C}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        x, z = s["x"].double(), s["z"].double()
        rms = ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + NORM_EPS).sqrt()
        return x / rms * s["weight"].double() * z / (1 + torch.exp(-z))
    if case["op"] == "conv":
        x, w, C = s["x"].double(), s["w"].double(), case["channels"]
        u, state = s["u"].double(), s["state"].double()
        begin = 0
        for slot, length in zip(s["slots"].tolist(), s["lengths"]):
            line = torch.cat([state[slot].T, x[begin:begin + length]])
            out = s["bias"].double() + sum(line[j:j + length] * w[:, j] for j in range(case["width"]))
            u[begin:begin + length] = out / (1 + torch.exp(-out))
            state[slot] = line[length:].T
            begin += length
        return u, state
    one_step = case["op"] == "step"
    q, k, v, dt, beta = (s[x].double() for x in ("q", "k", "v", "dt", "beta"))
    if one_step:
        q, k, v, dt, beta = (x[:, None] for x in (q, k, v, dt, beta))
    lengths, cache, slots = None, None, None
    if one_step:
        cache, slots = s["state"].double(), s["slots"].long()
        lengths = (slots >= 0).long()
    elif case["packed"]:
        lengths, slots = torch.tensor(s["lengths"], device="cuda"), s["slots"].long()
        cache = s["h_last"].double()
        q, k, v, dt, beta = (torch.nn.utils.rnn.pad_sequence(x[0].split(s["lengths"]), batch_first=True)
                             for x in (q, k, v, dt, beta))
    n, steps, h, V = v.shape
    K, per = k.shape[3], h // k.shape[2]
    if cache is not None:
        state = cache[slots.clamp(min=0)]
    else:
        state = s["h0"].double() if s["h0"] is not None else torch.zeros(n, h, K, V, dtype=torch.float64, device="cuda")
    decay = torch.exp(torch.log1p(torch.exp(dt + s["dt_bias"].double())) * s["A"].double())
    gain = 1 / (1 + torch.exp(-beta))
    y = torch.zeros_like(v)
    for t in range(steps):
        kt = (k[:, t] / (k[:, t].square().sum(-1, keepdim=True) + L2_EPS).sqrt()).repeat_interleave(per, 1)
        qt = (q[:, t] / (q[:, t].square().sum(-1, keepdim=True) + L2_EPS).sqrt()).repeat_interleave(per, 1)
        new = state * decay[:, t, :, None, None]
        u = gain[:, t, :, None] * (v[:, t] - torch.einsum("nhkv,nhk->nhv", new, kt))
        new = new + torch.einsum("nhk,nhv->nhkv", kt, u)
        y[:, t] = s["scale"] * torch.einsum("nhkv,nhk->nhv", new, qt)
        if lengths is not None:
            alive = (t < lengths)[:, None, None, None]
            state, y[:, t] = torch.where(alive, new, state), torch.where(alive[..., 0], y[:, t], 0)
        else:
            state = new
    if cache is None:
        return y, state
    cache[slots[lengths > 0]] = state[lengths > 0]
    if one_step:
        return y[:, 0], cache
    return torch.cat([y[i, :m] for i, m in enumerate(s["lengths"])])[None], cache
