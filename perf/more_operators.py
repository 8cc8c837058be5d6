"""The operators of a Gated DeltaNet layer and their plain forms, as cases to time and to compare.

Five entry points stand between the fused input projection (qkv | z | a | b) and
the output projection of a recurrent layer that is being served:

  conv       causal depthwise convolution with SiLU of ragged prompts, with a carried state
  conv_step  the same for one new token a request
  chunk      the gated delta rule over ragged prompts, in chunks, with a carried state
  step       the same for one new token a request
  norm       a norm over each head of the output, times the SiLU of the gate z

``own`` chooses what ``run`` computes: the plain forms below (False) or the
library's kernels (True).  ``prepare`` makes the same inputs for both.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6
CHUNK = 64  # of the plain chunked form


def listed():
    # Head layout of the hybrid 27B model that the workloads of this library are drawn from: qkv 8192, z 6144, a and b 48
    # columns, which is 8 key heads and 48 value heads of 128.
    wide = {"k_heads": 8, "v_heads": 48, "head_k": 128, "head_v": 128}
    return [
        # one decode step of 32 requests
        {"name": "conv_decode", "op": "conv_step", "seqs": 32, "channels": 8192, "width": 4, "bias": False, "rest": 6240, "dtype": "bf16"},
        # an 8K-token prompt, read from the columns of the fused projection
        {"name": "conv_prefill", "op": "conv", "seqs": 1, "most": 8192, "resumed": 0, "channels": 8192, "width": 4, "bias": False,
         "rest": 6240, "dtype": "bf16"},
        # prompts of odd lengths, some of them continued, one of a single token
        {"name": "conv_ragged", "op": "conv", "seqs": 13, "most": 1021, "resumed": 5, "channels": 2568, "width": 3, "bias": True, "rest": 0,
         "dtype": "f16"},
        # a few short prompts in float32: the latency of a call
        {"name": "chunk_small", "op": "chunk", "k_heads": 2, "v_heads": 4, "head_k": 64, "head_v": 64, "seqs": 3, "most": 100, "resumed": 1,
         "rest": 0, "dtype": "f32"},
        # an 8K-token prompt alone on the card
        {"name": "chunk_prompt", "op": "chunk", **wide, "seqs": 1, "most": 8192, "resumed": 0, "rest": 14336, "dtype": "bf16"},
        # a batch of ragged prompts, a few of them continued
        {"name": "chunk_batch", "op": "chunk", **wide, "seqs": 12, "most": 4096, "resumed": 3, "rest": 14336, "dtype": "bf16"},
        # a long prompt where the heads are dealt to eight cards
        {"name": "chunk_few_heads", "op": "chunk", "k_heads": 1, "v_heads": 6, "head_k": 128, "head_v": 128, "seqs": 1, "most": 16411,
         "resumed": 1, "rest": 0, "dtype": "f16"},
        # one request in float32: the latency of a call
        {"name": "step_small", "op": "step", "k_heads": 2, "v_heads": 4, "head_k": 64, "head_v": 64, "seqs": 1, "idle": 0, "rest": 0,
         "dtype": "f32"},
        # one decode step of 32 requests, two of them rows that pad the batch
        {"name": "step_decode", "op": "step", **wide, "seqs": 32, "idle": 2, "rest": 14336, "dtype": "bf16"},
        # one decode step of 32 requests
        {"name": "norm_decode", "op": "norm", "groups": 48, "dim": 128, "tokens": 32, "centred": False, "gate": True, "shared": True,
         "bias": False, "rest": 8288, "dtype": "bf16"},
        # an 8K-token prompt
        {"name": "norm_prefill", "op": "norm", "groups": 48, "dim": 128, "tokens": 8192, "centred": False, "gate": True, "shared": True,
         "bias": False, "rest": 8288, "dtype": "bf16"},
        # a group norm with its mean taken off, weights and bias for each channel, odd groups in float32
        {"name": "norm_centred", "op": "norm", "groups": 20, "dim": 121, "tokens": 4099, "centred": True, "gate": False, "shared": False,
         "bias": True, "rest": 0, "dtype": "f32"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["conv", "conv_step", "chunk", "chunk", "chunk", "step", "step", "norm"])
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    rest = rng.choice([0, 0, 48, 6240])  # columns of other things in the same rows
    if op in ("conv", "conv_step"):
        channels = 8 * _log(rng, 8, 1536) + rng.choice([0, 0, 0, 4, 1])
        case = {"op": op, "channels": channels, "width": rng.choice([2, 3, 4, 4]), "bias": rng.random() < 0.5, "rest": rest, "dtype": dtype}
        if op == "conv_step":
            return {**case, "seqs": _log(rng, 1, 512)}
        seqs = _log(rng, 1, 64)
        most = _log(rng, 1, max(2, min(32768, (1 << 25) // (seqs * channels))))
        return {**case, "seqs": seqs, "most": most, "resumed": rng.randint(0, seqs)}
    if op == "norm":
        groups, dim = rng.choice([1, 4, 6, 16, 20, 48]), rng.choice([64, 128, 128, 192, 256, rng.randint(1, 600)])
        return {"op": op, "groups": groups, "dim": dim, "tokens": _log(rng, 1, min(65536, (1 << 25) // (groups * dim))),
                "centred": rng.random() < 0.5, "gate": rng.random() < 0.6, "shared": rng.random() < 0.5, "bias": rng.random() < 0.5,
                "rest": rest, "dtype": dtype}
    k_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 6])
    head_k, head_v = rng.choice([64, 128, 128]), rng.choice([64, 128, 128, 192, 256])
    while k_heads * group * head_v > 6144:
        k_heads //= 2
    case = {"op": op, "k_heads": k_heads, "v_heads": k_heads * group, "head_k": head_k, "head_v": head_v, "rest": rest, "dtype": dtype}
    per_token = k_heads * group * head_k * head_v
    if op == "step":
        seqs = _log(rng, 1, max(2, min(256, 32 * 48 * 128 * 128 // per_token)))
        return {**case, "seqs": seqs, "idle": rng.choice([0, 0, 1, seqs // 5]) if seqs > 1 else 0}
    seqs = _log(rng, 1, 48)
    most = _log(rng, 1, max(2, min(16384, 12 * 2100 * 48 * 128 * 128 // (seqs * per_token))))
    return {**case, "seqs": seqs, "most": most, "resumed": rng.randint(0, seqs)}


# Lengths go by the case alone, so that its work is known; what they hold goes by the seed.

def _lens(case):
    """Lengths from a sixteenth of the longest up to it, the first the longest, out of order; the last of several a single token."""
    count, high = case["seqs"], case["most"]
    low = max(1, high // 16)
    at = np.modf(np.arange(1, count + 1) * 0.6180339887498949)[0]
    got = (low + np.floor(at * (high - low + 1))).astype(np.int64)
    got[0] = high
    if count > 2:
        got[-1] = 1
    return got


def _pad(case):
    """Rows behind the last sequence, as a batch padded to a round number has them."""
    return 0 if case["seqs"] == 1 else 5


def work(case):
    op, size = case["op"], BYTES[case["dtype"]]
    if op == "norm":
        t, n = case["tokens"], case["groups"] * case["dim"]
        rows = 3 if case["gate"] else 2
        params = (case["dim"] if case["shared"] else n) * (2 if case["bias"] else 1)
        return {"bytes": t * n * rows * size + 4 * params, "flops": t * n * (10 if case["gate"] else 8)}
    n = case["seqs"]
    if op in ("conv", "conv_step"):
        c, w = case["channels"], case["width"]
        t = n if op == "conv_step" else int(_lens(case).sum())
        read = n if op == "conv_step" else case["resumed"]
        params = c * (w + case["bias"])
        return {"bytes": size * c * (2 * t + (w - 1) * (read + n)) + 4 * params + 12 * n, "flops": t * c * (2 * w + 4)}
    hk, hv, dk, dv = case["k_heads"], case["v_heads"], case["head_k"], case["head_v"]
    if op == "step":
        t = read = written = n - case["idle"]
    else:
        t, read, written = int(_lens(case).sum()), case["resumed"], n
    # k and q against the state, and its update: three products of 2 dk dv, and the decay
    return {"bytes": t * size * (2 * hk * dk + 2 * hv * dv + 2 * hv) + 4 * hv * dk * dv * (read + written) + 8 * hv + 12 * n,
            "flops": 7 * t * hv * dk * dv}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _ints(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV, torch.int32)


def _rand(shape, g):
    return torch.randn(shape, generator=g, device=DEV)


def _projected(tokens, columns, g, dtype):
    """Rows of a projection: normal values with every 64th channel larger."""
    x = _rand((tokens, columns), g)
    x[:, ::64] *= 4.0
    return x.to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    s = {"case": case}
    if op == "norm":
        t, groups, dim = case["tokens"], case["groups"], case["dim"]
        n = groups * dim
        # outputs of the recurrence: heads of different sizes; some values far from the mean of their group
        x = (_rand((t, groups, dim), g) * torch.exp(_rand((t, groups, 1), g)) + 0.5 * _rand((1, groups, 1), g)).to(dtype)
        rows = _projected(t, n + case["rest"], g, dtype)
        gate = rows[:, case["rest"]:].view(t, groups, dim) if case["gate"] else None
        shape = (dim,) if case["shared"] else (groups, dim)
        s.update(x=x, gate=gate, weight=1.0 + 0.2 * _rand(shape, g), bias=0.1 * _rand(shape, g) if case["bias"] else None,
                 out=torch.empty_like(x))
        return s
    n = case["seqs"]
    slots = torch.randperm(n + 5, generator=g, device=DEV)[:n].to(torch.int32)
    if op in ("conv", "chunk"):
        lens = _lens(case)
        starts = np.concatenate([[0], np.cumsum(lens)])
        cached = np.zeros(n, np.int64)
        cached[n - case["resumed"]:] = 777
        s.update(starts=_ints(starts), cached=_ints(cached), tokens=int(starts[-1]))
        t = int(starts[-1]) + _pad(case)
    else:
        t = n
    if op in ("conv", "conv_step"):
        c, w = case["channels"], case["width"]
        x = _projected(t, c + case["rest"], g, dtype)[:, :c]
        s.update(x=x, weight=_rand((c, w), g) / w ** 0.5, bias=0.1 * _rand((c,), g) if case["bias"] else None, slots=slots,
                 state=_rand((n + 5, w - 1, c), g).to(dtype), state_out=torch.zeros((n + 5, w - 1, c), dtype=dtype, device=DEV),
                 out=torch.zeros((t, c), dtype=dtype, device=DEV))
        return s
    hk, hv, dk, dv = case["k_heads"], case["v_heads"], case["head_k"], case["head_v"]
    # what the convolution leaves: SiLU of normal values, q | k | v in one row
    qkv = torch.nn.functional.silu(_projected(t, 2 * hk * dk + hv * dv, g, torch.float32)).to(dtype)
    gates = _projected(t, case["rest"] + 2 * hv, g, dtype)
    s.update(q=qkv[:, :hk * dk].view(t, hk, dk), k=qkv[:, hk * dk:2 * hk * dk].view(t, hk, dk), v=qkv[:, 2 * hk * dk:].view(t, hv, dv),
             a=gates[:, case["rest"]:case["rest"] + hv], b=gates[:, case["rest"] + hv:])
    if op == "step" and case["idle"]:
        slots[n - case["idle"]:] = -1
    # decays as such layers are initialised: rates of 1 to 16 a unit of time, steps of 0.001 to 0.1
    dt = torch.exp(torch.rand(hv, generator=g, device=DEV) * math.log(100.0) + math.log(0.001))
    s.update(a_log=torch.log(1.0 + 15.0 * torch.rand(hv, generator=g, device=DEV)), dt_bias=dt + torch.log(-torch.expm1(-dt)), slots=slots,
             scale=dk ** -0.5, state=0.3 * _rand((n + 5, hv, dk, dv), g), state_out=torch.zeros((n + 5, hv, dk, dv), device=DEV),
             out=torch.zeros((t, hv, dv), dtype=dtype, device=DEV))
    if own and op == "chunk":
        import nvfp4_w4a4_block_quantize_amd as nv

        size = nv.nvfp4_gated_delta_workspace(t, n, hk, hv, dk, dv, dtype)
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return s


def run(s):
    return {"conv": _conv, "conv_step": _conv_step, "chunk": _chunk, "step": _step, "norm": _norm}[s["case"]["op"]](s)


def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _conv(s):
    if own:
        import nvfp4_w4a4_block_quantize_amd as nv

        nv.nvfp4_causal_conv(s["x"], s["weight"], s["state"], s["slots"], s["starts"], cached_lens=s["cached"], bias=s["bias"],
                             activation="silu", state_out=s["state_out"], out=s["out"])
        return {"out": s["out"], "state": s["state_out"]}
    x, w, t = s["x"].float(), s["case"]["width"], s["tokens"]
    starts, slots = s["starts"].long(), s["slots"].long()
    old = s["state"][slots].float() * (s["cached"] > 0)[:, None, None]
    at = torch.arange(t, device=DEV)
    r = torch.searchsorted(starts[1:], at, right=True)
    y = torch.zeros((t, x.shape[1]), device=DEV)
    for j in range(w):
        back = at - (w - 1) + j
        before = back - starts[r]  # negative: in the carried state
        row = torch.where((before < 0)[:, None], old[r, (w - 1 + before).clamp(0, w - 2)], x[back.clamp(min=0)])
        y += s["weight"][:, j] * row
    if s["bias"] is not None:
        y += s["bias"]
    out = s["out"]
    out[:t] = _silu(y).to(out.dtype)
    for j in range(w - 1):
        back = starts[1:] - (w - 1) + j
        before = back - starts[:-1]
        index = torch.arange(len(slots), device=DEV)
        row = torch.where((before < 0)[:, None], old[index, (w - 1 + before).clamp(0, w - 2)], x[back.clamp(min=0)])
        s["state_out"][slots, j] = row.to(out.dtype)
    return {"out": out, "state": s["state_out"]}


def _conv_step(s):
    if own:
        import nvfp4_w4a4_block_quantize_amd as nv

        nv.nvfp4_causal_conv_step(s["x"], s["weight"], s["state"], s["slots"], bias=s["bias"], activation="silu", state_out=s["state_out"],
                                  out=s["out"])
        return {"out": s["out"], "state": s["state_out"]}
    slots = s["slots"].long()
    seen = torch.cat([s["state"][slots], s["x"][:, None, :]], 1)
    y = (seen.float() * s["weight"].t()).sum(1)
    if s["bias"] is not None:
        y += s["bias"]
    s["out"].copy_(_silu(y))
    s["state_out"][slots] = seen[:, 1:]
    return {"out": s["out"], "state": s["state_out"]}


def _unit(x):
    x = x.float()
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS)


def _gates(s):
    """Log decays (in 64 bits: their sums are subtracted) and write strengths."""
    x = s["a"].double() + s["dt_bias"].double()
    decay = -torch.exp(s["a_log"].double()) * (x.clamp(min=0) + torch.log1p(torch.exp(-x.abs())))
    return decay, 1.0 / (1.0 + torch.exp(-s["b"].float()))


def _chunk(s):
    if own:
        import nvfp4_w4a4_block_quantize_amd as nv

        nv.nvfp4_gated_delta_chunked(s["q"], s["k"], s["v"], s["a"], s["b"], s["a_log"], s["dt_bias"], s["state"], s["slots"], s["starts"],
                                     cached_lens=s["cached"], scale=s["scale"], eps=EPS, state_out=s["state_out"], out=s["out"],
                                     workspace=s["workspace"])
        return {"out": s["out"], "state": s["state_out"]}
    c = s["case"]
    n, hk, hv, dk, dv = c["seqs"], c["k_heads"], c["v_heads"], c["head_k"], c["head_v"]
    group, chunks = hv // hk, -(-c["most"] // CHUNK)
    starts, slots = s["starts"].long(), s["slots"].long()
    at = torch.arange(chunks * CHUNK, device=DEV)
    here = at < (starts[1:] - starts[:-1])[:, None]  # [n, T]
    token = (starts[:-1, None] + at).clamp(max=s["tokens"] - 1)

    def laid(x, heads):  # [tokens, heads, ...] -> [n, heads, chunks, CHUNK, ...], zeros behind each sequence
        y = x[token].masked_fill(~here.view(n, -1, *[1] * (x.dim() - 1)), 0)
        y = y.view(n, chunks, CHUNK, heads, *x.shape[2:])
        return y.permute(0, 3, 1, 2, *range(4, y.dim())).contiguous()

    k, q, v = laid(_unit(s["k"]), hk), laid(_unit(s["q"]) * s["scale"], hk), laid(s["v"].float(), hv)
    decay, beta = _gates(s)
    total = laid(decay, hv).cumsum(-1)
    beta = laid(beta, hv)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEV).tril()
    ratio = torch.exp((total[..., :, None] - total[..., None, :]).masked_fill(~low, -math.inf).float())
    kk = torch.matmul(k, k.transpose(-1, -2)).repeat_interleave(group, 1)
    mixed = (beta[..., None] * ratio * kk).tril(-1)
    turn = torch.eye(CHUNK, device=DEV).expand_as(mixed).contiguous()
    for i in range(1, CHUNK):  # (1 + mixed) turn = 1, row by row
        turn[..., i, :i] = -torch.matmul(mixed[..., i:i + 1, :i], turn[..., :i, :i]).squeeze(-2)
    del mixed, kk
    inner = torch.matmul(q, k.transpose(-1, -2)).repeat_interleave(group, 1) * ratio
    del ratio
    since, until = torch.exp(total.float()), torch.exp((total[..., -1:] - total).float())
    state = (s["state"][slots] * (s["cached"] > 0)[:, None, None, None]).view(n, hk, group, dk, dv)
    rows = []
    for i in range(chunks):
        kc, qc = k[:, :, None, i], q[:, :, None, i]
        gain = since[:, :, i].view(n, hk, group, CHUNK, 1)
        x = beta[:, :, i].view(n, hk, group, CHUNK, 1) * (v[:, :, i].view(n, hk, group, CHUNK, dv) - gain * torch.matmul(kc, state))
        x = torch.matmul(turn[:, :, i].view(n, hk, group, CHUNK, CHUNK), x)
        rows.append(gain * torch.matmul(qc, state) + torch.matmul(inner[:, :, i].view(n, hk, group, CHUNK, CHUNK), x))
        state = gain[..., -1:, :] * state + torch.matmul(kc.transpose(-1, -2), until[:, :, i].view(n, hk, group, CHUNK, 1) * x)
    y = torch.stack(rows, 3).view(n, hv, -1, dv).permute(0, 2, 1, 3)  # [n, T, hv, dv]
    s["out"][:s["tokens"]] = y[here].to(s["out"].dtype)
    s["state_out"][slots] = state.reshape(n, hv, dk, dv)
    return {"out": s["out"], "state": s["state_out"]}


def _step(s):
    if own:
        import nvfp4_w4a4_block_quantize_amd as nv

        nv.nvfp4_gated_delta_step(s["q"], s["k"], s["v"], s["a"], s["b"], s["a_log"], s["dt_bias"], s["state"], s["slots"], scale=s["scale"],
                                  eps=EPS, state_out=s["state_out"], out=s["out"])
        return {"out": s["out"], "state": s["state_out"]}
    c = s["case"]
    live = c["seqs"] - c["idle"]
    slots, group = s["slots"][:live].long(), c["v_heads"] // c["k_heads"]
    decay, beta = _gates(s)
    k, q = (_unit(x[:live]).repeat_interleave(group, 1).unsqueeze(-2) for x in (s["k"], s["q"]))
    state = s["state"][slots] * torch.exp(decay[:live].float())[..., None, None]
    new = beta[:live, :, None, None] * (s["v"][:live].float().unsqueeze(-2) - torch.matmul(k, state))
    state = state + k.transpose(-1, -2) * new
    s["out"][:live] = (torch.matmul(q, state).squeeze(-2) * s["scale"]).to(s["out"].dtype)
    s["state_out"][slots] = state
    return {"out": s["out"], "state": s["state_out"]}


def _norm(s):
    c = s["case"]
    if own:
        import nvfp4_w4a4_block_quantize_amd as nv

        nv.nvfp4_group_norm(s["x"], s["weight"], bias=s["bias"], gate=s["gate"], activation="silu", centred=c["centred"], eps=EPS, out=s["out"])
        return s["out"]
    y = s["x"].float()
    if c["centred"]:
        y = y - y.mean(-1, keepdim=True)
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * s["weight"]
    if s["bias"] is not None:
        y = y + s["bias"]
    y = _silu(y) if s["gate"] is None else y * _silu(s["gate"].float())
    s["out"].copy_(y)
    return s["out"]


def _recurrence(s, steps, states):
    """Token by token in 64 bits.  `steps`: for each step the rows of q, k, v, a and b, and which of `states` they belong to."""
    c = s["case"]
    group, outs = c["v_heads"] // c["k_heads"], torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    x = s["a"].double() + s["dt_bias"].double()
    alpha = torch.exp(-torch.exp(s["a_log"].double()) * torch.logaddexp(x, torch.zeros_like(x)))
    beta = torch.sigmoid(s["b"].double())
    unit = []
    for name in ("k", "q"):
        y = s[name].double()
        unit.append(y / torch.sqrt((y * y).sum(-1, keepdim=True) + EPS))
    for rows, live in steps:
        k, q = (u[rows].repeat_interleave(group, 1) for u in unit)
        state = states[:live]
        state *= alpha[rows][:, :, None, None]
        new = beta[rows][..., None] * (s["v"][rows].double() - torch.matmul(k.unsqueeze(-2), state).squeeze(-2))
        state.addcmul_(k.unsqueeze(-1), new.unsqueeze(-2))
        outs[rows] = torch.matmul(q.unsqueeze(-2), state).squeeze(-2) * s["scale"]
    return outs


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "norm":
        y = s["x"].double()
        if case["centred"]:
            y = y - y.mean(-1, keepdim=True)
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * s["weight"].double()
        if s["bias"] is not None:
            y = y + s["bias"].double()
        if s["gate"] is None:
            return y * torch.sigmoid(y)
        z = s["gate"].double()
        return y * z * torch.sigmoid(z)
    slots = s["slots"].long()
    if op in ("conv", "conv_step"):
        out, after = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV), torch.zeros(s["state"].shape, dtype=torch.float64, device=DEV)
        w = case["width"]
        weight = s["weight"].double().t().unsqueeze(0)  # [1, width, channels]
        for r in range(case["seqs"]):
            low, high = (r, r + 1) if op == "conv_step" else (int(s["starts"][r]), int(s["starts"][r + 1]))
            old = s["state"][slots[r]].double()
            if op == "conv" and int(s["cached"][r]) == 0:
                old = torch.zeros_like(old)
            seen = torch.cat([old, s["x"][low:high].double()])
            y = (seen.unfold(0, w, 1).transpose(1, 2) * weight).sum(1)
            if s["bias"] is not None:
                y = y + s["bias"].double()
            out[low:high] = y * torch.sigmoid(y)
            after[slots[r]] = seen[len(seen) - (w - 1):]
        return {"out": out, "state": after}
    after = torch.zeros(s["state"].shape, dtype=torch.float64, device=DEV)
    if op == "step":
        live = case["seqs"] - case["idle"]
        states = s["state"][slots[:live]].double()
        out = _recurrence(s, [(torch.arange(live, device=DEV), live)], states)
        after[slots[:live]] = states
        return {"out": out, "state": after}
    lens, starts = _lens(case), s["starts"].long()
    if int(lens.max()) > 60000:
        return None
    order = np.argsort(-lens, kind="stable")  # the longest first, so that the live ones are a leading part
    first = starts[:-1][torch.from_numpy(order).to(DEV)]
    states = (s["state"][slots].double() * (s["cached"] > 0)[:, None, None, None])[torch.from_numpy(order).to(DEV)].contiguous()
    count = np.searchsorted(-lens[order], -np.arange(int(lens.max())), side="left")  # sequences longer than i
    out = _recurrence(s, ((first[:int(live)] + i, int(live)) for i, live in enumerate(count)), states)
    after[slots[torch.from_numpy(order).to(DEV)]] = states
    return {"out": out, "state": after}
