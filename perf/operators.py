"""The paged KV cache's operators and their plain forms, as cases to time and to compare.

Four operators stand between the qkv projection and the output projection of an
attention layer that is being served:

  table   block tables and slot maps, built on the GPU from the requests' lengths
  rope    rotary positions with several axes, on the query and key heads
  write   K and V rows to FP8 (E4M3, one static scale per tensor), into cache pages
  attend  one new token per sequence against its pages of that cache

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
E4M3_MAX = 448.0
# what a serving program keeps for the attention's partial results
WORKSPACE = 1 << 27


def listed():
    # Head layout of the hybrid 27B model that the workloads of this library are
    # drawn from: 24 gated query heads and 4 KV heads of 256, which is 14336
    # columns of the fused projection, 64 of the 256 rotated.
    wide = {"q_heads": 24, "kv_heads": 4, "head_dim": 256}
    return [
        # a decode step of 256 running requests: one token each, a few finished
        {"name": "table_decode", "op": "table", "requests": 256, "new": 1, "cached": 32768, "page": 16, "short": 0},
        # admission of 96 prompts of up to 32K tokens, some with a cached prefix; the free list is too short for the last
        {"name": "table_prompts", "op": "table", "requests": 96, "new": 32768, "cached": 4096, "page": 16, "short": 500},
        # one decode step of 32 requests
        {"name": "rope_decode", "op": "rope", **wide, "tokens": 32, "rot": 64, "gated": True, "adjacent": False, "turns": True,
         "far": 32768, "dtype": "bf16"},
        # an 8K-token prompt
        {"name": "rope_prefill", "op": "rope", **wide, "tokens": 8192, "rot": 64, "gated": True, "adjacent": False, "turns": True,
         "far": 32768, "dtype": "bf16"},
        # a long video in float32: the whole head rotated, neighbours paired, far positions, an odd count
        {"name": "rope_video", "op": "rope", "q_heads": 16, "kv_heads": 2, "head_dim": 128, "tokens": 4099, "rot": 128, "gated": False,
         "adjacent": True, "turns": False, "far": 1000000, "dtype": "f32"},
        # one decode step of 32 requests
        {"name": "write_decode", "op": "write", **wide, "gated": True, "tokens": 32, "page": 16, "prompt": False, "pad": 0, "dtype": "bf16"},
        # a 32K-token prompt
        {"name": "write_prefill", "op": "write", **wide, "gated": True, "tokens": 32768, "page": 64, "prompt": True, "pad": 0, "dtype": "bf16"},
        # an odd number of tokens in pages of 48, the batch padded with tokens that belong to no page
        {"name": "write_ragged", "op": "write", "q_heads": 32, "kv_heads": 8, "head_dim": 128, "gated": False, "tokens": 5003, "page": 48,
         "prompt": True, "pad": 77, "dtype": "f16"},
        # a few short sequences in float32: the latency of a call
        {"name": "attend_small", "op": "attend", "q_heads": 8, "kv_heads": 2, "head_dim": 64, "seqs": 3, "most": 200, "empty": 0,
         "page": 16, "window": 0, "lse": True, "dtype": "f32"},
        # one long context alone on the card
        {"name": "attend_long", "op": "attend", **wide, "seqs": 1, "most": 131072, "empty": 0, "page": 64, "window": 0, "lse": False,
         "dtype": "bf16"},
        # a full batch of ragged contexts
        {"name": "attend_batch", "op": "attend", **wide, "seqs": 64, "most": 16384, "empty": 0, "page": 64, "window": 0, "lse": False,
         "dtype": "bf16"},
        # sliding windows over odd pages, the batch padded with empty rows
        {"name": "attend_window", "op": "attend", "q_heads": 32, "kv_heads": 4, "head_dim": 128, "seqs": 33, "most": 20011, "empty": 3,
         "page": 24, "window": 4095, "lse": True, "dtype": "f16"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["table", "rope", "write", "attend", "attend"])
    page = rng.choice([8, 16, 24, 32, 48, 64, 128, 256])
    if op == "table":
        requests = _log(rng, 1, 4096)
        new = 1 if rng.random() < 0.4 else _log(rng, 1, max(2, min(32768, (3 << 20) // requests)))
        cached = _log(rng, 1, max(page, min(65536, (1 << 22) * page // requests)))
        return {"op": op, "requests": requests, "new": new, "cached": cached, "page": page, "short": rng.choice([0, 0, 7, 300])}
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 6, 8, 12, 16])
    head_dim = rng.choice([64, 128, 192, 256])
    if kv_heads * group * head_dim > 8192:
        group = max(1, 8192 // (kv_heads * head_dim))
        group -= group % 4 == 0 and group > 4  # an odd group now and then
    heads = {"q_heads": kv_heads * group, "kv_heads": kv_heads, "head_dim": head_dim}
    if op == "rope":
        row = BYTES[dtype] * head_dim * kv_heads * (group + 1)
        return {"op": op, **heads, "tokens": _log(rng, 1, (1 << 27) // row), "rot": 2 * rng.randint(4, head_dim // 2),
                "gated": rng.random() < 0.5, "adjacent": rng.random() < 0.5, "turns": rng.random() < 0.5,
                "far": rng.choice([1000, 32768, 1000000]), "dtype": dtype}
    if op == "write":
        tokens = _log(rng, 1, (1 << 25) // (kv_heads * head_dim))
        return {"op": op, **heads, "gated": rng.random() < 0.5, "tokens": tokens, "page": page, "prompt": rng.random() < 0.6,
                "pad": rng.choice([0, 0, tokens // 7]), "dtype": dtype}
    seqs = _log(rng, 1, 64)
    most = _log(rng, 1, min(131072, (1 << 28) // (seqs * kv_heads * head_dim)))
    return {"op": op, **heads, "seqs": seqs, "most": most, "empty": rng.choice([0, 0, 1]) if seqs > 1 else 0, "page": page,
            "window": rng.choice([0, 0, 0, 1 + most // 3]), "lse": rng.random() < 0.5, "dtype": dtype}


# Lengths go by the case alone, so that its work is known; what they hold goes by the seed.

def _spread(count, low, high):
    """`count` whole numbers over low..high, the first the highest, out of order."""
    at = np.modf(np.arange(1, count + 1) * 0.6180339887498949)[0]
    got = (low + np.floor(at * (high - low + 1))).astype(np.int64)
    if count:
        got[0] = high
    return got


def _ceil(a, b):
    return -(-a // b)


def _table_lens(case):
    n = case["requests"]
    cached = _spread(n, 0, case["cached"])
    new = np.ones(n, np.int64) if case["new"] == 1 else _spread(n + 1, 1, case["new"])[1:]
    if case["new"] == 1:
        new[np.arange(n) % 37 == 36] = 0  # finished requests that still hold their rows
    else:
        cached[np.arange(n) % 3 > 0] = 0  # most prompts have no cached prefix
    return cached, new


def _attend_lens(case):
    lens = _spread(case["seqs"], max(1, case["most"] // 16), case["most"])
    if case["empty"]:
        lens[-case["empty"]:] = 0  # the rows that pad a batch
    return lens


def work(case):
    op = case["op"]
    if op == "table":
        cached, new = _table_lens(case)
        n, tokens, page = case["requests"], int(new.sum()), case["page"]
        fresh = int((_ceil(cached + new, page) - _ceil(cached, page)).sum())
        # lengths in; free pages in, into the tables; lengths, starts and first pages out; a slot for each token; one entry read where a page is begun
        held = int(((cached % page > 0) & (new > 0)).sum())
        return {"bytes": 4 * (2 * n + 2 * fresh + held + 3 * n + 1 + tokens + 2), "flops": 0}
    width = case["head_dim"]
    if op == "rope":
        heads, t = case["q_heads"] + case["kv_heads"], case["tokens"]
        pairs = case["rot"] // 2
        return {"bytes": 2 * t * heads * width * BYTES[case["dtype"]] + 12 * t + 8 * pairs, "flops": t * heads * pairs * 6}
    if op == "write":
        t, row = case["tokens"] - case["pad"], case["kv_heads"] * width
        return {"bytes": 2 * t * row * (BYTES[case["dtype"]] + 1) + 4 * case["tokens"] + 8, "flops": 2 * t * row}
    lens = _attend_lens(case)
    seen = int((np.minimum(lens, case["window"]) if case["window"] else lens).sum())
    pages = int(_ceil(np.minimum(lens, case["window"]) if case["window"] else lens, case["page"]).sum())
    rows = case["seqs"] * case["q_heads"]
    return {"bytes": 2 * seen * case["kv_heads"] * width + 4 * pages + 4 * case["seqs"]
            + rows * (2 * width * BYTES[case["dtype"]] + (4 if case["lse"] else 0)),
            "flops": 4 * seen * case["q_heads"] * width}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _ints(a):
    return torch.from_numpy(np.asarray(a)).to(DEV, torch.int32)


def _activations(shape, g, dtype):
    """Normal values with every 64th channel of the last axis larger, as projections give them."""
    x = torch.randn(shape, generator=g, device=DEV)
    x[..., ::64] *= 4.0
    return x.to(dtype)


def _fused(case, g):
    """The rows of a fused qkv projection, and the query, key and value heads in them."""
    t, hq, hk, d = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"]
    span = 2 * d if case["gated"] else d  # a gated query head is followed by its gate
    rows = _activations((t, hq * span + 2 * hk * d), g, DTYPES[case["dtype"]])
    q = rows[:, :hq * span].view(t, hq, span)[:, :, :d]
    k = rows[:, hq * span:hq * span + hk * d].view(t, hk, d)
    v = rows[:, hq * span + hk * d:].view(t, hk, d)
    return q, k, v


def prepare(case, seed):
    g = _gen(seed)
    state = {"case": case}
    op = case["op"]
    if op == "table":
        cached, new = _table_lens(case)
        page, n = case["page"], case["requests"]
        held, all_ = _ceil(cached, page), _ceil(cached + new, page)
        columns = int(all_.max()) + 3
        ids = torch.randperm(int(all_.sum()) + 64, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
        at = torch.from_numpy(np.cumsum(held) - held).to(DEV)
        col = torch.arange(columns, device=DEV)
        inside = col[None, :] < torch.from_numpy(held).to(DEV)[:, None]
        table = torch.where(inside, ids[(at[:, None] + col[None, :]).clamp(max=ids.numel() - 1)], torch.full((), -1, dtype=torch.int32, device=DEV))
        used = 5  # entries of the free list that earlier steps took
        wanted = int((all_ - held).sum())
        free = ids[int(held.sum()):][:max(used, used + wanted - case["short"])].contiguous()
        tokens = int(new.sum()) + 9  # a few places behind the last token, as in a padded batch
        i32 = dict(dtype=torch.int32, device=DEV)
        state.update(cached=_ints(cached), new=_ints(new), free=free, used=_ints([used]), table=table.contiguous(), tokens=tokens,
                     slots=torch.empty(tokens, **i32), lens=torch.empty(n, **i32), starts=torch.empty(n + 1, **i32),
                     first=torch.empty(n, **i32), used_out=torch.empty(1, **i32))
        return state
    if op == "rope":
        q, k, _ = _fused(case, g)
        t, pairs = case["tokens"], case["rot"] // 2
        base = int(torch.randint(0, case["far"], (1,), generator=g, device=DEV))
        i = torch.arange(t, device=DEV)
        picture = (i // 1024) % 2 == 1  # text and pictures of 32 x 32 patches in turn
        time = torch.where(picture, base + i // 1024 * 1024, base + i)
        pos = torch.stack([time, torch.where(picture, time + i % 1024 // 32, time), torch.where(picture, time + i % 32, time)])
        axes = torch.arange(pairs, device=DEV)
        axes = axes % 3 if case["turns"] else axes * 3 // pairs
        inv_freq = (1e7 ** (-torch.arange(pairs, device=DEV, dtype=torch.float64) / pairs)).float()
        state.update(q=q, k=k, positions=pos.to(torch.int32), axes=axes.to(torch.int32), inv_freq=inv_freq,
                     q_out=torch.empty(q.shape, dtype=q.dtype, device=DEV), k_out=torch.empty(k.shape, dtype=k.dtype, device=DEV))
        return state
    hk, d, page = case["kv_heads"], case["head_dim"], case["page"]
    if op == "write":
        _, k, v = _fused(case, g)
        t, pad = case["tokens"], case["pad"]
        i = torch.arange(t, device=DEV)
        pages = (t // page + 2 if case["prompt"] else t) + 8
        ids = torch.randperm(pages, generator=g, device=DEV)
        if case["prompt"]:  # consecutive places, the first page already begun
            at = i + page // 3
            slots = ids[at // page] * page + at % page
        else:  # a place in a page of its own for each
            slots = ids[i] * page + torch.randint(0, page, (t,), generator=g, device=DEV)
        slots[t - pad:] = -1
        # one page more than the cache has, where the plain form sends the tokens without a place
        old = torch.randint(0, 120, (2, pages + 1, hk, page, d), generator=g, device=DEV, dtype=torch.uint8)
        scale = E4M3_MAX / torch.stack([k.abs().max(), v.abs().max()]).float() * 1.25  # a calibration that a few values pass
        state.update(k=k, v=v, slots=slots.to(torch.int32), k_cache=old[0], v_cache=old[1], pages=pages, k_scale=scale[0:1].clone(), v_scale=scale[1:2].clone())
        return state
    lens = _attend_lens(case)
    held = _ceil(lens, page)
    pages = int(held.sum()) + 3
    columns = int(held.max()) + 2
    ids = torch.randperm(pages, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    col = torch.arange(columns, device=DEV)
    at = torch.from_numpy(np.cumsum(held) - held).to(DEV)[:, None] + col[None, :]
    inside = col[None, :] < torch.from_numpy(held).to(DEV)[:, None]
    table = torch.where(inside, ids[at.clamp(max=pages - 1)], torch.full((), -1, dtype=torch.int32, device=DEV)).contiguous()
    caches, scales = [], []
    for _ in range(2):
        x = _activations((pages, hk, page, d), g, torch.float32)
        s = E4M3_MAX / x.abs().max()
        caches.append(x.mul_(s).to(torch.float8_e4m3fn).view(torch.uint8))
        scales.append(s.reshape(1))
        del x
    # queries whose scores spread enough for a few tokens to carry a row
    q = (2.0 * torch.randn((case["seqs"], case["q_heads"], d), generator=g, device=DEV)).to(DTYPES[case["dtype"]])
    state.update(q=q, k_cache=caches[0], v_cache=caches[1], k_scale=scales[0], v_scale=scales[1], table=table, lens=_ints(lens),
                 pages=pages, longest=int(lens.max()), scale=d ** -0.5, out=torch.empty_like(q),
                 lse=torch.empty((case["seqs"], case["q_heads"]), device=DEV) if case["lse"] else None,
                 workspace=torch.empty(WORKSPACE, dtype=torch.uint8, device=DEV))
    return state


def run(state):
    return {"table": _table, "rope": _rope, "write": _write, "attend": _attend}[state["case"]["op"]](state)


def _table(s):
    page, tokens = s["case"]["page"], s["tokens"]
    if own:
        import nvfp4_w4a4_block_quantize_amd as nv

        nv.nvfp4_kv_block_table(s["cached"], s["new"], page, s["free"], s["used"], s["table"], s["slots"], seq_lens=s["lens"],
                                token_starts=s["starts"], first_pages=s["first"], free_used_out=s["used_out"])
        return {"slots": s["slots"], "lens": s["lens"], "starts": s["starts"], "first": s["first"], "used": s["used_out"], "table": s["table"]}
    cached, new, table = s["cached"].long(), s["new"].long(), s["table"]
    used, free, columns = s["used"].long(), s["free"], s["table"].shape[1]
    ends = new.clamp(min=0).cumsum(0)
    held, all_ = (cached + page - 1) // page, (cached + new + page - 1) // page
    fits = (cached >= 0) & (new >= 0) & (all_ <= columns) & (ends <= tokens)
    need = torch.where(fits, all_ - held, 0)
    upto = used + need.cumsum(0)
    served = fits & ((need == 0) | (upto <= free.numel()))
    first = torch.where(served, (upto - need).clamp(max=free.numel()), -1)
    lens = torch.where(served, cached + new, cached)
    used_out = used + torch.where(served, need, 0).sum()
    starts = torch.cat([torch.zeros_like(used), ends]).clamp(max=tokens)
    # the fresh pages, into the rows of the table
    last = max(free.numel() - 1, 0)
    col = torch.arange(columns, device=DEV)[None, :]
    fresh = served[:, None] & (col >= held[:, None]) & (col < all_[:, None])
    table = torch.where(fresh, free[(first[:, None] + col - held[:, None]).clamp(0, last)], table)
    # a slot for each token
    t = torch.arange(tokens, device=DEV)
    r = torch.searchsorted(ends, t, right=True).clamp(max=cached.numel() - 1)
    at = cached[r] + t - starts[r]
    slot = table[r, (at // page).clamp(0, columns - 1)].long() * page + at % page
    slot = torch.where(served[r] & (t < ends[-1]), slot, -1)
    i32 = torch.int32
    return {"slots": slot.to(i32), "lens": lens.to(i32), "starts": starts.to(i32), "first": first.to(i32), "used": used_out.to(i32), "table": table}


def _turned(x, cos, sin, adjacent):
    h = cos.shape[-1]
    y = x.float()
    a, b = (y[..., 0:2 * h:2], y[..., 1:2 * h:2]) if adjacent else (y[..., :h], y[..., h:2 * h])
    u, w = a * cos - b * sin, b * cos + a * sin
    front = torch.stack([u, w], -1).flatten(-2) if adjacent else torch.cat([u, w], -1)
    return torch.cat([front, y[..., 2 * h:]], -1).to(x.dtype)


def _rope(s):
    adjacent = s["case"]["adjacent"]
    if own:
        import nvfp4_w4a4_block_quantize_amd as nv

        nv.nvfp4_rope(s["q"], s["k"], s["positions"], s["inv_freq"], s["axes"], adjacent=adjacent, q_out=s["q_out"], k_out=s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    # far positions times a frequency: the angle needs more than 32 bits
    angle = (s["positions"].double()[s["axes"].long()] * s["inv_freq"].double()[:, None]).t()[:, None, :]
    cos, sin = angle.cos().float(), angle.sin().float()
    return {"q": _turned(s["q"], cos, sin, adjacent), "k": _turned(s["k"], cos, sin, adjacent)}


def _write(s):
    page, pages = s["case"]["page"], s["pages"]
    if own:
        import nvfp4_w4a4_block_quantize_amd as nv

        k_cache, v_cache = s["k_cache"][:pages], s["v_cache"][:pages]
        nv.nvfp4_kv_cache_write(s["k"], s["v"], s["k_scale"], s["v_scale"], s["slots"], k_cache, v_cache)
        return {"k": k_cache.view(torch.float8_e4m3fn), "v": v_cache.view(torch.float8_e4m3fn)}
    slot = s["slots"].long()
    slot = torch.where((slot >= 0) & (slot < pages * page), slot, pages * page)
    out = {}
    for name, x, scale, cache in (("k", s["k"], s["k_scale"], s["k_cache"]), ("v", s["v"], s["v_scale"], s["v_cache"])):
        code = (x.float() * scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        cache[slot // page, :, slot % page] = code
        out[name] = cache[:pages].view(torch.float8_e4m3fn)
    return out


def _attend(s):
    c = s["case"]
    if own:
        import nvfp4_w4a4_block_quantize_amd as nv

        nv.nvfp4_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["lens"],
                                 softmax_scale=s["scale"], window=c["window"], out=s["out"], lse=s["lse"], workspace=s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    n, hk, d, page = c["seqs"], c["kv_heads"], c["head_dim"], c["page"]
    at = torch.arange(s["longest"], device=DEV)
    lens = s["lens"].long()[:, None]
    seen = at < lens
    if c["window"]:
        seen = seen & (at >= lens - c["window"])
    ids = s["table"][:, at // page].long()
    seen = seen & (ids >= 0) & (ids < s["pages"])
    ids = ids.clamp(0, s["pages"] - 1)
    k = s["k_cache"][ids, :, at % page].view(torch.float8_e4m3fn).float() / s["k_scale"]  # [seqs, tokens, heads, dim]
    scores = torch.matmul(s["q"].float().view(n, hk, -1, d), k.permute(0, 2, 3, 1).contiguous()) * s["scale"]
    del k
    scores = scores.masked_fill(~seen[:, None, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    v = s["v_cache"][ids, :, at % page].view(torch.float8_e4m3fn).float() / s["v_scale"]
    out = torch.matmul(p, v.permute(0, 2, 1, 3).contiguous()) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total)).view(n, -1) if c["lse"] else None
    return {"out": out.view(n, -1, d).to(s["q"].dtype), "lse": lse}


def _e4m3_values(codes):
    """What E4M3 bytes stand for, from the bits."""
    b = torch.arange(256, dtype=torch.float64, device=DEV)
    e, m = (b // 8) % 16, b % 8
    value = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e - 10))
    value = torch.where(b >= 128, -value, value)
    return value[codes.long()]


def exact(case, seed):
    op = case["op"]
    if op == "table":
        return None
    s = prepare(case, seed)
    if op == "rope":
        angle = (s["positions"].double() * 1.0)[s["axes"].long()].t() * s["inv_freq"].double()
        turn = torch.polar(torch.ones_like(angle), angle)[:, None, :]
        out = {}
        for name in ("q", "k"):
            x, h = s[name].double().clone(), turn.shape[-1]
            at = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if case["adjacent"] else (slice(0, h), slice(h, 2 * h))
            z = torch.complex(x[..., at[0]].contiguous(), x[..., at[1]].contiguous()) * turn
            x[..., at[0]], x[..., at[1]] = z.real, z.imag
            out[name] = x
        return out
    if op == "write":
        slot = s["slots"].long()
        there = ((slot >= 0) & (slot < s["pages"] * case["page"])).nonzero()[:, 0]
        slot = slot[there]
        out = {}
        for name in ("k", "v"):
            cache = _e4m3_values(s[name + "_cache"][:s["pages"]])
            y = (s[name][there].double() * s[name + "_scale"].double()).float().double()  # one rounding to 32 bits belongs to the rule
            size = y.abs().clamp(max=E4M3_MAX)
            step = torch.exp2((torch.frexp(size)[1].double() - 1).clamp(min=-6.0) - 3)
            cache[slot // case["page"], :, slot % case["page"]] = torch.copysign(torch.round(size / step) * step, y)
            out[name] = cache
        return out
    lens, page = _attend_lens(case), case["page"]
    n, hk, d = case["seqs"], case["kv_heads"], case["head_dim"]
    q = s["q"].double().view(n, hk, -1, d)
    out, lse = torch.zeros_like(q), torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device=DEV)
    for i in range(n):
        low, high = (max(0, int(lens[i]) - case["window"]) if case["window"] else 0), int(lens[i])
        if low == high:
            continue
        ids = s["table"][i, low // page:_ceil(high, page)].long()
        rows = slice(low % page, low % page + high - low)
        for h in range(hk):
            k = _e4m3_values(s["k_cache"][ids, h]).view(-1, d)[rows] / s["k_scale"].double()
            v = _e4m3_values(s["v_cache"][ids, h]).view(-1, d)[rows] / s["v_scale"].double()
            scores = (k @ q[i, h].t().contiguous()).t() * s["scale"]
            lse[i, h] = torch.logsumexp(scores, -1)
            out[i, h] = torch.exp(scores - lse[i, h][:, None]) @ v
    return {"out": out.view(n, -1, d), "lse": lse.view(n, -1) if case["lse"] else None}
