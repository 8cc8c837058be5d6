"""The paged FP8 KV cache on the GPU, through the binding, against plain
64-bit references (tests/kv_reference.py): block tables and slot maps exactly,
cache bytes exactly, rotary positions and attention within bounds that follow
from the roundings made.  Then the four together as a server runs them."""
import sys

import numpy as np
import pytest

from oracle import nvfp4_oracle as O
from tests import kv_reference as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def log(*a):
    print("[case]", *a, flush=True)
    sys.stdout.flush()


def dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda").to(dtype)


def host(t):
    return t.float().cpu().numpy().astype(np.float64) if t.is_floating_point() else t.cpu().numpy()


# ---------------------------------------------------------------- block tables

def table_case(rng, n, page, columns, cached_most, new_most, spare):
    cached = rng.integers(0, cached_most + 1, n)
    new = rng.integers(0, new_most + 1, n)
    held = -(-cached // page)
    ids = rng.permutation(int(held.sum()) + int((-(-(cached + new) // page) - held).sum()) + 50)
    table = np.full((n, columns), -1)
    at = 0
    for r in range(n):
        h = min(int(held[r]), columns)
        table[r, :h] = ids[at:at + h]
        at += int(held[r])
    need = int((-(-(cached + new) // page) - held).sum())
    return cached, new, table, ids[at:at + max(0, need + 4 + spare)]


def check_table(nv, cached, new, page, free, used, table, tokens, in_place=False):
    want = R.block_table(cached, new, page, free, used, table, tokens)
    c, t, u = dev(cached), dev(table), dev([used])
    slots = torch.full((tokens,), 77, dtype=torch.int32, device="cuda")
    extra = dict(seq_lens=c, free_used_out=u) if in_place else {}
    lens, starts, first, used_out = nv.nvfp4_kv_block_table(c, dev(new), page, dev(free), u, t, slots, **extra)
    torch.cuda.synchronize()
    for name, got, ref in (("lens", lens, want[1]), ("starts", starts, want[2]), ("first", first, want[3]),
                           ("used", used_out, want[4]), ("table", t, want[5]), ("slots", slots, want[0])):
        assert np.array_equal(host(got).reshape(np.shape(ref)), ref), name
    return want


@pytest.mark.parametrize("n,page,cached,new,tokens_over", [
    (1, 16, 0, 1, 0), (1, 8, 0, 40000, 3), (7, 16, 100, 1, 0), (64, 48, 300, 90, 5), (1023, 16, 40, 1, 1),
    (1024, 64, 200, 3, 0), (1025, 8, 20, 9, 9), (3001, 24, 50, 5, 2), (4096, 16, 30, 1, 0), (4100, 16, 30, 4, 0),
    (33, 1024, 5000, 3000, 100)])
def test_block_table_matches_serving_one_by_one(gpu_lib, n, page, cached, new, tokens_over):
    rng = np.random.default_rng([n, page])
    c, w, table, free = table_case(rng, n, page, -(-(cached + new) // page) + 1, cached, new, 0)
    tokens = int(w.sum()) + tokens_over
    log("block table", n, page, tokens)
    want = check_table(gpu_lib, c, w, page, free, 2, table, max(1, tokens))
    assert (want[3] >= 0).all()  # everyone is served


@pytest.mark.parametrize("n,page", [(5, 16), (200, 8), (1500, 16), (4500, 32)])
@pytest.mark.parametrize("in_place", [False, True])
def test_block_table_serves_what_fits(gpu_lib, n, page, in_place):
    """Short free lists, requests past their row or past the slot map, wrong lengths, unallocated held pages."""
    rng = np.random.default_rng([n, page, 1])
    c, w, table, free = table_case(rng, n, page, 5 + 60 // page, 50, 30, 0)
    w[rng.random(n) < 0.2] = 0
    for wrong, value in ((c, -3), (w, -7), (w, 10 ** 6), (c, 2 ** 31 - 1), (w, 2 ** 31 - 1)):
        wrong[rng.integers(0, n)] = value
    table[rng.integers(0, n), 0] = -1
    total = int(np.clip(w, 0, 100).sum())
    for share in (0.0, 0.4, 1.0):
        short = free[:int(len(free) * share)]
        for tokens in (max(1, total // 2), total + 10 ** 6 + 50):
            for used in (0, 3, len(short), len(short) + 5, -2):
                log("block table, short", n, page, len(short), tokens, used)
                check_table(gpu_lib, c, w, page, short, used, table, tokens, in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("long", [0, 9, 500])
def test_block_table_of_many_short_requests(gpu_lib, in_place, long):
    """More requests than a workgroup has threads, each with a few tokens, or one of them with more."""
    rng = np.random.default_rng([7, long])
    n, page = 2501, 8
    c, w, table, free = table_case(rng, n, page, 80, 50, 3, 70)
    w[rng.random(n) < 0.3] = 0
    if long:
        w[1700] = long
    w[40], c[2222] = -1, 2 ** 31 - 1
    total = int(np.clip(w, 0, 1000).sum())
    for share in (0.5, 1.0):
        short = free[:int(len(free) * share)]
        for tokens in (total // 2, total, total + 100):
            log("block table, many", in_place, long, len(short), tokens)
            check_table(gpu_lib, c, w, page, short, 3, table, tokens, in_place)


def test_block_table_slots_past_31_bits(gpu_lib):
    page = 1024
    free = np.array([2 ** 21 - 1, 2 ** 21, 2 ** 31 - 1, -5])
    check_table(gpu_lib, np.zeros(4, int), np.full(4, page), page, free, 0, np.full((4, 2), -1), 4 * page)


def test_block_table_leaves_the_rest_of_a_wide_table(gpu_lib):
    page, wide = 16, torch.full((3, 40), 9, dtype=torch.int32, device="cuda")
    gpu_lib.nvfp4_kv_block_table(dev([0, 5, 16]), dev([17, 11, 0]), page, dev(np.arange(100, 110)), dev([1]), wide[:, 3:8],
                                 torch.empty(30, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    want = np.full((3, 40), 9)
    want[0, 3:5] = [101, 102]
    assert np.array_equal(host(wide), want)


# ------------------------------------------------------------- rotary positions

def turn(nv, x, k, positions, inv_freq, axes, adjacent, **kw):
    got = nv.nvfp4_rope(x, k, dev(positions), dev(inv_freq, torch.float32), dev(axes), adjacent=adjacent, **kw)
    torch.cuda.synchronize()
    return got


def check_rope(got, x, positions, inv_freq, axes, adjacent, dtype):
    want, slack = R.rope(host(x), positions, inv_freq, axes, adjacent)
    slack += R.HALF_STEP[dtype] * 1.01 * np.abs(want) + 2.0 ** -25 * (dtype == "f16")
    pairs = 2 * len(inv_freq)
    off = np.abs(host(got) - want)
    assert np.array_equal(host(got)[..., pairs:], host(x)[..., pairs:])
    assert (off[..., :pairs] <= slack[..., :pairs]).all(), float((off[..., :pairs] / np.maximum(slack[..., :pairs], 1e-300)).max())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("tokens,q_heads,k_heads,dim,rot", [
    (1, 1, 1, 64, 64), (1, 24, 4, 256, 64), (37, 6, 2, 128, 128), (5, 3, 1, 80, 42), (260, 1, 0, 64, 2), (9, 2, 1, 130, 130),
    (3, 5, 5, 1024, 1024), (700, 1, 1, 256, 256), (65, 40, 8, 96, 24)])
def test_rope(gpu_lib, dtype, adjacent, tokens, q_heads, k_heads, dim, rot):
    rng = np.random.default_rng([tokens, dim, rot])
    pairs = rot // 2
    positions = rng.integers(-1000, 1000000, (3, tokens))
    positions[:, 0] = [0, 2 ** 31 - 1, -2 ** 31]
    inv_freq = (1e4 ** (-np.arange(pairs) / pairs)).astype(np.float32)
    axes = np.arange(pairs) % 3
    x = dev(rng.standard_normal((tokens, q_heads, dim)), DTYPES[dtype])
    k = dev(rng.standard_normal((tokens, k_heads, dim)), DTYPES[dtype]) if k_heads else None
    log("rope", dtype, adjacent, tokens, q_heads, k_heads, dim, rot)
    q_out, k_out = turn(gpu_lib, x, k, positions, inv_freq, axes, adjacent)
    check_rope(q_out, x, positions, inv_freq, axes, adjacent, dtype)
    if k_heads:
        check_rope(k_out, k, positions, inv_freq, axes, adjacent, dtype)
    # in place: the same values, the rest untouched
    again, key = x.clone(), None if k is None else k.clone()
    turn(gpu_lib, again, key, positions, inv_freq, axes, adjacent, q_out=again, k_out=key)
    assert torch.equal(again, q_out) and (k is None or torch.equal(key, k_out))


@pytest.mark.parametrize("in_place", [False, True])
def test_rope_of_more_than_one_launch(gpu_lib, in_place):
    tokens, q_heads, k_heads = (1 << 20) + 3, 250, 7
    g = torch.Generator("cuda").manual_seed(2)
    wide = torch.randn(tokens, q_heads + k_heads, 2, generator=g, device="cuda", dtype=torch.bfloat16)
    q, k = wide[:, :q_heads], wide[:, q_heads:]
    positions = torch.randint(-2 ** 31, 2 ** 31 - 1, (2, tokens), generator=g, device="cuda", dtype=torch.int32)
    at = torch.cat([torch.arange(a, b) for a, b in ((0, 3), (1044494 - 3, 1044494 + 3), (tokens - 3, tokens))]).cuda()
    was, out = wide[at], {"q_out": q, "k_out": k} if in_place else {}
    log("rope, pieces", in_place)
    q_out, k_out = gpu_lib.nvfp4_rope(q, k, positions, dev([0.37], torch.float32), dev([1]), **out)
    torch.cuda.synchronize()
    got = torch.cat([q_out[at], k_out[at]], 1)
    check_rope(got, was, host(positions[:, at]), np.array([0.37], np.float32), np.array([1]), False, "bf16")
    if in_place:  # every token turned once: lengths stay, to two roundings
        size = lambda x: x.double().square().sum()
        before = torch.Generator("cuda").manual_seed(2)
        before = size(torch.randn(tokens, q_heads + k_heads, 2, generator=before, device="cuda", dtype=torch.bfloat16))
        assert abs(size(wide) / before - 1) <= 2.0 ** -7
    del wide, q, k, q_out, k_out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("which", ["q", "k"])
def test_rope_one_tensor_in_place(gpu_lib, adjacent, which):
    """Only q, or only k, turned in place, with parts that 16 bytes do not divide."""
    rng = np.random.default_rng(31)
    tokens, dim, rot = 67, 96, 54
    positions, axes = rng.integers(0, 4000, (1, tokens)), np.zeros(rot // 2, int)
    inv_freq = (1e4 ** (-np.arange(rot // 2) / (rot // 2))).astype(np.float32)
    q, k = (dev(rng.standard_normal((tokens, h, dim)), torch.bfloat16) for h in (6, 2))
    before = q.clone(), k.clone()
    q_out, k_out = turn(gpu_lib, q, k, positions, inv_freq, axes, adjacent, **({"q_out": q} if which == "q" else {"k_out": k}))
    check_rope(q_out, before[0], positions, inv_freq, axes, adjacent, "bf16")
    check_rope(k_out, before[1], positions, inv_freq, axes, adjacent, "bf16")
    assert (q_out is q) == (which == "q") and (k_out is k) == (which == "k")
    assert torch.equal((k, q)[which == "k"], before[which == "q"])  # the other one's input stays


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("shift", [0, 1, 2, 4])
def test_rope_in_the_rows_of_a_projection(gpu_lib, adjacent, shift):
    """Heads with their gates between them, at every alignment; what lies between stays as it was."""
    rng = np.random.default_rng(shift)
    tokens, dim = 11, 64
    rows = dev(rng.standard_normal((tokens, 4 * 2 * dim + 2 * dim + 2 * shift)), torch.bfloat16)
    before = rows.clone()
    q = rows[:, shift:shift + 512].view(tokens, 4, 128)[:, :, :dim] if shift == 0 else \
        rows[:, shift:shift + 512].unflatten(1, (4, 128))[:, :, :dim]
    k = rows[:, shift + 512:shift + 640].unflatten(1, (2, dim))
    positions = rng.integers(0, 5000, (2, tokens))
    inv_freq = (1e4 ** (-np.arange(16) / 16)).astype(np.float32)
    axes = np.repeat([0, 1], 8)
    ref_q, ref_k = q.clone(), k.clone()
    log("rope rows", adjacent, shift)
    turn(gpu_lib, q, k, positions, inv_freq, axes, adjacent, q_out=q, k_out=k)
    check_rope(q, ref_q, positions, inv_freq, axes, adjacent, "bf16")
    check_rope(k, ref_k, positions, inv_freq, axes, adjacent, "bf16")
    q.copy_(ref_q)
    k.copy_(ref_k)
    assert torch.equal(rows, before)


def test_rope_axes_outside_count_as_the_nearest(gpu_lib):
    x = dev(np.random.default_rng(0).standard_normal((4, 2, 16)), torch.float32)
    positions, inv_freq = np.arange(8).reshape(2, 4), np.ones(4, np.float32)
    a, _ = turn(gpu_lib, x, None, positions, inv_freq, [-1, 0, 1, 9], False)
    b, _ = turn(gpu_lib, x, None, positions, inv_freq, [0, 0, 1, 1], False)
    assert torch.equal(a, b)


# ------------------------------------------------------------------ cache writes

@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("tokens,heads,dim,page,gap", [
    (1, 1, 8, 8, 0), (3, 2, 64, 16, 8), (32, 4, 256, 16, 0), (1000, 8, 128, 48, 16), (257, 1, 192, 1024, 0), (50, 3, 40, 24, 8)])
def test_cache_write(gpu_lib, dtype, tokens, heads, dim, page, gap):
    rng = np.random.default_rng([tokens, dim])
    pages = tokens // page + 5
    slots = rng.permutation(pages * page)[:tokens]
    slots[rng.random(tokens) < 0.1] = -1
    slots[rng.random(tokens) < 0.05] = pages * page
    slots[-1] = 2 ** 31 - 1 if tokens > 1 else slots[-1]
    x = rng.standard_t(3, (2, tokens, heads, dim + gap)).astype(np.float32) * 8
    x[0, 0, 0, :8] = [0.0, -0.0, 1e9, -1e9, 448.0, 2.0 ** -10, 3 * 2.0 ** -10, -2.0 ** -12]
    k, v = (dev(x[i], DTYPES[dtype])[:, :, :dim] for i in (0, 1))
    old = rng.integers(0, 256, (2, pages, heads, page, dim)).astype(np.uint8)
    ck, cv = dev(old[0], torch.uint8), dev(old[1], torch.uint8)
    ks, vs = np.float32(7.3), np.float32(0.61)
    log("cache write", dtype, tokens, heads, dim, page, gap)
    gpu_lib.nvfp4_kv_cache_write(k, v, dev([ks], torch.float32), dev([vs], torch.float32), dev(slots), ck, cv)
    torch.cuda.synchronize()
    for got, src, scale, was in ((ck, k, ks, old[0]), (cv, v, vs, old[1])):
        want = was.copy()
        code = O.kv_quantize_ref(src.float().cpu().numpy().reshape(tokens, heads * dim), scale).reshape(tokens, heads, dim)
        for t in range(tokens):
            if 0 <= slots[t] < pages * page:
                want[slots[t] // page, :, slots[t] % page] = code[t]
        assert np.array_equal(host(got), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("tokens,heads,dim,page", [(17001, 8, 128, 48), (4099, 16, 256, 8), (120011, 3, 48, 256)])
@pytest.mark.parametrize("strided", [False, True])
def test_cache_write_of_long_prompts(gpu_lib, dtype, tokens, heads, dim, page, strided):
    """Rows that do not fit the caches, alone or inside wider rows, against torch's cast of the same products."""
    g = torch.Generator("cuda").manual_seed(tokens)
    wide = torch.randn(tokens, heads * (3 if strided else 1), dim, generator=g, device="cuda").mul_(60).to(DTYPES[dtype])
    k, v = (wide[:, heads:2 * heads], wide[:, 2 * heads:]) if strided else (wide, wide.flip(0).contiguous())
    pages = tokens // page + 3
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:tokens].to(torch.int32)
    slots[::97] = -1
    scales = dev([2.3, 9.7], torch.float32)
    ck, cv = (torch.full((pages, heads, page, dim), 0x55, dtype=torch.uint8, device="cuda") for _ in range(2))
    log("cache write, long", dtype, tokens, heads, dim, page, strided)
    gpu_lib.nvfp4_kv_cache_write(k, v, scales[:1], scales[1:], slots, ck, cv)
    torch.cuda.synchronize()
    kept = slots >= 0
    at = slots[kept].long()
    for got, x, scale in ((ck, k, scales[0]), (cv, v, scales[1])):
        want = torch.full_like(got, 0x55)
        code = (x[kept].float() * scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        want[at // page, :, at % page] = code
        assert torch.equal(got, want)


@pytest.mark.parametrize("tokens,heads,dim,strided", [((1 << 18) + 5, 1024, 8, False), ((1 << 19) + 3, 32, 256, True)])
def test_cache_write_of_more_than_one_launch(gpu_lib, tokens, heads, dim, strided):
    g = torch.Generator("cuda").manual_seed(tokens)
    wide = torch.randn(tokens, heads * (2 if strided else 1), dim, generator=g, device="cuda", dtype=torch.bfloat16)
    k = wide[:, -heads:]
    at = np.unique(np.concatenate([[0, 1, tokens - 1], (1 << 18) + np.arange(-3, 5), (1 << 19) + np.arange(-2, 3)]))
    at = at[at < tokens]
    slots = torch.full((tokens,), -1, dtype=torch.int32, device="cuda")
    slots[torch.from_numpy(at).cuda()] = torch.arange(len(at), dtype=torch.int32, device="cuda") + 1
    scales = dev([100.0, 200.0], torch.float32)
    ck, cv = (torch.full((4, heads, 8, dim), 0x55, dtype=torch.uint8, device="cuda") for _ in range(2))
    log("cache write, pieces", tokens, heads, dim, strided)
    gpu_lib.nvfp4_kv_cache_write(k, k, scales[:1], scales[1:], slots, ck, cv)
    torch.cuda.synchronize()
    for got, scale in ((ck, 100.0), (cv, 200.0)):
        want = torch.full_like(got, 0x55)
        code = (k[torch.from_numpy(at).cuda()].float() * scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        slot = torch.arange(len(at), device="cuda") + 1
        want[slot // 8, :, slot % 8] = code
        assert torch.equal(got, want)
    del wide, k
    torch.cuda.empty_cache()


# --------------------------------------------------------------------- attention

def attention_case(rng, lens, heads, kv_heads, dim, page, dtype, sharpen=2.0, columns=None):
    """Pages in random order; whatever belongs to no token holds NaN bytes."""
    n = len(lens)
    held = [-(-max(int(x), 0) // page) for x in lens]
    columns = columns or max(held) + 1
    pages = sum(held) + 2
    ids, table = list(rng.permutation(pages)), np.full((n, columns), -1)
    k, v = (np.full((pages, kv_heads, page, dim), 0x7F, np.uint8) for _ in range(2))
    for r in range(n):
        for j in range(min(held[r], columns)):
            table[r, j] = ids.pop()
            rows = min(page, int(lens[r]) - j * page)
            for cache in (k, v):
                x = rng.standard_normal((kv_heads, rows, dim)) * np.where(np.arange(dim) % 64 == 5, 5, 1)
                cache[table[r, j], :, :rows] = O.kv_quantize_ref(x.reshape(-1, dim).astype(np.float32), np.float32(20.0)).reshape(x.shape)
    q = dev(rng.standard_normal((n, heads, dim)) * sharpen, DTYPES[dtype])
    return q, k, v, table


def check_attention(nv, q, k, v, table, lens, window=0, scale=None, dtype="bf16", out=None, workspace=None, ref=None):
    n, heads, dim = q.shape
    scale = dim ** -0.5 if scale is None else scale
    lse = torch.full((n, heads), 5.0, device="cuda")
    s = dev([20.0], torch.float32)
    if isinstance(k, np.ndarray):
        k, v = dev(k, torch.uint8), dev(v, torch.uint8)
    got = nv.nvfp4_paged_attention(q, k, v, s, s, dev(table), dev(lens), softmax_scale=scale, window=window, out=out, lse=lse,
                                   workspace=workspace)
    torch.cuda.synchronize()
    if ref is None:
        ref = R.attention(host(q), host(k), host(v), 20.0, 20.0, table, lens, np.float32(scale), window, k.shape[0])
    want, want_lse, reach, sharp = ref
    b_out, b_lse = R.attention_bounds(want, want_lse, reach, sharp, lens, dtype)
    off = np.abs(host(got) - want)
    assert (off <= b_out).all(), ("out", float((off / np.maximum(b_out, 1e-300)).max()))
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(host(lse)), empty)
    assert (host(got)[empty] == 0).all()
    off = np.abs(np.where(empty, 0, host(lse)) - np.where(empty, 0, want_lse))
    assert (off <= b_lse).all(), ("lse", float((off / b_lse).max()))
    return got, lse, ref


SHORT = [1, 0, 2, 7, 8, 9, 31, 32, 33, 63, 65, 127, 128, 129, 255, 257, -4]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("heads,kv_heads,page", [(1, 1, 8), (6, 1, 24), (16, 1, 16), (10, 2, 1024), (34, 2, 48), (40, 1, 64)])
def test_attention_short_lengths(gpu_lib, dtype, dim, heads, kv_heads, page):
    rng = np.random.default_rng([dim, heads, page])
    log("attention short", dtype, dim, heads, kv_heads, page)
    q, k, v, table = attention_case(rng, SHORT, heads, kv_heads, dim, page, dtype)
    check_attention(gpu_lib, q, k, v, table, SHORT, dtype=dtype)


@pytest.mark.parametrize("dtype,dim", [("bf16", 256), ("f16", 128), ("f32", 64), ("bf16", 64), ("f32", 256)])
@pytest.mark.parametrize("lens", [[40000], [3000, 1, 0, 9000, 128, 129, 0, 0, 5000], [700] * 40])
def test_attention_split_over_workers(gpu_lib, dtype, dim, lens):
    """Items spread over many workgroups, and workgroups spread over many items."""
    rng = np.random.default_rng([dim, len(lens)])
    log("attention split", dtype, dim, lens[:4])
    q, k, v, table = attention_case(rng, lens, 6, 2, dim, 16, dtype)
    check_attention(gpu_lib, q, k, v, table, lens, dtype=dtype)


@pytest.mark.parametrize("n,live", [(70, [0, 69]), (300, [5, 6, 250]), (1100, [0, 1, 600, 1099]), (2500, [2499]), (900, range(900)), (400, [])])
def test_attention_batches_with_few_live_rows(gpu_lib, n, live):
    """Long batches, most of whose rows are empty; and one of very many short sequences."""
    rng = np.random.default_rng(n)
    lens = np.zeros(n, int)
    lens[list(live)] = rng.integers(1, 900 if len(live) < 10 else 60, len(live))
    lens[::7] = np.where(lens[::7] == 0, -3, lens[::7])
    log("attention live rows", n, len(live))
    q, k, v, table = attention_case(rng, lens, 4, 2, 64, 16, "bf16")
    check_attention(gpu_lib, q, k, v, table, lens)


@pytest.mark.parametrize("dtype,dim,heads,kv_heads,page", [
    ("f32", 64, 6, 1, 8), ("bf16", 256, 10, 2, 24), ("f16", 128, 34, 2, 16), ("bf16", 192, 40, 1, 1024), ("f16", 256, 1, 1, 48)])
@pytest.mark.parametrize("window", [0, 40])
def test_attention_short_lengths_in_wide_tables(gpu_lib, dtype, dim, heads, kv_heads, page, window):
    """Tables with room for sequences that would be split."""
    rng = np.random.default_rng([dim, heads, page, 1])
    log("attention wide tables", dtype, dim, heads, kv_heads, page, window)
    q, k, v, table = attention_case(rng, SHORT, heads, kv_heads, dim, page, dtype, columns=20000 // page)
    check_attention(gpu_lib, q, k, v, table, SHORT, window=window, dtype=dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("heads,kv_heads", [(8, 2), (40, 2)])
def test_attention_of_many_short_sequences(gpu_lib, dtype, dim, heads, kv_heads):
    """More items than CUs, each short enough for a workgroup of its own."""
    rng = np.random.default_rng([dim, heads, 3])
    lens = rng.integers(-5, 140, 140)
    log("attention many short", dtype, dim, heads)
    q, k, v, table = attention_case(rng, lens, heads, kv_heads, dim, 16, dtype)
    check_attention(gpu_lib, q, k, v, table, lens, dtype=dtype)
    check_attention(gpu_lib, q, k, v, table, lens, window=33, dtype=dtype)


@pytest.mark.parametrize("n,live,by", [(1100, [0, 1, 600, 1099], 1), (2500, [2499], 7), (900, range(900), 3), (400, [], 1)])
def test_attention_batches_with_few_live_rows_in_wide_tables(gpu_lib, n, live, by):
    rng = np.random.default_rng([n, 1])
    lens = np.zeros(n, int)
    lens[list(live)] = rng.integers(1, 900 if len(live) < 10 else 60, len(live))
    lens[::by] = np.where(lens[::by] == 0, -3, lens[::by])
    log("attention live rows, wide tables", n, len(live))
    q, k, v, table = attention_case(rng, lens, 4, 2, 64, 16, "bf16", columns=600)
    check_attention(gpu_lib, q, k, v, table, lens)


@pytest.mark.parametrize("most,n,kv_heads", [(1200, 130, 8), (2500, 128, 4), (2600, 128, 4), (760, 3, 1), (770, 3, 1)])
@pytest.mark.parametrize("window", [0, 500])
def test_attention_of_items_that_may_be_split_or_not(gpu_lib, most, n, kv_heads, window):
    """Sizes to both sides of where items stop being split; the lengths stop at the table's end."""
    rng = np.random.default_rng([most, n])
    lens = rng.integers(0, 200, n)
    lens[:3] = [most, most - 1, most + 7]
    log("attention split or not", most, n, kv_heads, window)
    columns = -(-most // 16)
    q, k, v, table = attention_case(rng, lens, 2 * kv_heads, kv_heads, 128, 16, "bf16", columns=columns)
    check_attention(gpu_lib, q, k, v, table, np.minimum(lens, columns * 16), window=window)


def test_attention_of_a_million_sequences(gpu_lib):
    """More (sequence, KV head) items than one launch has workgroups."""
    n = (1 << 20) + 7
    g = torch.Generator("cuda").manual_seed(1)
    q = torch.randn(n, 1, 64, generator=g, device="cuda").to(torch.bfloat16)
    cache = torch.randint(0, 0x7F, (50, 1, 8, 64), generator=g, device="cuda", dtype=torch.uint8)
    table = torch.randint(0, 50, (n, 1), generator=g, device="cuda", dtype=torch.int32)
    lens = torch.randint(0, 2, (n,), generator=g, device="cuda", dtype=torch.int32)
    s = dev([20.0], torch.float32)
    log("attention, a million sequences")
    lse = torch.empty(n, 1, device="cuda")
    got = gpu_lib.nvfp4_paged_attention(q, cache, cache.clone(), s, s, table, lens, lse=lse)
    torch.cuda.synchronize()
    # one token: its value itself, which has 4 bits (a division by 20 and the output's rounding)
    want = torch.where((lens > 0)[:, None], cache.view(torch.float8_e4m3fn).double()[table[:, 0].long(), 0, 0] / 20, 0.0)
    assert ((got[:, 0].double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -20)).all()
    assert torch.equal(torch.isneginf(lse[:, 0]), lens == 0)


def test_attention_of_scales_next_to_nothing(gpu_lib):
    """All tokens weigh the same, and those behind the last one still nothing."""
    rng = np.random.default_rng(17)
    lens = [1, 45, 300, 0]
    for dtype in ("bf16", "f32"):
        q, k, v, table = attention_case(rng, lens, 4, 2, 128, 16, dtype)
        for scale in (1e-40, 1.5e-45):
            log("attention scale", dtype, scale)
            check_attention(gpu_lib, q, k, v, table, lens, scale=scale, dtype=dtype)


@pytest.mark.parametrize("window", [1, 5, 8, 100, 128, 1000, 2 ** 40, 2 ** 63 - 1])
def test_attention_window(gpu_lib, window):
    lens = [1, 3, 99, 100, 101, 900, 3001, 0]
    rng = np.random.default_rng(window)
    log("attention window", window)
    q, k, v, table = attention_case(rng, lens, 8, 2, 128, 24, "bf16")
    check_attention(gpu_lib, q, k, v, table, lens, window=window)
    # pages before the window may be gone
    for r, n in enumerate(lens):
        table[r, :max(0, n - window) // 24] = -1
    check_attention(gpu_lib, q, k, v, table, lens, window=window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_wrong_pages_and_lengths(gpu_lib, dtype):
    """Tokens of pages outside the cache are not seen; lengths stop at the table's last column."""
    rng = np.random.default_rng(7)
    lens = [200, 64, 1000, 33]
    q, k, v, table = attention_case(rng, lens, 4, 2, 128, 16, dtype)
    table[0, 3], table[0, 7], table[1, :], table[2, 5], table[2, 62] = -1, k.shape[0], 2 ** 31 - 1, -2 ** 31, 10 ** 6
    log("attention wrong pages", dtype)
    check_attention(gpu_lib, q, k, v, table, lens, dtype=dtype)
    most = table.shape[1] * 16
    check_attention(gpu_lib, q[2:3], k, v, table[2:3, :40], [2 ** 31 - 1], dtype=dtype,
                    ref=R.attention(host(q[2:3]), k, v, 20.0, 20.0, table[2:3, :40], [640], np.float32(128 ** -0.5), 0, k.shape[0]))
    assert most > 640


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_attention_one_token_carries_all_or_none_does(gpu_lib, dtype):
    rng = np.random.default_rng(3)
    lens = [2000, 17]
    for sharpen in (0.0, 40.0):  # equal weights; scores of hundreds
        log("attention sharpen", dtype, sharpen)
        q, k, v, table = attention_case(rng, lens, 4, 1, 64, 32, dtype, sharpen)
        check_attention(gpu_lib, q, k, v, table, lens, dtype=dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_attention_far_below_the_largest(gpu_lib, dtype):
    """One token takes nearly all; what thousands of small probabilities add is kept."""
    n, dim, page = 8000, 64, 16
    rng = np.random.default_rng(5)
    q, k, v, table = attention_case(rng, [n], 2, 1, dim, page, dtype, 0.0)
    q[:] = 0
    q[:, :, 0] = 1
    k[:, :, :, 0] = 0
    v[:] = O.kv_quantize_ref(np.full((1, 1), 1.0, np.float32), np.float32(20.0))[0, 0]
    k[table[0, 100], 0, 3, 0] = 0x7E  # 448 / 20 = 22.4 at scale 0.5: e^11.2 against 1
    v[table[0, 100], 0, 3] = 0
    log("attention far below", dtype)
    check_attention(gpu_lib, q, k, v, table, [n], scale=0.5, dtype=dtype)


def test_attention_strided_heads_and_rows_left_alone(gpu_lib):
    rng = np.random.default_rng(9)
    lens = [300, 0, 77]
    q, k, v, table = attention_case(rng, lens, 4, 2, 128, 16, "bf16")
    gated = torch.randn((3, 4, 2, 128), device="cuda").to(torch.bfloat16)
    gated[:, :, 0] = q
    room = torch.full((3, 4, 3, 128), 7.0, device="cuda").to(torch.bfloat16)
    wide = torch.full((3, table.shape[1] + 9), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = dev(table)
    _, _, ref = check_attention(gpu_lib, gated[:, :, 0], k, v, table, lens, out=room[:, :, 1])
    assert (room[:, :, 0] == 7).all() and (room[:, :, 2] == 7).all()
    s = dev([20.0], torch.float32)
    got = gpu_lib.nvfp4_paged_attention(q, dev(k, torch.uint8), dev(v, torch.uint8), s, s, wide[:, :table.shape[1]], dev(lens))
    assert torch.equal(got, room[:, :, 1])


def test_attention_cache_past_32_bits(gpu_lib):
    """Pages that lie more than 4 GiB into each cache."""
    rng = np.random.default_rng(11)
    heads, dim, page = 4, 256, 64
    lens = [500, 70]
    q, k, v, table = attention_case(rng, lens, 8, heads, dim, page, "bf16")
    page_bytes = heads * dim * page
    pages = (9 << 29) // page_bytes + 50
    far = np.where(table >= 0, table + pages - k.shape[0], -1)
    log("attention far pages", pages * page_bytes)
    big = [torch.empty((pages, heads, page, dim), dtype=torch.uint8, device="cuda") for _ in range(2)]
    # through the cache write: the tokens' own values, in slots past 2^32 bytes
    s = dev([20.0], torch.float32)
    for r, n in enumerate(lens):
        at = np.arange(n)
        rows = [dev(R.E4M3[c[table[r, at // page], :, at % page]] / 20.0, torch.float32) for c in (k, v)]
        gpu_lib.nvfp4_kv_cache_write(*rows, s, s, dev(far[r, at // page] * page + at % page), *big)
    ref = R.attention(host(q), k, v, 20.0, 20.0, table, lens, np.float32(dim ** -0.5), 0, k.shape[0])
    check_attention(gpu_lib, q, big[0], big[1], far, lens, ref=ref)
    del big
    torch.cuda.empty_cache()


def test_attention_is_the_same_whatever_the_workspace_holds(gpu_lib):
    rng = np.random.default_rng(13)
    lens = [5000, 40, 0, 20000]
    q, k, v, table = attention_case(rng, lens, 12, 2, 128, 16, "f16")
    size = gpu_lib.nvfp4_paged_attention_workspace(12, 2, 128)
    first = None
    for fill in (0, 0xFF, 0x7F):
        workspace = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        got, lse, _ = check_attention(gpu_lib, q, k, v, table, lens, dtype="f16", workspace=workspace)
        if first is None:
            first = got.clone(), lse.clone()
        assert torch.equal(got, first[0]) and torch.equal(lse, first[1])


# -------------------------------------------------- streams, graphs, all together

def test_graphs_that_share_a_workspace_follow_the_lengths(gpu_lib):
    nv, rng = gpu_lib, np.random.default_rng(17)
    most = [3000, 500, 64]
    cases = []
    for dim, heads in ((128, 8), (256, 6)):
        q, k, v, table = attention_case(rng, most, heads, 2, dim, 16, "bf16")
        cases.append((q, dev(k, torch.uint8), dev(v, torch.uint8), dev(table), torch.zeros(3, dtype=torch.int32, device="cuda"),
                      torch.empty_like(q)))
    workspace = torch.empty(nv.nvfp4_paged_attention_workspace(8, 2, 256), dtype=torch.uint8, device="cuda")
    s = dev([20.0], torch.float32)

    def step(c):
        nv.nvfp4_paged_attention(c[0], c[1], c[2], s, s, c[3], c[4], out=c[5], workspace=workspace)

    graphs = []
    for c in cases:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(c)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(c)
        graphs.append(g)
    for lens in ([3000, 500, 64], [1, 0, 64], [2999, 129, 0], [0, 0, 0], [128, 500, 7]):
        log("graph replay", lens)
        for c in cases:
            c[4].copy_(dev(lens))
            c[5].fill_(3.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        replayed = [c[5].clone() for c in cases]
        for c, got in zip(cases, replayed):
            step(c)  # eager work between replays
            torch.cuda.synchronize()
            assert torch.equal(c[5], got)
            assert not (c[5] == 3.0).any()


def test_two_streams_with_a_workspace_each(gpu_lib):
    nv, rng = gpu_lib, np.random.default_rng(19)
    work = []
    for lens, dim in (([9000, 30], 128), ([400] * 20, 256)):
        q, k, v, table = attention_case(rng, lens, 8, 2, dim, 16, "bf16")
        args = (q, dev(k, torch.uint8), dev(v, torch.uint8), dev([20.0], torch.float32), dev([20.0], torch.float32), dev(table), dev(lens))
        work.append((args, nv.nvfp4_paged_attention(*args).clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for turn_ in range(4):
        log("two streams", turn_)
        got = []
        for args, _, stream in work:
            with torch.cuda.stream(stream):
                got.append([nv.nvfp4_paged_attention(*args, stream=stream) for _ in range(4)])
        torch.cuda.synchronize()
        for outs, (_, want, _) in zip(got, work):
            assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("captured", [False, True])
def test_prompt_and_decode_steps_together(gpu_lib, captured):
    """Prompts, then decode steps: tables, positions, cache writes and attention on one cache, each step's result
    against the reference on the values that were cached.  The decode step also as a captured graph whose lengths
    and tables live on the device."""
    nv, rng = gpu_lib, np.random.default_rng(23)
    heads, kv_heads, dim, rot, page, n = 8, 2, 128, 32, 16, 5
    prompts = np.array([30, 1, 100, 0, 17])
    steps = 20
    pages, columns = 40, 10
    i32 = dict(dtype=torch.int32, device="cuda")
    ck, cv = (torch.full((pages, kv_heads, page, dim), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
    table, lens, used = torch.full((n, columns), -1, **i32), torch.zeros(n, **i32), torch.zeros(1, **i32)
    free = dev(rng.permutation(pages))
    ks, vs = dev([30.0], torch.float32), dev([25.0], torch.float32)
    inv_freq = dev((1e4 ** (-np.arange(rot // 2) / (rot // 2))).astype(np.float32), torch.float32)
    axes = dev(np.arange(rot // 2) % 3)
    workspace = torch.empty(nv.nvfp4_paged_attention_workspace(heads, kv_heads, dim), dtype=torch.uint8, device="cuda")
    kept = [[[], []] for _ in range(n)]  # the bytes that each sequence should hold

    def rows(tokens):
        x = dev(rng.standard_normal((tokens, (heads + 2 * kv_heads) * dim)), torch.bfloat16)
        return x, x[:, :heads * dim].view(tokens, heads, dim), x[:, heads * dim:(heads + kv_heads) * dim].view(tokens, kv_heads, dim), \
            x[:, (heads + kv_heads) * dim:].view(tokens, kv_heads, dim)

    def keep(k_turned, v, slots, new):
        at = 0
        for r, m in enumerate(new):
            for t in range(at, at + m):
                if host(slots)[t] >= 0:
                    for which, x, s in ((0, k_turned, 30.0), (1, v, 25.0)):
                        kept[r][which].append(O.kv_quantize_ref(x[t].float().cpu().numpy(), np.float32(s)))
            at += m

    # the prompts: all their tokens at once, the slot map padded
    total = int(prompts.sum())
    x, q, k, v = rows(total + 6)
    slots = torch.empty(total + 6, **i32)
    nv.nvfp4_kv_block_table(lens, dev(prompts), page, free, used, table, slots, seq_lens=lens, free_used_out=used)
    at = np.concatenate([np.arange(p) for p in prompts] + [np.zeros(6, int)])
    positions = dev(np.stack([at, at // 3, at % 7]))
    nv.nvfp4_rope(q, k, positions, inv_freq, axes, q_out=q, k_out=k)
    nv.nvfp4_kv_cache_write(k, v, ks, vs, slots, ck, cv)
    torch.cuda.synchronize()
    keep(k, v, slots, prompts)
    assert host(lens).tolist() == prompts.tolist()

    one, slots = torch.ones(n, **i32), torch.empty(n, **i32)
    x, q, k, v = rows(n)
    positions = torch.zeros((3, n), **i32)
    out = torch.empty((n, heads, dim), dtype=torch.bfloat16, device="cuda")

    def step():
        positions[:] = lens
        nv.nvfp4_kv_block_table(lens, one, page, free, used, table, slots, seq_lens=lens, free_used_out=used)
        nv.nvfp4_rope(q, k, positions, inv_freq, axes, q_out=q, k_out=k)
        nv.nvfp4_kv_cache_write(k, v, ks, vs, slots, ck, cv)
        nv.nvfp4_paged_attention(q, ck, cv, ks, vs, table, lens, out=out, workspace=workspace)

    graph = None
    if captured:
        state = [t.clone() for t in (lens, used, table, ck, cv)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for t, was in zip((lens, used, table, ck, cv), state):
            t.copy_(was)
    for i in range(steps):
        log("decode step", captured, i)
        x.copy_(rows(n)[0])
        q_in, k_in, before = q.clone(), k.clone(), host(lens)
        graph.replay() if captured else step()
        torch.cuda.synchronize()
        place = np.stack([before] * 3)
        freq, ax = host(inv_freq).astype(np.float32), host(axes)
        check_rope(q, q_in, place, freq, ax, False, "bf16")
        check_rope(k, k_in, place, freq, ax, False, "bf16")
        keep(k, v, slots, [1] * n)
        now = prompts + i + 1
        assert host(lens).tolist() == now.tolist()
        # the reference reads a cache of its own, one page per sequence
        room = 1 + int(now.max())
        mine = [np.full((n, kv_heads, room, dim), 0x7F, np.uint8) for _ in range(2)]
        for r in range(n):
            for which in (0, 1):
                mine[which][r, :, :now[r]] = np.stack(kept[r][which], 1)
        want, lse, reach, sharp = R.attention(host(q), mine[0], mine[1], 30.0, 25.0, np.arange(n)[:, None], now,
                                              np.float32(dim ** -0.5), 0, n)
        bound, _ = R.attention_bounds(want, lse, reach, sharp, now, "bf16")
        off = np.abs(host(out) - want)
        assert (off <= bound).all(), float((off / bound).max())
