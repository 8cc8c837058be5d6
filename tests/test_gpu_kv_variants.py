"""The variants of the paged FP8 KV cache's kernels that only long calls reach: two
items of a rotation to a thread, two tokens of a block table to a thread, calls in
several launches."""
import numpy as np
import pytest

from tests.test_gpu_paged_kv import DTYPES, check_rope, check_table, dev, host, log, table_case, turn

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype,adjacent,tokens,q_heads,k_heads,dim,rot", [
    ("bf16", False, 2803, 5, 2, 256, 64), ("f16", False, 2805, 7, 0, 256, 64), ("f32", True, 4001, 3, 2, 128, 128),
    ("bf16", True, 4003, 11, 5, 72, 40), ("f32", False, 1601, 3, 3, 256, 32), ("bf16", True, 4099, 9, 1, 128, 128)])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("in_place", [False, True])
def test_rope_of_long_prompts(gpu_lib, dtype, adjacent, tokens, q_heads, k_heads, dim, rot, shift, in_place):
    rng = np.random.default_rng([tokens, rot, shift])
    pairs = rot // 2
    positions = rng.integers(-1000, 1000000, (3, tokens))
    inv_freq = (1e4 ** (-np.arange(pairs) / pairs)).astype(np.float32)
    axes = np.arange(pairs) % 3
    rows = dev(rng.standard_normal((tokens, shift + (q_heads + k_heads) * (dim + shift))), DTYPES[dtype])
    heads = rows[:, shift:].unflatten(1, (q_heads + k_heads, dim + shift))[:, :, :dim]
    q, k = heads[:, :q_heads], heads[:, q_heads:] if k_heads else None
    before, was = rows.clone(), heads.clone()
    log("rope, long", dtype, adjacent, tokens, q_heads, k_heads, dim, rot, shift, in_place)
    out = dict(q_out=q, k_out=k) if in_place else {}
    q_out, k_out = turn(gpu_lib, q, k, positions, inv_freq, axes, adjacent, **out)
    got = q_out if k is None else torch.cat([q_out, k_out], 1)
    check_rope(got, was, positions, inv_freq, axes, adjacent, dtype)
    if in_place:
        heads.copy_(was)
    assert torch.equal(rows, before)


@pytest.mark.parametrize("n,new", [(700, 900), (3000, 210), (4096, 160)])
def test_block_table_of_two_tokens_a_thread(gpu_lib, n, new):
    rng = np.random.default_rng(n)
    c, w, table, free = table_case(rng, n, 16, 80, 300, new, 0)
    tokens = int(w.sum()) + 11
    log("block table, two a thread", n, tokens)
    assert 1 << 18 < tokens <= 1 << 19
    check_table(gpu_lib, c, w, 16, free, 2, table, tokens)
    check_table(gpu_lib, c, w, 16, free[:len(free) // 2], 2, table, tokens)


@pytest.mark.parametrize("in_place", [False, True])
def test_rope_of_neighbours_in_more_than_one_launch(gpu_lib, in_place):
    tokens, q_heads, k_heads = (1 << 20) + 3, 250, 7
    draw = lambda: torch.randn(tokens, q_heads + k_heads, 2, generator=torch.Generator("cuda").manual_seed(2), device="cuda", dtype=torch.bfloat16)
    wide = draw()
    q, k = wide[:, :q_heads], wide[:, q_heads:]
    positions = torch.arange(2 * tokens, device="cuda", dtype=torch.int32).view(2, tokens)
    # 2^28 items of 257 a token in a launch: the second one begins at token 1044495
    at = torch.cat([torch.arange(a, b) for a, b in ((0, 3), (1044495 - 3, 1044495 + 3), (tokens - 3, tokens))]).cuda()
    was, out = wide[at], {"q_out": q, "k_out": k} if in_place else {}
    log("rope, neighbours, pieces", in_place)
    q_out, k_out = gpu_lib.nvfp4_rope(q, k, positions, dev([0.37], torch.float32), dev([1]), adjacent=True, **out)
    torch.cuda.synchronize()
    check_rope(torch.cat([q_out[at], k_out[at]], 1), was, host(positions[:, at]), np.array([0.37], np.float32), np.array([1]), True, "bf16")
    size = lambda x: x.double().square().sum()
    turned = size(q_out) + size(k_out)
    del wide, q, k, q_out, k_out
    assert abs(turned / size(draw()) - 1) <= 2.0 ** -7  # every token turned once: lengths stay, to two roundings
    torch.cuda.empty_cache()
