"""Exactness of the paged FP8 KV cache's kernels where a worst-case bound over
whole rows would hide a lost part: cases in which sums cancel or have one term,
so that the bound is a few roundings of the result itself."""
import numpy as np
import pytest

from tests import kv_reference as R
from tests.test_gpu_paged_kv import DTYPES, dev, host, log, turn

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

ONE, LOWEST = 0x38, 0xFE  # E4M3 bytes of 1 and -448


def two_token_case(rng, lens, heads, kv_heads, dim, page, dtype):
    """Sequences whose first and last token share the weight (all between them have none), with values that
    nearly cancel: -1 for the last one, and for the first what e^-score comes to, to an E4M3 step."""
    n = len(lens)
    columns = max(-(-x // page) for x in lens)
    table = np.zeros((n, columns), int)  # page 0: tokens without weight
    k, v = (np.zeros((2 * n + 1, kv_heads, page, dim), np.uint8) for _ in range(2))
    k[..., 1] = LOWEST
    steps = 0x38 - 16 + np.arange(dim) % 32  # 1/4 up to 3.75
    for r, length in enumerate(lens):
        for at, place, key, value in ((0, 2 * r + 1, ONE, steps), (length - 1, 2 * r + 2, 0, ONE | 0x80)):
            place = table[r, at // page] or place
            table[r, at // page] = place
            k[place, :, at % page] = 0
            k[place, :, at % page, 0] = key
            v[place, :, at % page] = value
    q = np.zeros((n, heads, dim))
    q[..., 0] = rng.uniform(-1.2, 1.2, (n, heads))
    q[..., 1] = 1
    return dev(q, DTYPES[dtype]), k, v, table


def cancelling_bounds(q, k, v, table, lens, scale, dtype):
    one = np.float32(1)
    out, lse, reach, _ = R.attention(host(q), k, v, one, one, table, lens, scale, 0, len(k))
    # a score is one product, exact in 32 bits, times the scale: four roundings with log2(e) and the division by the
    # keys' scale; two tokens carry all the weight, and sums with zeros do not round
    sharp = 4 * 2.0 ** -24 * np.abs(host(q)[..., 0]) * scale
    b_out, b_lse = R.attention_bounds(out, lse, reach, sharp, [2] * len(lens), dtype)
    # a probability is held to 22 bits at least, whatever the output's type
    return out, lse, b_out - (2.0 ** -11 - 2.0 ** -22) * reach * (dtype == "bf16"), b_lse


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("heads,kv_heads,lens", [(8, 2, [2, 9, 33, 130]), (32, 1, [2, 9, 33, 130]), (6, 3, [20000, 4000])])
def test_attention_of_values_that_cancel(gpu_lib, dtype, dim, heads, kv_heads, lens):
    rng = np.random.default_rng([dim, heads])
    lens = lens * 4
    log("attention, cancelling", dtype, dim, heads, lens[:4])
    q, k, v, table = two_token_case(rng, lens, heads, kv_heads, dim, 16, dtype)
    want, want_lse, b_out, b_lse = cancelling_bounds(q, k, v, table, lens, 1.0, dtype)
    one, lse = torch.ones(1, device="cuda"), torch.empty((len(lens), heads), device="cuda")
    got = gpu_lib.nvfp4_paged_attention(q, dev(k, torch.uint8), dev(v, torch.uint8), one, one, dev(table), dev(lens),
                                        softmax_scale=1.0, lse=lse)
    torch.cuda.synchronize()
    off = np.abs(host(got) - want)
    assert (off <= b_out).all(), float((off / b_out).max())
    off = np.abs(host(lse) - want_lse)
    assert (off <= b_lse).all(), float((off / b_lse).max())


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("tokens", [40, 3000])
def test_rope_near_the_zeros_of_sine_and_cosine(gpu_lib, adjacent, tokens):
    """Pairs (1, 0) and (0, 1) become the cosine and sine themselves: each to a few steps of its own size."""
    rng = np.random.default_rng(tokens)
    pairs = 64
    positions = rng.integers(-1000000, 1000000, (2, tokens))
    inv_freq = (1e4 ** (-np.arange(pairs) / pairs)).astype(np.float32)
    axes = np.arange(pairs) % 2
    x = np.zeros((tokens, 2, 2 * pairs))
    first = slice(0, None, 2) if adjacent else slice(0, pairs)
    second = slice(1, None, 2) if adjacent else slice(pairs, None)
    x[:, 0, first] = x[:, 1, second] = 1
    log("rope, zeros", adjacent, tokens)
    got, _ = turn(gpu_lib, dev(x, torch.float32), None, positions, inv_freq, axes, adjacent)
    want, _ = R.rope(x, positions, inv_freq, axes, adjacent)
    # two steps of the 32-bit sine and cosine (2^-23 each) and a rounding where the angle's low part is added; the angle
    # itself to 2^-51, twice, of at most a million radians
    bound = 5 * 2.0 ** -24 * np.abs(want) + 2.0 ** -30
    off = np.abs(host(got) - want)
    assert (off <= bound).all(), float((off / bound).max())


@pytest.mark.parametrize("which", ["q", "k"])
@pytest.mark.parametrize("adjacent", [False, True])
def test_rope_leaves_the_rest_of_heads_in_place_alone(gpu_lib, adjacent, which):
    """One tensor in place and the other not, while another stream writes what lies behind rot_dim in the first."""
    rng = np.random.default_rng(41)
    tokens, dim, rot, rounds = 6000, 256, 64, 12
    positions, axes = dev(rng.integers(0, 4000, (1, tokens))), dev(np.zeros(rot // 2, int))
    inv_freq = dev(1e4 ** (-np.arange(rot // 2) / (rot // 2)), torch.float32)
    q, k = (dev(rng.standard_normal((tokens, h, dim)), torch.bfloat16) for h in (8, 8))
    mine, other = (q, k) if which == "q" else (k, q)
    out, before, side = torch.empty_like(other), mine.clone(), torch.cuda.Stream()
    torch.cuda.synchronize()
    log("rope, in place beside a writer", adjacent, which)
    for i in range(rounds):
        gpu_lib.nvfp4_rope(q, k, positions, inv_freq, axes, adjacent=adjacent, **{which + "_out": mine, "qk"[which == "q"] + "_out": out})
        with torch.cuda.stream(side):
            mine[:, :, rot:].fill_(float(i))
    torch.cuda.synchronize()
    assert (mine[:, :, rot:] == rounds - 1).all()
    assert torch.equal(out[:, :, rot:], other[:, :, rot:])
    assert torch.equal(out, gpu_lib.nvfp4_rope(other, None, positions, inv_freq, axes, adjacent=adjacent)[0])
    again = before.clone()
    for _ in range(rounds):
        gpu_lib.nvfp4_rope(again, None, positions, inv_freq, axes, adjacent=adjacent, q_out=again)
    torch.cuda.synchronize()
    assert torch.equal(again[:, :, :rot], mine[:, :, :rot])


def test_rope_with_one_row_of_positions(gpu_lib):
    rng = np.random.default_rng(43)
    x = dev(rng.standard_normal((50, 3, 64)), torch.bfloat16)
    row, axes = dev(rng.integers(0, 100000, (1, 50))), dev(np.arange(16) % 3)
    inv_freq = dev(1e4 ** (-np.arange(16) / 16), torch.float32)
    log("rope, one row of positions")
    got, _ = gpu_lib.nvfp4_rope(x, None, row.expand(3, -1), inv_freq, axes)
    want, _ = gpu_lib.nvfp4_rope(x, None, row.repeat(3, 1), inv_freq, axes)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_attention_of_the_largest_float32_queries(gpu_lib, dim):
    """Elements up to the type's largest, against keys of zero there; the rest of the row decides."""
    rng = np.random.default_rng(dim)
    heads, lens = 4, [1, 7, 40]
    most = np.finfo(np.float32).max
    q = np.zeros((3, heads, dim), np.float32)
    q[..., 0] = rng.uniform(-2, 2, (3, heads))
    q[..., 1:5] = [most, -most, most * 0.9985, np.float32(3.39e38)]
    k, v = (rng.integers(0x30, 0x50, (4, 1, 48, dim)).astype(np.uint8) for _ in range(2))
    k[..., 1:] = 0
    table, one = np.array([[2], [0], [3]]), torch.ones(1, device="cuda")
    lse = torch.empty((3, heads), device="cuda")
    log("attention, largest queries", dim)
    got = gpu_lib.nvfp4_paged_attention(dev(q, torch.float32), dev(k, torch.uint8), dev(v, torch.uint8), one, one, dev(table), dev(lens),
                                        softmax_scale=0.5, lse=lse)
    torch.cuda.synchronize()
    q[..., 1:5] = 0  # they meet zeros alone
    ref = R.attention(q, k, v, 1.0, 1.0, table, lens, 0.5, 0, len(k))
    b_out, b_lse = R.attention_bounds(*ref, lens, "f32")
    assert (np.abs(host(got) - ref[0]) <= b_out).all() and (np.abs(host(lse) - ref[1]) <= b_lse).all()


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("channel", [0, 37, 63])
def test_attention_holds_every_bit_of_a_float32_query(gpu_lib, dim, channel):
    rng = np.random.default_rng([dim, channel])
    heads, n = 16, 5
    x = rng.uniform(1, 2, (n, heads)).astype(np.float32)
    q = np.zeros((n, heads, dim), np.float32)
    q[..., channel] = x * np.where(rng.random((n, heads)) < 0.5, -1, 1)
    key = rng.integers(0x70, 0x7F, n).astype(np.uint8)  # 128 to 448
    k, v = (np.zeros((n, 1, 16, dim), np.uint8) for _ in range(2))
    k[:, 0, 0, channel] = key
    s = q[..., channel].astype(np.float64) * R.E4M3[key][:, None] * 4.0
    one, lse = torch.ones(1, device="cuda"), torch.empty((n, heads), device="cuda")
    log("attention, every bit", dim, channel)
    gpu_lib.nvfp4_paged_attention(dev(q, torch.float32), dev(k, torch.uint8), dev(v, torch.uint8), one, one, dev(np.arange(n)[:, None]),
                                  dev(np.ones(n)), softmax_scale=4.0, lse=lse)
    torch.cuda.synchronize()
    # the products of three parts and their sum: 3 roundings; times log2(e): one of the maximum and one of what is left;
    # back from base 2: 3, all of 2^-24 of the score, and the exponential and logarithm of one term: 2^-19.  Without its
    # last eight bits a query would be off by up to 2^-16 of itself, fifty times that.
    off, bound = np.abs(host(lse) - s), 8 * 2.0 ** -24 * np.abs(s) + 2.0 ** -19
    assert (off <= bound).all(), float((off / bound).max())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("scale", [1e4, 3e5, 1e6, 7.7e6, 1e8, 1.3e9, 1e12, 1e30])
@pytest.mark.parametrize("columns", [4, 1200])
def test_attention_of_very_large_scores(gpu_lib, dtype, scale, columns):
    """Scores whose neighbours in 32 bits lie more than one apart: the largest takes all, equal ones share."""
    rng = np.random.default_rng([columns, int(np.log10(scale))])
    n, heads, dim, page = 12, 6, 64, 16
    lens = rng.integers(1, 4 * page, n)
    k, v = (rng.integers(0x20, 0x70, (4 * n, 1, page, dim)).astype(np.uint8) for _ in range(2))
    k[..., 0] ^= (rng.random(k[..., 0].shape) < 0.5).astype(np.uint8) << 7
    k[..., 1:] = 0
    table = np.full((n, columns), -1)
    table[:, :4] = rng.permutation(4 * n).reshape(n, 4)
    q = np.zeros((n, heads, dim))
    q[..., 0] = rng.uniform(0.5, 2, (n, heads)) * np.where(rng.random((n, heads)) < 0.5, -1, 1)
    q = dev(q, DTYPES[dtype])
    one, lse = torch.ones(1, device="cuda"), torch.empty((n, heads), device="cuda")
    log("attention, large scores", dtype, scale, columns)
    got = gpu_lib.nvfp4_paged_attention(q, dev(k, torch.uint8), dev(v, torch.uint8), one, one, dev(table), dev(lens), softmax_scale=scale,
                                        lse=lse)
    torch.cuda.synchronize()
    scale = float(np.float32(scale))
    want, want_lse, reach, _ = R.attention(host(q), k, v, 1.0, 1.0, table, lens, scale, 0, len(k))
    # E4M3 keys and one channel: other tokens are a sixteenth of a score away (e^-625 at least) or equal, so weights are
    # 0 or 1 over the number of equal ones, a division and the type's own rounding
    bound = (R.HALF_STEP[dtype] * 1.01 + 2.0 ** -20) * reach
    assert (np.abs(host(got) - want) <= bound).all()
    assert (np.abs(host(lse) - want_lse) <= 2.0 ** -20 * np.abs(want_lse)).all()
