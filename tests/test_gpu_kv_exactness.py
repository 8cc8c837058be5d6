"""Exactness of the paged FP8 KV cache's kernels where a worst-case bound over
whole rows would hide a lost part: cases in which sums cancel or have one term,
so that the bound is a few roundings of the result itself."""
import numpy as np
import pytest

from tests import kv_reference as R
from tests.test_gpu_paged_kv import DTYPES, dev, host, log

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
