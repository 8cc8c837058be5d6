"""The gated delta layer's kernels that only larger calls reach: many columns of states, parts of long
sequences of every head size, more sequences than are put in order, and convolutions of many rows.
Checks, bounds and their reasons are those of test_gpu_gdn."""
import numpy as np
import pytest

from tests.test_gpu_gdn import Delta, check_conv, conv_inputs, delta_starts, log

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

LENS = [70, 1, 64, 0, 130, 63, 2, 65, 5, 128, 31, 64, 97]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("heads,n", [((2, 6, 128, 128), 13), ((2, 6, 128, 128), 25), ((1, 5, 64, 192), 20), ((1, 9, 64, 256), 9), ((3, 12, 64, 64), 14)])
def test_chunked_of_many_columns(gpu_lib, dtype, heads, n):
    """9984, 19200, 19200, 20736 and 10752 columns: workgroups of 64 and of 128 of them."""
    rng = np.random.default_rng([n, *heads, 2])
    starts = delta_starts([LENS[i % len(LENS)] for i in range(n)])
    log("many columns", dtype, heads, n)
    d = Delta(rng, dtype, int(starts[-1]) + 3, n, *heads, extra=8 * (n % 2))
    d.slots[5] = -1
    d.check(gpu_lib, starts, cached=rng.integers(0, 2, n) * 5, in_place=n % 2 == 1, out_extra=8 * (n % 2))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("heads,lens", [
    ((2, 2, 64, 192), [2700]), ((1, 3, 128, 64), [1100, 1700]), ((1, 1, 128, 256), [2600, 64]), ((1, 2, 64, 128), [513, 4000, 0, 3]),
    ((8, 24, 64, 128), [3100]), ((2, 12, 128, 128), [1700, 1500])])
def test_chunked_in_parts_of_every_size(gpu_lib, dtype, heads, lens):
    """Parts of sequences, the last two cases' in workgroups of 128 columns."""
    rng = np.random.default_rng([len(lens), *heads, 3])
    log("parts", dtype, heads, lens)
    starts = delta_starts(lens) + 2
    d = Delta(rng, dtype, int(starts[-1]) + 3, len(lens), *heads, decay=0.05)
    d.check(gpu_lib, starts, cached=np.arange(len(lens)) % 2 == 0, in_place=len(lens) == 1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [511, 512, 513, 700])
def test_chunked_of_many_sequences(gpu_lib, dtype, n):
    rng = np.random.default_rng([n, 4])
    starts = delta_starts([(0, 1, 2, 65)[i * 7 % 11 % 4] for i in range(n)])
    log("many sequences", dtype, n)
    Delta(rng, dtype, int(starts[-1]), n, 1, 1, 64, 64).check(gpu_lib, starts, cached=rng.integers(0, 2, n))


@pytest.mark.parametrize("dtype,channels", [("f32", 2056), ("f16", 2056), ("bf16", 4104)])
@pytest.mark.parametrize("width", [2, 4])
def test_conv_of_many_rows(gpu_lib, dtype, channels, width):
    """16 rows a thread, and 32 with outputs stored past the caches."""
    rng = np.random.default_rng([channels, width])
    lens = [1000, 1, 31, 32, 33, 0, 2, 1999, 3, 999]
    starts = np.concatenate([[0], np.cumsum(lens)])
    x, weight, bias, state, slots = conv_inputs(rng, int(starts[-1]) + 2, channels, width, dtype, len(lens))
    slots[3] = -1
    log("conv of many rows", dtype, channels, width)
    check_conv(gpu_lib, dtype, x, weight, bias, "silu", state, slots, starts, rng.integers(0, 2, len(lens)), in_place=width == 4)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("huge", [300.0, 1e9, 1e30, 3e38])
def test_tokens_after_one_that_forgets_all(gpu_lib, dtype, huge):
    """A token's decay of any size, also one that overflows, leaves the later tokens' decays exact."""
    rng = np.random.default_rng(21)
    starts = delta_starts([130, 200])
    log("forgets", dtype, huge)
    d = Delta(rng, dtype, int(starts[-1]), 2, 1, 2, 64, 64)
    d.a_log[:] = torch.tensor([0.0, 3.0], device="cuda")
    d.dt_bias.zero_()
    d.a[:] = torch.as_tensor(rng.uniform(-5, -2, d.a.shape), device="cuda").to(d.a.dtype)
    for token in (0, 5, 70, 71, 127, 140, 250):
        d.a[token] = huge
    for step in (False, True):
        if step:
            d.slots = np.concatenate([d.slots, [-1] * (len(d.q) - len(d.slots))])
        d.check(gpu_lib, np.arange(len(d.q) + 1) if step else starts, step=step)


@pytest.mark.parametrize("channels", [2 ** 26, 2 ** 26 - 3])
@pytest.mark.parametrize("step", [False, True])
def test_conv_of_the_widest_rows(gpu_lib, channels, step):
    """Two tokens of two sequences; three products of 2^-24 and their sum's roundings: 2^-22 of the sizes."""
    log("widest", channels, step)
    gen = torch.Generator("cuda").manual_seed(3)
    make = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")
    x, weight, state = make(2, channels), make(channels, 2), make(2, 1, channels)
    slots, starts = torch.tensor([1, 0], dtype=torch.int32, device="cuda"), torch.arange(3, dtype=torch.int32, device="cuda")
    was, after = state.flip(0)[:, 0], torch.zeros_like(state)
    args = (x, weight, state, slots) if step else (x, weight, state, slots, starts)
    out = (gpu_lib.nvfp4_causal_conv_step if step else gpu_lib.nvfp4_causal_conv)(*args, activation="none", state_out=after)
    assert torch.equal(after[:, 0].flip(0), x)
    for r in range(2):
        old, new = was[r].double() * weight[:, 0].double(), x[r].double() * weight[:, 1].double()
        assert ((out[r].double() - old - new).abs() <= 2.0 ** -22 * (old.abs() + new.abs()) + 1e-37).all()


def test_conv_in_two_launches(gpu_lib):
    """More tokens than one launch takes."""
    tokens, channels = 2 ** 24 + 50, 3
    log("conv in two launches")
    gen = torch.Generator("cuda").manual_seed(4)
    make = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")
    x, weight, state = make(tokens, channels), make(channels, 2), make(1, 1, channels)
    starts, slots = torch.tensor([0, tokens], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    after = torch.zeros_like(state)
    out = gpu_lib.nvfp4_causal_conv(x, weight, state, slots, starts, activation="none", state_out=after)
    assert torch.equal(after[0], x[-1:])
    old = torch.cat([state[0], x[:-1]]).double() * weight[:, 0].double()
    new = x.double() * weight[:, 1].double()
    assert ((out.double() - old - new).abs() <= 2.0 ** -22 * (old.abs() + new.abs()) + 1e-37).all()


def test_norm_in_two_launches(gpu_lib):
    """More groups than one launch takes; eight squares, their mean and its root, a product: 2^-19 of the value, and bf16's rounding."""
    tokens = 2 ** 24 + 100
    log("norm in two launches")
    x = torch.randn(tokens, 1, 8, generator=torch.Generator("cuda").manual_seed(5), device="cuda", dtype=torch.bfloat16)
    out = gpu_lib.nvfp4_group_norm(x, torch.ones(8, device="cuda"), activation="none", eps=1e-6)
    for rows in (slice(0, 1000), slice(2 ** 24 - 1000, tokens)):
        y = x[rows].double()
        want = y / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt()
        assert ((out[rows].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -19) * want.abs() + 1e-37).all()


def test_chunked_in_two_launches(gpu_lib):
    """More sequences than one launch takes, of a token each: out = scale (q~ . k~) beta v, S = k~ (beta v)^T."""
    n = 2 ** 20 + 100
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("needs 120 GiB")
    log("chunked in two launches")
    gen = torch.Generator("cuda").manual_seed(6)
    q, k, v = (torch.randn(n, 1, 64, generator=gen, device="cuda").half() for _ in range(3))
    a, b = torch.zeros(n, 1, device="cuda").half(), torch.randn(n, 1, generator=gen, device="cuda").half()
    zero = torch.zeros(1, device="cuda")
    state = torch.empty(n, 1, 64, 64, device="cuda")
    slots = torch.arange(n - 1, -1, -1, dtype=torch.int32, device="cuda")
    starts, cached = torch.arange(n + 1, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    out = gpu_lib.nvfp4_gated_delta_chunked(q, k, v, a, b, zero, zero, state, slots, starts, cached_lens=cached, scale=0.125, eps=1e-6)
    torch.cuda.synchronize()
    qn, kn = (x[:, 0].double() / (x[:, 0].double().square().sum(-1, keepdim=True) + 1e-6).sqrt() for x in (q, k))
    d = torch.sigmoid(b.double()) * v[:, 0].double()
    want = 0.125 * (qn * kn).sum(-1, keepdim=True) * d
    assert ((out[:, 0].double() - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -19 * 0.125 * d.abs() + 2.0 ** -25).all()
    for r in (*range(0, n, 65536), *range(n - 101, n)):
        got = state[n - 1 - r, 0].double()
        exact = kn[r][:, None] * d[r]
        assert ((got - exact).abs() <= 2.0 ** -19 * d[r].abs()).all(), r
