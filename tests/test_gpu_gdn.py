"""The gated delta layer on the GPU, through the binding, against plain 64-bit
references (tests/gdn_reference.py), within bounds that follow from the roundings
made.  Then the operators together, as a layer runs them."""
import sys

import numpy as np
import pytest

from tests import gdn_reference as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


def log(*a):
    print("[case]", *a, flush=True)
    sys.stdout.flush()


def dev(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda").to(dtype)


def ints(a):
    return dev(np.asarray(a, np.int64), torch.int32)


def host(t):
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def strided(t, extra=0, lead=0):
    """The same values in the middle of wider rows."""
    if not extra and not lead:
        return t
    wide = torch.full((t.shape[0], lead + t[0].numel() + extra), 7.0, dtype=t.dtype, device=t.device)
    part = wide[:, lead:lead + t[0].numel()]
    part.copy_(t.reshape(t.shape[0], -1))
    return part.unflatten(1, t.shape[1:]) if t.dim() > 2 else part


def within(got, want, slack, dtype, name):
    """One rounding to dtype beyond `slack`."""
    off = np.abs(host(got) - want)
    most = slack + R.HALF_STEP[dtype] * 1.01 * np.abs(want) + R.LEAST[dtype]
    assert np.isfinite(host(got)).all(), name
    assert (off <= most).all(), (name, float((off / np.maximum(most, 1e-300)).max()), np.unravel_index(np.argmax(off - most), off.shape))


# ------------------------------------------------------------------ convolution

# Sums of width + 1 products, each of five roundings at most 2^-24 of the sum of sizes; |silu'| <= 1.1; the sigmoid's
# exponential is off by 2^-22 (16-bit types: by |y| 2^-24 more), and y times the sigmoid's slope stays below 0.28 in size.
# 2^-21 of the sizes holds all of it.
CONV_SLACK = 2.0 ** -21


def conv_inputs(rng, tokens, channels, width, dtype, n, bias=True, num_slots=None):
    num_slots = n + 3 if num_slots is None else num_slots
    x = dev(rng.standard_normal((tokens, channels)) * np.exp(rng.standard_normal(channels)), DTYPES[dtype])
    weight = dev(rng.standard_normal((channels, width)))
    b = dev(rng.standard_normal(channels)) if bias else None
    state = dev(rng.standard_normal((num_slots, width - 1, channels)), DTYPES[dtype])
    slots = rng.permutation(num_slots)[:n]
    return x, weight, b, state, slots


def check_conv(nv, dtype, x, weight, bias, act, state, slots, starts, cached, step=False, in_place=False, out_stride=0):
    out = strided(torch.full(x.shape, 5.0, dtype=x.dtype, device="cuda"), out_stride)
    after = state.clone() if in_place else torch.full_like(state, 3.0)
    was = host(after)
    want, sizes, left = R.conv(host(x), host(weight), 0.0 if bias is None else host(bias), act == "silu", host(state), slots, starts,
                               cached, host(out))
    for _, _, _, slot in R.spans(starts, slots, len(state), len(x)):
        was[slot] = left[slot]
    given = after if in_place else state
    if step:
        got = nv.nvfp4_causal_conv_step(x, weight, given, ints(slots), bias=bias, activation=act, state_out=after, out=out)
    else:
        got = nv.nvfp4_causal_conv(x, weight, given, ints(slots), ints(starts), cached_lens=None if cached is None else ints(cached),
                                   bias=bias, activation=act, state_out=after, out=out)
    torch.cuda.synchronize()
    assert got is out
    assert np.array_equal(host(after), was)
    within(out, want, CONV_SLACK * sizes, dtype, "conv")
    left_out = sizes == 0
    assert np.array_equal(host(out)[left_out], want[left_out])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("lens,channels,stride", [
    ([1], 8, 0), ([2], 1, 0), ([0, 3, 0], 24, 8), ([1, 2, 3, 4, 5, 1, 1], 40, 3), ([31, 1, 1, 33, 2], 264, 0), ([30, 2, 64, 100], 2056, 16),
    ([70], 4100, 0), ([32, 32, 1, 63, 3, 29], 7, 1), ([500, 3, 77], 136, 8)])
@pytest.mark.parametrize("in_place", [False, True])
def test_conv(gpu_lib, dtype, width, lens, channels, stride, in_place):
    rng = np.random.default_rng([width, channels, len(lens)])
    starts = np.concatenate([[0], np.cumsum(lens)])
    tokens = int(starts[-1]) + 3  # rows behind the last sequence
    x, weight, bias, state, slots = conv_inputs(rng, tokens, channels, width, dtype, len(lens), bias=channels != 40)
    cached = rng.integers(0, 2, len(lens)) * 9 - 1
    log("conv", dtype, width, lens, channels, stride, in_place)
    act = "none" if channels == 264 else "silu"
    check_conv(gpu_lib, dtype, strided(x, stride), weight, bias, act, state, slots, starts, cached, in_place=in_place, out_stride=stride)
    check_conv(gpu_lib, dtype, x, weight, bias, act, state, slots, starts, None, in_place=in_place)


def test_conv_of_left_out_sequences_and_starts(gpu_lib):
    rng = np.random.default_rng(5)
    x, weight, bias, state, slots = conv_inputs(rng, 90, 16, 4, "bf16", 6)
    slots[1], slots[4] = -1, len(state)
    log("conv, left out")
    for starts in ([5, 20, 33, 34, 70, 80, 85], [0, 0, 0, 90, 90, 90, 90], [-3, 4, 9, 60, 61, 2 ** 31 - 1, 2 ** 31 - 1]):
        check_conv(gpu_lib, "bf16", x, weight, bias, "silu", state, slots, np.array(starts), np.array([1, 1, 0, 5, 5, -2]))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,channels,width", [(1, 8, 4), (5, 9, 3), (33, 2056, 4), (4, 30, 2), (300, 64, 4)])
@pytest.mark.parametrize("in_place", [False, True])
def test_conv_step(gpu_lib, dtype, n, channels, width, in_place):
    rng = np.random.default_rng([n, channels])
    x, weight, bias, state, slots = conv_inputs(rng, n, channels, width, dtype, n)
    if n > 4:
        slots[2], slots[4] = -1, len(state) + 7
    log("conv step", dtype, n, channels, width, in_place)
    check_conv(gpu_lib, dtype, x, weight, bias, "silu", state, slots, np.arange(n + 1), None, step=True, in_place=in_place)


def test_conv_large_and_small_values(gpu_lib):
    """SiLU far out: outputs go to the input and to zero, without infinities."""
    x = dev(np.array([[-3e38, -1e30, -200.0, -90.0, -87.0, -30.0, 30.0, 90.0, 1e30, 3e38, 0.0, -0.0, 1e-40, 2e-38, 1.0, -1.0]]))
    weight = torch.zeros((16, 2), device="cuda")
    weight[:, 1] = 1.0
    state, slots = torch.zeros((1, 1, 16), device="cuda"), np.array([0])
    for dtype in ("f32", "bf16"):
        with np.errstate(over="ignore"):
            check_conv(gpu_lib, dtype, x.to(DTYPES[dtype]), weight, None, "silu", state.to(DTYPES[dtype]), slots, np.array([0, 1]), None)


# ------------------------------------------------------------------- delta rule

# Each token's 32-bit evaluation makes a handful of roundings of 2^-24 relative to what R.delta adds up, in sums of head_k
# products (in the matrix units 2^-22 of the operands): 32 of them, 2^-19, hold a token's.
DELTA_SLACK = 2.0 ** -19
# Chunks of 64 tokens cut what a column's state and its tokens write at 2^-32 of the largest of them; a token's output and
# state are made of up to 192 such operands with weights of at most 1: less than 2^-24.
DELTA_LEAST = 2.0 ** -24 / DELTA_SLACK


class Delta:
    def __init__(self, rng, dtype, tokens, n, k_heads, v_heads, head_k, head_v, extra=0, size=1.0, spare=3, decay=1.0):
        def heads(shape, scale=1.0):
            return strided(dev(R.silu(rng.standard_normal(shape)) * scale, DTYPES[dtype]), extra, extra)
        self.dtype = dtype
        self.q, self.k = heads((tokens, k_heads, head_k)), heads((tokens, k_heads, head_k), 0.1)
        self.v = heads((tokens, v_heads, head_v), size)
        gates = dev(rng.standard_normal((tokens, 2 * v_heads + 1)), DTYPES[dtype])
        self.a, self.b = gates[:, :v_heads], gates[:, v_heads + 1:]
        self.a_log = dev(np.log(rng.uniform(0.01, 8, v_heads) * decay))
        self.dt_bias = dev(rng.uniform(-6, 1, v_heads))
        self.state = dev(rng.standard_normal((n + spare, v_heads, head_k, head_v)) * 0.2 * size)
        self.slots = rng.permutation(n + spare)[:n]
        self.scale = head_k ** -0.5
        self.in_place = False

    def want(self, starts, cached, out, least=0.0):
        return R.delta(*(host(t) for t in (self.q, self.k, self.v, self.a, self.b, self.a_log, self.dt_bias)), self.scale, EPS, host(self.state),
                       self.slots, starts, cached, out, least)

    def run(self, nv, starts, cached=None, step=False, state=None, after=None, out=None, **kw):
        state = self.state if state is None else state
        slots, starts = ints(self.slots), ints(starts)
        args = (self.q, self.k, self.v, self.a, self.b, self.a_log, self.dt_bias, state, slots)
        if step:
            return nv.nvfp4_gated_delta_step(*args, scale=self.scale, eps=EPS, state_out=after, out=out, **kw)
        return nv.nvfp4_gated_delta_chunked(*args, starts, cached_lens=None if cached is None else ints(cached), scale=self.scale, eps=EPS,
                                            state_out=after, out=out, **kw)

    def check(self, nv, starts, cached=None, step=False, in_place=False, out_extra=0):
        starts = np.asarray(starts)
        out = strided(torch.full(self.v.shape, 5.0, dtype=self.v.dtype, device="cuda"), out_extra)
        given = self.state.clone()
        after = given if in_place else torch.full_like(self.state, 3.0)
        was = host(after)
        want, slack, left, left_slack, floors = self.want(starts, cached, host(out), 0.0 if step else DELTA_LEAST)
        touched = [slot for _, _, _, slot in R.spans(starts, self.slots, len(self.state), len(self.q))]
        was[touched] = left[touched]
        got = self.run(nv, starts, cached, step, given, after, out)
        torch.cuda.synchronize()
        assert got is out
        within(out, want, DELTA_SLACK * slack, self.dtype, "out")
        within(after, was, DELTA_SLACK * left_slack, "f32", "state")
        # Independent roundings of 2^-22 in the operands of the three products that lead to a state, met by a rule that
        # shortens errors: their length is below 2^-20 of the state's, where nothing but decay G is left of it 2^-23 |G| more.
        # A lost part of an operand would leave 2^-12.  The columns' floors come on top.
        total = np.exp(host(self.a_log)) * np.logaddexp(0, host(self.a) + host(self.dt_bias)).sum(0)
        share = 2.0 ** -20 + 2.0 ** -23 * np.minimum(total, 64)
        for slot in touched:
            off = np.sqrt(((host(after)[slot] - left[slot]) ** 2).sum((1, 2)))
            length = np.sqrt((left[slot] ** 2).sum((1, 2)))
            least = DELTA_SLACK * np.sqrt((floors[slot] ** 2).sum(1))
            assert (off <= share * length + least + 1e-37).all(), ("state", slot, float((off / np.maximum(length, 1e-300)).max()))
        rows = np.ones(len(self.q), bool)
        for _, low, high, _ in R.spans(starts, self.slots, len(self.state), len(self.q)):
            rows[low:high] = False
        assert np.array_equal(host(out)[rows], want[rows])
        return out, after


def delta_starts(lens):
    return np.concatenate([[0], np.cumsum(lens)])


HEADS = [(1, 1, 64, 64), (2, 4, 128, 128), (1, 3, 128, 64), (3, 3, 64, 192), (1, 2, 128, 256), (2, 12, 64, 128)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("lens", [[1], [0, 2, 0, 1], [64], [63, 65, 1], [130, 7, 64, 128], [331]])
def test_chunked(gpu_lib, dtype, heads, lens):
    rng = np.random.default_rng([len(lens), *heads])
    starts = delta_starts(lens)
    log("chunked", dtype, heads, lens)
    d = Delta(rng, dtype, int(starts[-1]) + 3, len(lens), *heads, extra=8 * (len(lens) % 2))
    d.check(gpu_lib, starts, cached=rng.integers(0, 2, len(lens)) * 5, in_place=len(lens) > 1, out_extra=8 * (len(lens) % 2))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("n", [1, 5, 70])
def test_step(gpu_lib, dtype, heads, n):
    rng = np.random.default_rng([n, *heads])
    log("step", dtype, heads, n)
    d = Delta(rng, dtype, n, n, *heads, extra=8 * (n % 2))
    if n > 4:
        d.slots[2], d.slots[4] = -1, len(d.state)
    d.check(gpu_lib, np.arange(n + 1), step=True, in_place=n > 1)


def test_chunked_left_out_sequences_and_starts(gpu_lib):
    rng = np.random.default_rng(8)
    d = Delta(rng, "bf16", 300, 6, 1, 2, 64, 64)
    d.slots[1], d.slots[4] = -1, len(d.state)
    log("chunked, left out")
    for starts in ([5, 20, 133, 134, 170, 280, 285], [0, 0, 0, 300, 300, 300, 300], [-3, 4, 9, 160, 161, 2 ** 31 - 1, 2 ** 31 - 1]):
        d.check(gpu_lib, starts, cached=[1, 1, 0, 5, 5, -2])
        d.check(gpu_lib, starts, in_place=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [1e-20, 1e-6, 300.0, 1e15])
def test_values_of_any_size(gpu_lib, dtype, size):
    """Values and states far from 1: nothing overflows or vanishes in the 16-bit parts."""
    rng = np.random.default_rng(3)
    starts = delta_starts([150, 64, 3])
    log("size", dtype, size)
    for step in (False, True):
        Delta(rng, dtype, 217, 3 if not step else 217, 1, 2, 64, 64, size=size).check(gpu_lib, np.arange(218) if step else starts, step=step)


def test_values_that_grow_and_shrink(gpu_lib):
    """One sequence whose values pass 36 powers of ten, up and down, with strong decays between."""
    rng = np.random.default_rng(4)
    log("growing")
    d = Delta(rng, "f32", 700, 1, 1, 2, 64, 64)
    climb = np.concatenate([np.linspace(-18, 18, 350), np.linspace(18, -18, 350)])
    d.v *= dev(10.0 ** climb)[:, None, None]
    d.a += 4.0
    d.check(gpu_lib, [0, 700])


@pytest.mark.parametrize("case", ["no decay", "full decay", "mixed", "beta 0", "beta 1", "same key", "opposed keys", "zero keys", "zero all"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gates_and_keys_at_their_ends(gpu_lib, case, dtype):
    rng = np.random.default_rng(6)
    log("ends", case, dtype)
    d = Delta(rng, dtype, 200, 2, 1, 2, 128, 64)
    if case == "no decay":
        d.a.fill_(-100.0)
        d.dt_bias.fill_(-50.0)
    elif case == "full decay":
        d.a.fill_(100.0)
        d.a_log.fill_(4.0)
    elif case == "mixed":  # sums of log decays that pass 10^4 beside decays of almost 1
        d.a_log.fill_(2.5)
        d.a.copy_(torch.where(torch.rand(d.a.shape, device="cuda") < 0.3, 60.0, -12.0))
    elif case in ("beta 0", "beta 1"):
        d.b.fill_(-200.0 if case == "beta 0" else 200.0)
    elif case in ("same key", "opposed keys"):
        d.k.copy_(d.k[:1].clone().expand_as(d.k))
        d.b.fill_(200.0)
        d.a.fill_(-100.0)
        if case == "opposed keys":
            d.k[::2] *= -1.0
    elif case == "zero keys":
        d.k[::3] = 0.0
        d.q[1::3] = 0.0
    else:
        for t in (d.q, d.k, d.v, d.state):
            t.zero_()
    d.check(gpu_lib, [0, 129, 200])


def test_small_and_large_keys(gpu_lib):
    """Rows of keys and queries are normalised whatever their size."""
    rng = np.random.default_rng(9)
    log("key sizes")
    d = Delta(rng, "f32", 140, 1, 1, 1, 64, 64)
    sizes = dev(10.0 ** rng.uniform(-15, 15, 140))[:, None, None]
    d.k *= sizes
    d.q *= sizes.flip(0)
    d.check(gpu_lib, [0, 140])
    d.k[:, :, 5] *= 300.0  # one element far above the rest
    d.check(gpu_lib, [0, 140])


def test_a_long_sequence_stays_exact(gpu_lib):
    rng = np.random.default_rng(10)
    log("long")
    d = Delta(rng, "bf16", 3000, 1, 1, 1, 128, 64, decay=0.05)
    d.check(gpu_lib, [0, 3000])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("heads,lens", [
    ((1, 2, 128, 128), [2500, 513, 0, 700, 1]), ((1, 1, 64, 64), [4096]), ((2, 2, 64, 192), [2113]), ((1, 3, 128, 64), [600, 1600]),
    ((1, 1, 128, 256), [2049, 64])])
@pytest.mark.parametrize("in_place", [False, True])
def test_chunked_in_parts(gpu_lib, dtype, heads, lens, in_place):
    """Few heads and long sequences, which are taken in parts that run at once."""
    rng = np.random.default_rng([len(lens), *heads, 1])
    log("parts", dtype, heads, lens, in_place)
    starts = delta_starts(lens)
    d = Delta(rng, dtype, int(starts[-1]) + 3, len(lens), *heads, decay=0.05)
    if len(lens) == 5:
        d.slots[3] = -1
    d.check(gpu_lib, starts, cached=rng.integers(0, 2, len(lens)) * 5 if in_place else None, in_place=in_place)


def test_the_result_is_the_same_in_every_call(gpu_lib):
    rng = np.random.default_rng(11)
    d = Delta(rng, "bf16", 1000, 3, 2, 4, 128, 128)
    starts = [0, 300, 301, 990]
    log("same")
    first = None
    for fill in (0, 255, 77):
        size = gpu_lib.nvfp4_gated_delta_workspace(1000, 3, 2, 4, 128, 128, torch.bfloat16)
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")  # NaN bit patterns among them
        after = torch.zeros_like(d.state)
        out = d.run(gpu_lib, starts, after=after, out=torch.zeros_like(d.v), workspace=ws)
        torch.cuda.synchronize()
        first = first or (out, after)
        assert torch.equal(out, first[0]) and torch.equal(after, first[1])


def test_garbage_behind_and_between_sequences_is_not_seen(gpu_lib):
    rng = np.random.default_rng(12)
    d = Delta(rng, "bf16", 200, 2, 1, 2, 64, 64)
    starts = [10, 75, 140]
    log("garbage")
    want = d.run(gpu_lib, starts, after=torch.zeros_like(d.state), out=torch.zeros_like(d.v))
    for t in (d.q, d.k, d.v, d.a, d.b):
        t[:10] = float("nan")
        t[140:] = float("inf")
    spare = [s for s in range(len(d.state)) if s not in d.slots]
    d.state[spare] = float("nan")
    got = d.run(gpu_lib, starts, after=torch.zeros_like(d.state), out=torch.zeros_like(d.v))
    torch.cuda.synchronize()
    assert torch.equal(got, want)


# ------------------------------------------------------------------------- norm

# A sum of group_dim squares in runs of up to 32 and eight halvings: 40 roundings at most, halved by the root, and those of
# the mean as often; the rest is a handful.  2^-18 of the sizes holds them.
NORM_SLACK = 2.0 ** -18


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("tokens,groups,dim", [
    (1, 1, 1), (3, 2, 2), (5, 48, 128), (33, 20, 121), (7, 3, 64), (9, 4, 65), (2, 5, 200), (3, 2, 256), (4, 1, 511), (3, 2, 513), (2, 1, 1024),
    (2, 2, 1030), (2, 1, 4096), (1, 1, 8192), (2, 1, 8191), (1500, 3, 16)])
@pytest.mark.parametrize("centred", [False, True])
def test_norm(gpu_lib, dtype, tokens, groups, dim, centred):
    rng = np.random.default_rng([tokens, groups, dim])
    x = dev(rng.standard_normal((tokens, groups, dim)) * 3 + rng.standard_normal((tokens, groups, 1)), DTYPES[dtype])
    gate = dev(rng.standard_normal(x.shape) * 3, DTYPES[dtype])
    stride = 8 if dim % 8 == 0 else 3
    log("norm", dtype, tokens, groups, dim, centred)
    for gated, act, shared, biased in ((1, "silu", 1, 0), (0, "silu", 0, 1), (1, "none", 0, 1), (0, "none", 1, 0)):
        shape = (dim,) if shared else (groups, dim)
        weight = dev(1 + 0.3 * rng.standard_normal(shape))
        bias = dev(rng.standard_normal(shape)) if biased else None
        z = strided(gate, stride, stride) if gated else None
        want, sizes = R.norm(host(x), host(weight), 0.0 if bias is None else host(bias), host(z) if gated else None, act == "silu", centred, EPS)
        out = strided(torch.zeros_like(x), stride)
        got = gpu_lib.nvfp4_group_norm(strided(x, 0, stride), weight, bias=bias, gate=z, activation=act, centred=centred, eps=EPS, out=out)
        torch.cuda.synchronize()
        within(got, want, NORM_SLACK * sizes, dtype, (gated, act))
        for name in ("x", "gate") if gated else ("x",):  # over an input
            kw = {"x": x.clone(), "gate": gate.clone() if gated else None}
            again = gpu_lib.nvfp4_group_norm(kw["x"], weight, bias=bias, gate=kw["gate"], activation=act, centred=centred, eps=EPS, out=kw[name])
            torch.cuda.synchronize()
            assert torch.equal(again, got) and again is kw[name]


def test_norm_of_equal_and_zero_groups(gpu_lib):
    log("norm, equal")
    x = torch.full((4, 3, 128), 1000.0, device="cuda")
    x[1] = 0.0
    x[2] = -7.25
    w = torch.ones(128, device="cuda")
    got = gpu_lib.nvfp4_group_norm(x, w, activation="none", centred=True)
    assert torch.equal(got, torch.zeros_like(got))
    got = gpu_lib.nvfp4_group_norm(x, w, activation="none")
    want, sizes = R.norm(host(x), 1.0, 0.0, None, False, False, EPS)
    within(got, want, NORM_SLACK * sizes, "f32", "equal")


# ---------------------------------------------------------- streams, graphs, layer

def test_on_another_stream_and_in_a_graph(gpu_lib):
    """One decode step of a layer, captured; replays follow the slots and inputs of the moment."""
    rng = np.random.default_rng(20)
    n, hk, hv, dk, dv = 6, 1, 2, 64, 64
    d = Delta(rng, "bf16", n, n, hk, hv, dk, dv)
    x, weight, bias, conv_state, _ = conv_inputs(rng, n, 2 * hk * dk + hv * dv, 4, "bf16", n)
    gate, w = dev(rng.standard_normal((n, hv, dv)), torch.bfloat16), dev(rng.standard_normal(dv))
    slots = ints(d.slots)
    start = d.state.clone(), conv_state.clone()
    outs = {"conv": torch.zeros_like(x), "delta": torch.zeros_like(d.v), "norm": torch.zeros_like(d.v)}

    def step(stream=None):
        kw = {"stream": stream}
        y = gpu_lib.nvfp4_causal_conv_step(x, weight, conv_state, slots, bias=bias, out=outs["conv"], **kw)
        q, k, v = y[:, :64].view(n, 1, 64), y[:, 64:128].view(n, 1, 64), y[:, 128:].view(n, hv, dv)
        gpu_lib.nvfp4_gated_delta_step(q, k, v, d.a, d.b, d.a_log, d.dt_bias, d.state, slots, out=outs["delta"], **kw)
        gpu_lib.nvfp4_group_norm(outs["delta"], w, gate=gate, out=outs["norm"], **kw)

    def reset():
        d.state.copy_(start[0])
        conv_state.copy_(start[1])

    log("eager")
    want = []
    for i in range(4):
        slots.copy_(ints(np.roll(d.slots, i)))
        step()
        want.append(outs["norm"].clone())
    final = d.state.clone(), conv_state.clone()
    torch.cuda.synchronize()
    reset()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    log("another stream")
    slots.copy_(ints(d.slots))
    torch.cuda.synchronize()
    step(side)
    side.synchronize()
    assert torch.equal(outs["norm"], want[0])
    reset()
    torch.cuda.synchronize()
    log("graph")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        slots.copy_(ints(np.roll(d.slots, i)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs["norm"], want[i]), i
    assert torch.equal(d.state, final[0]) and torch.equal(conv_state, final[1])


def test_prompts_in_two_graphs_of_one_workspace(gpu_lib):
    """Two captured calls that run one after another may share a workspace; replays follow the starts."""
    rng = np.random.default_rng(21)
    d = Delta(rng, "bf16", 400, 2, 1, 2, 128, 64)
    ws = torch.empty(gpu_lib.nvfp4_gated_delta_workspace(400, 2, 1, 2, 128, 64, torch.bfloat16), dtype=torch.uint8, device="cuda")
    slots, starts, cached = ints(d.slots), ints([0, 0, 0]), ints([0, 0])
    after, out = torch.zeros_like(d.state), torch.zeros_like(d.v)

    def call():
        gpu_lib.nvfp4_gated_delta_chunked(d.q, d.k, d.v, d.a, d.b, d.a_log, d.dt_bias, d.state, slots, starts, cached_lens=cached, state_out=after,
                                          out=out, workspace=ws)

    graphs = []
    call()
    torch.cuda.synchronize()
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    log("two graphs")
    for i, (at, have) in enumerate((([0, 100, 400], [0, 3]), ([0, 1, 64], [1, 1]), ([30, 300, 390], [0, 0]), ([0, 400, 400], [2, 0]))):
        starts.copy_(ints(at))
        cached.copy_(ints(have))
        out.zero_(), after.zero_()
        call()
        want = out.clone(), after.clone()
        out.zero_(), after.zero_()
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(after, want[1])


def test_calls_on_two_streams_at_once(gpu_lib):
    rng = np.random.default_rng(22)
    ds = [Delta(rng, "bf16", 600, 2, 2, 4, 128, 64) for _ in range(2)]
    want = [d.run(gpu_lib, [0, 250, 600], after=torch.zeros_like(d.state), out=torch.zeros_like(d.v)) for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    log("two streams")
    afters, outs = [torch.zeros_like(d.state) for d in ds], [torch.zeros_like(d.v) for d in ds]
    starts, slots = ints([0, 250, 600]), [ints(d.slots) for d in ds]
    torch.cuda.synchronize()
    for _ in range(3):
        for d, s, after, out, slot in zip(ds, streams, afters, outs, slots):
            gpu_lib.nvfp4_gated_delta_chunked(d.q, d.k, d.v, d.a, d.b, d.a_log, d.dt_bias, d.state, slot, starts, state_out=after, out=out,
                                              stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(outs, want))


def layer(nv, rows, p, conv_state, state, slots, starts, cached, step=False):
    """From the fused projection's rows (q k v | z | a | b) to the output projection's input."""
    hk, hv, dk, dv = p["heads"]
    qkv_n, z_n = 2 * hk * dk + hv * dv, hv * dv
    t = rows.shape[0]
    x, z = rows[:, :qkv_n], rows[:, qkv_n:qkv_n + z_n].view(t, hv, dv)
    a, b = rows[:, qkv_n + z_n:qkv_n + z_n + hv], rows[:, qkv_n + z_n + hv:]
    out = torch.zeros((t, qkv_n), dtype=rows.dtype, device="cuda")
    if step:
        y = nv.nvfp4_causal_conv_step(x, p["conv"], conv_state, slots, out=out)
    else:
        y = nv.nvfp4_causal_conv(x, p["conv"], conv_state, slots, starts, cached_lens=cached, out=out)
    q, k = y[:, :hk * dk].view(t, hk, dk), y[:, hk * dk:2 * hk * dk].view(t, hk, dk)
    v = y[:, 2 * hk * dk:].view(t, hv, dv)
    o = torch.zeros((t, hv, dv), dtype=rows.dtype, device="cuda")
    if step:
        nv.nvfp4_gated_delta_step(q, k, v, a, b, p["a_log"], p["dt_bias"], state, slots, out=o)
    else:
        nv.nvfp4_gated_delta_chunked(q, k, v, a, b, p["a_log"], p["dt_bias"], state, slots, starts, cached_lens=cached, out=o)
    return nv.nvfp4_group_norm(o, p["norm"], gate=z).view(t, hv * dv)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_layer_in_parts_equals_the_layer_at_once(gpu_lib, dtype):
    """Prompts through quantised projections at once, or in two parts and then token by token, with states carried."""
    nv, rng = gpu_lib, np.random.default_rng(23)
    hk, hv, dk, dv = 2, 4, 64, 64
    hidden, columns = 256, 2 * hk * dk + 2 * hv * dv + 2 * hv
    lens = np.array([150, 90, 66])
    starts = delta_starts(lens)
    g = torch.zeros(2, device="cuda")
    w_in = nv.nvfp4_quantize(dev(rng.standard_normal((columns, hidden)) * 0.1, torch.bfloat16), g[:1], "dynamic")
    x = dev(rng.standard_normal((starts[-1], hidden)), torch.bfloat16)
    ac = nv.nvfp4_quantize(x, g[1:], "dynamic")
    rows = nv.nvfp4_gemm(ac[0], ac[1], g[1:], w_in[0], w_in[1], g[:1], DTYPES[dtype])
    p = dict(heads=(hk, hv, dk, dv), conv=dev(rng.standard_normal((2 * hk * dk + hv * dv, 4)) * 0.5), norm=dev(1 + 0.1 * rng.standard_normal(dv)),
             a_log=dev(np.log(rng.uniform(1, 16, hv))), dt_bias=dev(rng.uniform(-6, -2, hv)))
    slots = ints([4, 0, 2])
    def states():
        return torch.full((5, 3, 2 * hk * dk + hv * dv), 9.0, dtype=DTYPES[dtype], device="cuda"), torch.full((5, hv, dk, dv), 9.0, device="cuda")

    log("layer at once", dtype)
    conv_state, state = states()
    whole = layer(nv, rows, p, conv_state, state, slots, ints(starts), ints([0, 0, 0]))
    log("layer in parts", dtype)
    conv_part, state_part = states()
    got = torch.zeros_like(whole)
    cuts = [np.zeros(3, int), np.array([70, 1, 64]), lens - 2]
    for i in (0, 1):
        idx = [np.arange(starts[r] + cuts[i][r], starts[r] + cuts[i + 1][r]) for r in range(3)]
        at = torch.from_numpy(np.concatenate(idx)).to("cuda")
        got[at] = layer(nv, rows[at], p, conv_part, state_part, slots, ints(delta_starts([len(j) for j in idx])), ints(cuts[i]))
    for i in (0, 1):
        at = torch.from_numpy(starts[:-1] + lens - 2 + i).to("cuda")
        got[at] = layer(nv, rows[at], p, conv_part, state_part, slots, None, None, step=True)
    torch.cuda.synchronize()
    assert torch.equal(conv_part, conv_state)
    assert (host(state_part[1]) == 9.0).all() and (host(state[3]) == 9.0).all()
    # Both are the recurrence within the slacks above, so each is within them of the other.  A head's norm divides by the
    # size of its outputs: what is off is a few of dtype's half steps of the group's largest value.
    for r in (4, 0, 2):
        off = (host(state_part[r]) - host(state[r])) ** 2
        # bf16 inputs are the same in both; the states differ by 32-bit roundings alone
        assert (np.sqrt(off.sum((1, 2))) <= 2.0 ** -19 * np.sqrt((host(state[r]) ** 2).sum((1, 2)))).all()
    size = np.abs(host(whole)).reshape(-1, hv, dv).max(-1, keepdims=True)
    off = np.abs(host(got) - host(whole)).reshape(-1, hv, dv)
    most = 4 * R.HALF_STEP[dtype] if dtype == "bf16" else 2.0 ** -16
    assert (off <= most * size).all(), float((off / size).max())
    # and on into the output projection
    codes, scales = nv.nvfp4_quantize(whole, g[1:], "dynamic")
    w_out = nv.nvfp4_quantize(dev(rng.standard_normal((hidden, hv * dv)) * 0.1, torch.bfloat16), g[:1], "dynamic")
    y = nv.nvfp4_gemm(codes, scales, g[1:], w_out[0], w_out[1], g[:1], DTYPES[dtype])
    torch.cuda.synchronize()
    assert y.shape == (starts[-1], hidden) and torch.isfinite(y).all()
