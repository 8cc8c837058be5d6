"""The gated delta layer at the ends of its inputs' ranges: the same results from the call over prompts and
from the one for single tokens.  Checks, bounds and their reasons are those of test_gpu_gdn."""
import numpy as np
import pytest

from tests import gdn_reference as R
from tests.test_gpu_gdn import DELTA_LEAST, DELTA_SLACK, DTYPES, NORM_SLACK, Delta, delta_starts, dev, host, ints, log, within

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


class Ranged(Delta):
    """With an eps of its own."""
    eps = 1e-6

    def want(self, starts, cached, out, least=0.0):
        # at 0, as far below every square of a 32-bit number: rows of zeros are zeros then
        return R.delta(*(host(t) for t in (self.q, self.k, self.v, self.a, self.b, self.a_log, self.dt_bias)), self.scale,
                       max(self.eps, 1e-200), host(self.state), self.slots, starts, cached, out, least)

    def run(self, nv, starts, cached=None, step=False, state=None, after=None, out=None, **kw):
        args = (self.q, self.k, self.v, self.a, self.b, self.a_log, self.dt_bias, state, ints(self.slots))
        kw = dict(kw, scale=self.scale, eps=self.eps, state_out=after, out=out)
        return nv.nvfp4_gated_delta_step(*args, **kw) if step else nv.nvfp4_gated_delta_chunked(*args, ints(starts), **kw)


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("dtype,low,high", [("f32", -30, 30), ("bf16", -30, 30), ("f16", -6, 2)])
@pytest.mark.parametrize("head_k", [64, 128])
def test_keys_of_any_size(gpu_lib, step, eps, dtype, low, high, head_k):
    """Finite keys and queries are normalised whatever their size, rows of zeros stay zeros."""
    rng = np.random.default_rng([head_k, high])
    log("key sizes", step, eps, dtype, head_k)
    tokens, starts = 140, delta_starts([75, 65])
    d = Ranged(rng, dtype, tokens, tokens if step else 2, 1, 2, head_k, 64)
    d.eps = eps
    for t, sizes in ((d.k, 10.0 ** rng.uniform(low, high, tokens)), (d.q, 10.0 ** rng.uniform(low, high, tokens))):
        t *= torch.from_numpy(sizes).to("cuda")[:, None, None].to(t.dtype)
    d.k[::7] = 0.0
    d.q[1::5] = 0.0
    d.k[4] = d.q[4] = 0.0
    for _ in range(2):
        d.check(gpu_lib, np.arange(tokens + 1) if step else starts, step=step)
        d.k[:, :, 5] *= 100.0  # one element far above the rest
        d.q[:, :, 6] *= 100.0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,step", [([200, 130], False), ([2700, 65], False), ([1] * 7, True)])  # the second in parts
@pytest.mark.parametrize("which", ["a", "b", "k", "v"])
def test_a_nan_reaches_the_state(gpu_lib, dtype, lens, step, which):
    """And no other sequence, head or column of it."""
    rng = np.random.default_rng(len(lens))
    log("nan", dtype, lens, step, which)
    starts = delta_starts(lens)
    d = Delta(rng, dtype, int(starts[-1]), len(lens), 1, 2, 64, 64, decay=0.05)

    def call():
        after = torch.zeros_like(d.state)
        out = d.run(gpu_lib, starts, step=step, state=d.state, after=after, out=torch.zeros_like(d.v))
        torch.cuda.synchronize()
        return out, after

    clean = call()
    tensor = getattr(d, which)
    for token in {0, min(70, lens[0] - 1), lens[0] - 1}:
        where = {"a": (token, 1), "b": (token, 1), "k": (token, 0, 9), "v": (token, 1, 21)}[which]
        was = tensor[where].clone()
        tensor[where] = float("nan")
        out, after = call()
        tensor[where] = was
        at = (d.slots[0], slice(None) if which == "k" else 1) + ((slice(None), 21) if which == "v" else ())
        assert after[at].isnan().all(), token
        want = clean[1].clone()
        want[at] = after[at]
        assert torch.equal(after.nan_to_num(7.0), want.nan_to_num(7.0)), token
        assert torch.equal(out[lens[0]:], clean[0][lens[0]:]), token


@pytest.mark.parametrize("eps", [0.0, 1e-36, 1e-6, 1e30])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [1, 16, 121, 128, 200, 256, 300, 512, 1024, 4096, 4100, 8191, 8192])
@pytest.mark.parametrize("centred", [False, True])
def test_norm_of_groups_of_any_size(gpu_lib, eps, dtype, dim, centred):
    """From 10^-36 to 10^37, each group of a token another one, and a group of zeros: squares that overflow or vanish."""
    rng = np.random.default_rng([dim, 5])
    log("norm of any size", eps, dtype, dim, centred)
    tokens, groups = 5, 7
    sizes = 10.0 ** rng.uniform(-36, 37, (tokens, groups, 1))
    sizes[0, 0], sizes[1, 1], sizes[2, 2] = 0.0, 1e-36, 1e37
    x = rng.standard_normal((tokens, groups, dim)) * sizes
    x[3, 3], x[4, 4] = 3.3e38, -3.3e38  # sums overflow too
    x[3, 4, ::2], x[3, 4, 1::2] = 3.3e38, -3.3e38
    x = dev(x, DTYPES[dtype])
    weight, bias = dev(1 + 0.3 * rng.standard_normal((groups, dim))), dev(rng.standard_normal((groups, dim)))
    if centred:  # without differences beyond roundings, and eps nothing beside them, nothing is defined
        x[3, 3], x[4, 4] = x[3, 4], -x[3, 4]
        if dim == 1:
            x[:] = 0.0
    want, sizes = R.norm(host(x), host(weight), host(bias), None, False, centred, max(eps, 1e-200))
    got = gpu_lib.nvfp4_group_norm(x, weight, bias=bias, activation="none", centred=centred, eps=eps)
    torch.cuda.synchronize()
    within(got, want, NORM_SLACK * sizes, dtype, "norm")


IN_PARTS = 2113  # tokens of one sequence of few heads that are taken in parts


def check_without_shortening(d, nv, starts):
    """Delta.check for keys along one line that nothing decays.  Its bound on a state's length, 2^-20 of it, is that of a
    chunk's roundings, which the rule shortens from chunk to chunk.  Across such keys it shortens nothing: each of n chunks
    leaves its own rounding, at most 2^-20 and independent of the others', and their sum has a length of 2^-20 sqrt(n)."""
    out, after = torch.zeros_like(d.v), torch.full_like(d.state, 3.0)
    was = host(after)
    want, slack, left, left_slack, floors = d.want(np.asarray(starts), None, host(out), DELTA_LEAST)
    slot = d.slots[0]
    was[slot] = left[slot]
    d.run(nv, starts, None, False, d.state, after, out)
    torch.cuda.synchronize()
    within(out, want, DELTA_SLACK * slack, d.dtype, "out")
    within(after, was, DELTA_SLACK * left_slack, "f32", "state")
    off, length = (np.sqrt((x ** 2).sum((1, 2))) for x in (host(after)[slot] - left[slot], left[slot]))
    chunks = -(-(starts[1] - starts[0]) // 64)
    assert (off <= 2.0 ** -20 * chunks ** 0.5 * length + DELTA_SLACK * np.sqrt((floors[slot] ** 2).sum(1))).all(), (off / length)


@pytest.mark.parametrize("case", ["no decay", "full decay", "mixed", "beta 0", "beta 1", "same key", "opposed keys", "zero keys", "zero all"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gates_and_keys_at_their_ends_in_parts(gpu_lib, case, dtype):
    rng = np.random.default_rng(40)
    log("ends in parts", case, dtype)
    d = Delta(rng, dtype, IN_PARTS + 2, 1, 1, 2, 64, 64, extra=8)
    if case == "no decay":
        d.a.fill_(-100.0)
        d.dt_bias.fill_(-50.0)
    elif case == "full decay":
        d.a.fill_(100.0)
        d.a_log.fill_(4.0)
    elif case == "mixed":
        d.a_log.fill_(2.5)
        d.a.copy_(torch.where(torch.rand(d.a.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(1)) < 0.3, 60.0, -12.0))
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
    if case in ("same key", "opposed keys"):
        check_without_shortening(d, gpu_lib, [1, IN_PARTS + 1])
    else:
        d.check(gpu_lib, [1, IN_PARTS + 1], out_extra=8)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [1e-20, 300.0, 1e15])
def test_values_of_any_size_in_parts(gpu_lib, dtype, size):
    rng = np.random.default_rng(41)
    log("size in parts", dtype, size)
    Delta(rng, dtype, IN_PARTS, 1, 1, 2, 64, 64, size=size, decay=0.05).check(gpu_lib, [0, IN_PARTS])


@pytest.mark.parametrize("down", [False, True])
@pytest.mark.parametrize("strong", [False, True])
def test_values_that_grow_and_shrink_in_parts(gpu_lib, down, strong):
    """Values pass 36 powers of ten, states with them, so that parts start from states far from what they add."""
    rng = np.random.default_rng(42)
    log("growing in parts", down, strong)
    d = Delta(rng, "f32", IN_PARTS, 1, 1, 2, 64, 64)
    climb = np.linspace(18, -18, IN_PARTS) if down else np.linspace(-18, 18, IN_PARTS)
    d.v *= dev(10.0 ** climb)[:, None, None]
    d.a += 4.0 if strong else -2.0
    d.check(gpu_lib, [0, IN_PARTS])
