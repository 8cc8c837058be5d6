"""The gated delta layer at the ends of its inputs' ranges: the same results from the call over prompts and
from the one for single tokens.  Checks, bounds and their reasons are those of test_gpu_gdn."""
import numpy as np
import pytest

from tests import gdn_reference as R
from tests.test_gpu_gdn import DTYPES, NORM_SLACK, Delta, delta_starts, dev, host, ints, log, within

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
