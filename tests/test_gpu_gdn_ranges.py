"""The gated delta layer at the ends of its inputs' ranges: the same results from the call over prompts and
from the one for single tokens.  Checks, bounds and their reasons are those of test_gpu_gdn."""
import numpy as np
import pytest

from tests import gdn_reference as R
from tests.test_gpu_gdn import Delta, delta_starts, host, ints, log

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
