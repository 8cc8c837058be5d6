"""The gated delta layer's calls over batches of unusual make: many sequences without rows.  Checks, bounds and their
reasons are those of test_gpu_gdn."""
import numpy as np
import pytest

from tests.test_gpu_gdn import check_conv, conv_inputs, delta_starts, ints, log

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype,channels", [("bf16", 24), ("f32", 5)])
def test_conv_among_many_sequences_without_rows(gpu_lib, dtype, channels):
    """Sequences without rows, before, between and behind those that have some, are not walked over one by one."""
    rng = np.random.default_rng(30)
    lens = [0] * 20000 + [5] + [0] * 40000 + [1, 0, 2] + [0] * 30000 + [29] + [0] * 20000
    starts = delta_starts(lens)
    tokens = int(starts[-1]) + 3  # rows behind the last sequence
    log("conv, many without rows", dtype, channels)
    x, weight, bias, state, slots = conv_inputs(rng, tokens, channels, 4, dtype, len(lens))
    check_conv(gpu_lib, dtype, x, weight, bias, "silu", state, slots, starts, rng.integers(0, 2, len(lens)))
    given, at, out, after = ints(slots), ints(starts), torch.empty_like(x), torch.empty_like(state)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(10):
        gpu_lib.nvfp4_causal_conv(x, weight, state, given, at, bias=bias, state_out=after, out=out)
    end.record()
    torch.cuda.synchronize()
    # a step over a sequence is a load that waits, 0.1 us at least: 40000 of them, 4 ms; a bisection has 17
    assert begin.elapsed_time(end) / 10 < 1.0
