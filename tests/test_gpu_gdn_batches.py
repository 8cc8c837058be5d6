"""The gated delta layer's calls over batches of unusual make, and of the sizes at which variants
begin and end: many sequences without rows, convolutions of 8, 16 and 32 rows a thread,
sequences whole and in parts.  Checks, bounds and their
reasons are those of test_gpu_gdn."""
import numpy as np
import pytest

from tests.test_gpu_gdn import Delta, check_conv, conv_inputs, delta_starts, ints, log

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


# (type, channels, tokens, rows a thread): just below and from what takes more of them on, a card of 256 CUs supposed
CONV_ROWS = [("f32", 1032, 3279, 8), ("f32", 1032, 3280, 16), ("f32", 1032, 9023, 16), ("f32", 1032, 9024, 32),
             ("bf16", 1032, 5455, 8), ("bf16", 1032, 15039, 16), ("bf16", 1032, 15040, 32), ("f16", 1032, 5456, 8), ("f16", 1032, 15039, 16),
             ("f16", 1032, 16500, 32), ("bf16", 135, 40000, 16)]


def conv_columns(dtype, channels):
    """Waves of a row: vectors of 16 bytes where rows are made of them, 64 a wave."""
    each = (4 if dtype == "f32" else 8) if channels % 8 == 0 else 1
    return -(-channels // (64 * each))


@pytest.mark.parametrize("dtype,channels,tokens,rows", CONV_ROWS)
@pytest.mark.parametrize("width", [2, 3, 4])
def test_conv_of_every_number_of_rows(gpu_lib, dtype, channels, tokens, rows, width):
    """Sequences that begin and end around a thread's rows, one left out, rows behind the last."""
    rng = np.random.default_rng([channels, tokens, width])
    lens = [1000, 1, 31, 32, 33, 0, 2, 999, 3, 8, 16]
    lens.append(tokens - 5 - sum(lens))
    log("conv rows", dtype, channels, tokens, rows, width)
    x, weight, bias, state, slots = conv_inputs(rng, tokens, channels, width, dtype, len(lens))
    slots[3] = -1
    check_conv(gpu_lib, dtype, x, weight, bias, "silu", state, slots, delta_starts(lens), rng.integers(0, 2, len(lens)), in_place=width == 4)


# (heads, lengths, parts that a sequence may have): 0 where whole ones are faster
PARTS = [((1, 2, 128, 128), [2044], 0), ((1, 2, 128, 128), [2045], 4), ((2, 2, 64, 64), [2100], 4), ((1, 6, 128, 128), [300, 4000, 0, 700], 9),
         ((1, 3, 128, 64), [5, 513, 2600], 6), ((1, 1, 128, 256), [2500, 64], 5), ((2, 4, 64, 192), [2300], 4), ((20, 20, 64, 128), [3600], 7),
         ((1, 6, 64, 64), [150] * 8, 0), ((1, 6, 64, 64), [400] * 8, 0), ((1, 1, 64, 64), [260] * 16, 0), ((8, 24, 64, 128), [1536], 0)]
BEHIND = 3  # rows behind the last sequence


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("heads,lens,parts", PARTS)
def test_chunked_whole_and_in_parts(gpu_lib, dtype, heads, lens, parts):
    rng = np.random.default_rng([len(lens), *heads, 6])
    log("whole and in parts", dtype, heads, lens, parts)
    starts = delta_starts(lens)
    d = Delta(rng, dtype, int(starts[-1]) + BEHIND, len(lens), *heads, decay=0.05)
    if len(lens) > 3:
        d.slots[3] = -1
    d.check(gpu_lib, starts, cached=np.arange(len(lens)) % 2, in_place=len(lens) == 1)


def test_prompts_in_parts_in_graphs_of_one_workspace(gpu_lib):
    """Replays follow the starts, lengths of 0 and 1 among them, and share a workspace with eager calls between them."""
    rng = np.random.default_rng(31)
    tokens = 2600
    d = Delta(rng, "bf16", tokens, 2, 1, 2, 128, 64, decay=0.05)
    ws = torch.empty(gpu_lib.nvfp4_gated_delta_workspace(tokens, 2, 1, 2, 128, 64, torch.bfloat16), dtype=torch.uint8, device="cuda")
    slots, starts, cached = ints(d.slots), ints([0, 0, 0]), ints([0, 0])
    after, out = torch.zeros_like(d.state), torch.zeros_like(d.v)

    def call():
        gpu_lib.nvfp4_gated_delta_chunked(d.q, d.k, d.v, d.a, d.b, d.a_log, d.dt_bias, d.state, slots, starts, cached_lens=cached,
                                          state_out=after, out=out, workspace=ws)

    graphs = []
    call()
    torch.cuda.synchronize()
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    log("graphs in parts")
    for i, (at, have) in enumerate((([0, 2100, 2600], [0, 3]), ([0, 1, 2600], [1, 1]), ([30, 30, 2590], [0, 0]), ([0, 1300, 1300], [2, 0]))):
        starts.copy_(ints(at))
        cached.copy_(ints(have))
        out.zero_(), after.zero_()
        call()
        want = out.clone(), after.clone()
        out.zero_(), after.zero_()
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(after, want[1]), i
    checked = d.check(gpu_lib, [0, 1300, 1300], cached=[2, 0])
    assert torch.equal(checked[1][d.slots[0]], after[d.slots[0]])
