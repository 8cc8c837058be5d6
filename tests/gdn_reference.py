"""Plain references for the gated delta layer's tests: numpy in 64 bits, one token
after another.  TEST INFRASTRUCTURE ONLY.

Each returns the outputs and what sizes the roundings of a 32-bit evaluation are
relative to."""
import numpy as np

HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # of a rounding, relative to the value
LEAST = {"f32": 2.0 ** -150, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}  # half the smallest subnormal: a rounding below the normal range


def silu(x):
    return x / (1.0 + np.exp(-x))


def spans(starts, slots, num_slots, tokens):
    """(sequence, first row, end, slot) of the sequences that are not left out."""
    for r in range(len(slots)):
        low, high = (min(max(int(s), 0), tokens) for s in starts[r:r + 2])
        if low < high and 0 <= slots[r] < num_slots:
            yield r, low, high, int(slots[r])


def conv(x, weight, bias, act, state, slots, starts, cached, out):
    """(out, sizes, state_out); out: what stands there before the call."""
    out, after = np.array(out), np.array(state)
    sizes = np.zeros_like(out)
    w = weight.shape[1]
    for r, low, high, slot in spans(starts, slots, len(state), len(x)):
        old = state[slot] if cached is None or cached[r] > 0 else np.zeros_like(state[slot])
        seen = np.concatenate([old, x[low:high]])
        for t in range(low, high):
            rows = seen[t - low:t - low + w]
            y = (rows * weight.T).sum(0) + bias
            sizes[t] = np.abs(rows * weight.T).sum(0) + np.abs(bias)
            out[t] = silu(y) if act else y
        after[slot] = seen[len(seen) - (w - 1):]
    return out, sizes, after


def delta(q, k, v, a, b, a_log, dt_bias, scale, eps, state, slots, starts, cached, out, least=0.0):
    """(out, out_slack, state_out, state_slack, floors): slacks grow as a rounding of 1 relative to
    what is added would, a token: columns of the state are compared by their length, since
    each step mixes the rows.  (1 - beta k k^T) e^g shortens every error it meets.  e^g is off
    by |g| times g's own roundings.  Beside that, `least` of the largest beta v and state of a
    column within 64 tokens, which stays in the state behind them; `floors` are the last ones."""
    out, after = np.array(out), np.array(state)
    out_slack, state_slack, floors = np.zeros_like(out), np.zeros_like(state), np.zeros_like(state[:, :, 0])
    group = v.shape[1] // k.shape[1]
    x = a + dt_bias
    decay = np.exp(a_log) * np.logaddexp(0.0, x)
    alpha = np.exp(-decay)
    beta = 1.0 / (1.0 + np.exp(-b))
    unit = lambda y: np.repeat(y / np.sqrt((y * y).sum(-1, keepdims=True) + eps), group, 1)
    kn, qn = unit(k), unit(q)
    for r, low, high, slot in spans(starts, slots, len(state), len(q)):
        s = np.array(state[slot]) if cached is None or cached[r] > 0 else np.zeros_like(state[slot])
        off = floor = np.zeros(s.shape[::2])  # [heads, head_v]
        for t in range(low, high):
            if (t - low) % 64 == 0:
                rows = slice(t, min(t + 64, high))
                off = off + floor
                floor = least * np.maximum(np.abs(s).max(1), (beta[rows][..., None] * np.abs(v[rows])).max(0))
            was = np.sqrt((s * s).sum(1))
            s = s * alpha[t][:, None, None]
            d = beta[t][:, None] * (v[t] - np.einsum("hk,hkv->hv", kn[t], s))
            s = s + kn[t][:, :, None] * d[:, None, :]
            off = off * alpha[t][:, None] + was * (alpha[t] * (1.0 + decay[t]))[:, None] + beta[t][:, None] * np.abs(v[t])
            out[t] = scale * np.einsum("hk,hkv->hv", qn[t], s)
            out_slack[t] = scale * (off + np.sqrt((s * s).sum(1)) + floor)
        after[slot], state_slack[slot] = s, (off + floor)[:, None, :]
        floors[slot] = floor
    return out, out_slack, after, state_slack, floors


def norm(x, weight, bias, gate, act, centred, eps):
    """(out, sizes)"""
    m = x.mean(-1, keepdims=True) if centred else 0.0
    root = np.sqrt(((x - m) ** 2).mean(-1, keepdims=True) + eps)
    y = (x - m) / root * weight + bias
    # a mean of values that cancel is off by roundings of what is summed, not of itself
    sizes = (np.abs(x) + np.abs(x).mean(-1, keepdims=True)) / root * np.abs(weight) + np.abs(bias)
    f = silu if act else (lambda z: z)
    if gate is None:
        return f(y), sizes
    return y * f(gate), sizes * np.abs(gate)
