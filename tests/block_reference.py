"""The block operators (norm, short convolution, selective scan) and their backward
passes in fp64 numpy, straight from the formulas, and the error bounds they are held to.

Test infrastructure only; shares no code with the library.
"""
import numpy as np

from mlstm_matrix_memory_amd import inputs

# half a step of each storage type, relative to the value
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
U = 2.0 ** -24


def stored(a, dtype):
    """Values as the type holds them."""
    a = np.asarray(a, dtype=np.float32)
    return inputs.bf16_round(a) if dtype == "bf16" else a


def assert_within(name, got, ref, bound):
    """|got - ref| <= bound, element by element; NaN and infinities where ref has them."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{name}: NaN in other places"
    assert np.array_equal(got[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)]), f"{name}: infinities differ"
    over = np.where(fine, np.abs(np.where(fine, got, 0) - np.where(fine, ref, 0)), 0) - np.broadcast_to(bound, ref.shape)
    if over.size and over.max() > 0:
        at = np.unravel_index(int(np.argmax(over)), over.shape)
        raise AssertionError(f"{name}{list(at)}: {got[at]!r}, expected {ref[at]!r} within "
                             f"{np.broadcast_to(bound, ref.shape)[at]:.3g}")


# ---- norm ------------------------------------------------------------------------
def norm_sum(x, residual, res_dtype):
    """r: the fp32 sum rounded to the residual's type (float64 values)."""
    total = np.asarray(x, np.float32) + (np.float32(0) if residual is None else np.asarray(residual, np.float32))
    return stored(total, res_dtype).astype(np.float64)


def norm_fwd(r, weight, eps):
    k = 1 / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    return r * k * np.asarray(weight, np.float64)


def norm_bwd(r, weight, dy, dres, eps):
    r, w, dy = (np.asarray(a, np.float64) for a in (r, weight, dy))
    k = 1 / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    v = w * dy
    dr = k * (v - r * k ** 2 * (v * r).mean(-1, keepdims=True))
    if dres is not None:
        dr = dr + np.asarray(dres, np.float64)
    return dr, (dy * r * k).reshape(-1, r.shape[-1]).sum(0)


def quantise_groups(y, group):
    """(largest |y| / 448 per group, the same spread over the columns)."""
    d = y.shape[-1]
    n = group or d
    starts = np.arange(0, d, n)
    scale = np.maximum.reduceat(np.abs(y), starts, axis=-1) / 448.0
    return scale, np.repeat(scale, n, axis=-1)[..., :d]


# ---- sequences ---------------------------------------------------------------------
def sequences(B, S, seq_start=None):
    """[(first row, one past the last row)] of a batch."""
    if seq_start is None:
        return [(b * S, (b + 1) * S) for b in range(B)]
    return [(int(a), int(z)) for a, z in zip(seq_start[:-1], seq_start[1:])]


# ---- short causal convolution ----------------------------------------------------------
def _sigmoid(x):
    return 0.5 * (1 + np.tanh(0.5 * x))


def conv_fwd(x, weight, bias, state, spans, act):
    """x [rows,D], state [B,W-1,D]; returns (y [rows,D], final state, sum of |terms| of p)."""
    x, w, state = (np.asarray(a, np.float64) for a in (x, weight, state))
    bias = np.zeros(x.shape[1]) if bias is None else np.asarray(bias, np.float64)
    W = w.shape[1]
    y, final, size = np.zeros_like(x), state.copy(), np.zeros_like(x)
    for b, (lo, hi) in enumerate(spans):
        line = np.concatenate([state[b], x[lo:hi]])
        n = hi - lo
        taps = [w[:, j] * line[j:j + n] for j in range(W)]
        p = bias + sum(taps)
        size[lo:hi] = np.abs(bias) + sum(np.abs(t) for t in taps)
        y[lo:hi] = p * _sigmoid(p) if act else p
        final[b] = line[n:]
    return y, final, size


def conv_bwd(x, weight, bias, state, spans, act, dy, dfinal):
    """Returns dict of gradients x, weight, bias, state, and of the sums of the absolute
    values of each one's terms (size_*)."""
    x, w, state, dy = (np.asarray(a, np.float64) for a in (x, weight, state, dy))
    bias = np.zeros(x.shape[1]) if bias is None else np.asarray(bias, np.float64)
    W = w.shape[1]
    g = {"x": np.zeros_like(x), "weight": np.zeros_like(w), "bias": np.zeros_like(bias), "state": np.zeros_like(state)}
    g.update({f"size_{k}": np.zeros_like(v) for k, v in g.items()})
    for b, (lo, hi) in enumerate(spans):
        line = np.concatenate([state[b], x[lo:hi]])
        n = hi - lo
        p = bias + sum(w[:, j] * line[j:j + n] for j in range(W))
        s = _sigmoid(p)
        dp = dy[lo:hi] * (s * (1 + p * (1 - s))) if act else dy[lo:hi]
        dline, size = np.zeros_like(line), np.zeros_like(line)
        if dfinal is not None:
            dline[n:] += dfinal[b]
            size[n:] += np.abs(dfinal[b])
        for j in range(W):
            dline[j:j + n] += w[:, j] * dp
            size[j:j + n] += np.abs(w[:, j] * dy[lo:hi])
            g["weight"][:, j] += (dp * line[j:j + n]).sum(0)
            g["size_weight"][:, j] += np.abs(dy[lo:hi] * line[j:j + n]).sum(0)
        g["bias"] += dp.sum(0)
        g["size_bias"] += np.abs(dy[lo:hi]).sum(0)
        g["x"][lo:hi], g["state"][b] = dline[W - 1:], dline[:W - 1]
        g["size_x"][lo:hi], g["size_state"][b] = size[W - 1:], size[:W - 1]
    return g
