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
