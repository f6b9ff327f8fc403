"""The norm's e4m3 output is the quotient y / scale, rounded to the nearest e4m3 value, of the
y that the fp32 norm gives and the scale that it returns: whole values, no tolerance."""
import numpy as np
import pytest

import block_reference as ref
from gpu_helpers import announce, to_gpu, to_np

pytestmark = pytest.mark.gpu


def e4m3(v):
    """Nearest e4m3 value, ties to the even one: steps of 2^(exponent - 3), of 2^-9 below 2^-6."""
    v = np.asarray(v, np.float64)
    exponent = np.frexp(np.where(v == 0, 1, v))[1] - 1
    step = 2.0 ** (np.maximum(exponent, -6) - 3)
    return np.rint(v / step) * step


def beside_ties(largest):
    """126 values whose quotients by scale = largest / 448 lie beside the middle of two e4m3
    values, on one side or the other by at most a unit in the last place of the value."""
    scale = np.float32(largest) / np.float32(448)
    values = e4m3(np.concatenate([np.arange(8) * 2.0 ** -9] + [2.0 ** e * (1 + np.arange(8) / 8) for e in range(-6, 9)]))
    values = values[values <= 448]
    ties = ((values[1:] + values[:-1]) / 2)[:126]
    y = (ties * np.float64(scale)).astype(np.float32)
    return np.nextafter(y, np.where(np.arange(126) % 3 == 0, np.float32(0), np.where(np.arange(126) % 3 == 1, y, np.float32(1e38))),
                        dtype=np.float32)


@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("size", [1.0, 2.0 ** 100, 2.0 ** -60, 2.0 ** -100, 2.0 ** -115])
def test_values_beside_ties(size, group):
    import torch
    from mlstm_matrix_memory_amd import mlstm_rms_norm_quant
    announce(f"norm quant of quotients beside ties, group={group}, weights near {size:g}")
    # rows of +-1 with eps = 0 have k = 1 exactly, so y = +-weight
    rng = np.random.default_rng(3)
    for seed in range(20):
        n = group or 128
        w = np.concatenate([np.concatenate([[m], rng.permutation(beside_ties(m))[:n - 1]])[:n] for m in
                            (rng.uniform(0.5, 2, 128 // n) * size).astype(np.float32)]).astype(np.float32)
        x = rng.choice([-1.0, 1.0], (3, len(w))).astype(np.float32)
        q, scale, _ = mlstm_rms_norm_quant(to_gpu(x, "f32"), to_gpu(w, "f32"), eps=0.0, group=group)
        torch.cuda.synchronize()
        y = x * w
        starts = np.arange(0, len(w), n)
        s = np.maximum.reduceat(np.abs(y), starts, axis=-1) / np.float32(448)
        assert np.array_equal(to_np(scale), s)
        assert np.array_equal(to_np(q), e4m3(y / np.repeat(s, n, axis=-1)[:, :len(w)]))


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", [(2000, 500), (1000, 1001), (700, 2048), (500, 4096), (300, 8192), (150, 16384)])
def test_quotients_of_the_fp32_norm(rows, d, dtype, group):
    import torch
    from mlstm_matrix_memory_amd import mlstm_rms_norm_fwd, mlstm_rms_norm_quant
    announce(f"norm quant against the fp32 norm's values, rows={rows} d={d} residual {dtype} group={group}")
    rng = np.random.default_rng(d)
    x = rng.standard_normal((rows, d)).astype(np.float32)
    r = ref.stored(3 * rng.standard_normal((rows, d)), dtype)
    w = (1 + 0.3 * rng.standard_normal(d)).astype(np.float32)
    a = (to_gpu(x, "f32"), to_gpu(w, "f32"), to_gpu(r, dtype))
    y, _ = mlstm_rms_norm_fwd(*a)
    q, scale, _ = mlstm_rms_norm_quant(*a, group=group)
    torch.cuda.synchronize()
    y = y.cpu().numpy()
    n = group or d
    s = np.maximum.reduceat(np.abs(y), np.arange(0, d, n), axis=-1) / np.float32(448)
    assert np.array_equal(scale.cpu().numpy().reshape(s.shape), s)
    assert np.array_equal(to_np(q), e4m3(y / np.repeat(s, n, axis=-1)[:, :d]))


def test_a_scale_below_the_smallest_normal_number():
    """Its rounding would move the quotients: they are taken with max |y| / 448 unrounded."""
    import torch
    from mlstm_matrix_memory_amd import mlstm_rms_norm_quant
    announce("norm quant with scales below 2^-126")
    w = np.array([1, -0.5, 0.25, 1 / 448, 0, 0.7, -1, 0.125], np.float32) * np.float32(2.0 ** -130)
    x = np.ones((1, 8), np.float32)
    q, scale, _ = mlstm_rms_norm_quant(to_gpu(x, "f32"), to_gpu(w, "f32"), eps=0.0)
    torch.cuda.synchronize()
    want = w.astype(np.float64) / np.abs(w).max() * 448
    assert np.array_equal(to_np(q)[0], e4m3(want))
    assert abs(to_np(scale)[0, 0] - 2.0 ** -130 / 448) <= 2.0 ** -150


def test_infinities_and_nan():
    """A y that is infinite makes its group's scale infinite, its own q NaN and the others 0; a y that is NaN has
    a NaN q and does not enter the maximum.  Other groups and rows are as without them."""
    import torch
    from mlstm_matrix_memory_amd import mlstm_rms_norm_quant
    announce("norm quant with infinities and NaN in the weight and in x")
    rng = np.random.default_rng(5)
    x, w = rng.standard_normal((4, 128)).astype(np.float32), np.ones(128, np.float32)
    clean, clean_scale, _ = (to_np(t) for t in mlstm_rms_norm_quant(to_gpu(x, "f32"), to_gpu(w, "f32"), group=32))
    w[5], w[40] = np.inf, np.nan
    q, scale, _ = (to_np(t) for t in mlstm_rms_norm_quant(to_gpu(x, "f32"), to_gpu(w, "f32"), group=32))
    assert np.all(np.isnan(q[:, [5, 40]])) and np.all(scale[:, 0] == np.inf) and np.all(np.delete(q[:, :32], 5, 1) == 0)
    rest = np.delete(np.arange(32, 64), 8)
    largest = np.argmax(np.abs(x[:, 32:64]), 1) + 32
    for row in range(4):
        if largest[row] != 40:
            assert scale[row, 1] == clean_scale[row, 1] and np.array_equal(q[row, rest], clean[row, rest])
    assert np.array_equal(q[:, 64:], clean[:, 64:]) and np.array_equal(scale[:, 2:], clean_scale[:, 2:])
    x[1, 3] = np.nan
    w[:] = 1
    q, scale, _ = (to_np(t) for t in mlstm_rms_norm_quant(to_gpu(x, "f32"), to_gpu(w, "f32"), group=32))
    assert np.all(np.isnan(q[1])) and np.all(scale[1] == 0)
    keep = [0, 2, 3]
    assert np.array_equal(q[keep], clean[keep]) and np.array_equal(scale[keep], clean_scale[keep])
