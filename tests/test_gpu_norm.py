"""The residual norm on the GPU against fp64, element by element.

Bounds, in units u = 2^-24 of fp32.  A row's sum of squares is taken by threads that
add at most 32 terms each, over at most 6 + 16 levels of partial sums: relative error
below 64 u, half of that in k, and four roundings more to y.  Storing adds half a
step of the type.
"""
import numpy as np
import pytest

import block_reference as ref
from block_reference import HALF, U, assert_within
from gpu_helpers import announce, to_gpu, to_np

pytestmark = pytest.mark.gpu

SUM = 64 * U          # relative error of a row's sum of terms of one sign
# every variant of threads per row, both ends of its widths, and widths off the 8-column grid
WIDTHS = [1, 7, 8, 33, 512, 513, 1024, 1027, 2048, 2056, 4096, 4100, 8192, 8195, 16384]


def _make(rows, d, dtype, res_dtype, seed, residual=True):
    rng = np.random.default_rng(seed)
    x = ref.stored(rng.standard_normal((rows, d)), dtype)
    r = ref.stored(3 * rng.standard_normal((rows, d)), res_dtype) if residual else None
    w = (1 + 0.3 * rng.standard_normal(d)).astype(np.float32)
    return x, r, w


def _fwd(x, r, w, dtype, res_dtype, eps=1e-5):
    import torch
    from mlstm_matrix_memory_amd import mlstm_rms_norm_fwd
    y, s = mlstm_rms_norm_fwd(to_gpu(x, dtype), to_gpu(w, "f32"), None if r is None else to_gpu(r, res_dtype), eps=eps)
    torch.cuda.synchronize()
    return to_np(y), to_np(s)


def _check_fwd(x, r, w, dtype, res_dtype, y, s, eps=1e-5):
    total = ref.norm_sum(x, r, dtype if r is None else res_dtype)
    assert np.array_equal(s, total)
    want = ref.norm_fwd(total, w, eps)
    assert_within("y", y, want, np.abs(want) * (HALF[dtype] + SUM / 2 + 5 * U))


@pytest.mark.parametrize("dtype,res_dtype", [("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("d", WIDTHS)
def test_widths(d, dtype, res_dtype):
    announce(f"norm fwd rows=5 d={d} {dtype} residual {res_dtype}")
    x, r, w = _make(5, d, dtype, res_dtype, d)
    _check_fwd(x, r, w, dtype, res_dtype, *_fwd(x, r, w, dtype, res_dtype))


@pytest.mark.parametrize("dtype,res_dtype", [("bf16", "bf16"), ("f32", "f32")])
def test_without_residual(dtype, res_dtype):
    announce(f"norm fwd rows=3 d=100 {dtype} no residual")
    x, _, w = _make(3, 100, dtype, res_dtype, 1, residual=False)
    _check_fwd(x, None, w, dtype, res_dtype, *_fwd(x, None, w, dtype, res_dtype))


def test_rows_of_zeros_and_extremes():
    announce("norm fwd rows of zeros, tiny and huge values, infinities and NaN")
    x, _, w = _make(6, 64, "f32", "f32", 2, residual=False)
    x[0] = 0
    x[1] *= 1e-18
    x[2] *= 1e18
    x[3, 5] = np.inf
    x[4, 7] = np.nan
    y, _ = _fwd(x, None, w, "f32", "f32")
    want = ref.norm_fwd(x.astype(np.float64), w, 1e-5)
    assert np.array_equal(y[0], np.zeros(64))
    for k in (1, 2, 5):
        assert_within(f"y[{k}]", y[k], want[k], np.abs(want[k]) * (SUM + 6 * U) + 1e-37)
    assert np.isnan(y[3, 5]) and np.all(y[3, :5] == 0) and np.all(np.isnan(y[4]))


def test_strided_rows_in_place_and_untouched_neighbours():
    import torch
    from mlstm_matrix_memory_amd import mlstm_rms_norm_fwd
    announce("norm fwd of a column range, residual updated in place")
    rng = np.random.default_rng(3)
    wide = ref.stored(rng.standard_normal((9, 301)), "bf16")
    res = rng.standard_normal((9, 100)).astype(np.float32)
    w = np.ones(100, np.float32)
    g, r = to_gpu(wide, "bf16"), to_gpu(res, "f32")
    y, s = mlstm_rms_norm_fwd(g[:, 101:201], to_gpu(w, "f32"), r, residual_out=r)
    torch.cuda.synchronize()
    assert s is r and np.array_equal(to_np(g), wide)
    _check_fwd(wide[:, 101:201], res, w, "bf16", "f32", to_np(y), to_np(r))


@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("rows,d", [(1, 8), (3, 130), (7, 1000), (2, 4096), (2, 5001), (2, 16384)])
def test_quant(rows, d, group):
    import torch
    from mlstm_matrix_memory_amd import mlstm_rms_norm_quant
    announce(f"norm quant rows={rows} d={d} group={group}")
    x, r, w = _make(rows, d, "bf16", "bf16", 17 * d + group)
    x[0, :min(d, 128)] = 0
    r[0, :min(d, 128)] = 0            # a group (or a whole row) of zeros
    if rows > 1:
        x[1, :64] = r[1, :64] = 2.0 ** -100   # a group whose scale is far below the smallest normal 448 / max
    q, scale, s = mlstm_rms_norm_quant(to_gpu(x, "bf16"), to_gpu(w, "f32"), to_gpu(r, "bf16"), group=group)
    torch.cuda.synchronize()
    total = ref.norm_sum(x, r, "bf16")
    assert np.array_equal(to_np(s), total)
    y = ref.norm_fwd(total, w, 1e-5)
    want, _ = ref.quantise_groups(y, group)
    err = SUM / 2 + 6 * U
    assert_within("scale", to_np(scale), want, want * err + 2.0 ** -149)
    wide = np.repeat(to_np(scale), group or d, axis=-1)[:, :d]
    v = np.where(wide > 0, y / np.where(wide > 0, wide, 1), 0)
    # half a step: 2^-4 of the value, 2^-10 below the smallest normal 2^-6
    assert_within("q", to_np(q), v, np.maximum(np.abs(v) * 2.0 ** -4, 2.0 ** -10) * (1 + 2 ** -10) + np.abs(v) * err * 2)
    assert np.abs(to_np(q)).max() <= 448


@pytest.mark.parametrize("dtype,res_dtype", [("bf16", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,d", [(1, 1), (5, 7), (3, 520), (700, 129), (2100, 64), (4, 1030), (6, 4099), (3, 8200),
                                    (2, 16384)])
def test_backward(rows, d, dtype, res_dtype):
    import torch
    from mlstm_matrix_memory_amd import mlstm_rms_norm_bwd
    announce(f"norm bwd rows={rows} d={d} {dtype} residual {res_dtype}")
    rng = np.random.default_rng(rows + d)
    r = ref.stored(3 * rng.standard_normal((rows, d)), res_dtype)
    dy, dres = ref.stored(rng.standard_normal((rows, d)), dtype), ref.stored(rng.standard_normal((rows, d)), res_dtype)
    w = (1 + 0.3 * rng.standard_normal(d)).astype(np.float32)
    for add in (dres, None):
        gx, gr, gw = mlstm_rms_norm_bwd(to_gpu(r, res_dtype), to_gpu(w, "f32"), to_gpu(dy, dtype),
                                        None if add is None else to_gpu(add, res_dtype))
        torch.cuda.synchronize()
        dr, dw = ref.norm_bwd(r, w, dy, add, 1e-5)
        r64, v = r.astype(np.float64), np.abs(w.astype(np.float64) * dy)
        k = 1 / np.sqrt((r64 * r64).mean(-1, keepdims=True) + 1e-5)
        size = k * (v + np.abs(r64) * k ** 2 * (v * np.abs(r64)).mean(-1, keepdims=True))
        part = size * (2 * SUM + 10 * U) + U * (np.abs(dr) + size)
        assert_within("grad_x", to_np(gx), dr, part + HALF[dtype] * (np.abs(dr) + part))
        assert_within("grad_residual", to_np(gr), dr, part + HALF[res_dtype if res_dtype != dtype else dtype] * (np.abs(dr) + part))
        # rows / 512 terms per part at most 64 parts per thread of the second sum, then 16
        terms = -(-rows // 512) + 128 + 16
        assert_within("grad_weight", to_np(gw), dw, np.abs(dy * r64 * k).sum(0) * (SUM + (5 + terms) * U))


def test_backward_in_place_and_one_output():
    import torch
    from mlstm_matrix_memory_amd import mlstm_rms_norm_bwd
    announce("norm bwd with grad_residual in the place of dres")
    rng = np.random.default_rng(9)
    r, dres = rng.standard_normal((2, 10, 96)).astype(np.float32)
    dy = ref.stored(rng.standard_normal((10, 96)), "bf16")
    w = np.ones(96, np.float32)
    a = [to_gpu(r, "f32"), to_gpu(w, "f32"), to_gpu(dy, "bf16")]
    first = [t.clone() for t in mlstm_rms_norm_bwd(*a, to_gpu(dres, "f32"))]
    g = to_gpu(dres, "f32")
    second = mlstm_rms_norm_bwd(*a, g, grad_residual=g)
    torch.cuda.synchronize()
    assert second[1] is g
    for p, q in zip(first, second):
        assert torch.equal(p, q)
