"""Packed sequences of which the first does not start at row 0, on the GPU against fp64:
the rows in front of it stay as they are and enter no sum.  Bounds as in the operators' own tests."""
import numpy as np
import pytest

import scan_cases
import test_gpu_conv as conv
import test_gpu_scan as scan
import test_gpu_scan_bwd as scan_bwd
from gpu_helpers import announce, to_gpu, to_np

pytestmark = pytest.mark.gpu

# rows in front: more than a piece of any of the kernels, and some with pieces of few rows
GAPS = [[700, 705, 705, 738, 1100], [700, 701, 706], [40, 45, 78]]


def sevens(*shape, dtype):
    return to_gpu(np.full(shape, 7.0, np.float32), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("packed", GAPS)
def test_conv(packed, dtype):
    import torch
    from mlstm_matrix_memory_amd import ssm_conv_bwd, ssm_conv_fwd
    announce(f"conv fwd and bwd packed {packed} {dtype}")
    c = conv.make(77, 4, dtype, 3, packed=packed)
    x, w, bias, state = (conv.dev(c, k) for k in ("x", "weight", "bias", "state"))
    y, final = ssm_conv_fwd(x, w, bias, 1, state, y_out=sevens(*x.shape, dtype=dtype), **conv.plan(c))
    got = ssm_conv_bwd(x, w, conv.dev(c, "dy"), bias, 1, state, dstate_final=conv.dev(c, "df"),
                       grad_x=sevens(*x.shape, dtype=dtype), **conv.plan(c))
    torch.cuda.synchronize()
    assert np.all(conv.check_fwd(c, 1, to_np(y), to_np(final)) == 7)
    assert np.all(conv.check_bwd(c, 1, got, packed[-1]) == 7)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("packed", GAPS)
@pytest.mark.parametrize("N", [4, 16, 32])
def test_scan(N, packed, dtype):
    import torch
    announce(f"scan fwd and bwd packed {packed} N={N} {dtype}")
    c = scan_cases.make(37, N, dtype, 4, packed=packed)
    rows = len(c["x"])
    y, final = scan_cases.forward(c, y_out=sevens(rows, 37, dtype=dtype))
    outs = {k: sevens(rows, 37, dtype=dtype) for k in ("grad_x", "grad_z", "grad_dt")}
    outs |= {k: sevens(rows, 1, N, dtype=dtype) for k in ("grad_B", "grad_C")}
    got = scan_bwd.backward(c, **outs)
    torch.cuda.synchronize()
    assert np.all(scan.check(c, y, final, joins=True) == 7)
    assert all(np.all(r == 7) for r in scan_bwd.check(c, got, joins=True))
