"""The short causal convolution on the GPU against fp64, element by element.

Bounds, in units u = 2^-24: p is a chain of W multiply-adds, each within u of the sum
of its terms' absolute values (size), so within (W + 1) u size.  |d swish| <= 1.1 and
the sigmoid (hardware exponential and reciprocal, their argument's rounding included)
is within (4 + |p|) u, so y is within (1.1 (W + 1) size + (6 + |p|) |p|) u; storing adds
half a step.  A derivative of swish carries the same errors, on dy.
"""
import numpy as np
import pytest

import block_reference as ref
from block_reference import HALF, U, assert_within
from gpu_helpers import announce, to_gpu, to_np

pytestmark = pytest.mark.gpu

PACKED = [0, 5, 5, 6, 39, 41, 44, 177]            # lengths 5, 0, 1, 33, 2, 3, 133


def make(D, W, dtype, seed, B=2, S=9, packed=None, bias=True, state=True):
    rng = np.random.default_rng(seed)
    rows = (packed[-1] + 3) if packed else B * S  # packed: three rows behind the last sequence
    B = len(packed) - 1 if packed else B
    c = {"x": ref.stored(rng.standard_normal((rows, D)), dtype), "weight": rng.standard_normal((D, W)).astype(np.float32),
         "bias": rng.standard_normal(D).astype(np.float32) if bias else None,
         "state": ref.stored(rng.standard_normal((B, W - 1, D)), dtype) if state else None,
         "dy": ref.stored(rng.standard_normal((rows, D)), dtype),
         "df": ref.stored(rng.standard_normal((B, W - 1, D)), dtype) if state else None,
         "spans": ref.sequences(B, S, packed), "B": B, "S": S, "W": W, "D": D, "dtype": dtype, "packed": packed}
    c["state64"] = c["state"] if state else np.zeros((B, W - 1, D))
    return c


def dev(c, key):
    a = c[key]
    if a is None:
        return None
    t = to_gpu(a, "f32" if key in ("weight", "bias") else c["dtype"])
    return t if c["packed"] or key not in ("x", "dy") else t.view(c["B"], c["S"], c["D"])


def plan(c):
    import torch
    if not c["packed"]:
        return {}
    return {"seq_start": torch.tensor(c["packed"], dtype=torch.int32, device="cuda"),
            "max_len": int(np.diff(c["packed"]).max())}


def bound_y(c, y, size, act):
    e = (c["W"] + 1) * size
    if act:
        e = 1.1 * e + (6 + size) * size
    return e * U + HALF[c["dtype"]] * (np.abs(y) + e * U)


def check_fwd(c, act, y, final):
    want, last, size = ref.conv_fwd(c["x"], c["weight"], c["bias"], c["state64"], c["spans"], act)
    inside = np.zeros(len(want), bool)
    for lo, hi in c["spans"]:
        inside[lo:hi] = True
    y = y.reshape(want.shape)
    assert_within("y", y[inside], want[inside], bound_y(c, want, size, act)[inside])
    assert np.array_equal(final, last)
    return y[~inside]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("D", [1, 8, 13, 200, 4096])
def test_forward(D, W, dtype):
    import torch
    from mlstm_matrix_memory_amd import ssm_conv_fwd
    for act, bias, state, S in ((1, True, True, 9), (0, False, False, 1), (1, False, True, 2), (1, True, False, 131)):
        announce(f"conv fwd B=2 S={S} D={D} W={W} {dtype} act={act} bias={bias} state={state}")
        c = make(D, W, dtype, D + W, S=S, bias=bias, state=state)
        y, final = ssm_conv_fwd(dev(c, "x"), dev(c, "weight"), dev(c, "bias"), act, dev(c, "state"))
        torch.cuda.synchronize()
        check_fwd(c, act, to_np(y), to_np(final))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [24, 515])
def test_packed_strided_and_rows_left_alone(D, dtype):
    import torch
    from mlstm_matrix_memory_amd import ssm_conv_fwd
    announce(f"conv fwd packed {PACKED} D={D} {dtype}, x and y column ranges of one buffer")
    c = make(D, 4, dtype, D, packed=PACKED)
    rows = len(c["x"])
    wide = to_gpu(np.full((rows, 2 * D + 3), 7.0, np.float32), dtype)
    x, y = wide[:, 1:D + 1], wide[:, D + 2:2 * D + 2]
    x.copy_(to_gpu(c["x"], dtype))
    got, final = ssm_conv_fwd(x, dev(c, "weight"), dev(c, "bias"), 1, dev(c, "state"), y_out=y, **plan(c))
    torch.cuda.synchronize()
    assert got is y
    assert np.all(check_fwd(c, 1, to_np(y), to_np(final)) == 7)
    assert np.all(to_np(wide)[:, [0, D + 1, 2 * D + 2]] == 7) and np.array_equal(to_np(x), c["x"])


def test_starts_outside_the_tensor_are_clamped():
    import torch
    from mlstm_matrix_memory_amd import ssm_conv_fwd
    announce("conv fwd with seq_start entries below 0, above rows and a length above max_len")
    c = make(16, 4, "f32", 5, packed=[0, 4, 30])
    start = torch.tensor([-5, 4, 1000], dtype=torch.int32, device="cuda")
    y = torch.full((33, 16), 7.0, device="cuda")
    y, final = ssm_conv_fwd(dev(c, "x"), dev(c, "weight"), dev(c, "bias"), 1, dev(c, "state"), seq_start=start, max_len=20,
                            y_out=y)
    torch.cuda.synchronize()
    c["spans"] = [(0, 4), (4, 24)]
    assert np.all(check_fwd(c, 1, to_np(y), to_np(final)) == 7)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W,D,B", [(2, 5, 3), (3, 64, 1), (4, 1027, 2), (4, 2048, 256)])
def test_step_continues_the_forward(W, D, B, dtype):
    import torch
    from mlstm_matrix_memory_amd import ssm_conv_fwd, ssm_conv_step
    announce(f"conv step after fwd B={B} D={D} W={W} {dtype}")
    c = make(D, W, dtype, D, B=B, S=7)
    x, w, bias = dev(c, "x"), dev(c, "weight"), dev(c, "bias")
    y, state = ssm_conv_fwd(x[:, :3].contiguous(), w, bias, 1, dev(c, "state"))
    rest = [ssm_conv_step(x[:, t], w, state, bias, 1) for t in range(3, 7)]
    torch.cuda.synchronize()
    check_fwd(c, 1, to_np(torch.cat([y, torch.stack(rest, 1)], 1)), to_np(state))


def check_bwd(c, act, got, runs):
    g = ref.conv_bwd(c["x"], c["weight"], c["bias"], c["state64"], c["spans"], act, c["dy"], c["df"])
    _, _, size = ref.conv_fwd(c["x"], c["weight"], c["bias"], c["state64"], c["spans"], act)
    # error of act'(p), relative to dy: act' is within (8 + |p|) u and moves by at most half of p's error
    slope = ((8 + size.max()) + 0.5 * (c["W"] + 1) * size.max()) * U if act else 0.0
    inside = np.zeros(len(c["x"]), bool)
    for lo, hi in c["spans"]:
        inside[lo:hi] = True
    for name, t, dtype, terms in (("x", got[0], c["dtype"], c["W"] + 2), ("weight", got[1], "f32", runs),
                                  ("bias", got[2], "f32", runs), ("state", got[3], c["dtype"], c["W"] + 2)):
        if t is None:
            continue
        e = g["size_" + name] * (1.1 * terms * U + slope)
        a, want, e = to_np(t), g[name], e + HALF[dtype] * (np.abs(g[name]) + e)
        if name == "x":
            a, want, e = a.reshape(want.shape)[inside], want[inside], e[inside]
        assert_within("grad_" + name, a, want, e)
    return to_np(got[0]).reshape(len(inside), -1)[~inside]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("D", [1, 8, 13, 520])
def test_backward(D, W, dtype):
    import torch
    from mlstm_matrix_memory_amd import ssm_conv_bwd
    for act, bias, state, B, S in ((1, True, True, 2, 9), (0, False, False, 3, 1), (1, True, False, 1, 300),
                                   (0, True, True, 2, 2)):
        announce(f"conv bwd B={B} S={S} D={D} W={W} {dtype} act={act} bias={bias} state={state}")
        c = make(D, W, dtype, D + W, B=B, S=S, bias=bias, state=state)
        got = ssm_conv_bwd(dev(c, "x"), dev(c, "weight"), dev(c, "dy"), dev(c, "bias"), act, dev(c, "state"),
                           dstate_final=dev(c, "df"))
        torch.cuda.synchronize()
        assert (got[2] is None) == (not bias) and (got[3] is None) == (not state)
        check_bwd(c, act, got, B * S)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_packed_into_a_column_range(dtype):
    import torch
    from mlstm_matrix_memory_amd import ssm_conv_bwd
    announce(f"conv bwd packed {PACKED} D=77 {dtype}, gradient into a column range")
    c = make(77, 4, dtype, 77, packed=PACKED)
    wide = to_gpu(np.full((len(c["x"]), 160), 7.0, np.float32), dtype)
    got = ssm_conv_bwd(dev(c, "x"), dev(c, "weight"), dev(c, "dy"), dev(c, "bias"), 1, dev(c, "state"),
                       dstate_final=dev(c, "df"), grad_x=wide[:, 80:157], **plan(c))
    torch.cuda.synchronize()
    assert np.all(check_bwd(c, 1, got, PACKED[-1]) == 7)
    assert np.all(to_np(wide)[:, :80] == 7) and np.all(to_np(wide)[:, 157:] == 7)


def test_saturated_gates_stay_finite():
    import torch
    from mlstm_matrix_memory_amd import ssm_conv_bwd, ssm_conv_fwd
    announce("conv with pre-activations of +-1000 and +-1e30")
    c = make(8, 2, "f32", 3, S=6, bias=False, state=False)
    c["x"][:] = np.array([1000.0, -1000.0, 1e30, -1e30, 90.0, -90.0] * 2, np.float32)[:, None]
    c["weight"][:] = [0, 1]
    y, _ = ssm_conv_fwd(dev(c, "x"), dev(c, "weight"))
    g = ssm_conv_bwd(dev(c, "x"), dev(c, "weight"), dev(c, "dy"))
    torch.cuda.synchronize()
    assert np.all(np.isfinite(to_np(y))) and np.all(np.isfinite(to_np(g[0])))
    want = np.maximum(c["x"], 0)
    assert_within("y", to_np(y).reshape(want.shape), want, 1e-30 + 1e-6 * np.abs(want))
