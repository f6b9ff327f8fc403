"""Seeded cases of the selective scan for the GPU tests: host arrays, device tensors, comparison."""
import numpy as np

import block_reference as ref
from block_reference import HALF, TINY, assert_within
from gpu_helpers import to_gpu, to_np

PACKED = [0, 5, 5, 6, 39, 41, 44, 177]            # lengths 5, 0, 1, 33, 2, 3, 133
F32 = ("A", "D", "dt_bias", "h")
PER_ROW = ("x", "dt", "z", "dy", "B", "C")


def make(D, N, dtype, seed, B=2, S=9, G=1, packed=None, gate=True, skip=True, bias=True, state=True, softplus=1):
    rng = np.random.default_rng(seed)
    rows = (packed[-1] + 3) if packed else B * S  # packed: three rows behind the last sequence
    B = len(packed) - 1 if packed else B
    st = lambda *shape: ref.stored(rng.standard_normal(shape), dtype)  # noqa: E731
    c = {"x": st(rows, D), "dt": ref.stored(0.7 * rng.standard_normal((rows, D)) + (0 if softplus else 0.05), dtype),
         "z": st(rows, D) if gate else None,
         "A": (-np.arange(1, N + 1) * np.exp(0.2 * rng.standard_normal((D, N)))).astype(np.float32),
         "B": st(rows, G, N), "C": st(rows, G, N), "D": rng.standard_normal(D).astype(np.float32) if skip else None,
         "dt_bias": np.log(np.expm1(np.exp(rng.uniform(np.log(1e-3), np.log(0.3), D)))).astype(np.float32) if bias else None,
         "h": rng.standard_normal((B, D, N)).astype(np.float32) if state else None, "dy": st(rows, D),
         "dh": rng.standard_normal((B, D, N)).astype(np.float32) if state else None,
         "spans": ref.sequences(B, S, packed), "softplus": softplus, "batch": B, "S": S, "dtype": dtype, "packed": packed}
    if not softplus:
        c["dt"] = ref.stored(np.abs(c["dt"]) * 0.1, dtype)
        c["dt_bias"] = None if not bias else np.full(D, 0.01, np.float32)
    return c


def dev(c, key):
    a = c[key]
    if a is None:
        return None
    t = to_gpu(a, "f32" if key in F32 + ("dh",) else c["dtype"])
    if key in PER_ROW and not c["packed"]:
        t = t.view(c["batch"], c["S"], *t.shape[1:])
    return t


def plan(c):
    import torch
    if not c["packed"]:
        return {}
    return {"seq_start": torch.tensor(c["packed"], dtype=torch.int32, device="cuda"),
            "max_len": int(np.diff(c["packed"]).max())}


def inside(c):
    m = np.zeros(len(c["x"]), bool)
    for lo, hi in c["spans"]:
        m[lo:hi] = True
    return m


def compare(c, name, tensor, want, dtype):
    """Compares with {name: (value, bound)}; per-row results within the sequences only.
    Returns the rows outside of them."""
    value, bound = want
    got = to_np(tensor).reshape(value.shape)
    e = bound + HALF[dtype] * (np.abs(value) + bound) + TINY
    if len(value) != len(c["x"]) or name in ("h_final", "grad_h", "grad_A", "grad_D", "grad_dt_bias"):
        assert_within(name, got, value, e)
        return None
    m = inside(c)
    assert_within(name, got[m], value[m], e[m])
    return got[~m]


def forward(c, **kw):
    from mlstm_matrix_memory_amd import ssm_scan_fwd
    return ssm_scan_fwd(*(dev(c, k) for k in ("x", "dt", "A", "B", "C")), D=dev(c, "D"), z=dev(c, "z"),
                        dt_bias=dev(c, "dt_bias"), softplus=bool(c["softplus"]), h_init=dev(c, "h"), **plan(c), **kw)
