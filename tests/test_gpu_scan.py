"""The selective scan on the GPU, over sequences and single rows, against fp64.

The bounds come from the reference itself, which follows the rounding errors of a fp32
evaluation through the recurrence (block_reference.scan).
"""
import numpy as np
import pytest

import block_reference as ref
from gpu_helpers import announce, to_gpu, to_np
from scan_cases import PACKED, compare, dev, forward, make

pytestmark = pytest.mark.gpu


def check(c, y, final, joins=False):
    want = ref.scan(c, joins=joins)
    compare(c, "h_final", final, want["h_final"], "f32")
    return compare(c, "y", y, want["y"], c["dtype"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,N,G", [(1, 1, 1), (64, 4, 1), (70, 5, 2), (130, 8, 1), (33, 12, 1), (96, 16, 3), (17, 24, 1),
                                   (64, 32, 1), (20, 50, 2), (65, 64, 1)])
def test_shapes(D, N, G, dtype):
    import torch
    for S, gate, skip, bias, state in ((9, True, True, True, True), (1, False, False, False, False),
                                       (70, True, False, True, False)):
        announce(f"scan fwd B=2 S={S} D={D} N={N} G={G} {dtype} gate={gate} skip={skip} bias={bias} state={state}")
        c = make(D, N, dtype, D + N, S=S, G=G, gate=gate, skip=skip, bias=bias, state=state)
        y, final = forward(c)
        torch.cuda.synchronize()
        check(c, y, final)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_plain_step_sizes(dtype):
    import torch
    announce(f"scan fwd without softplus {dtype}")
    c = make(40, 16, dtype, 4, S=33, softplus=0)
    y, final = forward(c)
    torch.cuda.synchronize()
    check(c, y, final)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_packed_column_ranges_and_rows_left_alone(dtype):
    import torch
    from mlstm_matrix_memory_amd import ssm_scan_fwd
    from scan_cases import plan
    announce(f"scan fwd packed {PACKED} {dtype}, inputs and output column ranges of wider rows")
    D, N, G = 75, 12, 3
    c = make(D, N, dtype, 6, G=G, packed=PACKED)
    rows = len(c["x"])
    wide = to_gpu(np.full((rows, 4 * D + 5), 7.0, np.float32), dtype)
    x, z, y, dt = (wide[:, k * (D + 1):k * (D + 1) + D] for k in range(4))
    bc = to_gpu(np.full((rows, 2 * G * N + 3), 7.0, np.float32), dtype)
    Bm, Cm = bc[:, 1:1 + G * N].view(rows, G, N), bc[:, 2 + G * N:2 + 2 * G * N].view(rows, G, N)
    for t, k in ((x, "x"), (z, "z"), (dt, "dt"), (Bm, "B"), (Cm, "C")):
        t.copy_(dev(c, k))
    got, final = ssm_scan_fwd(x, dt, dev(c, "A"), Bm, Cm, dev(c, "D"), z, dev(c, "dt_bias"), h_init=dev(c, "h"), y_out=y,
                              **plan(c))
    torch.cuda.synchronize()
    assert got is y and np.all(check(c, y.contiguous(), final) == 7)
    assert np.all(to_np(wide)[:, [D, 2 * D + 1, 3 * D + 2, 4 * D + 3, 4 * D + 4]] == 7)


def test_starts_outside_the_tensor_are_clamped():
    import torch
    from mlstm_matrix_memory_amd import ssm_scan_fwd
    announce("scan fwd with seq_start entries below 0, above rows and a length above max_len")
    c = make(20, 16, "f32", 5, packed=[0, 4, 30])
    start = torch.tensor([-5, 4, 1000], dtype=torch.int32, device="cuda")
    y = torch.full((33, 20), 7.0, device="cuda")
    y, final = ssm_scan_fwd(*(dev(c, k) for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")), h_init=dev(c, "h"),
                            seq_start=start, max_len=20, y_out=y)
    torch.cuda.synchronize()
    c["spans"] = [(0, 4), (4, 24)]
    assert np.all(check(c, y, final) == 7)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,N,G,B", [(1, 1, 1, 1), (65, 4, 1, 3), (50, 7, 2, 2), (512, 16, 1, 256), (96, 33, 3, 2),
                                     (40, 64, 1, 5)])
def test_steps_continue_the_forward(D, N, G, B, dtype):
    import torch
    from mlstm_matrix_memory_amd import ssm_scan_fwd, ssm_step
    announce(f"scan steps after fwd B={B} D={D} N={N} G={G} {dtype}")
    c = make(D, N, dtype, D, B=B, S=6, G=G)
    t = {k: dev(c, k) for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h")}
    first = {k: t[k][:, :3].contiguous() for k in ("x", "dt", "z", "B", "C")}
    par = dict(D=t["D"], dt_bias=t["dt_bias"])
    y, h = ssm_scan_fwd(first["x"], first["dt"], t["A"], first["B"], first["C"], z=first["z"], h_init=t["h"], **par)
    ys = [ssm_step(t["x"][:, k], t["dt"][:, k], t["A"], t["B"][:, k], t["C"][:, k], h, z=t["z"][:, k], **par)
          for k in range(3, 6)]
    torch.cuda.synchronize()
    check(c, torch.cat([y, torch.stack(ys, 1)], 1), h)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_sequences_cut_into_pieces(dtype):
    import torch
    for B, S, D, packed in ((1, 1500, 70, None), (3, 0, 40, [0, 700, 701, 1300])):
        announce(f"scan fwd B={B} S={S} D={D} packed={packed} {dtype}")
        c = make(D, 16, dtype, 11, B=B, S=S, packed=packed)
        y, final = forward(c)
        torch.cuda.synchronize()
        check(c, y, final, joins=True)


def test_extreme_step_sizes_and_gates():
    import torch
    announce("scan fwd with dt of +-1e4, z of +-1e30 and a state that must vanish")
    c = make(8, 16, "f32", 12, S=8, bias=False)
    c["dt"][::2] = -1e4                            # step size 0: the state stays
    c["dt"][1] = 1e4                               # step size 1e4: full forgetting, input times 1e4
    c["z"][3], c["z"][5] = 1e30, -1e30
    y, final = forward(c)
    torch.cuda.synchronize()
    assert np.all(np.isfinite(to_np(y))) and np.all(np.isfinite(to_np(final)))
    check(c, y, final)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_short_and_one_long_sequence(dtype):
    import torch
    # piece numbers of packed sequences: empty ones first, last and in a row, single rows, one long
    lengths = [0, 0, 1, 900, 0, 17, 64, 63, 65, 1, 1, 128, 0]
    starts = list(np.cumsum([0] + lengths))
    announce(f"scan fwd packed {lengths} {dtype}")
    c = make(37, 8, dtype, 15, packed=starts)
    y, final = forward(c)
    torch.cuda.synchronize()
    check(c, y, final, joins=True)


def test_repeated_calls_give_the_same_bits():
    import torch
    announce("scan fwd three times, B=1 S=900 D=200 N=16")
    c = make(200, 16, "bf16", 13, B=1, S=900)
    first = [t.clone() for t in forward(c)]
    for _ in range(2):
        for p, q in zip(first, forward(c)):
            assert torch.equal(p, q)


def test_rows_far_apart():
    """Rows 8.4 million elements apart: offsets past 32 bits in every tensor give the bits of dense rows."""
    import torch
    from mlstm_matrix_memory_amd import ssm_conv_bwd, ssm_conv_fwd, ssm_scan_bwd, ssm_scan_fwd
    announce("scan and convolution, forward and backward, over rows 8.4 million elements apart (300 rows)")
    c = make(64, 16, "bf16", 16, B=1, S=300, state=False)
    t = {k: dev(c, k) for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "dy")}
    apart = 8_400_000
    wide = torch.zeros(1, 300, apart, dtype=torch.bfloat16, device="cuda")

    def far(place, like):
        v = wide[:, :, place * 64:place * 64 + like[0, 0].numel()].view(like.shape)
        v.copy_(like)
        return v

    f = {k: far(i, t[k]) for i, k in enumerate(("x", "dt", "z", "dy", "B", "C"))}
    out = [far(6 + i, torch.zeros_like(t["x"])) for i in range(6)]
    outB, outC = far(12, torch.zeros_like(t["B"])), far(13, torch.zeros_like(t["C"]))
    par = dict(D=t["D"], dt_bias=t["dt_bias"])
    w = torch.randn(64, 4, device="cuda")
    a = [ssm_scan_fwd(t["x"], t["dt"], t["A"], t["B"], t["C"], z=t["z"], **par)[0],
         ssm_conv_fwd(t["x"], w)[0], ssm_conv_bwd(t["x"], w, t["dy"])[0],
         *ssm_scan_bwd(t["x"], t["dt"], t["A"], t["B"], t["C"], t["dy"], z=t["z"], **par)[:8]]
    g = ssm_scan_bwd(f["x"], f["dt"], t["A"], f["B"], f["C"], f["dy"], z=f["z"], grad_x=out[3], grad_dt=out[4],
                     grad_z=out[5], grad_B=outB, grad_C=outC, **par)
    b = [ssm_scan_fwd(f["x"], f["dt"], t["A"], f["B"], f["C"], z=f["z"], y_out=out[0], **par)[0],
         ssm_conv_fwd(f["x"], w, y_out=out[1])[0], ssm_conv_bwd(f["x"], w, f["dy"], grad_x=out[2])[0], *g[:8]]
    torch.cuda.synchronize()
    for i, (u, v) in enumerate(zip(a, b)):
        assert torch.equal(u, v), i
