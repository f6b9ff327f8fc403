"""The selective scan's gradients on the GPU against fp64, within the bounds that the
reference follows through both recurrences (block_reference.scan)."""
import numpy as np
import pytest

import block_reference as ref
from gpu_helpers import announce, to_gpu, to_np
from scan_cases import PACKED, compare, dev, make, plan

pytestmark = pytest.mark.gpu

NAMES = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h")


def backward(c, **kw):
    from mlstm_matrix_memory_amd import ssm_scan_bwd
    return ssm_scan_bwd(*(dev(c, k) for k in ("x", "dt", "A", "B", "C", "dy", "D", "z", "dt_bias")),
                        softplus=bool(c["softplus"]), h_init=dev(c, "h"), dh_final=dev(c, "dh"), **plan(c), **kw)


def check(c, got, joins=False):
    """Compares every gradient; returns the rows of per-row ones outside the sequences."""
    want = ref.scan(c, c["dy"], c["dh"], joins=joins)
    left = []
    for name, t in zip(NAMES, got):
        if c[name] is None:
            assert t is None
            continue
        rows = compare(c, "grad_" + name, t, want["grad_" + name], c["dtype"] if name in ("x", "dt", "B", "C", "z") else "f32")
        if rows is not None:
            left.append(rows)
    return left


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,N,G", [(1, 1, 1), (64, 4, 1), (70, 5, 2), (130, 8, 1), (33, 12, 1), (96, 16, 3), (17, 24, 1),
                                   (64, 32, 1), (20, 50, 2), (65, 64, 1)])
def test_shapes(D, N, G, dtype):
    import torch
    for S, gate, skip, bias, state in ((9, True, True, True, True), (1, False, False, False, False),
                                       (70, True, False, True, False), (16, False, True, False, True)):
        announce(f"scan bwd B=2 S={S} D={D} N={N} G={G} {dtype} gate={gate} skip={skip} bias={bias} state={state}")
        c = make(D, N, dtype, D + N, S=S, G=G, gate=gate, skip=skip, bias=bias, state=state)
        got = backward(c)
        torch.cuda.synchronize()
        check(c, got)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_plain_step_sizes(dtype):
    import torch
    announce(f"scan bwd without softplus {dtype}")
    c = make(40, 16, dtype, 4, S=33, softplus=0)
    got = backward(c)
    torch.cuda.synchronize()
    check(c, got)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_packed_into_column_ranges_and_rows_left_alone(dtype):
    import torch
    announce(f"scan bwd packed {PACKED} {dtype}, gradients into column ranges of wider rows")
    D, N, G = 75, 12, 3
    c = make(D, N, dtype, 6, G=G, packed=PACKED)
    rows = len(c["x"])
    wide = to_gpu(np.full((rows, 3 * D + 7), 7.0, np.float32), dtype)
    bc = to_gpu(np.full((rows, 2 * G * N + 3), 7.0, np.float32), dtype)
    gx, gz, gdt = (wide[:, k * (D + 1):k * (D + 1) + D] for k in range(3))
    gB, gC = bc[:, 1:1 + G * N].view(rows, G, N), bc[:, 2 + G * N:2 + 2 * G * N].view(rows, G, N)
    got = backward(c, grad_x=gx, grad_z=gz, grad_dt=gdt, grad_B=gB, grad_C=gC)
    torch.cuda.synchronize()
    assert got[0] is gx and got[3] is gB
    assert all(np.all(r == 7) for r in check(c, got))
    assert np.all(to_np(wide)[:, [D, 2 * D + 1]] == 7) and np.all(to_np(bc)[:, [0, 1 + G * N, 2 + 2 * G * N]] == 7)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_sequences_cut_into_pieces(dtype):
    import torch
    for B, S, D, packed in ((1, 1500, 70, None), (3, 0, 40, [0, 700, 701, 1300])):
        announce(f"scan bwd B={B} S={S} D={D} packed={packed} {dtype}")
        c = make(D, 16, dtype, 11, B=B, S=S, packed=packed)
        got = backward(c)
        torch.cuda.synchronize()
        check(c, got, joins=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_short_and_one_long_sequence(dtype):
    import torch
    lengths = [0, 0, 1, 900, 0, 17, 64, 63, 65, 1, 1, 128, 0]
    starts = list(np.cumsum([0] + lengths))
    announce(f"scan bwd packed {lengths} {dtype}")
    c = make(37, 8, dtype, 15, packed=starts)
    got = backward(c)
    torch.cuda.synchronize()
    check(c, got, joins=True)


def test_starts_outside_the_tensor_are_clamped():
    import torch
    from mlstm_matrix_memory_amd import ssm_scan_bwd
    announce("scan bwd with seq_start entries below 0, above rows and a length above max_len")
    c = make(20, 16, "f32", 5, packed=[0, 4, 30])
    start = torch.tensor([-5, 4, 1000], dtype=torch.int32, device="cuda")
    left = {f"grad_{k}": torch.full(c[k].shape, 7.0, device="cuda") for k in ("x", "dt", "z", "B", "C")}
    got = ssm_scan_bwd(*(dev(c, k) for k in ("x", "dt", "A", "B", "C", "dy", "D", "z", "dt_bias")), h_init=dev(c, "h"),
                       dh_final=dev(c, "dh"), seq_start=start, max_len=20, **left)
    torch.cuda.synchronize()
    c["spans"] = [(0, 4), (4, 24)]
    assert all(np.all(r == 7) for r in check(c, got))


def test_repeated_calls_give_the_same_bits():
    import torch
    announce("scan bwd three times, B=2 S=300 D=200 N=16")
    c = make(200, 16, "bf16", 13, S=300)
    first = [t.clone() for t in backward(c)]
    for _ in range(2):
        for p, q in zip(first, backward(c)):
            assert torch.equal(p, q)


def test_gradients_are_differences_of_the_gpu_forward():
    # a directional difference of the fp32 forward: the loss moves by about 2 h |g . v|, and each
    # loss carries rounding errors near 1e-6 of the sum of its terms' sizes
    import torch
    from mlstm_matrix_memory_amd import ssm_scan_fwd
    announce("scan bwd against directional differences of the forward, f32")
    c = make(48, 16, "f32", 14, S=40)
    t = {k: dev(c, k) for k in NAMES}
    dy, dh = dev(c, "dy").double(), dev(c, "dh").double()
    g = dict(zip(NAMES, backward(c)))

    def loss(**kw):
        a = dict(t, **kw)
        y, h = ssm_scan_fwd(a["x"], a["dt"], a["A"], a["B"], a["C"], a["D"], a["z"], a["dt_bias"], h_init=a["h"])
        return (y.double() * dy).sum() + (h.double() * dh).sum(), (y.double() * dy).abs().sum() + (h.double() * dh).abs().sum()

    for name in NAMES:
        v = torch.randn(t[name].shape, generator=torch.Generator().manual_seed(1)).cuda()
        if name == "A":
            v = v * t[name].abs() * 0.1
        h = 2.0 ** -7
        (up, size), (down, _) = loss(**{name: t[name] + h * v}), loss(**{name: t[name] - h * v})
        want = float((g[name].double() * v.double()).sum())
        scale = float((g[name].double() * v.double()).abs().sum())
        # the cubic term of the difference: h^2 times a third derivative, at most a few times the
        # size of the first derivative's terms
        assert abs(float(up - down) / (2 * h) - want) <= 10 * h * h * scale + 1e-6 * float(size) / h, name
