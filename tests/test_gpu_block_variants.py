"""The block operators at the sizes where another kernel, tile or number of pieces is taken than at
small ones.  Bounds as in the operators' own tests.

Batches large enough for that repeat a few sequences: copies have to give the same bits as
the first ones, which are compared with fp64, and sums over sequences are that many times theirs.
"""
import numpy as np
import pytest

import scan_cases
import test_gpu_conv as conv
import test_gpu_norm as norm
import test_gpu_scan as scan
import test_gpu_scan_bwd as scan_bwd
import block_reference as ref
from block_reference import HALF, TINY, assert_within
from gpu_helpers import announce, to_np

pytestmark = pytest.mark.gpu


# ---- selective scan over repeated sequences ---------------------------------------------
def repeated(c, times):
    """The case with all of its sequences `times` times (packed: without rows behind the last)."""
    rows = c["spans"][-1][1]
    big = dict(c, batch=c["batch"] * times)
    for k in scan_cases.PER_ROW:
        if c[k] is not None:
            big[k] = np.concatenate([c[k][:rows]] * times)
    for k in ("h", "dh"):
        if c[k] is not None:
            big[k] = np.concatenate([c[k]] * times)
    if c["packed"]:
        big["packed"] = [0] + [int(p) + i * rows for i in range(times) for p in c["packed"][1:]]
    return big


def first(t, times, name):
    """The first copy of a result; all others have its bits."""
    copies = t.reshape(times, -1)
    assert bool((copies == copies[:1]).all()), f"{name}: copies differ"
    return copies[0]


def trimmed(c):
    """Without the rows behind the last packed sequence."""
    rows = c["spans"][-1][1]
    return dict(c, **{k: c[k][:rows] for k in scan_cases.PER_ROW if c[k] is not None})


def run_forward(c, times, joins):
    import torch
    y, final = scan_cases.forward(repeated(c, times))
    torch.cuda.synchronize()
    scan.check(trimmed(c), first(y, times, "y"), first(final, times, "h_final"), joins=joins)


# (sequences, rows, channels, states), and what the forward takes
FORWARD = [
    (162, 130, 33, 16),      # 32-row tiles, uncut, five turns of which the last is short
    (162, 128, 33, 8),       # 32-row tiles, uncut, four whole turns
    (150, 161, 9, 64),       # 32-row tiles, six turns, 16 states a wave
    (51, 97, 130, 24),       # 32-row tiles over three channel tiles, of which the last has two channels
    (300, 130, 33, 16),      # 16-row tiles, uncut, nine turns
    (330, 100, 5, 3),        # the same with one wave of states
    (258, 145, 6, 40),       # the same with 16 states a wave
    (141, 800, 5, 16),       # eight pieces of 112 rows
    (141, 805, 3, 4),        # likewise with one wave of states
    (60, 1300, 4, 32),       # seventeen pieces of 80 rows
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("B,S,D,N", FORWARD)
def test_scan_forward(B, S, D, N, gate, dtype):
    announce(f"scan fwd B={B} S={S} D={D} N={N} {dtype} gate={gate}")
    c = scan_cases.make(D, N, dtype, B + S, B=3, S=S, gate=gate, skip=gate, state=gate)
    run_forward(c, B // 3, joins=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [16, 64])
def test_scan_forward_packed_uncut(N, dtype):
    # 7 sequences of 4 tiles' rows and more, 100 times: more than 256 workgroups, 16-row tiles
    packed = [0, 130, 130, 131, 228, 230, 320, 420]
    announce(f"scan fwd 100 times packed {packed} N={N} {dtype}")
    run_forward(scan_cases.make(13, N, dtype, 2, packed=packed), 100, joins=True)


def run_backward(c, times, joins=True):
    import torch
    got = scan_bwd.backward(repeated(c, times))
    torch.cuda.synchronize()
    c = trimmed(c)
    want = ref.scan(c, c["dy"], c["dh"], joins=joins)
    for name, t in zip(scan_bwd.NAMES, got):
        if c[name] is None:
            assert t is None
            continue
        value, bound = want["grad_" + name]
        if name in ("A", "D", "dt_bias"):
            # a sum of `times` equal parts; its additions one after another (rows of a piece, a part of
            # the pieces, 16 of these) are fewer than the rows of c, which the bound counts
            assert_within("grad_" + name, to_np(t), times * value, times * (bound + HALF["f32"] * np.abs(value) + TINY))
        else:
            scan_cases.compare(c, "grad_" + name, first(t, times, name), want["grad_" + name],
                               "f32" if name == "h" else c["dtype"])


BACKWARD = [
    (450, 130, 5, 16),       # uncut, nine tiles of rows, the last short
    (451, 96, 66, 12),       # uncut over two channel tiles
    (900, 100, 5, 8),        # uncut, two waves
    (897, 83, 3, 2),         # uncut, one wave
    (225, 130, 5, 32),       # uncut, 8 states a lane
    (225, 100, 4, 64),       # uncut, 16 states a lane
    (150, 400, 5, 16),       # three pieces of 144 rows
    (150, 405, 3, 4),        # pieces of one wave
    (60, 330, 4, 40),        # pieces of 16 states a lane
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,S,D,N", BACKWARD)
def test_scan_backward(B, S, D, N, dtype):
    announce(f"scan bwd B={B} S={S} D={D} N={N} {dtype}")
    c = scan_cases.make(D, N, dtype, B + S, B=3, S=S, gate=B % 2 == 0)
    run_backward(c, B // 3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scan_backward_packed(dtype):
    packed = [0, 130, 130, 131, 228, 230, 320, 420]
    for times in (200, 60):                            # uncut, and in pieces of 80 rows
        announce(f"scan bwd {times} times packed {packed} {dtype}")
        run_backward(scan_cases.make(13, 16, dtype, 2, packed=packed), times)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,D,N,G", [(257, 512, 16, 1), (129, 1026, 16, 2), (131, 512, 24, 1), (1025, 517, 3, 1),
                                     (65, 513, 64, 3)])
def test_step_of_two_sequences_a_thread(B, D, N, G, dtype):
    import torch
    from mlstm_matrix_memory_amd import ssm_step
    assert B % 2 == 1 and B * D * N >= 1 << 20
    announce(f"scan step B={B} D={D} N={N} G={G} {dtype}")
    c = scan_cases.make(D, N, dtype, B, B=B, S=1, G=G)
    t = {k: scan_cases.dev(c, k) for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h")}
    y = ssm_step(t["x"][:, 0], t["dt"][:, 0], t["A"], t["B"][:, 0], t["C"][:, 0], t["h"], z=t["z"][:, 0], D=t["D"],
                 dt_bias=t["dt_bias"])
    torch.cuda.synchronize()
    scan.check(c, y, t["h"])


# ---- one of the two states' gradients -----------------------------------------------------
@pytest.mark.parametrize("S", [9, 300])
def test_scan_backward_with_one_state(S):
    import torch
    for given in ("h", "dh"):
        announce(f"scan bwd B=2 S={S} with {given} only")
        c = scan_cases.make(33, 16, "f32", 8, S=S)
        c["dh" if given == "h" else "h"] = None
        got = scan_bwd.backward(c)
        torch.cuda.synchronize()
        scan_bwd.check(c, got, joins=True)


@pytest.mark.parametrize("S", [2, 9, 300])
def test_conv_backward_with_one_state(S):
    import torch
    from mlstm_matrix_memory_amd import ssm_conv_bwd
    for given in ("state", "df"):
        announce(f"conv bwd B=2 S={S} with {given} only")
        c = conv.make(13, 4, "f32", 8, S=S)
        if given == "state":
            c["df"] = None
        else:
            c["state"], c["state64"] = None, np.zeros_like(c["state64"])
        got = ssm_conv_bwd(conv.dev(c, "x"), conv.dev(c, "weight"), conv.dev(c, "dy"), conv.dev(c, "bias"), 1,
                           conv.dev(c, "state"), dstate_final=conv.dev(c, "df"))
        torch.cuda.synchronize()
        assert (got[3] is None) == (given == "df")
        conv.check_bwd(c, 1, got, 2 * S)


# ---- short convolution: runs of eight rows ---------------------------------------------------
LONG = list(np.cumsum([0, 2, 0, 1, 1500, 64, 63, 65, 1, 0, 3, 2350, 0]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W,act,D", [(2, 0, 4099), (3, 1, 4096), (4, 1, 4099), (4, 0, 4103)])
def test_conv_runs_of_eight(W, act, D, dtype):
    import torch
    from mlstm_matrix_memory_amd import ssm_conv_fwd
    for packed in (None, LONG):
        announce(f"conv fwd D={D} W={W} {dtype} act={act} " + (f"packed {LONG}" if packed else "B=3 S=1367"))
        c = conv.make(D, W, dtype, D + W, B=3, S=1367, packed=packed, bias=act == 1, state=W != 3)
        y = torch.full(conv.dev(c, "x").shape, 7.0, device="cuda", dtype=conv.dev(c, "x").dtype)
        y, final = ssm_conv_fwd(conv.dev(c, "x"), conv.dev(c, "weight"), conv.dev(c, "bias"), act, conv.dev(c, "state"),
                                y_out=y, **conv.plan(c))
        torch.cuda.synchronize()
        assert np.all(conv.check_fwd(c, act, to_np(y), to_np(final)) == 7)


# ---- norm backward: more rows than workgroups, a workgroup to a row --------------------------------
@pytest.mark.parametrize("dtype,res_dtype", [("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rows,d", [(1100, 1030), (1100, 4099), (1100, 8200), (700, 16384)])
def test_norm_backward(rows, d, dtype, res_dtype):
    norm.test_backward(rows, d, dtype, res_dtype)


# ---- a bound of the lengths above the rows -------------------------------------------------------
def test_max_len_above_the_rows():
    import torch
    from mlstm_matrix_memory_amd import ssm_conv_bwd, ssm_conv_fwd, ssm_scan_bwd, ssm_scan_fwd
    announce(f"packed {scan_cases.PACKED} with max_len 100000")
    c = conv.make(20, 4, "f32", 4, packed=scan_cases.PACKED)
    a = [conv.dev(c, k) for k in ("x", "weight", "bias", "state", "dy", "df")]
    plan = dict(conv.plan(c), max_len=100000)
    y, final = ssm_conv_fwd(a[0], a[1], a[2], 1, a[3], **plan)
    got = ssm_conv_bwd(a[0], a[1], a[4], a[2], 1, a[3], dstate_final=a[5], **plan)
    torch.cuda.synchronize()
    conv.check_fwd(c, 1, to_np(y), to_np(final))
    conv.check_bwd(c, 1, got, scan_cases.PACKED[-1])
    c = scan_cases.make(20, 16, "f32", 4, packed=scan_cases.PACKED)
    t = {k: scan_cases.dev(c, k) for k in ("x", "dt", "A", "B", "C", "dy", "D", "z", "dt_bias", "h", "dh")}
    par = dict(D=t["D"], z=t["z"], dt_bias=t["dt_bias"], h_init=t["h"], **plan)
    y, final = ssm_scan_fwd(t["x"], t["dt"], t["A"], t["B"], t["C"], **par)
    got = ssm_scan_bwd(t["x"], t["dt"], t["A"], t["B"], t["C"], t["dy"], dh_final=t["dh"], **par)
    torch.cuda.synchronize()
    scan.check(c, y, final, joins=True)
    scan_bwd.check(c, got, joins=True)


# ---- NaN and infinities ---------------------------------------------------------------------------
def same_elsewhere(name, got, clean, touched):
    """NaN (or infinite) at the touched places, the clean run's bits at all others."""
    got, clean = to_np(got), to_np(clean)
    touched = np.broadcast_to(touched, got.shape)
    assert np.array_equal(got[~touched], clean[~touched]), name
    assert not np.any(np.isfinite(got[touched])), name


@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.parametrize("B,S,N", [(3, 40, 16), (3, 300, 12), (162, 70, 16)])
def test_scan_forward_with_a_value_that_is_not_finite(B, S, N, bad):
    import torch
    announce(f"scan fwd B={B} S={S} D=70 N={N} with {bad} in x, z and B")
    D, row, ch = 70, 21, 66
    c = scan_cases.make(D, N, "f32", 5, B=B, S=S, G=2)
    clean = scan_cases.forward(c)
    rows, chans = np.arange(S)[:, None], np.arange(D)
    here = (np.arange(B) == 1)[:, None, None]
    for key, at, touched_y, touched_h in (
            ("x", (S + row, ch), (rows >= row) & (chans == ch), chans == ch),
            ("z", (S + row, ch), (rows == row) & (chans == ch), np.zeros(D, bool)),
            ("B", (S + row, 1), (rows >= row) & (chans >= D // 2), chans >= D // 2)):
        d = dict(c, **{key: c[key].copy()})
        d[key][at] = bad
        y, h = scan_cases.forward(d)
        torch.cuda.synchronize()
        same_elsewhere("y " + key, y, clean[0], here & touched_y)
        same_elsewhere("h " + key, h, clean[1], here & touched_h[:, None])


def test_backward_with_nan_in_one_channel():
    """x: what the formulas carry it to in the rows, and nothing of other sequences' rows or channels' parameters."""
    import torch
    from mlstm_matrix_memory_amd import ssm_conv_bwd
    D, N, row, ch = 70, 12, 21, 66
    for B, S in ((3, 40), (3, 300), (3, 22)):          # in the middle, in a piece, in the last row
        announce(f"scan and conv bwd B={B} S={S} D={D} with NaN in x")
        c = scan_cases.make(D, N, "f32", 5, B=B, S=S)
        d = dict(c, x=c["x"].copy())
        d["x"][S + row, ch] = np.nan
        clean, got = scan_bwd.backward(c), scan_bwd.backward(d)
        torch.cuda.synchronize()
        seq, rows, chans = (np.arange(B) == 1)[:, None, None], np.arange(S)[None, :, None], np.arange(D)
        one = seq & (chans == ch)
        touched = {"x": one & (rows < 0), "dt": one & (rows >= row), "z": one & (rows >= row), "h": np.zeros(1, bool),
                   "B": (seq & (rows == row))[..., None], "C": (seq & (rows >= row))[..., None]}
        for name, a, b in zip(scan_bwd.NAMES, got, clean):
            if name in touched:
                same_elsewhere("grad_" + name, a, b, touched[name])
            else:
                other = np.arange(D) != ch
                assert np.array_equal(to_np(a)[other], to_np(b)[other]), name
        c = conv.make(D, 4, "f32", 5, B=B, S=S)
        d = dict(c, x=c["x"].copy())
        d["x"][S + row, ch] = np.nan
        clean, got = (ssm_conv_bwd(conv.dev(k, "x"), conv.dev(k, "weight"), conv.dev(k, "dy"), conv.dev(k, "bias"), 1,
                                   conv.dev(k, "state"), dstate_final=conv.dev(k, "df")) for k in (c, d))
        torch.cuda.synchronize()
        # row t's pre-activation enters the gradients of rows t - 3 .. t; this x those of rows row .. row + 3
        same_elsewhere("conv grad_x", got[0], clean[0], one & (rows >= row - 3) & (rows <= row + 3))
        same_elsewhere("conv grad_state", got[3], clean[3], np.zeros((B, 3, D), bool))
        other = np.arange(D) != ch
        for a, b in zip(got[1:3], clean[1:3]):
            assert np.array_equal(to_np(a)[other], to_np(b)[other])


def test_rows_of_no_sequence_may_hold_anything():
    import torch
    from mlstm_matrix_memory_amd import ssm_conv_bwd, ssm_conv_fwd
    announce("packed sequences between rows of NaN")
    packed = [40, 45, 45, 78, 200]
    c = scan_cases.make(37, 16, "f32", 4, packed=packed)
    k = conv.make(37, 4, "f32", 4, packed=packed)
    for key in scan_cases.PER_ROW:
        c[key][:40] = c[key][200:] = np.nan
    for key in ("x", "dy"):
        k[key][:40] = k[key][200:] = np.nan
    y, final = scan_cases.forward(c)
    got = scan_bwd.backward(c)
    cy, cfinal = ssm_conv_fwd(conv.dev(k, "x"), conv.dev(k, "weight"), conv.dev(k, "bias"), 1, conv.dev(k, "state"),
                              **conv.plan(k))
    cgot = ssm_conv_bwd(conv.dev(k, "x"), conv.dev(k, "weight"), conv.dev(k, "dy"), conv.dev(k, "bias"), 1,
                        conv.dev(k, "state"), dstate_final=conv.dev(k, "df"), **conv.plan(k))
    torch.cuda.synchronize()
    for key in scan_cases.PER_ROW:
        c[key][:40] = c[key][200:] = 0
    for key in ("x", "dy"):
        k[key][:40] = k[key][200:] = 0
    scan.check(c, y, final, joins=True)
    scan_bwd.check(c, got, joins=True)
    conv.check_fwd(k, 1, to_np(cy), to_np(cfinal))
    conv.check_bwd(k, 1, cgot, 160)
