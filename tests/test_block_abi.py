"""Argument validation of the block operators on the CPU: every refusal happens before
any HIP call, with a status and a reason."""
import pytest

from mlstm_matrix_memory_amd import binding as b

P = [0x10000000 * (k + 1) for k in range(32)]     # far apart, aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    return b.load_library()


def refused(status, words, code=b.MLSTM_ERR_INVALID_ARG):
    assert status == code, (status, b.mlstm_error_detail())
    assert words in b.mlstm_error_detail()


def _norm(lib, quant=False, **kw):
    a = dict(x=P[0], xs=64, res=P[1], rs=64, w=P[2], rows=4, d=64, eps=1e-5, dt=1, rdt=0, group=0, rout=P[3], y=P[4],
             scale=P[5])
    a.update(kw)
    head = (a["x"], a["xs"], a["res"], a["rs"], a["w"], a["rows"], a["d"], a["eps"], a["dt"], a["rdt"])
    if quant:
        return lib.mlstm_rms_norm_quant(*head, a["group"], a["rout"], a["y"], a["scale"], None)
    return lib.mlstm_rms_norm_fwd(*head, a["rout"], a["y"], None)


NORM_BAD = [
    (dict(rows=0), "rows=0"), (dict(d=0), "d=0"), (dict(d=16385, xs=16385, rs=16385), "d=16385"),
    (dict(eps=-1.0), "eps=-1"), (dict(eps=float("nan")), "eps=nan"), (dict(eps=float("inf")), "eps=inf"),
    (dict(dt=2), "dtype=2"), (dict(rdt=5), "res_dtype=5"),
    (dict(x=None), "x is NULL"), (dict(w=None), "weight is NULL"), (dict(x=P[0] + 1), "x is not 2-byte aligned"),
    (dict(rout=P[3] + 2), "residual_out is not 4-byte aligned"),
    (dict(xs=63), "x_stride=63"), (dict(rs=-64), "residual_stride"),
    (dict(rout=P[1] + 4), "residual_out overlaps residual"), (dict(rout=P[0]), "overlaps"),
]


@pytest.mark.parametrize("kw,words", NORM_BAD + [(dict(y=None), "y_out is NULL"), (dict(y=P[0]), "y_out overlaps x")])
def test_norm_refusals(lib, kw, words):
    if "rout" in kw and kw["rout"] == P[0]:
        words = "residual_out overlaps x"
    refused(_norm(lib, **kw), words)


@pytest.mark.parametrize("kw,words", NORM_BAD + [
    (dict(group=16), "group=16"), (dict(group=-32), "group=-32"), (dict(y=None), "q_out is NULL"),
    (dict(scale=None), "scale_out is NULL"), (dict(scale=P[4] + 4), "overlaps")])
def test_norm_quant_refusals(lib, kw, words):
    refused(_norm(lib, quant=True, **kw), words)


def _norm_bwd(lib, **kw):
    a = dict(r=P[0], rs=64, w=P[1], dy=P[2], ds=64, dres=P[3], rows=4, d=64, eps=1e-5, dt=1, rdt=0, gx=P[4], gr=P[5],
             gw=P[6], ws=P[7], n=1 << 20)
    a.update(kw)
    return lib.mlstm_rms_norm_bwd(*a.values(), None)


@pytest.mark.parametrize("kw,words", [
    (dict(rows=-1), "rows=-1"), (dict(d=0), "d=0"), (dict(r=None), "r is NULL"), (dict(dy=None), "dy is NULL"),
    (dict(gw=None), "grad_weight is NULL"), (dict(gx=None, gr=None), "both NULL"), (dict(ds=5), "dy_stride=5"),
    (dict(gx=P[2]), "grad_x overlaps dy"), (dict(gr=P[0]), "grad_residual overlaps r"), (dict(gx=P[3]), "overlaps"),
    (dict(gw=P[7] + 64), "overlaps"), (dict(ws=P[7] + 2), "workspace is not 4-byte aligned"),
])
def test_norm_bwd_refusals(lib, kw, words):
    refused(_norm_bwd(lib, **kw), words)


def test_norm_bwd_workspace(lib):
    need = b.mlstm_rms_norm_bwd_workspace_bytes(4, 64)
    assert need >= 64 * 4
    refused(_norm_bwd(lib, n=need - 1), "needed", b.MLSTM_ERR_WORKSPACE)
    refused(_norm_bwd(lib, ws=None), "needed", b.MLSTM_ERR_WORKSPACE)
    assert b.mlstm_rms_norm_bwd_workspace_bytes(0, 64) == 0
    assert b.mlstm_rms_norm_bwd_workspace_bytes(4, 20000) == 0


def _conv(lib, **kw):
    a = dict(x=P[0], xs=64, w=P[1], bias=P[2], start=None, init=P[3], B=2, S=8, rows=16, D=64, W=4, act=1, dt=1, y=P[4],
             ys=64, final=P[5])
    a.update(kw)
    return lib.ssm_conv_fwd(*a.values(), None)


BATCH_BAD = [
    (dict(B=0, rows=0), "B=0"), (dict(S=0), "S=0"), (dict(rows=15), "rows=15 is not B*S=16"), (dict(D=0), "D=0"),
    (dict(start=P[20], S=17), "S=17 exceeds rows=16"), (dict(start=P[20] + 2), "seq_start is not 4-byte aligned"),
    (dict(dt=7), "dtype=7"), (dict(x=None), "x is NULL"), (dict(xs=63), "x_stride=63"),
    (dict(x=P[0] + 1), "x is not 2-byte aligned"),
]


@pytest.mark.parametrize("kw,words", BATCH_BAD + [
    (dict(W=1), "width=1"), (dict(W=5), "width=5"), (dict(act=2), "act=2"), (dict(w=None), "weight is NULL"),
    (dict(y=None), "y_out is NULL"), (dict(y=P[0]), "y_out overlaps x"), (dict(final=P[3]), "state_final overlaps state_init"),
    (dict(y=P[0] + 2 * 32, ys=64), "y_out overlaps x"), (dict(start=P[4] + 64), "y_out overlaps seq_start"),
])
def test_conv_refusals(lib, kw, words):
    refused(_conv(lib, **kw), words)


def test_too_many_sequences(lib):
    refused(_conv(lib, B=65536, S=1, rows=65536), "65536", b.MLSTM_ERR_UNSUPPORTED)


def test_sizes_past_the_kernels_indexes(lib):
    unsupported = b.MLSTM_ERR_UNSUPPORTED
    refused(_conv(lib, D=(1 << 24) + 1, xs=1 << 25, ys=1 << 25), "too large", unsupported)
    refused(_conv(lib, B=1, S=(1 << 30) + 1, rows=(1 << 30) + 1), "too large", unsupported)
    refused(_conv(lib, xs=1 << 58), "x_stride")
    refused(_conv(lib, xs=(1 << 62) + 64), "x_stride=46116860184273879")      # its bytes wrap to a small number
    refused(_conv(lib, xs=-64), "x_stride=-64")
    refused(_scan(lib, B=65535, S=1, rows=65535, D=1 << 24, xs=1 << 24, dts=1 << 24, zs=1 << 24, ys=1 << 24), "too large",
            unsupported)
    assert b.ssm_conv_bwd_workspace_bytes(2, 16, (1 << 24) + 1, 4) == 0
    assert b.ssm_scan_bwd_workspace_bytes(1, 1 << 30, 1 << 30, 1 << 24, 1, 16) == 0


def test_column_ranges_of_one_buffer_are_apart(lib):
    # y behind x in rows of one width: accepted so far as to reach the next check
    refused(_conv(lib, xs=128, y=P[0] + 2 * 64, ys=128, final=P[3]), "state_final overlaps state_init")
    refused(_conv(lib, xs=127, y=P[0] + 2 * 64, ys=127), "y_out overlaps x")


@pytest.mark.parametrize("kw,words", [
    (dict(B=0), "B=0"), (dict(D=0), "D=0"), (dict(W=5), "width=5"), (dict(state=None), "state is NULL"),
    (dict(y=P[2]), "overlaps"), (dict(xs=1), "x_stride=1"), (dict(act=-1), "act=-1"), (dict(dt=3), "dtype=3"),
])
def test_conv_step_refusals(lib, kw, words):
    a = dict(x=P[0], xs=64, w=P[1], bias=None, B=2, D=64, W=4, act=1, dt=1, state=P[2], y=P[3], ys=64)
    a.update(kw)
    refused(lib.ssm_conv_step(*a.values(), None), words)


def _conv_bwd(lib, **kw):
    a = dict(x=P[0], xs=64, w=P[1], bias=P[2], start=None, init=P[3], dy=P[4], ds=64, df=P[5], B=2, S=8, rows=16, D=64,
             W=4, act=1, dt=1, gx=P[6], gs=64, gw=P[7], gb=P[8], gi=P[9], ws=P[10], n=1 << 24)
    a.update(kw)
    return lib.ssm_conv_bwd(*a.values(), None)


@pytest.mark.parametrize("kw,words", BATCH_BAD + [
    (dict(W=0), "width=0"), (dict(dy=None), "dy is NULL"), (dict(gx=None), "grad_x is NULL"),
    (dict(gw=None), "grad_weight is NULL"), (dict(gb=None), "grad_bias is NULL"),
    (dict(bias=None), "grad_bias is given without bias"), (dict(gi=P[3]), "grad_state_init overlaps state_init"),
    (dict(gx=P[4]), "grad_x overlaps dy"), (dict(gw=P[10] + 4), "grad_weight overlaps workspace"),
])
def test_conv_bwd_refusals(lib, kw, words):
    refused(_conv_bwd(lib, **kw), words)


def test_conv_bwd_workspace(lib):
    need = b.ssm_conv_bwd_workspace_bytes(2, 16, 64, 4)
    assert need >= 5 * 64 * 4
    refused(_conv_bwd(lib, n=need - 1), "needed", b.MLSTM_ERR_WORKSPACE)
    assert b.ssm_conv_bwd_workspace_bytes(2, 0, 64, 4) == 0 and b.ssm_conv_bwd_workspace_bytes(2, 16, 64, 9) == 0


SCAN = dict(x=P[0], xs=64, dtp=P[1], dts=64, A=P[2], Bm=P[3], bs=16, Cm=P[4], cs=16, skip=P[5], bias=P[6], z=P[7],
            zs=64, start=None, h0=P[8], B=2, S=8, rows=16, D=64, G=1, N=16, softplus=1, dt=1)
SCAN_BAD = [
    (dict(D=63, G=2, xs=63, dts=63, zs=63), "D=63 is not a multiple of G=2"), (dict(G=0), "G=0"), (dict(N=0), "N=0"),
    (dict(N=65, bs=65, cs=65), "N=65"), (dict(softplus=2), "softplus=2"), (dict(dtp=None), "dt is NULL"),
    (dict(A=None), "A is NULL"), (dict(Bm=None), "Bm is NULL"), (dict(Cm=None), "Cm is NULL"), (dict(bs=15), "Bm_stride=15"),
    (dict(zs=1), "z_stride=1"), (dict(A=P[2] + 2), "A is not 4-byte aligned"),
]


def _scan(lib, **kw):
    a = dict(SCAN, y=P[9], ys=64, final=P[10], ws=P[11], n=1 << 30)
    a.update(kw)
    return lib.ssm_scan_fwd(*a.values(), None)


@pytest.mark.parametrize("kw,words", BATCH_BAD + SCAN_BAD + [
    (dict(y=None), "y_out is NULL"), (dict(y=P[1]), "y_out overlaps dt"), (dict(final=P[8]), "h_final overlaps h_init"),
    (dict(y=P[7], ys=64), "y_out overlaps z")])
def test_scan_refusals(lib, kw, words):
    refused(_scan(lib, **kw), words)


def test_scan_workspace(lib):
    big = dict(B=1, S=65536, rows=65536)
    need = b.ssm_scan_fwd_workspace_bytes(1, 65536, 65536, 64, 1, 16)
    assert need > 0
    refused(_scan(lib, n=need - 1, **big), "needed", b.MLSTM_ERR_WORKSPACE)
    refused(_scan(lib, ws=P[11] + 4, **big), "workspace is not 16-byte aligned")
    for bad in ((0, 8, 16, 64, 1, 16), (2, 0, 16, 64, 1, 16), (2, 8, 16, 64, 3, 16), (2, 8, 16, 64, 1, 65), (2, 8, 0, 64, 1, 16)):
        assert b.ssm_scan_fwd_workspace_bytes(*bad) == 0


@pytest.mark.parametrize("kw,words", SCAN_BAD + [
    (dict(B=0), "B=0"), (dict(h=None), "h is NULL"), (dict(y=P[10]), "overlaps"), (dict(h=P[2]), "h overlaps A")])
def test_ssm_step_refusals(lib, kw, words):
    a = {k: v for k, v in SCAN.items() if k not in ("start", "h0", "S", "rows")}
    a.update(h=P[10], y=P[9], ys=64)
    a.update(kw)
    refused(lib.ssm_step(*a.values(), None), words)


def _scan_bwd(lib, **kw):
    a = dict(SCAN, dy=P[9], ds=64, dh=P[10], gx=P[11], gxs=64, gdt=P[12], gdts=64, gz=P[13], gzs=64, gB=P[14], gBs=16,
             gC=P[15], gCs=16, gA=P[16], gD=P[17], gb=P[18], gh=P[19], ws=P[20], n=1 << 30)
    a.update(kw)
    order = ["x", "xs", "dtp", "dts", "A", "Bm", "bs", "Cm", "cs", "skip", "bias", "z", "zs", "start", "h0", "dy", "ds", "dh",
             "B", "S", "rows", "D", "G", "N", "softplus", "dt"]
    rest = [k for k in a if k not in order]
    return lib.ssm_scan_bwd(*(a[k] for k in order + rest), None)


@pytest.mark.parametrize("kw,words", [(dict(k, start=P[21]) if "start" in k and k["start"] == P[20] else k, w)
                                      for k, w in BATCH_BAD] + SCAN_BAD + [
    (dict(dy=None), "dy is NULL"), (dict(gx=None), "grad_x is NULL"), (dict(gz=None), "grad_z is NULL"),
    (dict(gD=None), "grad_Dskip is NULL"), (dict(gb=None), "grad_dt_bias is NULL"), (dict(gA=None), "grad_A is NULL"),
    (dict(z=None), "grad_z is given without z"), (dict(skip=None), "grad_Dskip is given without Dskip"),
    (dict(bias=None), "grad_dt_bias is given without dt_bias"), (dict(gh=P[10]), "overlaps"),
    (dict(gB=P[15]), "overlaps"), (dict(gx=P[9]), "overlaps"), (dict(gCs=15), "grad_C_stride=15"),
])
def test_scan_bwd_refusals(lib, kw, words):
    refused(_scan_bwd(lib, **kw), words)


def test_scan_bwd_workspace(lib):
    need = b.ssm_scan_bwd_workspace_bytes(2, 8, 16, 64, 1, 16)
    assert need > 0
    refused(_scan_bwd(lib, n=need - 1), "needed", b.MLSTM_ERR_WORKSPACE)
    refused(_scan_bwd(lib, ws=P[20] + 4), "workspace is not 16-byte aligned")
    assert b.ssm_scan_bwd_workspace_bytes(2, 8, 0, 64, 1, 16) == 0


def test_block_operators_exported(lib):
    import mlstm_matrix_memory_amd as pkg
    for name in ("mlstm_rms_norm_fwd", "mlstm_rms_norm_quant", "mlstm_rms_norm_bwd",
                 "mlstm_rms_norm_bwd_workspace_bytes", "ssm_conv_fwd", "ssm_conv_step", "ssm_conv_bwd",
                 "ssm_conv_bwd_workspace_bytes", "ssm_scan_fwd", "ssm_step", "ssm_scan_fwd_workspace_bytes",
                 "ssm_scan_bwd", "ssm_scan_bwd_workspace_bytes"):
        assert name in b.header_symbols() and hasattr(lib, name) and callable(getattr(pkg, name))


def test_binding_refuses_before_any_call():
    """Shapes, dtypes and layouts are checked on any device; these calls reach no library function."""
    import torch
    import mlstm_matrix_memory_amd as pkg
    x, w = torch.zeros(2, 8, 64), torch.zeros(64, 4)
    with pytest.raises(ValueError, match="GPU"):
        pkg.ssm_conv_fwd(x, w)
    with pytest.raises(ValueError, match="GPU"):
        pkg.mlstm_rms_norm_fwd(x, torch.ones(64))
    assert b._row_stride(torch.zeros(5, 7), "t") == 7 and b._row_stride(torch.zeros(5, 14)[:, :7], "t") == 14
    assert b._row_stride(torch.zeros(1, 14)[:, :7], "t") == 7
    assert b._row_stride(torch.zeros(2, 3, 2, 8), "t", 2) == 16
    assert b._row_stride(torch.zeros(2, 3, 40)[..., 8:24].view(2, 3, 2, 8), "t", 2) == 40
    assert b._row_stride(torch.zeros(3, 1, 9), "t") == 9 and b._row_stride(torch.zeros(3, 2, 9)[:, :1], "t") == 18
    for bad in (torch.zeros(7, 5).t(), torch.zeros(2, 8, 64)[:, :, ::2]):
        with pytest.raises(ValueError, match="contiguous"):
            b._row_stride(bad, "t")
    with pytest.raises(ValueError, match="uniform"):
        b._row_stride(torch.zeros(2, 8, 64)[:, :4], "t")
    with pytest.raises(ValueError, match="contiguous"):
        b._row_stride(torch.zeros(4, 1).expand(4, 6), "t")       # a broadcast row
    assert b._row_stride(torch.zeros(1, 6).expand(4, 6), "t") == 0     # a broadcast batch: refused by the library (stride)


def _far(a, **kw):
    """The call's pointers 2^46 bytes apart (never dereferenced), for tensors larger than their usual distance."""
    a = {k: (v // 0x10000000 << 46) if isinstance(v, int) and v >= 0x10000000 and v % 0x10000000 == 0 else v
         for k, v in a.items()}
    return dict(a, **kw)


def test_norm_rows_past_32_bit_indexes(lib):
    rows = (1 << 31) - 1
    refused(_norm(lib, rows=rows, d=1, xs=1, rs=1), "exceeds", b.MLSTM_ERR_UNSUPPORTED)
    refused(_norm_bwd(lib, rows=rows, d=1, rs=1, ds=1), "exceeds", b.MLSTM_ERR_UNSUPPORTED)
    assert b.mlstm_rms_norm_bwd_workspace_bytes(rows, 1) == 0


def test_more_threads_than_a_launch_takes(lib):
    """Refused before any kernel: 2^32 threads or more."""
    words, code = "more threads than one launch takes", b.MLSTM_ERR_UNSUPPORTED
    far = _far(dict(x=P[0], res=P[1], w=P[2], rout=P[3], y=P[4], scale=P[5]))
    for quant in (False, True):                      # a wave to a row: 2^26 rows
        refused(_norm(lib, quant=quant, rows=1 << 26, d=8, xs=8, rs=8, **far), words, code)
    # 65535 sequences of one row: a workgroup each for every 64 channels (256 of the convolution)
    B, D, wide = 65535, 1 << 14, dict(xs=1 << 14, ys=1 << 14)
    conv = _far(dict(x=P[0], w=P[1], bias=P[2], init=P[3], y=P[4], final=P[5]))
    refused(_conv(lib, B=B, S=1, rows=B, D=1 << 17, **dict(conv, xs=1 << 17, ys=1 << 17)), words, code)
    scan = _far(dict(x=P[0], dtp=P[1], A=P[2], Bm=P[3], Cm=P[4], skip=P[5], bias=P[6], z=P[7], h0=P[8], y=P[9],
                     final=P[10], ws=P[11]))
    refused(_scan(lib, B=B, S=1, rows=B, D=D, dts=D, zs=D, **wide, **scan, n=1 << 45), words, code)
