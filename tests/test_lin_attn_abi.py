"""Argument validation of linear attention on the CPU: every refusal happens before any HIP call, with
a status and a reason."""
import pytest

from mlstm_matrix_memory_amd import binding as b

P = [0x100000000 * (k + 1) for k in range(32)]    # far apart, aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    return b.load_library()


def refused(status, words, code=b.MLSTM_ERR_INVALID_ARG):
    assert status == code, (status, b.mlstm_error_detail())
    assert words in b.mlstm_error_detail()


BASE = dict(q=P[0], qs=2 * 32, k=P[1], ks=2 * 32, v=P[2], vs=4 * 48, g=P[3], ss=None, h=P[4], B=2, S=100, rows=200, H=4, G=2,
            dk=32, dv=48, scale=1.0, dt=1)


def _head(a):
    return a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["g"]


def _sizes(a):
    return a["B"], a["S"], a["rows"], a["H"], a["G"], a["dk"], a["dv"], a["scale"], a["dt"]


def _fwd(lib, **kw):
    a = dict(BASE, o=P[5], os=4 * 48, hf=P[6], ws=P[7], wb=1 << 31)
    a.update(kw)
    return lib.lin_attn_fwd(*_head(a), a["ss"], a["h"], *_sizes(a), a["o"], a["os"], a["hf"], a["ws"], a["wb"], None)


def _bwd(lib, **kw):
    a = dict(BASE, do=P[5], dos=4 * 48, dhf=P[6], gq=P[8], gqs=64, gk=P[9], gks=64, gv=P[10], gvs=192, gh=P[11], ws=P[7],
             wb=1 << 31)
    a.update(kw)
    return lib.lin_attn_bwd(*_head(a), a["ss"], a["h"], a["do"], a["dos"], a["dhf"], *_sizes(a), a["gq"], a["gqs"], a["gk"],
                            a["gks"], a["gv"], a["gvs"], a["gh"], a["ws"], a["wb"], None)


def _step(lib, **kw):
    a = dict(BASE, rows=2, o=P[5], os=4 * 48)
    a.update(kw)
    return lib.lin_attn_step(*_head(a), a["B"], a["H"], a["G"], a["dk"], a["dv"], a["scale"], a["dt"], a["h"], a["o"], a["os"],
                             None)


BAD = [
    (dict(B=0), "B=0"), (dict(H=3), "H=3 is not a multiple of G=2"), (dict(G=0), "G=0"), (dict(dk=0), "dk=0"),
    (dict(dv=1025), "dv=1025"), (dict(dk=2000, qs=4000, ks=4000), "dk=2000"), (dict(scale=float("nan")), "scale=nan"),
    (dict(scale=float("inf")), "scale=inf"), (dict(dt=4), "dtype=4"), (dict(q=None), "q is NULL"), (dict(k=None), "k is NULL"),
    (dict(v=None), "v is NULL"), (dict(g=None), "log_decay is NULL"), (dict(qs=63), "q_stride=63"), (dict(vs=191), "v_stride=191"),
    (dict(k=P[1] + 1), "k is not 2-byte aligned"), (dict(g=P[3] + 2), "log_decay is not 4-byte aligned"),
]
SEQUENCES = [(dict(rows=201), "rows=201 is not B*S"), (dict(ss=P[12], S=300), "S=300 exceeds rows"), (dict(ss=P[12] + 1), "seq_start"),
             (dict(S=0), "S=0"), (dict(wb=1000), "workspace of 1000"), (dict(ws=None), "workspace of 0"),
             (dict(ws=P[7] + 8), "workspace is not 16-byte aligned"), (dict(h=P[4] + 1), "h_init is not 4-byte aligned")]


@pytest.mark.parametrize("kw,words", BAD + SEQUENCES + [
    (dict(o=None), "o_out is NULL"), (dict(o=P[2]), "o_out overlaps v"), (dict(hf=P[4]), "h_final overlaps h_init"),
    (dict(os=100), "o_out_stride=100"), (dict(hf=P[7] + 64), "overlaps"), (dict(ws=P[0]), "overlaps"),
])
def test_forward_refusals(lib, kw, words):
    refused(_fwd(lib, **kw), words, b.MLSTM_ERR_WORKSPACE if "workspace of" in words else b.MLSTM_ERR_INVALID_ARG)


@pytest.mark.parametrize("kw,words", BAD + [
    (dict(h=None), "h is NULL"), (dict(o=None), "o_out is NULL"), (dict(o=P[0]), "o_out overlaps q"), (dict(h=P[2]), "h overlaps v"),
])
def test_step_refusals(lib, kw, words):
    refused(_step(lib, **kw), words)


@pytest.mark.parametrize("kw,words", BAD + SEQUENCES + [
    (dict(do=None), "do is NULL"), (dict(dos=1), "do_stride=1"), (dict(gq=None), "grad_q is NULL"), (dict(gk=None), "grad_k is NULL"),
    (dict(gv=None), "grad_v is NULL"), (dict(gq=P[0]), "grad_q overlaps q"), (dict(gk=P[8]), "grad_q overlaps grad_k"),
    (dict(gh=P[6]), "grad_h_init overlaps dh_final"), (dict(gvs=10), "grad_v_stride=10"),
])
def test_backward_refusals(lib, kw, words):
    refused(_bwd(lib, **kw), words, b.MLSTM_ERR_WORKSPACE if "workspace of" in words else b.MLSTM_ERR_INVALID_ARG)


def test_too_large(lib):
    far = dict(q=1 << 40, k=1 << 44, v=1 << 48, h=None, o=1 << 50, hf=None, ws=1 << 55, wb=1 << 62)
    refused(_fwd(lib, B=1, S=1 << 30, rows=1 << 30, **far), "more threads", b.MLSTM_ERR_UNSUPPORTED)  # of the output kernel
    wide = dict(H=512, G=512, dk=1024, dv=1024, qs=1 << 19, ks=1 << 19, vs=1 << 19)
    refused(_fwd(lib, B=60000, S=1, rows=60000, **dict(far, os=1 << 19), **wide), "more threads", b.MLSTM_ERR_UNSUPPORTED)  # of the states'
    refused(_fwd(lib, B=65536, S=1, rows=65536, **far), "65535", b.MLSTM_ERR_UNSUPPORTED)
    refused(_fwd(lib, H=1 << 20, G=1 << 20, qs=1 << 25, ks=1 << 25, vs=1 << 26, **far), "too many heads", b.MLSTM_ERR_UNSUPPORTED)


def test_workspace_bytes(lib):
    f, g = lib.lin_attn_fwd_workspace_bytes, lib.lin_attn_bwd_workspace_bytes
    assert f(2, 100, 200, 4, 3, 32, 48, 1) == 0 and f(0, 100, 200, 4, 2, 32, 48, 1) == 0 and f(2, 100, 200, 4, 2, 32, 48, 9) == 0
    # one bf16 state of 64 x 64 per chunk and head; a packed batch has up to rows / 128 + B chunks
    assert f(2, 100, 200, 4, 2, 32, 48, 1) == 3 * 4 * 64 * 64 * 2
    assert f(2, 130, 150, 4, 2, 32, 48, 0) == 3 * 4 * 64 * 64 * 4
    # the gradients of q or k by head, where heads share them
    assert g(2, 100, 200, 4, 2, 32, 48, 1) == f(2, 100, 200, 4, 2, 32, 48, 1) + 200 * 4 * 32 * 4
    assert g(2, 100, 200, 4, 4, 32, 48, 1) == f(2, 100, 200, 4, 4, 32, 48, 1)


def test_python_checks():
    import torch
    from mlstm_matrix_memory_amd import lin_attn_bwd, lin_attn_fwd, lin_attn_step
    q, v, g = torch.zeros(1, 4, 2, 8), torch.zeros(1, 4, 2, 8), torch.zeros(2)
    for f, a in ((lin_attn_fwd, (q, q, v, g)), (lin_attn_step, (q, q, v, g, q)), (lin_attn_bwd, (q, q, v, g, v))):
        with pytest.raises(ValueError, match="GPU"):
            f(*a)


def test_calls_that_keep_no_states_need_no_workspace_for_them(lib):
    """Sequences of one chunk without a state at their start (in the backward: at either end) keep none: the
    call goes on to its next check with no workspace, or with that of the gradients by head alone."""
    short = dict(S=100, rows=200, h=None, ws=None, wb=0)
    refused(_fwd(lib, **short, o=None), "o_out is NULL")
    refused(_fwd(lib, **dict(short, S=128, rows=256), o=None), "o_out is NULL")
    refused(_fwd(lib, **dict(short, S=129, rows=258)), "workspace of 0", b.MLSTM_ERR_WORKSPACE)
    refused(_fwd(lib, **dict(short, h=P[4])), "workspace of 0", b.MLSTM_ERR_WORKSPACE)
    back = dict(short, dhf=None, gq=None)
    refused(_bwd(lib, **back), "workspace of 0", b.MLSTM_ERR_WORKSPACE)              # two heads share q and k
    refused(_bwd(lib, **dict(back, ws=P[7], wb=200 * 4 * 32 * 4)), "grad_q is NULL")
    refused(_bwd(lib, **dict(back, G=4, qs=128, ks=128)), "grad_q is NULL")
    for one in (dict(h=P[4]), dict(dhf=P[6])):
        refused(_bwd(lib, **dict(back, G=4, qs=128, ks=128, **one)), "workspace of 0", b.MLSTM_ERR_WORKSPACE)


def test_workspace_bytes_of_a_call(lib):
    """What one call takes, by whether it is packed and has states at its ends; the plain query is the largest of them."""
    from mlstm_matrix_memory_amd import lin_attn_bwd_call_workspace_bytes, lin_attn_fwd_call_workspace_bytes
    f, g = lin_attn_fwd_call_workspace_bytes, lin_attn_bwd_call_workspace_bytes
    state = 64 * 64 * 2
    assert f(2, 100, 200, 4, 2, 32, 48, 1, False, False) == 0 and f(2, 100, 200, 4, 2, 32, 48, 1, True, False) == 0
    assert f(2, 100, 200, 4, 2, 32, 48, 1, False, True) == 2 * 4 * state and f(2, 100, 200, 4, 2, 32, 48, 1, True, True) == 3 * 4 * state
    assert f(2, 130, 260, 4, 2, 32, 48, 1, False, False) == f(2, 130, 260, 4, 2, 32, 48, 1, False, True) == 4 * 4 * state
    assert g(2, 100, 200, 4, 4, 32, 48, 1, False, False) == 0 and g(2, 100, 200, 4, 2, 32, 48, 1, False, False) == 200 * 4 * 32 * 4
    assert g(2, 100, 200, 4, 4, 32, 48, 1, False, True) == 2 * 4 * state
    for call, most in ((f, lib.lin_attn_fwd_workspace_bytes), (g, lib.lin_attn_bwd_workspace_bytes)):
        for sizes in ((2, 100, 200, 4, 2, 32, 48, 1), (1, 5000, 5000, 2, 1, 40, 40, 0), (9, 700, 6300, 3, 3, 130, 70, 1)):
            assert most(*sizes) == max(call(*sizes, packed, states) for packed in (False, True) for states in (False, True))
    # sizes that make no batch
    assert f(2, 100, 201, 4, 2, 32, 48, 1, False, True) == 0 and f(2, 100, 200, 4, 3, 32, 48, 1, True, True) == 0
    assert g(0, 100, 200, 4, 2, 32, 48, 1, True, True) == 0


def test_declared_exported_and_in_the_package(lib):
    """The header's functions of these operators are among those that the export check goes through."""
    import mlstm_matrix_memory_amd as pkg
    names = b.header_symbols()
    for name in ("lin_attn_fwd", "lin_attn_step", "lin_attn_bwd", "lin_attn_fwd_workspace_bytes", "lin_attn_bwd_workspace_bytes",
                 "lin_attn_fwd_call_workspace_bytes", "lin_attn_bwd_call_workspace_bytes", "mlstm_quant_e4m3", "mlstm_mm_e4m3"):
        assert name in names and hasattr(lib, name) and callable(getattr(pkg, name))
    # every function that the header declares, whatever its prefix, is one of them
    import re
    text = re.sub(r"/\*.*?\*/", "", open(b.HEADER).read(), flags=re.S)
    assert set(re.findall(r"^(?:mlstm_status|size_t|const char *\*) *(\w+)\s*\(", text, flags=re.M)) <= set(names)
