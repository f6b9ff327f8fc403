"""Linear attention with a decay for each head on the GPU against 64 bits: forward, backward and
single rows, at the lengths, widths and batches where the kernels take another way."""
import numpy as np
import pytest

import block_reference as ref
import lin_attn_reference as la
from gpu_helpers import announce, to_gpu, to_np

pytestmark = pytest.mark.gpu


def on_gpu(c, packed):
    """Device tensors of a case: q, k, v, do as column ranges of one projection, each at an odd column."""
    import torch
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    lead = (c["rows"],) if packed else (c["B"], c["S"])
    names = [n for n in ("q", "k", "v", "do") if c[n] is not None]
    widths = [int(np.prod(c[n].shape[1:])) for n in names]
    whole = torch.full((*lead, sum(widths) + 3), float("nan"), dtype=dt, device="cuda")
    t, at = {}, 1
    for n, w in zip(names, widths):
        part = whole[..., at:at + w]
        part.copy_(to_gpu(c[n], c["dtype"]).reshape(*lead, w))
        t[n] = part.unflatten(-1, c[n].shape[1:])
        at += w
    t["g"] = to_gpu(c["g"], "f32")
    for n in ("h", "dh"):
        t[n] = None if c[n] is None else to_gpu(c[n], "f32")
    t["plan"] = dict(seq_start=torch.tensor(c["at"], device="cuda"), max_len=c["S"]) if packed else {}
    return t


def run(c, packed, backward=True):
    """{name: array} of all outputs; rows of sequences only are compared, the others must stay."""
    import torch
    from mlstm_matrix_memory_amd import lin_attn_bwd, lin_attn_fwd
    t = on_gpu(c, packed)
    o_room = torch.full((*t["v"].shape[:-2], c["v"].shape[1] * c["v"].shape[2] + 5), 9.0, dtype=t["v"].dtype, device="cuda")
    o = o_room[..., 2:-3].unflatten(-1, c["v"].shape[1:])
    _, final = lin_attn_fwd(t["q"], t["k"], t["v"], t["g"], scale=c["scale"], h_init=t["h"], o_out=o, **t["plan"])
    torch.cuda.synchronize()
    assert (o_room[..., :2] == 9).all() and (o_room[..., -3:] == 9).all()
    got = {"o": to_np(o).reshape(c["v"].shape), "h_final": to_np(final)}
    if backward:
        room = {n: torch.full((*t[n].shape[:-2], t[n].shape[-2] * t[n].shape[-1] + 2), 9.0, dtype=t[n].dtype, device="cuda")
                for n in ("q", "k", "v")}
        part = {n: r[..., 1:-1].unflatten(-1, c[n].shape[1:]) for n, r in room.items()}
        grads = lin_attn_bwd(t["q"], t["k"], t["v"], t["g"], t["do"], scale=c["scale"], h_init=t["h"], dh_final=t["dh"],
                             grad_q=part["q"], grad_k=part["k"], grad_v=part["v"], **t["plan"])
        torch.cuda.synchronize()
        for r in room.values():
            assert (r[..., 0] == 9).all() and (r[..., -1] == 9).all()
        for n, x, like in zip(("dq", "dk", "dv"), grads, ("q", "k", "v")):
            got[n] = to_np(x).reshape(c[like].shape)
        if grads[3] is not None:
            got["dh0"] = to_np(grads[3])
    return got


def check(c, packed=False, backward=True):
    got, want = run(c, packed, backward), la.reference(c)
    for n, x in got.items():
        ref.assert_within(n, x, *want[n])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S", [1, 2, 17, 63, 64, 65, 127, 128, 129, 191, 257])
def test_lengths(S, dtype):
    announce(f"lin_attn lengths S={S} {dtype}")
    check(la.make(2, S, 2, 2, 32, 48, dtype, seed=S))


WIDTHS = [(1, 1), (3, 5), (8, 16), (40, 77), (64, 64), (65, 63), (66, 130), (128, 96), (129, 200), (256, 256), (384, 40), (24, 520),
          (1024, 65), (70, 1024)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", WIDTHS)
def test_widths(dk, dv, dtype):
    announce(f"lin_attn widths dk={dk} dv={dv} {dtype}")
    check(la.make(1, 150, 2, 1, dk, dv, dtype, seed=dk + dv))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,G", [(1, 1), (6, 3), (6, 2), (5, 1), (8, 8)])
def test_heads(H, G, dtype):
    announce(f"lin_attn heads H={H} G={G} {dtype}")
    check(la.make(2, 140, H, G, 20, 36, dtype, seed=H * G, init=H != 5))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("init", [False, True])
def test_packed(init, dtype):
    announce(f"lin_attn packed sequences init={init} {dtype}")
    check(la.make(7, 0, 4, 2, 24, 40, dtype, seed=3, lengths=[130, 0, 1, 260, 128, 0, 77], init=init), packed=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_segments(dtype):
    """Few tiles over long sequences: cut into segments, of which the last is shorter."""
    from mlstm_matrix_memory_amd import binding
    announce(f"lin_attn segments {dtype}")
    code = binding.MLSTM_BF16 if dtype == "bf16" else binding.MLSTM_F32
    kept = (1300 // 128 + 1) * 2 * 64 * 64 * (2 if dtype == "bf16" else 4)
    assert binding.lin_attn_fwd_workspace_bytes(1, 1300, 1300, 2, 2, 32, 40, code) > kept  # sums of segments beside
    check(la.make(1, 1300, 2, 2, 32, 40, dtype, seed=5))
    check(la.make(3, 0, 2, 1, 16, 20, dtype, seed=6, lengths=[1100, 3, 1024]), packed=True)
    check(la.make(1, 1153, 1, 1, 20, 24, dtype, seed=7, init=False))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decays(dtype):
    """No memory at all, a single row's, all rows' alike."""
    announce(f"lin_attn decays {dtype}")
    check(la.make(1, 300, 5, 5, 16, 24, dtype, seed=8, decay=[-np.inf, -30.0, -1.5, -1e-5, 0.0]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("back", [False, True])
def test_nan_and_infinities_reach_only_what_follows(back, dtype):
    """A value of v (its gradient's do) does not reach rows before (behind) it, other columns, heads or sequences."""
    import torch
    from mlstm_matrix_memory_amd import lin_attn_bwd, lin_attn_fwd
    announce(f"lin_attn NaN and infinities back={back} {dtype}")
    c = la.make(2, 200, 2, 2, 20, 72, dtype, seed=9, init=False)
    name = "do" if back else "v"
    for row, col, value in ((30, 5, np.inf), (70, 6, np.nan), (140, 70, -np.inf)):
        clean = la.reference(c)
        d = dict(c)
        d[name] = c[name].copy()
        d[name][row, 1, col] = value
        t = on_gpu(d, False)
        if back:
            grads = lin_attn_bwd(t["q"], t["k"], t["v"], t["g"], t["do"], scale=c["scale"])
            torch.cuda.synchronize()
            got, n = to_np(grads[2]).reshape(c["v"].shape), "dv"
            hit = np.zeros(got.shape, bool)
            hit[:row + 1, 1, col] = True
            for x, m in ((grads[0], "dq"), (grads[1], "dk")):
                x = to_np(x).reshape(c["q"].shape)
                ok = np.ones(c["rows"], bool)
                ok[row if m == "dq" else slice(0, row + 1)] = False
                ref.assert_within(m, x[ok][:, 1], clean[m][0][ok][:, 1], clean[m][1][ok][:, 1])
                ref.assert_within(m, x[:, 0], clean[m][0][:, 0], clean[m][1][:, 0])
                assert not np.isfinite(x[~ok][:, 1]).any()
        else:
            o, _ = lin_attn_fwd(t["q"], t["k"], t["v"], t["g"], scale=c["scale"])
            torch.cuda.synchronize()
            got, n = to_np(o).reshape(c["v"].shape), "o"
            hit = np.zeros(got.shape, bool)
            hit[row:200, 1, col] = True
        value, bound = clean[n]
        ref.assert_within(n, np.where(hit, 0, got), np.where(hit, 0, value), bound)
        assert not np.isfinite(got[hit]).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(1, 1), (16, 7), (33, 64), (64, 64), (100, 130), (256, 48), (512, 512), (700, 20), (1024, 33)])
def test_step(dk, dv, dtype):
    import torch
    from mlstm_matrix_memory_amd import lin_attn_step
    announce(f"lin_attn step dk={dk} dv={dv} {dtype}")
    c = la.make(3, 1, 4, 2, dk, dv, dtype, seed=dk, grads=False)
    t = on_gpu(c, True)
    room = torch.full((3, 4 * dv + 3), 9.0, dtype=t["v"].dtype, device="cuda")
    o = lin_attn_step(t["q"], t["k"], t["v"], t["g"], t["h"], scale=c["scale"], o_out=room[:, 1:-2].unflatten(-1, (4, dv)))
    torch.cuda.synchronize()
    want = la.reference(c)
    ref.assert_within("h", to_np(t["h"]), *want["h_final"])
    # the step rounds its result only
    T = c["scale"] * np.einsum("bhvk,bhk->bhv", np.abs(want["h_final"][0]), np.repeat(np.abs(c["q"].astype(np.float64)), 2, 1))
    S = c["scale"] * np.einsum("bhvk,bhk->bhv", want["h_final"][1], np.repeat(np.abs(c["q"].astype(np.float64)), 2, 1))
    b = (dk + 4) * ref.U * T + S
    ref.assert_within("o", to_np(o), want["o"][0], b + ref.HALF[dtype] * (np.abs(want["o"][0]) + b))
    assert (room[:, 0] == 9).all() and (room[:, -2:] == 9).all()


def test_gradients_against_differences():
    """The fp32 backward against central differences of the forward in 64 bits (through the recurrence)."""
    import torch
    announce("lin_attn gradients against differences")
    c = la.make(1, 140, 1, 1, 5, 6, "f32", seed=11)
    got = run(c, False)
    rng = np.random.default_rng(12)

    def loss(d):
        o, f = la.recurrence(*(torch.tensor(d[n][:, 0], dtype=torch.float64) for n in ("q", "k", "v")),
                             torch.tensor(float(c["g"][0]), dtype=torch.float64), c["scale"],
                             torch.tensor(d["h"][0, 0], dtype=torch.float64))
        return float((o.numpy() * c["do"][:, 0]).sum() + (f.numpy() * c["dh"][0, 0]).sum())
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("h", "dh0")):
        way = rng.standard_normal(c[name].shape)
        step = 1e-4
        sides = [loss({**{n: np.asarray(c[n], np.float64) for n in ("q", "k", "v", "h")},
                       name: np.asarray(c[name], np.float64) + s * step * way}) for s in (1, -1)]
        want, have = (sides[0] - sides[1]) / (2 * step), float((got[grad] * way).sum())
        # the loss is bilinear in each: the difference is exact to its rounding, 2^-52 of the loss over the step
        size = float(np.abs(got[grad] * way).sum())
        assert abs(want - have) <= 1e-9 * max(map(abs, sides)) / step * 1e-3 + 400 * ref.U * size


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S", [100, 140])
@pytest.mark.parametrize("absent", ["h", "dh"])
def test_only_one_of_the_states(absent, S, dtype):
    """An initial state without a gradient of the final one, and the other way round; over one chunk and two."""
    announce(f"lin_attn without {absent} S={S} {dtype}")
    c = la.make(2, S, 2, 1, 24, 20, dtype, seed=60 + S)
    c[absent] = None
    check(c)


def test_empty_sequences_return_their_states():
    import torch
    from mlstm_matrix_memory_amd import lin_attn_bwd, lin_attn_fwd
    announce("lin_attn of empty sequences only")
    q, v = torch.full((5, 1, 16), float("nan"), device="cuda"), torch.full((5, 2, 24), float("nan"), device="cuda")
    h, dh = torch.randn(2, 2, 24, 16, device="cuda"), torch.randn(2, 2, 24, 16, device="cuda")
    plan = dict(seq_start=torch.tensor([2, 2, 2], dtype=torch.int32, device="cuda"), max_len=1)
    g = torch.tensor([-0.1, -0.2], device="cuda")
    o, final = lin_attn_fwd(q, q, v, g, h_init=h, o_out=torch.full_like(v, 3.0), **plan)
    grads = lin_attn_bwd(q, q, v, g, v, h_init=h, dh_final=dh, **plan)
    _, zero = lin_attn_fwd(q, q, v, g, **plan)
    torch.cuda.synchronize()
    assert (o == 3).all() and torch.equal(final, h) and torch.equal(grads[3], dh) and (zero == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_segments_of_wide_states(dtype):
    """The tiles of 256 columns and those of 128, cut into segments, forwards and backwards."""
    announce(f"lin_attn segments of wide states {dtype}")
    check(la.make(1, 1100, 1, 1, 72, 200, dtype, seed=70))
    check(la.make(1, 1050, 1, 1, 136, 264, dtype, seed=71, init=False))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("packed", [False, True])
def test_short_sequences_take_no_workspace(packed, dtype):
    """Sequences of one chunk without states: the wrappers allocate their outputs and, where heads share q and k, the
    gradients by head; results as ever."""
    import torch
    from mlstm_matrix_memory_amd import lin_attn_bwd, lin_attn_fwd
    announce(f"lin_attn of short sequences without a workspace packed={packed} {dtype}")
    for G in (4, 2):
        c = la.make(5, 128, 4, G, 24, 40, dtype, seed=80 + G, init=False, lengths=[128, 0, 1, 77, 128] if packed else None)
        check(c, packed)
        t = on_gpu(c, packed)
        t = {n: x.contiguous() if n in ("q", "k", "v", "do") else x for n, x in t.items()}
        outputs = c["v"].size * t["v"].element_size() + 5 * 4 * 40 * 24 * 4
        grads = (2 * c["q"].size + c["v"].size) * t["v"].element_size() + (0 if G == 4 else c["rows"] * 4 * 24 * 4)
        for f, need in ((lambda: lin_attn_fwd(t["q"], t["k"], t["v"], t["g"], **t["plan"]), outputs),
                        (lambda: lin_attn_bwd(t["q"], t["k"], t["v"], t["g"], t["do"], **t["plan"]), grads)):
            torch.cuda.synchronize()
            torch.cuda.reset_peak_memory_stats()
            before = torch.cuda.memory_allocated()
            f()
            assert torch.cuda.max_memory_allocated() - before <= need + 4 * 512  # (allocations are whole 512 bytes)
        torch.cuda.synchronize()


def in_c(c, final=True, grad_h=True):
    """A case through the C entry points: h_final NULL unless `final`, grad_h_init NULL unless `grad_h`, whatever h_init is."""
    import torch
    from mlstm_matrix_memory_amd import MLSTM_BF16, MLSTM_F32, binding
    lib, t = binding.load_library(), on_gpu(c, False)
    B, S, H, G, dk, dv = c["B"], c["S"], c["v"].shape[1], c["q"].shape[1], c["q"].shape[2], c["v"].shape[2]
    code, f32 = (MLSTM_BF16 if c["dtype"] == "bf16" else MLSTM_F32), dict(dtype=torch.float32, device="cuda")
    row, ptr = t["q"].stride(1), lambda x: None if x is None else x.data_ptr()  # noqa: E731
    head = [y for n in ("q", "k", "v") for y in (ptr(t[n]), row)] + [ptr(t["g"]), None, ptr(t["h"])]
    sizes = [B, S, B * S, H, G, dk, dv, c["scale"], code]
    bytes_of = lambda f, states: f(B, S, B * S, H, G, dk, dv, code, 0, states)  # noqa: E731
    need = [bytes_of(lib.lin_attn_fwd_call_workspace_bytes, int(c["h"] is not None)),
            bytes_of(lib.lin_attn_bwd_call_workspace_bytes, int(c["h"] is not None or c["dh"] is not None))]
    ws = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None for n in need]
    o, gv = (torch.empty(B, S, H, dv, dtype=t["v"].dtype, device="cuda") for _ in range(2))
    gq, gk = (torch.empty(B, S, G, dk, dtype=t["v"].dtype, device="cuda") for _ in range(2))
    h_final, gh = (torch.empty(B, H, dv, dk, **f32) if wanted else None for wanted in (final, grad_h))
    stream = torch.cuda.current_stream().cuda_stream
    st = lib.lin_attn_fwd(*head, *sizes, ptr(o), H * dv, ptr(h_final), ptr(ws[0]), need[0], stream)
    assert st == 0, binding.mlstm_error_detail()
    st = lib.lin_attn_bwd(*head, ptr(t["do"]), row, ptr(t["dh"]), *sizes, ptr(gq), G * dk, ptr(gk), G * dk, ptr(gv), H * dv, ptr(gh),
                          ptr(ws[1]), need[1], stream)
    assert st == 0, binding.mlstm_error_detail()
    torch.cuda.synchronize()
    like = {"o": c["v"], "dq": c["q"], "dk": c["q"], "dv": c["v"]}
    got = {"o": o, "dq": gq, "dk": gk, "dv": gv, "h_final": h_final, "dh0": gh}
    return {n: to_np(x).reshape(like[n].shape) if n in like else to_np(x) for n, x in got.items() if x is not None}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S", [100, 300, 1100])
@pytest.mark.parametrize("final,h,dh,grad_h", [(False, True, True, True), (False, False, False, False), (True, True, True, False),
                                               (True, False, True, True), (False, False, False, True), (False, True, False, False)])
def test_final_states_and_gradients_that_are_not_wanted(final, h, dh, grad_h, S, dtype):
    """The C entry points without h_final, without grad_h_init though there is an h_init, with it though there is none; in
    one chunk, in several, in segments, from workspaces of exactly the call's bytes that hold NaN."""
    announce(f"lin_attn in C final={final} h={h} dh={dh} grad_h={grad_h} S={S} {dtype}")
    c = la.make(1, S, 2, 1, 24, 40, dtype, seed=90 + S)
    want_of = dict(c, h=c["h"] if h else None, dh=c["dh"] if dh else None)
    got, want = in_c(want_of, final, grad_h), la.reference(want_of)
    assert ("h_final" in got) == final and ("dh0" in got) == grad_h
    for n, x in got.items():
        ref.assert_within(n, x, *want[n])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [np.nan, np.inf])
@pytest.mark.parametrize("name", ["q", "k"])
def test_nan_and_infinities_in_later_rows_of_q_and_k(name, value, dtype):
    """A value in a row of q or k reaches no earlier row of the output, nor rows, columns and heads of the gradients that do
    not read it; rows that read it are not finite."""
    import torch
    from mlstm_matrix_memory_amd import lin_attn_bwd, lin_attn_fwd
    announce(f"lin_attn with {value} in {name} {dtype}")
    c = la.make(2, 200, 4, 2, 20, 72, dtype, seed=19, init=False)
    clean = la.reference(c)
    for row, col in ((0, 3), (37, 5), (63, 19), (130, 0), (199, 7)):
        d = dict(c)
        d[name] = c[name].copy()
        d[name][row, 1, col] = value             # of the first sequence, and of the heads 2 and 3
        t = on_gpu(d, False)
        o, final = lin_attn_fwd(t["q"], t["k"], t["v"], t["g"], scale=c["scale"])
        grads = lin_attn_bwd(t["q"], t["k"], t["v"], t["g"], t["do"], scale=c["scale"])
        torch.cuda.synchronize()
        got = {"o": to_np(o).reshape(c["v"].shape), "h_final": to_np(final)}
        got.update((n, to_np(x).reshape(c[s].shape)) for n, x, s in zip(("dq", "dk", "dv"), grads, "qkv"))
        hit = {n: np.zeros(x.shape, bool) for n, x in got.items()}
        if name == "q":                          # o_row, dv and one column of dk up to the row
            hit["o"][row, 2:], hit["dv"][:row + 1, 2:], hit["dk"][:row + 1, 1, col] = True, True, True
        else:                                    # o and one column of dq from the row on, dv of the row, one column of the state
            hit["o"][row:200, 2:], hit["dq"][row:200, 1, col], hit["dv"][row, 2:], hit["h_final"][0, 2:, :, col] = True, True, True, True
        for n, x in got.items():
            ref.assert_within(f"{n} row {row}", np.where(hit[n], 0, x), np.where(hit[n], 0, clean[n][0]), clean[n][1])
            assert not np.isfinite(x[hit[n]]).any(), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_states_behind_nan_and_infinities(dtype):
    """Rows of the final state that a NaN or infinity of v reaches are not finite, the others as without it; through
    chunks and segments."""
    import torch
    from mlstm_matrix_memory_amd import lin_attn_fwd
    announce(f"lin_attn states behind NaN and infinities {dtype}")
    for S in (90, 200, 1200):
        c = la.make(1, S, 2, 1, 24, 40, dtype, seed=95, grads=False, decay=[-1e-3, -0.002])
        clean = la.reference(c)
        c["v"][S // 3, 0, 7], c["v"][S // 2, 1, 30] = np.inf, np.nan
        t = on_gpu(c, False)
        _, final = lin_attn_fwd(t["q"], t["k"], t["v"], t["g"], scale=c["scale"], h_init=t["h"])
        torch.cuda.synchronize()
        hit = np.zeros((1, 2, 40, 24), bool)
        hit[0, 0, 7], hit[0, 1, 30] = True, True
        final = to_np(final)
        ref.assert_within("h", np.where(hit, 0, final), np.where(hit, 0, clean["h_final"][0]), clean["h_final"][1])
        assert not np.isfinite(final[hit]).any()
