"""Linear attention and the e4m3 operators as they are used together: a block's forward and backward,
a prompt followed by single tokens, sequences in pieces, graphs, streams, packed batches with gaps."""
import numpy as np
import pytest

import block_reference as ref
import lin_attn_reference as la
from gpu_helpers import announce, to_gpu, to_np

pytestmark = pytest.mark.gpu


def _normal(shape, seed, sd=1.0, dtype=None):
    import torch
    x = torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") * sd
    return x.to(dtype or torch.bfloat16)


def _block(x, p, h, step=False):
    """norm to e4m3 -> projection -> linear attention -> quantiser -> projection back; x [..., d]."""
    import mlstm_matrix_memory_amd as m
    q8, s8, _ = m.mlstm_rms_norm_quant(x, p["norm"], group=128)
    proj = m.mlstm_mm_e4m3(q8, s8, *p["w_in"])
    q, k, v = proj.split([p["G"] * p["dk"]] * 2 + [p["H"] * p["dv"]], -1)
    heads = q.unflatten(-1, (p["G"], p["dk"])), k.unflatten(-1, (p["G"], p["dk"])), v.unflatten(-1, (p["H"], p["dv"])), p["g"]
    if step:
        o = m.lin_attn_step(*heads, h)
    else:
        o, h = m.lin_attn_fwd(*heads, h_init=h)
    return m.mlstm_mm_e4m3(*m.mlstm_quant_e4m3(o.flatten(-2)), *p["w_out"]), o, proj, h


def _weights(d=256, H=4, G=2, dk=48, dv=64):
    import torch
    import mlstm_matrix_memory_amd as m
    wide = 2 * G * dk + H * dv
    return dict(H=H, G=G, dk=dk, dv=dv, norm=torch.ones(d, device="cuda"), g=torch.tensor([-0.5, -0.1, -0.01, -0.002], device="cuda"),
                w_in=m.mlstm_quant_e4m3(_normal((wide, d), 1, d ** -0.5), block_rows=128),
                w_out=m.mlstm_quant_e4m3(_normal((d, H * dv), 2, (H * dv) ** -0.5), block_rows=128))


def test_a_block_over_a_prompt_and_then_token_by_token():
    """Every stage against 64 bits from the values that entered it; the tokens after the prompt against one long run."""
    import torch
    announce("chain: norm e4m3 -> mm -> lin_attn -> quant -> mm, a prompt and steps")
    p = _weights()
    x = _normal((2, 150, 256), 3)
    y, o, proj, h = _block(x[:, :140].contiguous(), p, None)
    c = {"q": None}
    flat = to_np(proj).reshape(280, -1)
    c = dict(q=flat[:, :96].reshape(280, 2, 48), k=flat[:, 96:192].reshape(280, 2, 48), v=flat[:, 192:].reshape(280, 4, 64), h=None,
             do=None, dh=None, g=to_np(p["g"]).astype(np.float32), spans=[(0, 140), (140, 280)], B=2, S=140, rows=280, dtype="bf16",
             scale=48 ** -0.5)
    want = la.reference(c)
    ref.assert_within("o", to_np(o).reshape(280, 4, 64), *want["o"])
    ref.assert_within("h", to_np(h), *want["h_final"])
    whole = to_np(_block(x, p, None)[1])
    for t in range(140, 150):
        y, o, _, h = _block(x[:, t].contiguous(), p, h, step=True)
        # the step rounds its result once; the long run its operands too, each by half a step of sums as large as
        # sqrt(terms) times the result: compared as a whole, to two roundings of 2^-8 and the result's own
        a, b = to_np(o), whole[:, t]
        assert np.linalg.norm(a - b) <= 3 * 2.0 ** -8 * np.linalg.norm(b)
    assert y.shape == (2, 256) and torch.isfinite(y).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sequences_in_pieces(dtype):
    """A sequence cut anywhere, each piece from the state before it.  States are rounded as operands where a piece's
    chunks begin, so the bounds are those of the pieces, from the exact state at each one's start; the
    state handed over adds its own, far smaller, error: twice the bound covers it."""
    from mlstm_matrix_memory_amd import lin_attn_fwd
    announce(f"lin_attn in pieces {dtype}")
    c = la.make(2, 333, 3, 3, 32, 40, dtype, seed=21, grads=False)
    whole = la.reference(c)
    split = {n: c[n].reshape(2, 333, *c[n].shape[1:]) for n in ("q", "k", "v")}
    g, h, exact = to_gpu(c["g"], "f32"), to_gpu(c["h"], "f32"), c["h"]
    for a, b in ((0, 1), (1, 130), (130, 131), (131, 333)):
        part = {n: x[:, a:b].reshape(-1, *x.shape[2:]) for n, x in split.items()}
        n = b - a
        want = la.reference(dict(c, **part, h=exact, spans=[(0, n), (n, 2 * n)], rows=2 * n, S=n))
        o, h = lin_attn_fwd(*(to_gpu(part[x], dtype).view(2, n, *part[x].shape[1:]) for x in ("q", "k", "v")), g, scale=c["scale"],
                            h_init=h)
        ref.assert_within("o", to_np(o).reshape(part["v"].shape), want["o"][0], 2 * want["o"][1])
        exact = want["h_final"][0]
    ref.assert_within("h", to_np(h), whole["h_final"][0], 2 * whole["h_final"][1])


@pytest.mark.parametrize("back", [False, True])
def test_packed_with_a_gap_in_front_and_behind(back):
    """Rows that belong to no sequence are neither read nor written, whatever they hold."""
    import torch
    from mlstm_matrix_memory_amd import lin_attn_bwd, lin_attn_fwd
    announce(f"lin_attn packed behind a gap back={back}")
    c = la.make(3, 0, 4, 2, 24, 32, "bf16", seed=22, lengths=[200, 0, 131])
    front, behind = 300, 77
    pad = lambda a: np.concatenate([np.full((front, *a.shape[1:]), np.nan), a, np.full((behind, *a.shape[1:]), np.nan)])  # noqa: E731
    t = {n: to_gpu(pad(c[n]), "bf16") for n in ("q", "k", "v", "do")}
    plan = dict(seq_start=torch.tensor(c["at"] + front, dtype=torch.int32, device="cuda"), max_len=10 ** 6)
    h, dh, g = (to_gpu(c[n], "f32") for n in ("h", "dh", "g"))
    want = la.reference(c)
    room = {n: torch.full_like(t[n], 5.0) for n in ("q", "k", "v")}
    if back:
        out = lin_attn_bwd(t["q"], t["k"], t["v"], g, t["do"], scale=c["scale"], h_init=h, dh_final=dh, grad_q=room["q"],
                           grad_k=room["k"], grad_v=room["v"], **plan)
        got = dict(zip(("dq", "dk", "dv"), (to_np(x) for x in out[:3])))
        ref.assert_within("dh0", to_np(out[3]), *want["dh0"])
    else:
        o, final = lin_attn_fwd(t["q"], t["k"], t["v"], g, scale=c["scale"], h_init=h, o_out=room["v"], **plan)
        got = {"o": to_np(o)}
        ref.assert_within("h", to_np(final), *want["h_final"])
    for n, x in got.items():
        ref.assert_within(n, x[front:-behind], *want[n])
        assert (x[:front] == 5).all() and (x[-behind:] == 5).all()


def test_starts_that_no_host_check_has_seen_stay_inside():
    """Entries of seq_start out of range or out of order change which rows are read, never to others than the tensor's."""
    import torch
    from mlstm_matrix_memory_amd import lin_attn_bwd, lin_attn_fwd
    announce("lin_attn with starts out of range")
    rows = 300
    room = {n: torch.full((rows + 512, *s), 7.0, dtype=torch.bfloat16, device="cuda") for n, s in (("q", (2, 32)), ("v", (2, 48)))}
    q, v = (_normal((rows, 2, d), 30 + d) for d in (32, 48))
    g = torch.tensor([-0.1, -0.01], device="cuda")
    for starts in ([-50, 100, 10 ** 9], [200, 100, 300], [0, 0, 2 ** 31 - 1], [-2 ** 31, -5, 40]):
        plan = dict(seq_start=torch.tensor(starts, dtype=torch.int32, device="cuda"), max_len=rows)
        lin_attn_fwd(q, q, v, g, o_out=room["v"][256:256 + rows], **plan)
        lin_attn_bwd(q, q, v, g, v, grad_q=room["q"][256:256 + rows], grad_v=room["v"][256:256 + rows], **plan)
        torch.cuda.synchronize()
        for r in room.values():
            assert (r[:256] == 7).all() and (r[256 + rows:] == 7).all()


def _calls(dtype, S=1200, H=2, G=1):
    import torch
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q, k, v, do = (_normal((1, S, n, 40), 40 + i, dtype=dt) for i, n in enumerate((G, G, H, H)))
    return q, k, v, torch.tensor([-0.2, -0.004], device="cuda"), do


def test_calls_repeat_bit_for_bit_on_any_stream_and_at_once():
    import torch
    from mlstm_matrix_memory_amd import lin_attn_bwd, lin_attn_fwd
    announce("lin_attn repeated, on two streams at once")
    q, k, v, g, do = _calls("bf16")
    first = [*lin_attn_fwd(q, k, v, g), *lin_attn_bwd(q, k, v, g, do)[:3]]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    results = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        results.append([*lin_attn_fwd(q, k, v, g, stream=s), *lin_attn_bwd(q, k, v, g, do, stream=s)[:3]])
    for s in streams:
        s.synchronize()
    for r in results:
        for a, b in zip(first, r):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_and_replayed(dtype):
    """Forward, backward and step in graphs that share one workspace, replayed on new inputs with eager calls between."""
    import torch
    from mlstm_matrix_memory_amd import (MLSTM_BF16, MLSTM_F32, lin_attn_bwd, lin_attn_bwd_workspace_bytes, lin_attn_fwd,
                                         lin_attn_step)
    announce(f"lin_attn captured {dtype}")
    q, k, v, g, do = _calls(dtype)
    ws = torch.empty(lin_attn_bwd_workspace_bytes(1, 1200, 1200, 2, 1, 40, 40, MLSTM_BF16 if dtype == "bf16" else MLSTM_F32),
                     dtype=torch.uint8, device="cuda")
    h = torch.zeros(1, 2, 40, 40, device="cuda")

    def eager():
        return [*lin_attn_fwd(q, k, v, g), *lin_attn_bwd(q, k, v, g, do)[:3]]
    eager()
    torch.cuda.synchronize()
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        fwd = lin_attn_fwd(q, k, v, g, workspace=ws)
        lin_attn_step(q[:, 0], k[:, 0], v[:, 0], g, h)
    with torch.cuda.graph(two):
        bwd = lin_attn_bwd(q, k, v, g, do, workspace=ws)[:3]
    state = torch.zeros_like(h)
    for seed in range(3):
        for i, t in enumerate((q, k, v, do)):
            t.copy_(_normal(t.shape, 100 * seed + i, dtype=t.dtype))
        two.replay()
        one.replay()
        want = eager()
        lin_attn_step(q[:, 0], k[:, 0], v[:, 0], g, state)
        torch.cuda.synchronize()
        for a, b in zip([*fwd, *bwd], want):
            assert torch.equal(a, b)
        assert torch.equal(h, state)


def test_widths_whose_rows_are_far_apart():
    """Rows whose offsets pass 32 bits: two sequences of a few rows in a tensor of strides of 2^30 elements."""
    import torch
    from mlstm_matrix_memory_amd import lin_attn_fwd
    announce("lin_attn rows 2^30 elements apart")
    c = la.make(1, 5, 2, 2, 16, 24, "bf16", seed=50, grads=False, init=False)
    stride = 1 << 30
    whole = torch.empty(4 * stride + 200, dtype=torch.bfloat16, device="cuda")
    parts = {}
    at = 0
    for n in ("q", "k", "v"):
        w = c[n].shape[1:]
        parts[n] = whole.as_strided((1, 5, *w), (5 * stride, stride, w[1], 1), at)
        parts[n].copy_(to_gpu(c[n], "bf16").view(1, 5, *w))
        at += int(np.prod(w))
    o, h = lin_attn_fwd(parts["q"], parts["k"], parts["v"], to_gpu(c["g"], "f32"), scale=c["scale"])
    want = la.reference(c)
    ref.assert_within("o", to_np(o).reshape(c["v"].shape), *want["o"])
    ref.assert_within("h", to_np(h), *want["h_final"])


@pytest.mark.parametrize("rows", [140, 1])
def test_every_stage_of_a_block(rows):
    """The block's five calls over a prompt of two sequences, or (rows = 1) one row each after it: every stage against 64 bits
    from the values that entered it."""
    import torch
    import mlstm_matrix_memory_amd as m
    from test_gpu_e4m3 import expected, expected_of_cut_terms, quantised
    announce(f"chain: every stage, rows={rows}")
    p = _weights()
    step, flat = rows == 1, lambda t: to_np(t).reshape(2 * rows, -1)  # noqa: E731
    x = _normal((2, 256) if step else (2, rows, 256), 300 + rows)
    g = to_np(p["g"]).astype(np.float32)
    h = _normal((2, 4, 64, 48), 301, dtype=torch.float32) if step else None
    before = None if h is None else to_np(h).astype(np.float32)
    for (w, s), raw in ((p["w_in"], _normal((448, 256), 1, 256 ** -0.5)), (p["w_out"], _normal((256, 256), 2, 256 ** -0.5))):
        q, scale, _ = quantised(to_np(raw), 128)
        assert np.array_equal(to_np(w), q) and np.array_equal(to_np(s), scale)

    q8, s8, _ = m.mlstm_rms_norm_quant(x, p["norm"], group=128)
    proj = m.mlstm_mm_e4m3(q8, s8, *p["w_in"])
    q, k, v = proj.split([96, 96, 256], -1)
    heads = q.unflatten(-1, (2, 48)), k.unflatten(-1, (2, 48)), v.unflatten(-1, (4, 64)), p["g"]
    if step:
        o = m.lin_attn_step(*heads, h)
    else:
        o, h = m.lin_attn_fwd(*heads)
    o8, os8 = m.mlstm_quant_e4m3(o.flatten(-2))
    y = m.mlstm_mm_e4m3(o8, os8, *p["w_out"])
    torch.cuda.synchronize()

    # the norm: fp32's 1 / sqrt is 140 steps off at most (256 squares, half of whose sum's error is the root's, and 12 more
    # roundings); e4m3 rounds by 2^-4 of a value or half its smallest step
    r = ref.norm_fwd(ref.norm_sum(to_np(x).reshape(-1, 256), None, "f32"), np.ones(256), 1e-5)
    scale = np.abs(r).reshape(-1, 2, 128).max(2) / 448
    ref.assert_within("norm scale", flat(s8), scale, 140 * ref.U * scale)
    wide = np.repeat(scale, 128, 1)
    ref.assert_within("norm", flat(q8) * np.repeat(flat(s8), 128, 1), r, (1 + 1e-4) * np.maximum(2.0 ** -4 * np.abs(r), 2.0 ** -10 * wide))

    def product(a, b):
        """(y, bound) of a bf16 product; few rows sum in fp32."""
        if not step:
            return expected_of_cut_terms(*map(flat, a), *map(to_np, b), 128)
        value, bound = expected(*map(flat, a), *map(to_np, b), 128, "f32")
        return value, bound + 2.0 ** -8 * (np.abs(value) + bound)
    ref.assert_within("projection", flat(proj), *product((q8, s8), p["w_in"]))
    # the cell
    at = flat(proj)
    c = dict(q=at[:, :96].reshape(-1, 2, 48), k=at[:, 96:192].reshape(-1, 2, 48), v=at[:, 192:].reshape(-1, 4, 64), h=before, do=None,
             dh=None, g=g, spans=[(0, rows), (rows, 2 * rows)], B=2, S=rows, rows=2 * rows, dtype="bf16", scale=48 ** -0.5)
    want = la.reference(c)
    ref.assert_within("o", flat(o).reshape(-1, 4, 64), *want["o"])
    ref.assert_within("h", to_np(h), *want["h_final"])
    # its quantiser, whole values, and the product back
    value, scale, _ = quantised(flat(o), 1)
    assert np.array_equal(flat(o8), value) and np.array_equal(flat(os8), scale)
    ref.assert_within("y", flat(y), *product((o8, os8), p["w_out"]))
