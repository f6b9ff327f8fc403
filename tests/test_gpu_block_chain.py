"""The block operators together, as a block runs them: norm, projection, convolution,
projections, scan, projection, residual; over a prompt and then token by token, forward
and backward; beside the mLSTM cell; in captured graphs, on other streams, side by side.
"""
import numpy as np
import pytest

import block_reference as ref
from block_reference import U
from gpu_helpers import announce, to_gpu, to_np

pytestmark = pytest.mark.gpu

B, S, E, D, N, W, LOW = 2, 50, 48, 96, 16, 4, 8


def _block(seed=1):
    rng = np.random.default_rng(seed)
    f = lambda *s, sd=1.0: (sd * rng.standard_normal(s)).astype(np.float32)  # noqa: E731
    return {"norm_w": 1 + f(E, sd=0.1), "w_in": f(2 * D, E, sd=E ** -0.5), "conv_w": f(D, W, sd=0.5), "conv_b": f(D, sd=0.1),
            "w_x": f(LOW + 2 * N, D, sd=D ** -0.5), "w_dt": f(D, LOW, sd=LOW ** -0.5),
            "dt_bias": np.log(np.expm1(np.exp(rng.uniform(np.log(1e-3), np.log(0.1), D)))).astype(np.float32),
            "A": (-np.arange(1, N + 1) * np.ones((D, 1))).astype(np.float32), "skip": np.ones(D, np.float32),
            "w_out": f(E, D, sd=D ** -0.5), "x": f(B, S, E), "residual": f(B, S, E), "dout": f(B, S, E)}


def _forward_gpu(p, x, residual, conv_state=None, h=None, step=False, keep=None):
    """x, residual [B, n, E] (or [B, E] with step) -> (block output, new residual)."""
    import torch
    import mlstm_matrix_memory_amd as m
    y, r = m.mlstm_rms_norm_fwd(x, p["norm_w"], residual=residual)
    xz = y @ p["w_in"].t()
    xi, z = xz[..., :D], xz[..., D:]
    if step:
        c = m.ssm_conv_step(xi, p["conv_w"], conv_state, bias=p["conv_b"])
    else:
        c, conv_state = m.ssm_conv_fwd(xi, p["conv_w"], bias=p["conv_b"], state_init=conv_state)
    q = c @ p["w_x"].t()
    dt = q[..., :LOW] @ p["w_dt"].t()
    Bm, Cm = q[..., LOW:LOW + N].unsqueeze(-2), q[..., LOW + N:].unsqueeze(-2)
    if step:
        o = m.ssm_step(c, dt, p["A"], Bm, Cm, h, D=p["skip"], z=z, dt_bias=p["dt_bias"])
    else:
        o, h = m.ssm_scan_fwd(c, dt, p["A"], Bm, Cm, D=p["skip"], z=z, dt_bias=p["dt_bias"], h_init=h)
    if keep is not None:
        keep.update(y=y, r=r, xi=xi, z=z, c=c, q=q, dt=dt, Bm=Bm, Cm=Cm, o=o)
    return o @ p["w_out"].t(), r, conv_state, h


def _forward_ref(b, x, residual, softplus=1):
    """The same in fp64 over whole sequences [B, n, E]."""
    n = x.shape[1]
    spans = ref.sequences(len(x), n)
    r = ref.norm_sum(x, residual, "f32").reshape(-1, E)
    y = ref.norm_fwd(r, b["norm_w"], 1e-5)
    xz = y @ b["w_in"].T.astype(np.float64)
    c = ref.conv_fwd(xz[:, :D], b["conv_w"], b["conv_b"], np.zeros((len(x), W - 1, D)), spans, True)[0]
    q = c @ b["w_x"].T.astype(np.float64)
    case = {"x": c, "dt": q[:, :LOW] @ b["w_dt"].T.astype(np.float64), "z": xz[:, D:], "A": b["A"],
            "B": q[:, None, LOW:LOW + N], "C": q[:, None, LOW + N:], "D": b["skip"], "dt_bias": b["dt_bias"], "h": None,
            "spans": spans, "softplus": softplus}
    o = ref.scan(case)["y"][0]
    return (o @ b["w_out"].T.astype(np.float64)).reshape(len(x), n, E), case, y, r, xz


def _params(b):
    return {k: to_gpu(v, "f32") for k, v in b.items() if k not in ("x", "residual", "dout")}


# The chain in fp32: five operators and fp32 products of at most 100 terms in a row, each adding
# below 200 u of the size of what it sums; sums of mixed sign can be tenfold smaller than that
# size, twice over in the backward's products of products.  These checks are for the wiring;
# the operators' own tests hold them to their last bits.
CHAIN = 5 * 200 * 10 * 10 * U


def _near(name, got, want):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    rms = np.sqrt((want ** 2).mean())
    assert np.all(np.isfinite(got)), name
    worst = np.abs(got - want).max() / rms
    assert worst <= CHAIN, f"{name}: {worst:.2e} of its root mean square off"


def test_prompt_then_tokens():
    import torch
    announce("block chain: 37 rows of prompt, 13 single rows, against whole sequences in fp64")
    b = _block()
    p, x, res = _params(b), to_gpu(b["x"], "f32"), to_gpu(b["residual"], "f32")
    n = 37
    out, r, cs, h = _forward_gpu(p, x[:, :n].contiguous(), res[:, :n].contiguous())
    outs, rs = [out], [r]
    for t in range(n, S):
        out, r, cs, h = _forward_gpu(p, x[:, t].contiguous(), res[:, t].contiguous(), cs, h, step=True)
        outs.append(out.unsqueeze(1))
        rs.append(r.unsqueeze(1))
    torch.cuda.synchronize()
    want, _, _, r64, _ = _forward_ref(b, b["x"], b["residual"])
    _near("out", to_np(torch.cat(outs, 1)), want)
    assert np.array_equal(to_np(torch.cat(rs, 1)).reshape(-1, E), r64)


def _backward_gpu(p, k, dout):
    import torch
    import mlstm_matrix_memory_amd as m
    do = dout @ p["w_out"]
    dxz = torch.empty(B, S, 2 * D, device="cuda")
    dq = torch.empty(B, S, LOW + 2 * N, device="cuda")
    g = m.ssm_scan_bwd(k["c"], k["dt"], p["A"], k["Bm"], k["Cm"], do, D=p["skip"], z=k["z"], dt_bias=p["dt_bias"],
                       grad_z=dxz[..., D:], grad_B=dq[..., LOW:LOW + N].unsqueeze(-2),
                       grad_C=dq[..., LOW + N:].unsqueeze(-2))
    dc, ddt, dA, dskip, dbias = g[0], g[1], g[2], g[5], g[7]
    dq[..., :LOW] = ddt @ p["w_dt"]
    dc = dc + dq @ p["w_x"]
    _, dcw, dcb, _ = m.ssm_conv_bwd(k["xi"], p["conv_w"], dc, bias=p["conv_b"], grad_x=dxz[..., :D])
    dy = dxz @ p["w_in"]
    dx, dres, dnw = m.mlstm_rms_norm_bwd(k["r"], p["norm_w"], dy)
    return {"x": dx, "A": dA, "skip": dskip, "dt_bias": dbias, "conv_w": dcw, "conv_b": dcb, "norm_w": dnw,
            "w_in": dxz.reshape(-1, 2 * D).t() @ k["y"].reshape(-1, E),
            "w_x": dq.reshape(-1, LOW + 2 * N).t() @ k["c"].reshape(-1, D),
            "w_dt": ddt.reshape(-1, D).t() @ k["q"].reshape(-1, LOW + 2 * N)[:, :LOW]}


def _backward_ref(b):
    want, case, y, r, xz = _forward_ref(b, b["x"], b["residual"])
    spans = case["spans"]
    w = {k: v.astype(np.float64) for k, v in b.items()}
    do = b["dout"].reshape(-1, E).astype(np.float64) @ w["w_out"]
    g = {k: v[0] for k, v in ref.scan(case, do).items()}
    dq = np.concatenate([g["grad_dt"] @ w["w_dt"], g["grad_B"][:, 0], g["grad_C"][:, 0]], 1)
    dc = g["grad_x"] + dq @ w["w_x"]
    q = case["x"] @ w["w_x"].T
    cg = ref.conv_bwd(xz[:, :D], b["conv_w"], b["conv_b"], np.zeros((B, W - 1, D)), spans, True, dc, None)
    dxz = np.concatenate([cg["x"], g["grad_z"]], 1)
    dx, dnw = ref.norm_bwd(r, b["norm_w"], dxz @ w["w_in"], None, 1e-5)
    return {"x": dx.reshape(B, S, E), "A": g["grad_A"], "skip": g["grad_D"], "dt_bias": g["grad_dt_bias"],
            "conv_w": cg["weight"], "conv_b": cg["bias"], "norm_w": dnw, "w_in": dxz.T @ y, "w_x": dq.T @ case["x"],
            "w_dt": g["grad_dt"].T @ q[:, :LOW]}


def test_training_step():
    import torch
    announce("block chain: forward and backward of 2 x 50 rows against fp64")
    b = _block(2)
    p, keep = _params(b), {}
    _forward_gpu(p, to_gpu(b["x"], "f32"), to_gpu(b["residual"], "f32"), keep=keep)
    got = _backward_gpu(p, keep, to_gpu(b["dout"], "f32"))
    torch.cuda.synchronize()
    want = _backward_ref(b)
    for k in want:
        _near("grad " + k, to_np(got[k]), want[k])


def test_captured_forward_and_backward_replay():
    """A graph of the whole step, replayed with new inputs and with the program's own eager
    calls between the replays, gives the bits of the eager step each time."""
    import torch
    announce("block chain captured, three replays with eager steps between them")
    b = _block(3)
    p = _params(b)
    x, res, dout = (to_gpu(b[k], "f32") for k in ("x", "residual", "dout"))

    def step():
        keep = {}
        out = _forward_gpu(p, x, res, keep=keep)
        return [out[0], out[1], out[2], out[3], *_backward_gpu(p, keep, dout).values()]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(3):
        x.copy_(to_gpu(np.random.default_rng(30 + k).standard_normal((B, S, E)).astype(np.float32), "f32"))
        eager = [t.clone() for t in step()]
        torch.cuda.synchronize()
        for t in held:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for i, (u, v) in enumerate(zip(held, eager)):
            assert torch.equal(u, v), f"replay {k}, output {i}"


def test_captured_token_steps_update_the_states():
    import torch
    announce("captured single-row steps: 4 replays against 4 eager steps")
    b = _block(4)
    p = _params(b)
    x, res = to_gpu(b["x"][:, 0], "f32"), to_gpu(b["residual"][:, 0], "f32")
    states = [(torch.zeros(B, W - 1, D, device="cuda"), torch.zeros(B, D, N, device="cuda")) for _ in range(2)]
    _forward_gpu(p, x, res, torch.zeros(B, W - 1, D, device="cuda"), torch.zeros(B, D, N, device="cuda"), step=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _forward_gpu(p, x, res, *states[0], step=True)[0]
    for t in range(4):
        x.copy_(to_gpu(b["x"][:, t], "f32"))
        graph.replay()
        want = _forward_gpu(p, x, res, *states[1], step=True)[0]
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert torch.equal(states[0][0], states[1][0]) and torch.equal(states[0][1], states[1][1])


def test_two_streams_at_once():
    """Calls side by side on two streams, memory reused at once on the current one."""
    import torch
    import mlstm_matrix_memory_amd as m
    from scan_cases import dev, make
    announce("scan and convolution forward and backward on two streams at once")
    cs = [make(200, 16, "bf16", 40 + k, B=2, S=700) for k in range(2)]
    args = [[dev(c, k) for k in ("x", "dt", "A", "B", "C")] for c in cs]
    more = [dict(D=dev(c, "D"), z=dev(c, "z"), dt_bias=dev(c, "dt_bias")) for c in cs]
    dys = [dev(c, "dy") for c in cs]
    w = torch.randn(200, 4, device="cuda")

    def both(k, stream):
        f = m.ssm_scan_fwd(*args[k], **more[k], stream=stream)
        g = m.ssm_scan_bwd(*args[k], dys[k], **more[k], stream=stream)
        c = m.ssm_conv_fwd(args[k][0], w, stream=stream)
        d = m.ssm_conv_bwd(args[k][0], w, dys[k], stream=stream)
        n = m.mlstm_rms_norm_bwd(args[k][0], w[:, 0].contiguous(), dys[k], stream=stream)
        return [t for t in (*f, *g, *c, *d, *n) if t is not None]

    want = [[t.clone() for t in both(k, None)] for k in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [both(k, streams[k]) for k in range(2)]
    junk = [torch.full((1 << 22,), 7.0, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    del junk
    for k in range(2):
        for u, v in zip(got[k], want[k]):
            assert torch.equal(u, v)


def test_in_front_of_the_mlstm_cell():
    """Norm and convolution feed the cell, the cell's output goes through the epilogue."""
    import torch
    import oracle
    import mlstm_matrix_memory_amd as m
    from gpu_helpers import TOL, rel_err
    announce("norm -> conv -> mlstm_fwd_parallel -> epilogue, B=1 NH=2 S=128 d=64")
    NH, d, n = 2, 64, 128
    rng = np.random.default_rng(50)
    x = ref.stored(rng.standard_normal((1, n, NH * d)), "bf16")
    w, cw = np.ones(NH * d, np.float32), (0.5 * rng.standard_normal((NH * d, 4))).astype(np.float32)
    y, _ = m.mlstm_rms_norm_fwd(to_gpu(x, "bf16"), to_gpu(w, "f32"))
    c, _ = m.ssm_conv_fwd(y, to_gpu(cw, "f32"))
    heads = lambda t: t.view(1, n, NH, d).transpose(1, 2).contiguous()  # noqa: E731
    q, k, v = heads(c), (heads(c).float() / 8).to(torch.bfloat16), heads(y)
    gates = rng.standard_normal((2, 1, NH, n)).astype(np.float32)
    o = rng.standard_normal((1, NH, n, d)).astype(np.float32)
    h = m.mlstm_fwd_parallel(q, k, v, to_gpu(gates[0], "f32"), to_gpu(gates[1] + 3, "f32"), to_gpu(o, "f32"), 64)[0]
    torch.cuda.synchronize()
    r = oracle.Oracle().fwd(to_np(q), to_np(k), to_np(v), gates[0], gates[1] + np.float32(3), o)[0]
    assert rel_err(to_np(h), r) <= TOL["bf16"]
