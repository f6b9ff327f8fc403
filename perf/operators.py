"""The recurrent block's operators and the sizes they are timed at.

Three families, in the order a block of a recurrent language model runs them:
  norm   residual addition and root-mean-square norm, optionally with an e4m3 output and scales
  conv   short causal depthwise convolution with an optional swish
  scan   selective state space scan, its backward, and its single-token step

A case names the family (``op``) and the direction (``dir``: fwd, bwd or step).  Sequences of
a batch either have one length (``S``) or are packed behind each other (``packed``: lengths
between 0 and ``S``).  ``run`` computes the operators in elementary torch operations in
32 bits, or, where ``own`` is true, calls the library.  A single-token step updates the
state it is given in place, in both forms.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ELEM = {"bf16": 2, "f32": 4}
E4M3_MAX = 448.0


# ---- cases -----------------------------------------------------------------------
def listed():
    return [
        # a training or prompt batch of the 125M-class layer (inner width 4 * 384)
        {"name": "scan_fwd_125m", "op": "scan", "dir": "fwd", "dtype": "bf16", "B": 8, "S": 2048, "D": 1536, "G": 1,
         "N": 16, "gate": True, "half": False, "init": False, "packed": False},
        # one very long prompt (the long-context layer: 8 heads of 256), its gate read from one half of a projection
        {"name": "scan_fwd_long", "op": "scan", "dir": "fwd", "dtype": "bf16", "B": 1, "S": 32768, "D": 2048, "G": 1,
         "N": 16, "gate": True, "half": True, "init": False, "packed": False},
        # prompts of unequal length continued from earlier states, odd width, two groups, fp32
        {"name": "scan_fwd_packed", "op": "scan", "dir": "fwd", "dtype": "f32", "B": 12, "S": 700, "D": 1002, "G": 2,
         "N": 12, "gate": False, "half": False, "init": True, "packed": True},
        # the backward of a training batch of the 125M-class layer
        {"name": "scan_bwd_125m", "op": "scan", "dir": "bwd", "dtype": "bf16", "B": 4, "S": 2048, "D": 1536, "G": 1,
         "N": 16, "gate": True, "half": False, "init": False, "packed": False},
        # the backward of packed sequences in fp32, from given states, odd width
        {"name": "scan_bwd_packed", "op": "scan", "dir": "bwd", "dtype": "f32", "B": 7, "S": 391, "D": 517, "G": 1,
         "N": 16, "gate": True, "half": False, "init": True, "packed": True},
        # decoding one token for each of 256 sequences (the decode layer: 4 heads of 512)
        {"name": "scan_step_256", "op": "scan", "dir": "step", "dtype": "bf16", "B": 256, "S": 1, "D": 2048, "G": 1,
         "N": 16, "gate": True, "half": False, "init": True, "packed": False},
        # the convolution in front of the 1.3B-class layer (4 * 1024), read from one half of a projection
        {"name": "conv_fwd_1_3b", "op": "conv", "dir": "fwd", "dtype": "bf16", "B": 4, "S": 2048, "D": 4096, "W": 4,
         "act": True, "init": False, "half": True, "packed": False},
        # its backward over packed sequences of unequal length, odd width, from given states
        {"name": "conv_bwd_packed", "op": "conv", "dir": "bwd", "dtype": "bf16", "B": 9, "S": 1500, "D": 1537, "W": 4,
         "act": True, "init": True, "half": False, "packed": True},
        # decoding a few sequences: latency
        {"name": "conv_step_4", "op": "conv", "dir": "step", "dtype": "bf16", "B": 4, "S": 1, "D": 4096, "W": 4,
         "act": True, "init": True, "half": True, "packed": False},
        # decoding one sequence: latency (1.3B-class embedding)
        {"name": "norm_fwd_1", "op": "norm", "dir": "fwd", "dtype": "bf16", "res": "f32", "R": 1, "D": 2048, "group": -1},
        # the norm in front of an 8-bit projection, a prompt batch of the 1.3B-class model
        {"name": "norm_fwd_e4m3", "op": "norm", "dir": "fwd", "dtype": "bf16", "res": "bf16", "R": 8192, "D": 4096,
         "group": 128},
        # its backward over a training batch of the 125M-class model (embedding 768)
        {"name": "norm_bwd_125m", "op": "norm", "dir": "bwd", "dtype": "bf16", "res": "f32", "R": 16384, "D": 768,
         "group": -1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "conv", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        c = {"op": "norm", "dir": rng.choice(["fwd", "fwd", "bwd"]), "dtype": dtype, "res": rng.choice(["bf16", "f32"]),
             "R": _log(rng, 1, 16384), "D": _log(rng, 64, 4096), "group": -1}
        if c["dir"] == "fwd":
            c["group"] = rng.choice([-1, 0, 32, 128])
        return c
    c = {"op": op, "dir": rng.choice(["fwd", "bwd", "step"]), "dtype": dtype, "packed": False, "init": rng.random() < 0.5,
         "half": rng.random() < 0.5}
    if c["dir"] == "step":
        c.update(B=_log(rng, 1, 256), S=1, D=_log(rng, 64, 4096), init=True)
    else:
        c.update(B=_log(rng, 1, 16), S=_log(rng, 1, 4096), D=_log(rng, 64, 4096), packed=rng.random() < 0.5)
        most = (1 << 24) if op == "conv" or c["dir"] == "fwd" else (1 << 23)
        c["S"] = max(1, min(c["S"], most // (c["B"] * c["D"])))
    if op == "scan":
        c.update(G=rng.choice([1, 1, 2]), N=rng.choice([4, 7, 8, 16, 16, 24]), gate=rng.random() < 0.7)
        c["D"] += c["D"] % c["G"]
    else:
        c.update(W=rng.choice([2, 3, 4, 4]), act=rng.random() < 0.7)
    return c


# ---- inputs ----------------------------------------------------------------------
def _lengths(case):
    """Lengths of packed sequences: the longest first, an empty one and a single row, the others spread evenly."""
    B, S = case["B"], case["S"]
    n = [1 + int(S * (0.618034 * b % 1.0)) for b in range(B)]
    n[0] = S
    if B > 2:
        n[1], n[2] = 0, 1
    return n


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = DT[case["dtype"]]

    def normal(*shape, sd=1.0, mu=0.0, dtype=t):
        return (torch.randn(*shape, generator=g, device="cuda") * sd + mu).to(dtype)

    s = {"case": case}
    D = case["D"]
    if case["op"] == "norm":
        R, rt = case["R"], DT[case["res"]]
        s.update(weight=normal(D, sd=0.1, mu=1.0, dtype=torch.float32), eps=1e-6)
        if case["dir"] == "fwd":
            s.update(x=normal(R, D), residual=normal(R, D, sd=3.0, dtype=rt))
        else:
            s.update(r=normal(R, D, sd=3.0, dtype=rt), dy=normal(R, D), dres=normal(R, D, dtype=rt))
        return s
    B, S = case["B"], case["S"]
    step = case["dir"] == "step"
    lead = (B,) if step else (B, S)
    s["seq_start"] = None
    if case["packed"]:
        at = [0]
        for n in _lengths(case):
            at.append(at[-1] + n)
        s["seq_start"] = torch.tensor(at, dtype=torch.int32, device="cuda")
        lead = (at[-1],)
    if case["op"] == "conv":
        W = case["W"]
        s["x"] = normal(*lead, 2 * D)[..., :D] if case["half"] else normal(*lead, D)
        s["weight"] = (torch.rand(D, W, generator=g, device="cuda") * 2 - 1) / math.sqrt(W)
        s["bias"] = normal(D, sd=0.1, dtype=torch.float32)
        s["state"] = normal(B, W - 1, D) if case["init"] else None
        if case["dir"] == "bwd":
            s["dy"] = normal(*lead, D)
        return s
    G, N = case["G"], case["N"]
    s["x"] = normal(*lead, D)
    # step sizes around 0.001 .. 0.1, as such layers learn them
    s["dt"] = normal(*lead, D, sd=0.5)
    size = torch.exp(torch.rand(D, generator=g, device="cuda") * math.log(100.0) + math.log(0.001))
    s["dt_bias"] = torch.log(torch.expm1(size))
    s["A"] = -torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * torch.exp(normal(D, N, sd=0.1, dtype=torch.float32))
    # B and C are column ranges of one projection, behind the low-rank step sizes
    low = 8 * (-(-D // 128))
    bc = normal(*lead, low + 2 * G * N)
    s["B"] = bc[..., low:low + G * N].unflatten(-1, (G, N))
    s["C"] = bc[..., low + G * N:].unflatten(-1, (G, N))
    s["D"] = normal(D, sd=0.1, mu=1.0, dtype=torch.float32)
    s["z"] = None
    if case["gate"]:
        s["z"] = normal(*lead, 2 * D)[..., D:] if case["half"] else normal(*lead, D)
    s["h"] = normal(B, D, N, dtype=torch.float32) if case["init"] else None
    if case["dir"] == "bwd":
        s["dy"] = normal(*lead, D)
    return s


# ---- what one pass has to move and compute ------------------------------------------
def _rows(case):
    return sum(_lengths(case)) if case["packed"] else case["B"] * case["S"]


def work(case):
    e, D = ELEM[case["dtype"]], case["D"]
    if case["op"] == "norm":
        R, r = case["R"], ELEM[case["res"]]
        if case["dir"] == "fwd":
            out = e if case["group"] < 0 else 1 + 4 / (case["group"] or D)
            return {"bytes": R * D * (e + 2 * r + out) + 4 * D, "flops": 6 * R * D}
        return {"bytes": R * D * (e + r + r + e + r) + 8 * D, "flops": 14 * R * D}
    R, B = _rows(case), case["B"]
    if case["op"] == "conv":
        W = case["W"]
        state, par = B * (W - 1) * D * e, 4 * D * (W + 1)
        act = 6 if case["act"] else 0
        if case["dir"] == "step":
            return {"bytes": 2 * R * D * e + 2 * state + par, "flops": R * D * (2 * W + act)}
        if case["dir"] == "fwd":
            return {"bytes": 2 * R * D * e + (2 if case["init"] else 1) * state + par, "flops": R * D * (2 * W + act)}
        return {"bytes": 3 * R * D * e + (2 * state if case["init"] else 0) + 2 * par, "flops": R * D * (6 * W + 2 * act)}
    G, N = case["G"], case["N"]
    state, par, gate = 4 * B * D * N, 4 * D * (N + 2), 1 if case["gate"] else 0
    if case["dir"] == "bwd":
        return {"bytes": R * D * e * (5 + 2 * gate) + 4 * R * G * N * e + (2 * state if case["init"] else 0) + 2 * par,
                "flops": R * D * (20 * N + 30)}
    init = state if case["init"] else 0
    return {"bytes": R * D * e * (3 + gate) + 2 * R * G * N * e + init + state + par, "flops": R * D * (7 * N + 15)}


# ---- plain forms -----------------------------------------------------------------
def _place(s, rows):
    """Of each row its sequence and its place in it; of each sequence its first and its last row."""
    case, at = s["case"], torch.arange(rows, device="cuda")
    if s["seq_start"] is None:
        S = rows // case["B"]
        start = torch.arange(case["B"] + 1, device="cuda") * S
    else:
        start = s["seq_start"].long()
    seq = torch.searchsorted(start[1:], at, right=True)
    return seq, at - start[seq], start[:-1], start[1:]


def _silu(z):
    return z / (1 + torch.exp(-z))


def _dsilu(z):
    g = 1 / (1 + torch.exp(-z))
    return g * (1 + z * (1 - g))


def _taps(x, state, seq, pos, W):
    """[rows, W, D]: the inputs that each row's taps meet."""
    rows, D = x.shape
    B = state.shape[0]
    j = torch.arange(W, device="cuda")
    back = W - 1 - j
    at = torch.arange(rows, device="cuda")[:, None] - back
    held = B * (W - 1) + at
    kept = seq[:, None] * (W - 1) + (W - 1) + pos[:, None] - back
    return torch.cat([state.reshape(-1, D), x])[torch.where(pos[:, None] >= back, held, kept)]


def _last_inputs(x, state, first, end, W):
    """[B, W-1, D]: the last W-1 inputs of each sequence, the given state's among them."""
    B, D = state.shape[0], x.shape[1]
    back = torch.arange(W - 1, 0, -1, device="cuda")
    at = end[:, None] - back
    kept = torch.arange(B, device="cuda")[:, None] * (W - 1) + (W - 1) + at - first[:, None]
    return torch.cat([state.reshape(-1, D), x])[torch.where(at >= first[:, None], B * (W - 1) + at, kept)]


def _conv(s):
    case, x = s["case"], s["x"]
    B, D, W, t = case["B"], case["D"], case["W"], x.dtype
    shape = x.shape
    x = x.reshape(-1, D)
    state = s["state"] if s["state"] is not None else x.new_zeros(B, W - 1, D)
    seq, pos, first, end = _place(s, x.shape[0])
    taps = _taps(x.float(), state.float(), seq, pos, W)
    pre = (taps * s["weight"].t()).sum(1) + s["bias"]
    if case["dir"] != "bwd":
        y = _silu(pre) if case["act"] else pre
        last = _last_inputs(x, state, first, end, W)
        if case["dir"] == "step":
            last = s["state"].copy_(last)
        return y.to(t).reshape(shape), last
    dy = s["dy"].reshape(-1, D).float()
    dp = dy * _dsilu(pre) if case["act"] else dy
    j = torch.arange(W, device="cuda")
    ahead = W - 1 - j
    n = (end - first)[seq]
    rows = x.shape[0]
    at = torch.arange(rows, device="cuda")[:, None] + ahead
    inside = (pos[:, None] + ahead < n[:, None]).unsqueeze(-1)
    dx = (torch.where(inside, dp[at.clamp(max=rows - 1)], 0.0) * s["weight"].t()).sum(1)
    dw = (taps * dp[:, None, :]).sum(0).t().contiguous()
    out = [dx.to(t).reshape(shape), dw, dp.sum(0)]
    if s["state"] is not None:
        back = torch.arange(W - 1, 0, -1, device="cuda")
        q = ahead - back[:, None]
        at = first[:, None, None] + q
        inside = ((q >= 0) & (q < (end - first)[:, None, None])).unsqueeze(-1)
        got = torch.where(inside, dp[at.clamp(0, rows - 1)], 0.0)
        out.append((got * s["weight"].t()).sum(2).to(t))
    return tuple(out)


def _recur(a, b, most):
    """h_t = a_t h_{t-1} + b_t along the first axis, in steps of doubling length."""
    n = 1
    while n < most:
        b = torch.cat([b[:n], b[n:] + a[n:] * b[:-n]])
        a = torch.cat([a[:n], a[n:] * a[:-n]])
        n *= 2
    return b


def _scan(s):
    case, t, shape = s["case"], s["x"].dtype, s["x"].shape
    B, D, G, N = case["B"], case["D"], case["G"], case["N"]
    x = s["x"].reshape(-1, D).float()
    rows = x.shape[0]
    v = s["dt"].reshape(-1, D).float() + s["dt_bias"]
    size = torch.where(v > 20, v, torch.log1p(torch.exp(v.clamp(max=20))))
    Bm, Cm = (s[k].reshape(rows, G, 1, N).float() for k in ("B", "C"))
    seq, pos, first, end = _place(s, rows)
    full = end > first
    at, last = first[full], end[full] - 1
    a = torch.exp(size[:, :, None] * s["A"])
    u = size * x
    b = (u.view(rows, G, -1, 1) * Bm).reshape(rows, D, N)
    h0 = s["h"] if s["h"] is not None else x.new_zeros(B, D, N)
    b[at] += a[at] * h0[full]
    stop = a.clone()
    stop[at] = 0
    h = _recur(stop, b, int(case["S"]))
    y = (h.view(rows, G, -1, N) * Cm).sum(-1).reshape(rows, D) + s["D"] * x
    z = s["z"].reshape(rows, D).float() if s["z"] is not None else None
    if case["dir"] != "bwd":
        final = h0.clone()
        final[full] = h[last]
        if z is not None:
            y = y * _silu(z)
        if case["dir"] == "step":
            final = s["h"].copy_(final)
        return y.to(t).reshape(shape), final
    dy = s["dy"].reshape(-1, D).float()
    ds = dy * _silu(z) if z is not None else dy
    back = torch.cat([a[1:], a[:1]])
    back[last] = 0
    grad = (ds.view(rows, G, -1, 1) * Cm).reshape(rows, D, N)
    grad = _recur(back.flip(0), grad.flip(0), int(case["S"])).flip(0)
    before = torch.cat([h[:1], h[:-1]])
    before[at] = h0[full]
    w = grad * a * before
    du = (grad.view(rows, G, -1, N) * Bm).sum(-1).reshape(rows, D)
    dsize = x * du + (w * s["A"]).sum(-1)
    ddt = dsize / (1 + torch.exp(-v))
    out = {"x": (size * du + s["D"] * ds).to(t).reshape(shape), "dt": ddt.to(t).reshape(shape),
           "A": (w * size[:, :, None]).sum(0),
           "B": (grad * u[:, :, None]).view(rows, G, -1, N).sum(2).to(t).reshape(s["B"].shape),
           "C": (h * ds[:, :, None]).view(rows, G, -1, N).sum(2).to(t).reshape(s["C"].shape),
           "D": (ds * x).sum(0), "dt_bias": ddt.sum(0)}
    if z is not None:
        out["z"] = (dy * y * _dsilu(z)).to(t).reshape(shape)
    if s["h"] is not None:
        out["h"] = torch.zeros_like(h0)
        out["h"][full] = a[at] * grad[at]
    return out


def _norm(s):
    case = s["case"]
    t, rt = DT[case["dtype"]], DT[case["res"]]
    if case["dir"] == "bwd":
        r, dy = s["r"].float(), s["dy"].float()
        rstd = 1 / torch.sqrt((r * r).mean(-1, keepdim=True) + s["eps"])
        v = dy * s["weight"]
        dr = rstd * (v - r * (rstd * rstd) * (v * r).mean(-1, keepdim=True)) + s["dres"].float()
        return dr.to(t), dr.to(rt), (dy * r * rstd).sum(0)
    r = (s["x"].float() + s["residual"].float()).to(rt)
    f = r.float()
    y = f * (1 / torch.sqrt((f * f).mean(-1, keepdim=True) + s["eps"])) * s["weight"]
    if case["group"] < 0:
        return y.to(t), r
    n = case["group"] or case["D"]
    fill = -y.shape[1] % n
    parts = torch.cat([y, y.new_zeros(y.shape[0], fill)], 1).unflatten(1, (-1, n))
    scale = parts.abs().amax(-1) / E4M3_MAX
    q = torch.where(scale[..., None] > 0, parts / scale[..., None], 0.0).flatten(1)[:, :case["D"]]
    return q.to(torch.float8_e4m3fn), scale, r


# ---- the library's calls ------------------------------------------------------------
def _own(s):
    import mlstm_matrix_memory_amd as m
    case = s["case"]
    if case["op"] == "norm":
        if case["dir"] == "bwd":
            return m.mlstm_rms_norm_bwd(s["r"], s["weight"], s["dy"], dres=s["dres"], eps=s["eps"])
        if case["group"] < 0:
            return m.mlstm_rms_norm_fwd(s["x"], s["weight"], residual=s["residual"], eps=s["eps"])
        return m.mlstm_rms_norm_quant(s["x"], s["weight"], residual=s["residual"], eps=s["eps"], group=case["group"])
    if case["op"] == "conv":
        act = m.SSM_ACT_SWISH if case["act"] else m.SSM_ACT_NONE
        if case["dir"] == "step":
            return m.ssm_conv_step(s["x"], s["weight"], s["state"], bias=s["bias"], act=act), s["state"]
        plan = {"seq_start": s["seq_start"], "max_len": case["S"]} if case["packed"] else {}
        if case["dir"] == "fwd":
            return m.ssm_conv_fwd(s["x"], s["weight"], bias=s["bias"], act=act, state_init=s["state"], **plan)
        got = m.ssm_conv_bwd(s["x"], s["weight"], s["dy"], bias=s["bias"], act=act, state_init=s["state"], **plan)
        return tuple(g for g in got if g is not None)
    args = (s["x"], s["dt"], s["A"], s["B"], s["C"])
    more = {"D": s["D"], "z": s["z"], "dt_bias": s["dt_bias"]}
    if case["dir"] == "step":
        return m.ssm_step(*args, s["h"], **more), s["h"]
    if case["packed"]:
        more.update(seq_start=s["seq_start"], max_len=case["S"])
    if case["dir"] == "fwd":
        return m.ssm_scan_fwd(*args, h_init=s["h"], **more)
    got = m.ssm_scan_bwd(*args, s["dy"], h_init=s["h"], **more)
    names = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h")
    return {k: g for k, g in zip(names, got) if g is not None}


def run(state):
    if own:
        return _own(state)
    return {"norm": _norm, "conv": _conv, "scan": _scan}[state["case"]["op"]](state)


# ---- the definitions in 64 bits, row by row -------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "conv": _exact_conv, "scan": _exact_scan}[case["op"]](s)


def _exact_norm(s):
    case, w = s["case"], s["weight"].double()
    if case["dir"] == "bwd":
        r, dy, D = s["r"].double(), s["dy"].double(), case["D"]
        ms = r.pow(2).sum(1, keepdim=True) / D + s["eps"]
        dot = (dy * w * r).sum(1, keepdim=True) / D
        dr = dy * w * ms.pow(-0.5) - r * dot * ms.pow(-1.5) + s["dres"].double()
        return dr, dr, (dy * r * ms.pow(-0.5)).sum(0)
    total = s["x"].double() + s["residual"].double()
    r = total.to(DT[case["res"]]).double()
    y = r * w / (r.pow(2).mean(1, keepdim=True) + s["eps"]).sqrt()
    if case["group"] < 0:
        return y, total
    n = case["group"] or case["D"]
    scale = torch.stack([c.abs().amax(1) for c in y.split(n, 1)], 1) / E4M3_MAX
    wide = scale.repeat_interleave(n, 1)[:, :case["D"]]
    return torch.where(wide > 0, y / wide, 0.0), scale, total


def _sequences(s, rows):
    if s["seq_start"] is None:
        S = rows // s["case"]["B"]
        return [(b * S, b * S + S) for b in range(s["case"]["B"])]
    at = s["seq_start"].tolist()
    return list(zip(at[:-1], at[1:]))


def _exact_conv(s):
    case, x = s["case"], s["x"]
    B, D, W = case["B"], case["D"], case["W"]
    shape, x = x.shape, x.reshape(-1, D).double()
    w, bias = s["weight"].double(), s["bias"].double()
    dy = s["dy"].reshape(-1, D).double() if case["dir"] == "bwd" else None
    out, finals, dstates = torch.zeros_like(x), [], []
    dw, db = torch.zeros_like(w), torch.zeros_like(bias)
    for b, (lo, hi) in enumerate(_sequences(s, x.shape[0])):
        before = s["state"][b].double() if s["state"] is not None else x.new_zeros(W - 1, D)
        line = torch.cat([before, x[lo:hi]])
        n = hi - lo
        finals.append(line[n:])
        pre = bias + sum(w[:, j] * line[j:j + n] for j in range(W))
        gate = torch.sigmoid(pre)
        if dy is None:
            out[lo:hi] = pre * gate if case["act"] else pre
            continue
        dp = dy[lo:hi] * (gate + pre * gate * (1 - gate)) if case["act"] else dy[lo:hi]
        dline = torch.zeros_like(line)
        for j in range(W):
            dline[j:j + n] += w[:, j] * dp
            dw[:, j] += (dp * line[j:j + n]).sum(0)
        db += dp.sum(0)
        out[lo:hi] = dline[W - 1:]
        dstates.append(dline[:W - 1])
    if dy is None:
        return out.reshape(shape), torch.stack(finals)
    got = [out.reshape(shape), dw, db]
    return tuple(got + ([torch.stack(dstates)] if s["state"] is not None else []))


def _exact_scan(s):
    case, shape = s["case"], s["x"].shape
    B, D, G, N = case["B"], case["D"], case["G"], case["N"]
    x = s["x"].reshape(-1, D).double()
    rows = x.shape[0]
    v = s["dt"].reshape(-1, D).double() + s["dt_bias"].double()
    size, A = torch.nn.functional.softplus(v, threshold=50.0), s["A"].double()
    Bm, Cm = (s[k].reshape(rows, G, N).double() for k in ("B", "C"))
    seqs = _sequences(s, rows)
    order = sorted(range(B), key=lambda b: seqs[b][0] - seqs[b][1])  # the longest first
    lo = torch.tensor([seqs[b][0] for b in order], device="cuda")
    n = [seqs[b][1] - seqs[b][0] for b in order]
    h = (s["h"].double() if s["h"] is not None else x.new_zeros(B, D, N))[torch.tensor(order, device="cuda")]
    put = torch.argsort(torch.tensor(order, device="cuda"))
    most = max(n)
    bwd = case["dir"] == "bwd"
    if bwd and most * B * D * N > (1 << 30):
        return None
    heads = D // G
    out, trace, live = torch.zeros_like(x), [], [sum(m > t for m in n) for t in range(most)]
    wide = lambda m: m.repeat_interleave(heads, 1)  # noqa: E731
    for t in range(most):
        k = live[t]
        r = lo[:k] + t
        d = size[r]
        if bwd:
            trace.append(h[:k].clone())
        h[:k] = torch.exp(d.unsqueeze(2) * A) * h[:k] + (d * x[r]).unsqueeze(2) * wide(Bm[r])
        out[r] = (h[:k] * wide(Cm[r])).sum(2) + s["D"].double() * x[r]
    z = s["z"].reshape(rows, D).double() if s["z"] is not None else None
    if not bwd:
        if z is not None:
            out *= z * torch.sigmoid(z)
        return out.reshape(shape), h[put]
    dy = s["dy"].reshape(-1, D).double()
    ds, gate = dy, None
    if z is not None:
        gate = torch.sigmoid(z)
        ds = dy * z * gate
    got = {"x": torch.zeros_like(x), "dt": torch.zeros_like(x), "A": torch.zeros_like(A), "B": torch.zeros_like(Bm),
           "C": torch.zeros_like(Cm), "D": (ds * x).sum(0)}
    G_next = torch.zeros_like(h)  # the gradient that reaches each sequence's state from later rows
    for t in reversed(range(most)):
        k = live[t]
        r = lo[:k] + t
        d, xr, old = size[r], x[r], trace.pop()
        a = torch.exp(d.unsqueeze(2) * A)
        new = a * old + (d * xr).unsqueeze(2) * wide(Bm[r])
        g = G_next[:k] + ds[r].unsqueeze(2) * wide(Cm[r])
        got["C"][r] = (new * ds[r].unsqueeze(2)).unflatten(1, (G, heads)).sum(2)
        got["B"][r] = (g * (d * xr).unsqueeze(2)).unflatten(1, (G, heads)).sum(2)
        drive = (g * wide(Bm[r])).sum(2)
        decay = g * a * old
        got["A"] += (decay * d.unsqueeze(2)).sum(0)
        got["x"][r] = d * drive + s["D"].double() * ds[r]
        got["dt"][r] = (xr * drive + (decay * A).sum(2)) * torch.sigmoid(v[r])
        G_next[:k] = g * a
    got["dt_bias"] = got["dt"].sum(0)
    for k, like in (("x", shape), ("dt", shape), ("B", s["B"].shape), ("C", s["C"].shape)):
        got[k] = got[k].reshape(like)
    if z is not None:
        got["z"] = (dy * out * (gate + z * gate * (1 - gate))).reshape(shape)
    if s["h"] is not None:
        got["h"] = G_next[put]
    return got
