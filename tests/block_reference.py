"""The block operators (norm, short convolution, selective scan) and their backward
passes in fp64 numpy, straight from the formulas, and the error bounds they are held to.

Test infrastructure only; shares no code with the library.
"""
import numpy as np

from mlstm_matrix_memory_amd import inputs

# half a step of each storage type, relative to the value
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
U = 2.0 ** -24
# the smallest normal fp32 number: the hardware exponential gives zero below it, and results
# below it may be flushed, so each such result is off by at most this much
TINY = 2.0 ** -126


def stored(a, dtype):
    """Values as the type holds them."""
    a = np.asarray(a, dtype=np.float32)
    return inputs.bf16_round(a) if dtype == "bf16" else a


def assert_within(name, got, ref, bound):
    """|got - ref| <= bound, element by element; NaN and infinities where ref has them."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{name}: NaN in other places"
    assert np.array_equal(got[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)]), f"{name}: infinities differ"
    over = np.where(fine, np.abs(np.where(fine, got, 0) - np.where(fine, ref, 0)), 0) - np.broadcast_to(bound, ref.shape)
    if over.size and over.max() > 0:
        at = np.unravel_index(int(np.argmax(over)), over.shape)
        raise AssertionError(f"{name}{list(at)}: {got[at]!r}, expected {ref[at]!r} within "
                             f"{np.broadcast_to(bound, ref.shape)[at]:.3g}")


# ---- norm ------------------------------------------------------------------------
def norm_sum(x, residual, res_dtype):
    """r: the fp32 sum rounded to the residual's type (float64 values)."""
    total = np.asarray(x, np.float32) + (np.float32(0) if residual is None else np.asarray(residual, np.float32))
    return stored(total, res_dtype).astype(np.float64)


def norm_fwd(r, weight, eps):
    k = 1 / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    return r * k * np.asarray(weight, np.float64)


def norm_bwd(r, weight, dy, dres, eps):
    r, w, dy = (np.asarray(a, np.float64) for a in (r, weight, dy))
    k = 1 / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    v = w * dy
    dr = k * (v - r * k ** 2 * (v * r).mean(-1, keepdims=True))
    if dres is not None:
        dr = dr + np.asarray(dres, np.float64)
    return dr, (dy * r * k).reshape(-1, r.shape[-1]).sum(0)


def quantise_groups(y, group):
    """(largest |y| / 448 per group, the same spread over the columns)."""
    d = y.shape[-1]
    n = group or d
    starts = np.arange(0, d, n)
    scale = np.maximum.reduceat(np.abs(y), starts, axis=-1) / 448.0
    return scale, np.repeat(scale, n, axis=-1)[..., :d]


# ---- sequences ---------------------------------------------------------------------
def sequences(B, S, seq_start=None):
    """[(first row, one past the last row)] of a batch."""
    if seq_start is None:
        return [(b * S, (b + 1) * S) for b in range(B)]
    return [(int(a), int(z)) for a, z in zip(seq_start[:-1], seq_start[1:])]


# ---- short causal convolution ----------------------------------------------------------
def _sigmoid(x):
    return 0.5 * (1 + np.tanh(0.5 * x))


def conv_fwd(x, weight, bias, state, spans, act):
    """x [rows,D], state [B,W-1,D]; returns (y [rows,D], final state, sum of |terms| of p)."""
    x, w, state = (np.asarray(a, np.float64) for a in (x, weight, state))
    bias = np.zeros(x.shape[1]) if bias is None else np.asarray(bias, np.float64)
    W = w.shape[1]
    y, final, size = np.zeros_like(x), state.copy(), np.zeros_like(x)
    for b, (lo, hi) in enumerate(spans):
        line = np.concatenate([state[b], x[lo:hi]])
        n = hi - lo
        taps = [w[:, j] * line[j:j + n] for j in range(W)]
        p = bias + sum(taps)
        size[lo:hi] = np.abs(bias) + sum(np.abs(t) for t in taps)
        y[lo:hi] = p * _sigmoid(p) if act else p
        final[b] = line[n:]
    return y, final, size


def conv_bwd(x, weight, bias, state, spans, act, dy, dfinal):
    """Returns dict of gradients x, weight, bias, state, and of the sums of the absolute
    values of each one's terms (size_*)."""
    x, w, state, dy = (np.asarray(a, np.float64) for a in (x, weight, state, dy))
    bias = np.zeros(x.shape[1]) if bias is None else np.asarray(bias, np.float64)
    W = w.shape[1]
    g = {"x": np.zeros_like(x), "weight": np.zeros_like(w), "bias": np.zeros_like(bias), "state": np.zeros_like(state)}
    g.update({f"size_{k}": np.zeros_like(v) for k, v in g.items()})
    for b, (lo, hi) in enumerate(spans):
        line = np.concatenate([state[b], x[lo:hi]])
        n = hi - lo
        p = bias + sum(w[:, j] * line[j:j + n] for j in range(W))
        s = _sigmoid(p)
        dp = dy[lo:hi] * (s * (1 + p * (1 - s))) if act else dy[lo:hi]
        dline, size = np.zeros_like(line), np.zeros_like(line)
        if dfinal is not None:
            dline[n:] += dfinal[b]
            size[n:] += np.abs(dfinal[b])
        for j in range(W):
            dline[j:j + n] += w[:, j] * dp
            size[j:j + n] += np.abs(w[:, j] * dy[lo:hi])
            g["weight"][:, j] += (dp * line[j:j + n]).sum(0)
            g["size_weight"][:, j] += np.abs(dy[lo:hi] * line[j:j + n]).sum(0)
        g["bias"] += dp.sum(0)
        g["size_bias"] += np.abs(dy[lo:hi]).sum(0)
        g["x"][lo:hi], g["state"][b] = dline[W - 1:], dline[:W - 1]
        g["size_x"][lo:hi], g["size_state"][b] = size[W - 1:], size[:W - 1]
    return g


# ---- selective state space scan ------------------------------------------------------------
def softplus(v):
    return np.where(v > 30, v, np.log1p(np.exp(np.minimum(v, 30))))


def _wide(m, D):
    """[G,N] -> [D,N]: each channel's group."""
    return np.repeat(m, D // m.shape[0], axis=0)


def scan(c, dy=None, dh_final=None, joins=False):
    """Forward (and, with dy, backward) of the scan, with a bound on a fp32 evaluation's error.

    c: dict with x, dt, z (or None) [rows,D], A [D,N], B, C [rows,G,N], D, dt_bias [D] (or
    None), h [batch,D,N] (or None), spans, softplus.  Returns {name: (value, bound)}; the
    bounds hold before a result is rounded to its storage type.

    Errors are followed through the recurrences.  Units u = 2^-24.  v = dt + bias is
    rounded once (|v| u); exp2 of LOG2E v adds 2 |v| u + 2 u; the logarithm, the reciprocal and four products
    7 u more: s is within es = (3 |v| + 10) u, relative, and v's own rounding where there
    is no softplus.  The decay's exponent s A log2(e) adds two roundings, its exp2 one:
    a is within ea = |s A| (es + 3 u) + 2 u.  Each step of h then adds the errors of its two
    terms and of their sum.  joins: the sequence may be cut into pieces, whose step
    sizes are summed (at most one u per row, times x e^-x <= 0.37 of what enters).
    """
    f = lambda k: None if c.get(k) is None else np.asarray(c[k], np.float64)  # noqa: E731
    x, dt, A, Bm, Cm = (f(k) for k in ("x", "dt", "A", "B", "C"))
    rows, D = x.shape
    N = A.shape[1]
    skip = f("D") if c.get("D") is not None else np.zeros(D)
    bias = f("dt_bias") if c.get("dt_bias") is not None else np.zeros(D)
    h0 = f("h") if c.get("h") is not None else np.zeros((len(c["spans"]), D, N))
    v = dt + bias
    s = softplus(v) if c["softplus"] else v
    es = (3 * np.abs(v) + 10) * U if c["softplus"] else np.full_like(v, 0.0)
    abs_s = np.abs(s) * es if c["softplus"] else np.abs(dt) * U + np.abs(bias) * U   # absolute error of s
    u = s * x
    eu = abs_s * np.abs(x) + U * np.abs(u)
    z = f("z")
    o, Eo = np.zeros((rows, D)), np.zeros((rows, D))
    H, EH = np.zeros((rows, D, N)), np.zeros((rows, D, N))
    before, Ebefore = np.zeros((rows, D, N)), np.zeros((rows, D, N))
    a_all = np.exp(s[:, :, None] * A)
    ea = np.abs(A) * abs_s[:, :, None] + np.abs(s[:, :, None] * A) * 3 * U + 2 * U
    final, Efinal = h0.copy(), np.zeros_like(h0)
    for b, (lo, hi) in enumerate(c["spans"]):
        h, E, most = h0[b], np.zeros((D, N)), np.abs(h0[b])
        for t in range(lo, hi):
            before[t], Ebefore[t] = h, E
            a, ub = a_all[t], u[t][:, None] * _wide(Bm[t], D)
            E = a * E + np.abs(a * h) * (ea[t] + U) + eu[t][:, None] * np.abs(_wide(Bm[t], D)) + 2 * U * np.abs(ub)
            h = a * h + ub
            E = E + U * np.abs(h) + TINY * (1 + np.abs(before[t]))
            most = np.maximum(most, np.abs(h))
            if joins:
                E = np.maximum(E, 0) + (0.4 * U * most if t > lo else 0)
            H[t], EH[t] = h, E
            Ct = _wide(Cm[t], D)
            o[t] = (h * Ct).sum(1) + skip * x[t]
            Eo[t] = (np.abs(Ct) * (E + (N + 3) * U * np.abs(h))).sum(1) + 3 * U * np.abs(skip * x[t])
        final[b], Efinal[b] = h, E
    out = {"h_final": (final, Efinal)}
    if z is None:
        out["y"] = (o, Eo)
    else:
        sg = _sigmoid(z)
        gate = z * sg
        eg = (6 + np.abs(z)) * U
        out["y"] = (o * gate, np.abs(gate) * (Eo + (eg + 2 * U) * np.abs(o)))
    if dy is None:
        return out
    dy = np.asarray(dy, np.float64)
    ds, eds = dy, np.zeros_like(dy)
    if z is not None:
        ds = dy * gate
        eds = np.abs(ds) * (eg + 2 * U)
        slope = sg * (1 + z * (1 - sg))
        out["grad_z"] = (dy * o * slope, np.abs(dy) * (Eo * np.abs(slope) + np.abs(o) * (12 + 2 * np.abs(z)) * U))
    g = {k: np.zeros(sh) for k, sh in (("x", x.shape), ("dt", x.shape), ("A", A.shape), ("B", Bm.shape), ("C", Cm.shape),
                                       ("h", h0.shape))}
    e = {k: np.zeros_like(val) for k, val in g.items()}
    G = Bm.shape[1]
    for b, (lo, hi) in enumerate(c["spans"]):
        nxt = np.zeros((D, N)) if dh_final is None else np.asarray(dh_final[b], np.float64)
        En, most = np.zeros((D, N)), np.abs(nxt)
        for t in range(hi - 1, lo - 1, -1):
            Ct, Bt, a = _wide(Cm[t], D), _wide(Bm[t], D), a_all[t]
            q = ds[t][:, None] * Ct
            gr = nxt + q
            E = En + eds[t][:, None] * np.abs(Ct) + U * np.abs(q) + U * np.abs(gr) + TINY
            most = np.maximum(most, np.abs(gr))
            if joins:
                E = E + 0.4 * U * most
            w = gr * a * before[t]
            ew = (E * np.abs(a * before[t]) + np.abs(gr * a) * Ebefore[t] + np.abs(w) * (ea[t] + 3 * U)
                  + TINY * (1 + np.abs(gr) + np.abs(gr * before[t])))
            du = (gr * Bt).sum(1)
            edu = (E * np.abs(Bt) + np.abs(gr * Bt) * (N + 3) * U).sum(1)
            das = (w * A).sum(1)
            edas = (ew * np.abs(A) + np.abs(w * A) * (N + 3) * U).sum(1)
            g["x"][t] = s[t] * du + skip * ds[t]
            e["x"][t] = np.abs(s[t]) * edu + abs_s[t] * np.abs(du) + np.abs(skip) * eds[t] + 3 * U * (
                np.abs(s[t] * du) + np.abs(skip * ds[t]))
            dsz = x[t] * du + das
            sgm = _sigmoid(v[t]) if c["softplus"] else 1.0
            g["dt"][t] = dsz * sgm
            e["dt"][t] = sgm * (np.abs(x[t]) * edu + edas + (12 + np.abs(v[t])) * U * (np.abs(x[t] * du) + np.abs(das)))
            g["A"] += w * s[t][:, None]
            e["A"] += ew * np.abs(s[t][:, None]) + np.abs(w) * abs_s[t][:, None] + (rows + 3) * U * np.abs(w * s[t][:, None])
            dB, dC = gr * u[t][:, None], H[t] * ds[t][:, None]
            eB = E * np.abs(u[t][:, None]) + np.abs(gr) * eu[t][:, None] + (D // G + 3) * U * np.abs(dB)
            eC = EH[t] * np.abs(ds[t][:, None]) + np.abs(H[t]) * eds[t][:, None] + (D // G + 3) * U * np.abs(dC)
            for k, val, er in (("B", dB, eB), ("C", dC, eC)):
                g[k][t], e[k][t] = val.reshape(G, D // G, N).sum(1), er.reshape(G, D // G, N).sum(1)
            nxt = gr * a
            En = E * a + np.abs(nxt) * (ea[t] + U) + TINY * (1 + np.abs(gr))
        g["h"][b], e["h"][b] = nxt, En
    inside = np.zeros((rows, 1))
    for lo, hi in c["spans"]:
        inside[lo:hi] = 1
    ds, eds = ds * inside, eds * inside
    g["D"], e["D"] = (ds * x).sum(0), ((eds + (rows + 3) * U * np.abs(ds)) * np.abs(x)).sum(0)
    g["dt_bias"], e["dt_bias"] = g["dt"].sum(0), (e["dt"] + (rows + 3) * U * np.abs(g["dt"])).sum(0)
    out.update({f"grad_{k}": (g[k], e[k]) for k in g})
    return out
