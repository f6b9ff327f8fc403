"""The e4m3 quantiser and product on the GPU against 64 bits: odd and ragged sizes, both kinds of
blocks, strides, every tile that the sizes choose, special values, streams, graphs.

The quantiser's values are whole: no tolerance.  The product's bound, per element, with T the sum of
the absolute terms: fp32 results sum exact products in fp32, 128 in a block and then the blocks with
two rounded factors, so at most (128 + blocks + 4) 2^-24 T.  The instruction of the bf16 results
keeps fewer bits; its sums are taken as good to 2^-14 of a block's T, and the result is rounded
once, by at most 2^-8 of its value."""
import numpy as np
import pytest

import block_reference as ref
from gpu_helpers import announce, to_gpu, to_np
from test_gpu_norm_e4m3 import e4m3

pytestmark = pytest.mark.gpu

BLOCK = 128


def quantised(x, block_rows):
    """(q, scale, scale of each element) of x [rows, cols], as the header defines them."""
    x = np.asarray(x, np.float32)
    rows, cols = x.shape
    big = np.where(np.isnan(x), 0, np.abs(x))
    m = np.maximum.reduceat(np.maximum.reduceat(big, np.arange(0, cols, BLOCK), axis=1), np.arange(0, rows, block_rows), axis=0)
    scale = m / np.float32(448)
    # quotients by the fp32 scale, rounded to fp32; by max / 448 unrounded where that is below the smallest normal number
    by = np.where(scale >= 2.0 ** -126, scale.astype(np.float64), m.astype(np.float64) / 448)
    wide = np.repeat(np.repeat(by, block_rows, 0)[:rows], BLOCK, 1)[:, :cols]
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        q = e4m3(np.where(wide > 0, (x.astype(np.float64) / np.where(wide > 0, wide, 1)).astype(np.float32), 0))
    return np.where(np.isnan(x), np.nan, q), scale, wide


QUANT_SIZES = [(1, 1), (1, 128), (3, 130), (2, 4096), (127, 129), (128, 128), (129, 127), (130, 257), (1000, 77), (257, 1001)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("turn", [False, True])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantiser(block_rows, turn, dtype):
    import torch
    from mlstm_matrix_memory_amd import mlstm_quant_e4m3
    for rows, cols in QUANT_SIZES:
        announce(f"quant rows={rows} cols={cols} blocks of {block_rows} turn={turn} {dtype}")
        rng = np.random.default_rng(rows * cols)
        x = ref.stored(rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal(cols)), dtype)
        x[rows // 2:, cols // 3] = 0
        q, scale = mlstm_quant_e4m3(to_gpu(x, dtype), block_rows=block_rows, transpose=turn)
        torch.cuda.synchronize()
        rq, rs, _ = quantised(x.T if turn else x, block_rows)
        assert np.array_equal(to_np(scale).reshape(rs.shape), rs)
        assert np.array_equal(to_np(q), rq)


@pytest.mark.parametrize("turn", [False, True])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantiser_of_a_column_range_leaves_what_surrounds_its_outputs(block_rows, turn):
    import torch
    from mlstm_matrix_memory_amd import mlstm_quant_e4m3
    announce(f"quant of a column range, blocks of {block_rows} turn={turn}")
    rows, cols = 133, 201
    x = ref.stored(np.random.default_rng(1).standard_normal((rows, 3 * cols)), "bf16")
    part = to_gpu(x, "bf16")[:, cols + 1:2 * cols + 1]
    rq, rs, _ = quantised(x[:, cols + 1:2 * cols + 1].T if turn else x[:, cols + 1:2 * cols + 1], block_rows)
    room = torch.full((rq.size + 64,), 7, dtype=torch.uint8, device="cuda")
    sroom = torch.full((rs.size + 64,), 7.0, device="cuda")
    q = room[33:33 + rq.size].view(torch.float8_e4m3fn).view(rq.shape)
    scale = sroom[33:33 + rs.size].view(rs.shape)
    mlstm_quant_e4m3(part, block_rows=block_rows, transpose=turn, q_out=q, scale_out=scale)
    torch.cuda.synchronize()
    assert np.array_equal(to_np(q), rq) and np.array_equal(to_np(scale), rs)
    assert (room[:33] == 7).all() and (room[33 + rq.size:] == 7).all()
    assert (sroom[:33] == 7).all() and (sroom[33 + rs.size:] == 7).all()


@pytest.mark.parametrize("turn", [False, True])
def test_quantiser_of_nan_infinities_and_tiny_values(turn):
    import torch
    from mlstm_matrix_memory_amd import mlstm_quant_e4m3
    announce(f"quant of special values turn={turn}")
    x = np.random.default_rng(2).standard_normal((140, 150)).astype(np.float32)
    x[3, 5], x[7, 9], x[130, 140] = np.nan, np.inf, -np.inf
    x[20] *= np.float32(2.0 ** -110)
    x[21] *= np.float32(2.0 ** -125)
    x[22] = 0
    t = x.T if turn else x
    q, scale = mlstm_quant_e4m3(to_gpu(np.ascontiguousarray(x), "f32"), transpose=turn)
    torch.cuda.synchronize()
    q, scale = to_np(q), to_np(scale)
    for i in range(t.shape[0]):
        for j in range(0, t.shape[1], BLOCK):
            line, got = t[i, j:j + BLOCK], q[i, j:j + BLOCK]
            fine = line[~np.isnan(line)]
            m = np.abs(fine).max()
            if np.isinf(m):
                assert np.isinf(scale[i, j // BLOCK])
                assert np.array_equal(np.isnan(got), ~np.isfinite(line)) and (got[np.isfinite(line)] == 0).all()
            else:
                assert scale[i, j // BLOCK] == m / np.float32(448) or abs(scale[i, j // BLOCK] - m / 448) <= 2.0 ** -126
                r = quantised(np.where(np.isnan(line), 0, line)[None], 1)[0][0]
                assert np.array_equal(np.isnan(got), np.isnan(line))
                assert np.array_equal(got[~np.isnan(line)], r[~np.isnan(line)])


def operands(M, N, K, block_rows, seed=0):
    rng = np.random.default_rng(seed + M + N + K)
    a, b = rng.standard_normal((M, K)) * np.exp(rng.standard_normal(K)), rng.standard_normal((N, K))
    (qa, sa, _), (qb, sb, _) = quantised(a, 1), quantised(b, block_rows)
    return qa, sa, qb, sb


def expected(qa, sa, qb, sb, block_rows, out):
    (M, K), N = qa.shape, qb.shape[0]
    wa = np.repeat(sa.astype(np.float64), BLOCK, 1)[:, :K]
    wb = np.repeat(np.repeat(sb.astype(np.float64), block_rows, 0)[:N], BLOCK, 1)[:, :K]
    with np.errstate(invalid="ignore"):
        a, b = qa * wa, qb * wb
        y, T = a @ b.T, np.abs(a) @ np.abs(b).T
        if out == "bf16":
            return y, 2.0 ** -14 * T + 2.0 ** -8 * np.abs(y) * (1 + 2.0 ** -14)
        return y, (128 + sa.shape[1] + 4) * 2.0 ** -24 * T


def e4m3_gpu(q):
    return to_gpu(q, "f32").to(__import__("torch").float8_e4m3fn)


MM_SIZES = [
    (1, 1, 1), (1, 16, 16), (2, 17, 15), (3, 130, 128), (16, 100, 257), (17, 40, 1040), (33, 50, 130), (64, 300, 520),
    (65, 64, 16), (100, 129, 257), (130, 260, 384), (300, 201, 1000), (129, 65, 4100),
    # 128 x 128 tiles, whole blocks straight to LDS and bytes by registers
    (2048, 2100, 400), (2050, 2051, 131),
    # 256 x 256 tiles, the last block shorter
    (4100, 4090, 144),
]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("M,N,K", MM_SIZES)
def test_product(M, N, K, block_rows, out):
    import torch
    from mlstm_matrix_memory_amd import mlstm_mm_e4m3
    announce(f"mm M={M} N={N} K={K} blocks of {block_rows} {out}")
    qa, sa, qb, sb = operands(M, N, K, block_rows)
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    # a column range of a wider tensor whose other columns stay as they are
    room = torch.full((M, N + 9), 3.0, dtype=dt, device="cuda")
    y = mlstm_mm_e4m3(e4m3_gpu(qa), to_gpu(sa, "f32"), e4m3_gpu(qb), to_gpu(sb, "f32"), block_rows=block_rows,
                      y_out=room[:, 5:5 + N])
    torch.cuda.synchronize()
    r, bound = expected(qa, sa, qb, sb, block_rows, out)
    ref.assert_within("y", to_np(y), r, bound)
    assert (room[:, :5] == 3).all() and (room[:, 5 + N:] == 3).all()


def test_product_of_unaligned_operands_and_leading_dimensions():
    import torch
    from mlstm_matrix_memory_amd import mlstm_mm_e4m3
    announce("mm with operands at odd addresses, a of three dimensions")
    qa, sa, qb, sb = operands(2 * 45, 70, 256, 128)
    whole = torch.empty(2 * 45 * 256 + 3, dtype=torch.float8_e4m3fn, device="cuda")
    a = whole[3:].view(2, 45, 256)
    a.copy_(e4m3_gpu(qa).view(2, 45, 256))
    y = mlstm_mm_e4m3(a, to_gpu(sa, "f32").view(2, 45, 2), e4m3_gpu(qb), to_gpu(sb, "f32"), out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert y.shape == (2, 45, 70)
    r, bound = expected(qa, sa, qb, sb, 128, "f32")
    ref.assert_within("y", to_np(y).reshape(90, 70), r, bound)


@pytest.mark.parametrize("M", [5, 200])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_nan_and_infinities_stay_in_their_row_and_column(M, out):
    import torch
    from mlstm_matrix_memory_amd import mlstm_mm_e4m3
    announce(f"mm with NaN and infinities M={M} {out}")
    qa, sa, qb, sb = operands(M, 140, 300, 1)
    qa[2, 290] = np.nan
    sa[M - 1, 1] = np.nan
    sb[139, 2] = np.inf
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    y = to_np(mlstm_mm_e4m3(e4m3_gpu(qa), to_gpu(sa, "f32"), e4m3_gpu(qb), to_gpu(sb, "f32"), block_rows=1, out_dtype=dt))
    r, bound = expected(np.where(np.isnan(qa), 0, qa), np.where(np.isnan(sa), 0, sa), qb, np.where(np.isinf(sb), 0, sb), 1, out)
    rows = np.setdiff1d(np.arange(M), [2, M - 1])
    ref.assert_within("y", y[rows][:, :139], r[rows][:, :139], bound[rows][:, :139])
    assert np.isnan(y[[2, M - 1]]).all() and not np.isfinite(y[:, 139]).any()


def test_the_norm_s_output_feeds_the_product_and_calls_repeat_bit_for_bit():
    import torch
    from mlstm_matrix_memory_amd import mlstm_mm_e4m3, mlstm_quant_e4m3, mlstm_rms_norm_quant
    announce("norm quant -> mm, twice and on another stream")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(70, 3, 384, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(500, 384, generator=g, device="cuda")
    q, s, _ = mlstm_rms_norm_quant(x, torch.ones(384, device="cuda"), group=128)
    wq, ws = mlstm_quant_e4m3(w, block_rows=128)
    y = mlstm_mm_e4m3(q, s, wq, ws)
    assert y.shape == (70, 3, 500)
    r, bound = expected(to_np(q).reshape(210, 384), to_np(s).reshape(210, 3), to_np(wq), to_np(ws), 128, "bf16")
    ref.assert_within("y", to_np(y).reshape(210, 500), r, bound)
    assert torch.equal(y, mlstm_mm_e4m3(q, s, wq, ws))
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    z = mlstm_mm_e4m3(q, s, wq, ws, stream=other)
    other.synchronize()
    assert torch.equal(y, z)


def test_gradients_of_a_linear_layer():
    """dx = dy W and dW = dy^T x from quantised operands, against the same operands in 64 bits."""
    import torch
    from mlstm_matrix_memory_amd import mlstm_mm_e4m3, mlstm_quant_e4m3
    announce("mm: both gradients of a linear layer")
    g = torch.Generator(device="cuda").manual_seed(2)
    T, K, N = 333, 200, 140
    x, dy, w = (torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16) for s in ((T, K), (T, N), (N, K)))
    for name, (a, turn_a), (b, turn_b), rows in (("dx", (dy, False), (w, True), 128), ("dw", (dy, True), (x, True), 1)):
        qa, sa = mlstm_quant_e4m3(a, transpose=turn_a)
        qb, sb = mlstm_quant_e4m3(b, block_rows=rows, transpose=turn_b)
        y = mlstm_mm_e4m3(qa, sa, qb, sb, block_rows=rows, out_dtype=torch.float32)
        r, bound = expected(to_np(qa), to_np(sa), to_np(qb), to_np(sb), rows, "f32")
        ref.assert_within(name, to_np(y), r, bound)
        plain = (dy.double() @ w.double() if name == "dx" else dy.double().t() @ x.double()).cpu().numpy()
        # e4m3 rounds each factor by at most 2^-4 of its value, or half its smallest step 2^-10 of a block's scale
        assert np.linalg.norm(to_np(y) - plain) <= 2 * 2.0 ** -4 * 1.1 * np.linalg.norm(plain)


def test_captured_and_replayed():
    import torch
    from mlstm_matrix_memory_amd import mlstm_mm_e4m3, mlstm_quant_e4m3
    announce("quant -> mm captured into a graph, replayed on new inputs")
    x = torch.randn(300, 260, device="cuda").to(torch.bfloat16)
    w = torch.randn(200, 260, device="cuda")
    wq, ws = mlstm_quant_e4m3(w, block_rows=128)

    def pair():
        q, s = mlstm_quant_e4m3(x)
        return mlstm_mm_e4m3(q, s, wq, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pair()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = pair()
    for seed in range(3):
        x.copy_(torch.randn(300, 260, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, pair())


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("M,N,K", [(1, 20, 300), (16, 40, 256), (40, 33, 1000), (64, 50, 400), (65, 70, 400), (200, 140, 304), (130, 70, 301)])
def test_terms_that_cancel(M, N, K, block_rows, out):
    """Values of 14 powers of two whose second half of a block takes the first half back, but for its last eight.  fp32
    sums in fp32 results and up to 64 rows; above that a bf16 result's eight neighbouring terms are each cut by less than 2^-13
    of the largest one's power of two: 7 of them, as the largest is whole."""
    import torch
    from mlstm_matrix_memory_amd import mlstm_mm_e4m3
    announce(f"mm of terms that cancel M={M} N={N} K={K} blocks of {block_rows} {out}")
    rng = np.random.default_rng(M + N + K)
    qa, qb = (e4m3(np.clip(rng.standard_normal((n, K)) * 2.0 ** rng.integers(-6, 8, K), -448, 448)) for n in (M, N))
    for j in range(0, K - 127, BLOCK):
        qa[:, j + 64:j + 120], qb[:, j + 64:j + 120] = qa[:, j:j + 56], -qb[:, j:j + 56]
    blocks = -(-K // BLOCK)
    sa, sb = (np.exp(rng.standard_normal((n, blocks))).astype(np.float32) for n in (M, -(-N // block_rows)))
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    y = mlstm_mm_e4m3(e4m3_gpu(qa), to_gpu(sa, "f32"), e4m3_gpu(qb), to_gpu(sb, "f32"), block_rows=block_rows, out_dtype=dt)
    torch.cuda.synchronize()
    r, bound = expected(qa, sa, qb, sb, block_rows, "f32")
    if out == "bf16":
        if M > 64:
            wide = lambda x: np.pad(x, ((0, 0), (0, -K % 8))).reshape(len(x), -1, 8)  # noqa: E731
            for i in range(0, -(-K // 8)):
                a, b = wide(qa)[:, i], wide(qb)[:, i]
                scale = sa[:, None, 8 * i // BLOCK] * np.repeat(sb, block_rows, 0)[None, :N, 8 * i // BLOCK].astype(np.float64)
                bound = bound + 7 * 2.0 ** -13 * np.abs(a[:, None] * b[None]).max(2) * scale
        bound = bound + 2.0 ** -8 * (np.abs(r) + bound)
    ref.assert_within("y", to_np(y), r, bound)


@pytest.mark.parametrize("M", [1, 16, 17, 33, 64])
def test_small_terms_beside_two_that_cancel(M):
    """126 equal terms beside 448^2 and -448^2, which the eight neighbours of one or of both must not lose."""
    import torch
    from mlstm_matrix_memory_amd import mlstm_mm_e4m3
    announce(f"mm of small terms beside two large ones M={M}")
    for small in (4.0, 1.0):
        for first, second in ((0, 1), (0, 127), (3, 64)):
            qa, qb = np.full((M, 128), small), np.ones((20, 128))
            qa[:, [first, second]] = 448
            qb[:, first], qb[:, second] = 448, -448
            ones = lambda n: to_gpu(np.ones((n, 1)), "f32")  # noqa: E731
            for dt in (torch.bfloat16, torch.float32):
                y = to_np(mlstm_mm_e4m3(e4m3_gpu(qa), ones(M), e4m3_gpu(qb), ones(20), block_rows=1, out_dtype=dt))
                bound = 129 * 2.0 ** -24 * (2 * 448.0 ** 2 + 126 * small)
                ref.assert_within("y", y, np.full((M, 20), 126 * small), bound + (2.0 ** -8 * (126 * small + bound) if dt == torch.bfloat16 else 0))


@pytest.mark.parametrize("M", [5, 70])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("a_size,b_size", [(-70, -50), (-110, 4), (100, -90), (60, 40), (-90, 100)])
def test_scales_far_from_one(a_size, b_size, out, M):
    """Scales whose products are normal numbers, and a block of zeros, whose scale is zero."""
    import torch
    from mlstm_matrix_memory_amd import mlstm_mm_e4m3
    announce(f"mm with scales of 2^{a_size} and 2^{b_size} M={M} {out}")
    qa, sa, qb, sb = operands(M, 140, 300, 128)
    qa[:, 128:256], sa[:, 1] = 0, 0
    sa, sb = sa * np.float32(2.0) ** a_size, sb * np.float32(2.0) ** b_size
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    y = mlstm_mm_e4m3(e4m3_gpu(qa), to_gpu(sa, "f32"), e4m3_gpu(qb), to_gpu(sb, "f32"), out_dtype=dt)
    torch.cuda.synchronize()
    r, bound = expected(qa, sa, qb, sb, 128, out)
    ref.assert_within("y", to_np(y), r, bound)


def expected_of_cut_terms(qa, sa, qb, sb, block_rows):
    """(y, bound) of bf16 results of more than 64 rows: cut terms as in test_terms_that_cancel, the largest of eight being at
    most the largest factors' product."""
    K = qa.shape[1]
    r, bound = expected(qa, sa, qb, sb, block_rows, "f32")
    most = lambda q, s, rows: np.maximum.reduceat(np.abs(q), np.arange(0, K, 8), 1) * np.repeat(  # noqa: E731
        np.repeat(s.astype(np.float64), rows, 0)[:len(q)], 16, 1)[:, :-(-K // 8)]
    bound = bound + 7 * 2.0 ** -13 * most(qa, sa, 1) @ most(qb, sb, block_rows).T
    return r, bound + 2.0 ** -8 * (np.abs(r) + bound)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("M,N,K", [(4100, 4090, 528), (4096, 4100, 640), (2048, 2100, 656)])
def test_product_of_several_blocks_in_large_tiles(M, N, K, block_rows):
    """256 x 256 and 128 x 128 tiles over five and six blocks, the last whole or shorter: both LDS buffers filled again
    and again beside the products, with other scales in every block."""
    import torch
    from mlstm_matrix_memory_amd import mlstm_mm_e4m3
    announce(f"mm of several blocks M={M} N={N} K={K} blocks of {block_rows}")
    qa, sa, qb, sb = operands(M, N, K, block_rows)
    rng = np.random.default_rng(7)
    sa, sb = ((s * np.exp2(rng.integers(-4, 5, s.shape))).astype(np.float32) for s in (sa, sb))
    y = mlstm_mm_e4m3(e4m3_gpu(qa), to_gpu(sa, "f32"), e4m3_gpu(qb), to_gpu(sb, "f32"), block_rows=block_rows)
    torch.cuda.synchronize()
    ref.assert_within("y", to_np(y), *expected_of_cut_terms(qa, sa, qb, sb, block_rows))
