// e4m3 values with a scale for each block of 128: the quantiser and the matrix product.
//
// Quantiser, of x or of its transpose, for blocks of 1 x 128 or 128 x 128:
//   scale = max |x| / 448 over the block,  q = round(x / scale)
// One pass: a workgroup holds 128 x 128 elements of x in registers, 8 x 8 a thread, so both
// kinds of block and both directions are whole in it; the transpose turns in LDS as bytes.
// Bound by HBM: 16384 x 1536 bf16 transposed in 18.2 us, 4.2 TB/s.
//
// Product of a [M,K] and b [N,K], K in blocks of 128:
//   y[m][n] = sum over blocks j of a_scale[m][j] b_scale[n or n/128][j] (a[m] . b[n] over block j)
// A block's inner products run on the matrix cores (16 x 16 x 128 e4m3, fp32 sums), and its scales
// enter as one multiply-add per element and block, from registers: an instruction of 32 cycles is
// followed by 4 multiply-adds of 4 cycles, which the other wave of the SIMD's matrix
// instructions cover in part: 8192 x 8192 x 2048 takes 183 us (1.5 PFLOP/s; traced 185, without the multiply-adds
// 143, without the loads 163).  b is the instruction's row operand, so that a lane holds four neighbouring
// columns of one row of y: one scale of a for them, and stores of four elements.
#include "block_internal.h"
#include "e4m3_common.h"

namespace mlstm {
namespace {

typedef int int2_u __attribute__((ext_vector_type(2), aligned(1)));
typedef int int2v __attribute__((ext_vector_type(2)));
typedef int int4v __attribute__((ext_vector_type(4)));
typedef int int4_u __attribute__((ext_vector_type(4), aligned(1)));
typedef int int8v __attribute__((ext_vector_type(8)));

__device__ __forceinline__ int pack4(float a, float b, float c, float d) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return __builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true);
}

// the first n (<= 8) of eight bytes to p
__device__ __forceinline__ void store_bytes8(unsigned char* p, int lo, int hi, int n) {
    if (n >= 8) {
        *reinterpret_cast<int2_u*>(p) = int2_u{lo, hi};
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < n) p[e] = (unsigned char)((e < 4 ? lo : hi) >> (8 * (e & 3)));
    }
}

// ---- quantiser ------------------------------------------------------------------
constexpr int QT = 128;                          // tile edge
constexpr int TURN_STRIDE = QT + 8;              // bytes between columns of the turned tile

// Thread t holds rows 8 (t / 16) + i, columns 8 (t % 16) + e of the tile, i, e < 8.
template <typename T, bool BLOCK, bool TURN>
__global__ __launch_bounds__(256) void quant_kernel(const T* __restrict__ x, long long x_stride, int rows, int cols,
                                                    unsigned char* __restrict__ q, float* __restrict__ scale)
{
    __shared__ float red[4][QT];
    __shared__ __align__(16) unsigned char turned[TURN ? QT * TURN_STRIDE : 16];
    const int tc = threadIdx.x & 15, tr = threadIdx.x >> 4, wave = wave_id(), lane = threadIdx.x & 63;
    const int row_tiles = (rows + QT - 1) / QT, col_tiles = (cols + QT - 1) / QT;
    const int c0 = (int)(blockIdx.x % col_tiles) * QT, r0 = (int)(blockIdx.x / col_tiles) * QT;
    const int col = c0 + 8 * tc, row = r0 + 8 * tr, n = cols - col;
    Raw8<T> v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = load_row8(x + (long long)(row + i < rows ? row + i : 0) * x_stride + col, row + i < rows ? n : 0);
    float m[8];                                  // of rows (as it is) or of columns (turned)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        m[j] = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m[j] = fmaxf(m[j], fabsf(TURN ? v[e].get(j) : v[j].get(e)));
    }
    if (BLOCK) {
#pragma unroll
        for (int j = 1; j < 8; ++j) m[0] = fmaxf(m[0], m[j]);
        m[0] = wave_max(m[0]);
        if (lane == 0) red[wave][0] = m[0];
        __syncthreads();
        m[0] = fmaxf(fmaxf(red[0][0], red[1][0]), fmaxf(red[2][0], red[3][0]));
        if (threadIdx.x == 0) {
            const size_t at = TURN ? (size_t)(c0 / QT) * row_tiles + r0 / QT : (size_t)(r0 / QT) * col_tiles + c0 / QT;
            scale[at] = m[0] / E4M3_MAX;
        }
    } else if (!TURN) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
            for (int off = 1; off < 16; off <<= 1) m[j] = fmaxf(m[j], __shfl_xor(m[j], off, 64));
            if (tc == 0 && row + j < rows) scale[(size_t)(row + j) * col_tiles + c0 / QT] = m[j] / E4M3_MAX;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            m[j] = fmaxf(m[j], __shfl_xor(m[j], 16, 64));
            m[j] = fmaxf(m[j], __shfl_xor(m[j], 32, 64));
            if (lane < 16) red[wave][8 * tc + j] = m[j];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = 8 * tc + j;
            m[j] = fmaxf(fmaxf(red[0][c], red[1][c]), fmaxf(red[2][c], red[3][c]));
            if (tr == 0 && c0 + c < cols) scale[(size_t)(c0 + c) * row_tiles + r0 / QT] = m[j] / E4M3_MAX;
        }
    }
    const Quotient whole(m[0]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const Quotient quotient = BLOCK ? whole : Quotient(m[j]);
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = quotient(TURN ? v[e].get(j) : v[j].get(e));
        const int lo = pack4(y[0], y[1], y[2], y[3]), hi = pack4(y[4], y[5], y[6], y[7]);
        if (!TURN) {
            if (row + j < rows) store_bytes8(q + (size_t)(row + j) * cols + col, lo, hi, n);
        } else {
            *reinterpret_cast<int2v*>(&turned[(8 * tc + j) * TURN_STRIDE + 8 * tr]) = int2v{lo, hi};
        }
    }
    if (TURN) {
        __syncthreads();
        // 16 lanes write the 128 bytes of one column of x
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = 16 * i + tr;
            const int2v b = *reinterpret_cast<const int2v*>(&turned[c * TURN_STRIDE + 8 * tc]);
            if (c0 + c < cols) store_bytes8(q + (size_t)(c0 + c) * rows + r0 + 8 * tc, b[0], b[1], rows - r0 - 8 * tc);
        }
    }
}

template <typename T>
void launch_quant_t(const QuantArgs& a, unsigned groups) {
#define QUANT(BLOCK, TURN)                                                                                       \
    hipLaunchKernelGGL((quant_kernel<T, BLOCK, TURN>), dim3(groups), dim3(256), 0, a.stream, (const T*)a.x,      \
                       a.x_stride, a.rows, a.cols, (unsigned char*)a.q, a.scale)
    if (a.block_rows == 1) {
        if (a.transpose) QUANT(false, true);
        else QUANT(false, false);
    } else {
        if (a.transpose) QUANT(true, true);
        else QUANT(true, false);
    }
#undef QUANT
}

// ---- product: tiles through LDS -----------------------------------------------------
constexpr int KB = 128;                          // bytes of a row in one block

// Eight e4m3 bytes as bf16 (exact).
__device__ __forceinline__ bf16x8 widen(int lo, int hi) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Inner products of a block.  The e4m3 instructions do not sum in fp32: 2.1e-5 of the result is lost over 40 blocks
// of random values, by 16 x 16 x 128 and by 16 x 16 x 32 alike.  Of eight neighbouring terms, k = 8 i .. 8 i + 7,
// the first cuts each towards zero to a multiple of 2^-13 of the largest one's power of two (that of its
// factors), and adds the eights in fp32: up to 7 / 8192 of the largest term of each eight.  A factor's own rounding
// to e4m3 is 2^-4 of the same term, and a bf16 result (rounding 1.7e-3) shows it only where large terms cancel.
// Fragment<bf16> feeds that instruction, for bf16 results of more than 64 rows: there fp32 sums cost up to
// 1.7 times the time (8192 x 8192 x 2048: 174 us against 301).  Fragment<float> widens the operands to
// bf16, whose instruction keeps fp32's bits at half the rate: for fp32 results, and for up to 64 rows, where the time is
// mostly that of b's bytes (16 x 8192 x 8192 22.8 us either way, 64 x 8192 x 2048 17.2 against 16.7).
template <typename T> struct Fragment;
template <> struct Fragment<bf16> {
    int8v v;
    __device__ __forceinline__ void set(int4v lo, int4v hi) { v = int8v{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]}; }
};
template <> struct Fragment<float> {
    bf16x8 v[4];
    __device__ __forceinline__ void set(int4v lo, int4v hi) {
        v[0] = widen(lo[0], lo[1]);
        v[1] = widen(lo[2], lo[3]);
        v[2] = widen(hi[0], hi[1]);
        v[3] = widen(hi[2], hi[3]);
    }
};
__device__ __forceinline__ f32x4 mfma_e4m3(const Fragment<bf16>& a, const Fragment<bf16>& b) {
    // (no scales of the instruction's own)
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_e4m3(const Fragment<float>& a, const Fragment<float>& b) {
    f32x4 c = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) c = mfma(a.v[i], b.v[i], c);
    return c;
}

// 16 bytes of a row from column k on, zero past K
__device__ __forceinline__ int4v row_bytes(const unsigned char* row, int k, int K) {
    if (k + 16 <= K) return *reinterpret_cast<const int4_u*>(row + k);
    int4v v = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 15; ++e)
        if (k + e < K) v[e >> 2] |= (int)row[k + e] << (8 * (e & 3));
    return v;
}

struct MmShape {
    const unsigned char* a; const float* as; const unsigned char* b; const float* bs;
    int M, N, K, block_rows;
};

// Rows of the tile lie in LDS as 128 bytes, their 16-byte pieces in another order: piece c of row r
// at place c ^ (r / 2 % 8), so that the 16 rows a fragment's read meets lie in different banks.
__device__ __forceinline__ int place(int r, int c) { return r * KB + ((c ^ (r >> 1)) & 7) * 16; }

// 16 bytes per lane from base + offset to LDS at `to` + 16 lane, with no register between.  The
// compiler does not count this load: arrived() waits for it.
__device__ __forceinline__ void load_to_lds(const void* base, unsigned offset, const void* to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :: "s"((unsigned)(uintptr_t)(__attribute__((address_space(3))) const void*)to), "v"(offset), "s"(base)
                 : "memory");
}
__device__ __forceinline__ void arrived() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// WN x WM waves, each NT x MT tiles of 16 x 16 (b's rows x a's rows).  ALIGNED: rows of a and b
// start at multiples of 16 bytes and are at most MM_ALIGNED_MAX_K long; whole blocks then go from
// HBM to LDS without registers between.
constexpr int MM_ALIGNED_MAX_K = 1 << 22;        // 256 rows' offsets stay within 32 bits
template <typename T, int WN, int WM, int NT, int MT, bool BLOCK, bool ALIGNED>
__global__ __launch_bounds__(64 * WN * WM, 2) void mm_tile_kernel(MmShape s, T* __restrict__ y, long long y_stride)
{
    constexpr int THREADS = 64 * WN * WM, BN = 16 * NT * WN, BM = 16 * MT * WM, ROWS = BN + BM, STEP = THREADS / 8;
    constexpr int PIECES = ROWS / STEP;          // 16-byte pieces a thread moves per block
    static_assert(BN % STEP == 0 && BM % STEP == 0, "whole pieces");
    __shared__ __align__(16) unsigned char tile[2][ROWS * KB];
    __shared__ __align__(16) float scales[2][ROWS];
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int wn = wave % WN, wm = wave / WN;
    // neighbouring workgroups go to different dies: each die takes a run of tiles, in bands of 8 tile rows of y, so
    // that the 32 tiles it runs at once are about 8 x 4 and share rows of a and b in its L2 (down columns of y 208 us,
    // so 186 then)
    const int m_tiles = (s.M + BM - 1) / BM, n_tiles = (s.N + BN - 1) / BN, tiles = m_tiles * n_tiles;
    const int per = (tiles + 7) / 8, id = (int)(blockIdx.x % 8) * per + blockIdx.x / 8;
    if (id >= tiles) return;
    const int band = id / (8 * n_tiles), in = id % (8 * n_tiles), high = min(8, m_tiles - 8 * band);
    const int n0 = in / high * BN, m0 = (8 * band + in % high) * BM;
    const int blocks = (s.K + KB - 1) / KB;

    // Thread t moves piece t % 8 (as it lies in LDS) of the tile's rows t / 8 + STEP i: b's for rows
    // below BN, then a's; rows past the end repeat the last.  Its piece of a row is the same in every
    // one of them, as STEP is a multiple of 16.
    static_assert(STEP % 16 == 0, "one piece for all rows of a thread");
    const int row = threadIdx.x / 8, piece = 16 * ((threadIdx.x ^ (row >> 1)) & 7);
    const unsigned char* from_b = s.b + (size_t)n0 * s.K;
    const unsigned char* from_a = s.a + (size_t)m0 * s.K;
    unsigned offset[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int r = row + STEP * i;
        offset[i] = (unsigned)((r < BN ? min(r, s.N - 1 - n0) : min(r - BN, s.M - 1 - m0)) * s.K + piece);
    }
    // a scale per thread (with fewer rows than threads some are moved twice)
    static_assert(THREADS % ROWS == 0, "a scale per thread");
    const int scale_row = threadIdx.x % ROWS;
    const float* scale_at = scale_row < BN ? s.bs + (size_t)(min(n0 + scale_row, s.N - 1) / s.block_rows) * blocks
                                           : s.as + (size_t)min(m0 + scale_row - BN, s.M - 1) * blocks;
    int4v held[ALIGNED ? 1 : PIECES];
    float held_scale = 0.0f;
    auto begin = [&](int kb, int buf) {
        if (!ALIGNED) {
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                const int r = row + STEP * i;
                const unsigned char* p = r < BN ? s.b + (size_t)min(n0 + r, s.N - 1) * s.K
                                                : s.a + (size_t)min(m0 + r - BN, s.M - 1) * s.K;
                held[i] = row_bytes(p, kb * KB + piece, s.K);
            }
        } else if ((kb + 1) * KB <= s.K) {
            // a wave's 64 pieces lie one after the other
#pragma unroll
            for (int i = 0; i < PIECES; ++i)
                load_to_lds((STEP * i < BN ? from_b : from_a) + (size_t)kb * KB, offset[i],
                            &tile[buf][(THREADS * i + 64 * wave) * 16]);
        } else {
            // the last, shorter block: K is a multiple of 16, so a piece is whole or past the end
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                int4v v = {0, 0, 0, 0};
                if (kb * KB + piece < s.K)
                    v = *reinterpret_cast<const int4v*>((STEP * i < BN ? from_b : from_a) + (size_t)kb * KB + offset[i]);
                *reinterpret_cast<int4v*>(&tile[buf][(THREADS * i + threadIdx.x) * 16]) = v;
            }
        }
        held_scale = scale_at[kb];
    };
    auto end = [&](int buf) {
        if (!ALIGNED) {
#pragma unroll
            for (int i = 0; i < PIECES; ++i) *reinterpret_cast<int4v*>(&tile[buf][(THREADS * i + threadIdx.x) * 16]) = held[i];
        }
        scales[buf][scale_row] = held_scale;
    };

    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    begin(0, 0);
    end(0);
    const int lr = lane & 15, lg = lane >> 4;
    for (int kb = 0; kb < blocks; ++kb) {
        const int buf = kb & 1;
        if (ALIGNED) arrived();
        __syncthreads();                         // this block is there, the one before it is read
        if (kb + 1 < blocks) begin(kb + 1, buf ^ 1);
        auto fragment = [&](int r) {
            const int4v lo = *reinterpret_cast<const int4v*>(&tile[buf][place(r, 2 * lg)]);
            const int4v hi = *reinterpret_cast<const int4v*>(&tile[buf][place(r, 2 * lg + 1)]);
            Fragment<T> f;
            f.set(lo, hi);
            return f;
        };
        Fragment<T> fb[NT];
        f32x4 sb[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int r = 16 * (NT * wn + j);
            fb[j] = fragment(r + lr);
            if (BLOCK) sb[j][0] = scales[buf][r];
            else sb[j] = *reinterpret_cast<const f32x4*>(&scales[buf][r + 4 * lg]);
        }
        // a row of tiles' matrix instructions beside the multiply-adds of the row before; the order is
        // fixed, as the compiler's own kept every tile's products at once and spilled them.  256 x 256 still has 18
        // registers too few: 76 bytes a lane go to scratch before the loop (40 of the 172 MB that 8192 x 8192 x 2048
        // writes), addresses that only a last, shorter block reads again, and two values of the end.
        f32x4 p[2][NT];
        float sa[2];
        Fragment<T> fa = fragment(BN + 16 * MT * wm + lr);
#pragma unroll
        for (int i = 0; i <= MT; ++i) {
            if (i < MT) {
                const int r = BN + 16 * (MT * wm + i) + lr;
                sa[i & 1] = scales[buf][r];
#pragma unroll
                for (int j = 0; j < NT; ++j) p[i & 1][j] = mfma_e4m3(fb[j], fa);
                if (i + 1 < MT) fa = fragment(r + 16);
            }
            if (i > 0) {
                const int h = (i - 1) & 1;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[i - 1][j][e] = fmaf(p[h][j][e], BLOCK ? sa[h] * sb[j][0] : sa[h] * sb[j][e], acc[i - 1][j][e]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        // (after the last block too, where nothing reads it: a branch here would let the compiler move
        // the multiply-adds behind it)
        end(buf ^ 1);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int m = m0 + 16 * (MT * wm + i) + lr;
        if (m >= s.M) continue;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int n = n0 + 16 * (NT * wn + j) + 4 * lg;
            Raw4<T> out;
#pragma unroll
            for (int e = 0; e < 4; ++e) out.set(e, acc[i][j][e]);
            store_row4(y + (long long)m * y_stride + n, out, s.N - n);
        }
    }
}

// ---- product: few rows of a ----------------------------------------------------------
// (4 x 2048 x 4096: 6.4 us traced, 9.1 with the host's call.)
// A workgroup takes 16 rows of b and all of a (16 MT rows); its waves take every WAVES-th block and
// load fragments as they are, with no LDS between: the time is that of b's bytes and of one
// trip to HBM.  Their sums are added in wave order.
template <typename T, int MT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void mm_row_kernel(MmShape s, T* __restrict__ y, long long y_stride)
{
    __shared__ f32x4 part[WAVES][MT][64];
    const int lane = threadIdx.x & 63, wave = wave_id(), lr = lane & 15, lg = lane >> 4;
    const int n0 = blockIdx.x * 16, blocks = (s.K + KB - 1) / KB;
    const unsigned char* b = s.b + (size_t)min(n0 + lr, s.N - 1) * s.K;
    const unsigned char* a[MT];
    const float* as[MT];
    const float* bs[4];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int m = min(16 * i + lr, s.M - 1);
        a[i] = s.a + (size_t)m * s.K;
        as[i] = s.as + (size_t)m * blocks;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) bs[e] = s.bs + (size_t)(min(n0 + 4 * lg + e, s.N - 1) / s.block_rows) * blocks;
    f32x4 acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = f32x4{0, 0, 0, 0};
    auto bytes32 = [&](const unsigned char* row, int kb) {
        const int k = kb * KB + 32 * lg;
        const int4v lo = row_bytes(row, k, s.K), hi = row_bytes(row, k + 16, s.K);
        return int8v{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    };
    auto whole = [](int8v v) {
        Fragment<float> f;
        f.set(int4v{v[0], v[1], v[2], v[3]}, int4v{v[4], v[5], v[6], v[7]});
        return f;
    };
    constexpr int AHEAD = MT <= 2 ? 4 : 2;       // blocks whose loads are in flight together
    for (int k0 = wave; k0 < blocks; k0 += AHEAD * WAVES) {
        int8v fb[AHEAD], fa[AHEAD][MT];
        float sa[AHEAD][MT], sb[AHEAD][4];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            // blocks past the last are read as zero bytes, with the last one's scales
            const int kb = k0 + u * WAVES, ks = min(kb, blocks - 1);
            fb[u] = bytes32(b, kb);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                fa[u][i] = bytes32(a[i], kb);
                sa[u][i] = as[i][ks];
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) sb[u][e] = bs[e][ks];
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            if (k0 + u * WAVES >= blocks) break;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const f32x4 p = mfma_e4m3(whole(fb[u]), whole(fa[u][i]));
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][e] = fmaf(p[e], sa[u][i] * sb[u][e], acc[i][e]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    for (int i = wave; i < MT; i += WAVES) {
        f32x4 sum = part[0][i][lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] += part[w][i][lane][e];
        const int m = 16 * i + lr, n = n0 + 4 * lg;
        if (m < s.M) {
            Raw4<T> out;
#pragma unroll
            for (int e = 0; e < 4; ++e) out.set(e, sum[e]);
            store_row4(y + (long long)m * y_stride + n, out, s.N - n);
        }
    }
}

template <typename T, int WN, int WM, int NT, int MT, bool BLOCK, bool ALIGNED>
hipError_t tile_launch(const MmArgs& a, const MmShape& s) {
    const long long tiles = (long long)((a.M + 16 * MT * WM - 1) / (16 * MT * WM)) * ((a.N + 16 * NT * WN - 1) / (16 * NT * WN));
    const long long groups = (tiles + 7) / 8 * 8;
    if (!launchable(groups, 64 * WN * WM)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((mm_tile_kernel<T, WN, WM, NT, MT, BLOCK, ALIGNED>), dim3((unsigned)groups), dim3(64 * WN * WM), 0,
                       a.stream, s, (T*)a.y, a.y_stride);
    return hipGetLastError();
}

template <typename T, bool BLOCK>
hipError_t tile_pick(const MmArgs& a, const MmShape& s) {
    const bool aligned = a.K % 16 == 0 && a.K <= MM_ALIGNED_MAX_K && (((uintptr_t)a.a | (uintptr_t)a.b) & 15) == 0;
    const long long tiles128 = (long long)((a.M + 127) / 128) * ((a.N + 127) / 128);
    if (!aligned) {
        // 3000 x 3000 x 2051, 128 x 128 against 64 x 64: bf16 67 us and 73; fp32, whose loads in flight then spill 12 to 25
        // registers beside the widened operands, 116 and 77
        if constexpr (sizeof(T) == 2) {
            if (tiles128 >= 256) return tile_launch<T, 2, 2, 4, 4, BLOCK, false>(a, s);
        }
        return tile_launch<T, 2, 2, 2, 2, BLOCK, false>(a, s);
    }
    // 256 x 256 where that fills the chip (8192 x 8192 x 2048 164.5 us, with 128 x 128 182; 4096 x 4096 x 8192 140 and 173),
    // 64 x 64 where 128 x 128 does not (1536 x 1536 x 4096 29 us, with 128 x 128 34; 2048 x 2048 x 2048 19.8 and 19.0; fp32 at
    // 4096 x 4096 x 2048 88 and 75).  Not 256 x 256 for scales of single rows, four factors a lane and tile: they spill 42
    // registers (8192 x 8192 x 2048 330 us, with 128 x 128 201), nor for fp32 results, whose widened operands do not fit
    // beside the sums.
    if constexpr (sizeof(T) == 2 && BLOCK) {
        const long long tiles256 = (long long)((a.M + 255) / 256) * ((a.N + 255) / 256);
        if (tiles256 >= 256) return tile_launch<T, 4, 2, 4, 8, BLOCK, true>(a, s);
    }
    return tiles128 >= 256 ? tile_launch<T, 2, 2, 4, 4, BLOCK, true>(a, s) : tile_launch<T, 2, 2, 2, 2, BLOCK, true>(a, s);
}

template <typename T>
hipError_t mm_launch(const MmArgs& a) {
    const MmShape s = {(const unsigned char*)a.a, a.a_scale, (const unsigned char*)a.b, a.b_scale, a.M, a.N, a.K, a.block_rows};
    if (a.M <= 64) {
        const long long groups = (a.N + 15) / 16;
#define MM_ROW(MT, WAVES)                                                                                          \
    do {                                                                                                           \
        if (!launchable(groups, 64 * WAVES)) return hipErrorInvalidConfiguration;                                  \
        hipLaunchKernelGGL((mm_row_kernel<T, MT, WAVES>), dim3((unsigned)groups), dim3(64 * WAVES), 0, a.stream, s, \
                           (T*)a.y, a.y_stride);                                                                   \
        return hipGetLastError();                                                                                  \
    } while (0)
        if (a.M <= 16) MM_ROW(1, 8);
        if (a.M <= 32) MM_ROW(2, 8);
        MM_ROW(4, 8);
#undef MM_ROW
    }
    return a.block_rows == 1 ? tile_pick<T, false>(a, s) : tile_pick<T, true>(a, s);
}

}  // namespace

hipError_t launch_quant(const QuantArgs& a) {
    const long long groups = (long long)((a.rows + QT - 1) / QT) * ((a.cols + QT - 1) / QT);
    if (!launchable(groups, 256)) return hipErrorInvalidConfiguration;
    if (a.dtype == MLSTM_BF16) launch_quant_t<bf16>(a, (unsigned)groups);
    else launch_quant_t<float>(a, (unsigned)groups);
    return hipGetLastError();
}

hipError_t launch_mm(const MmArgs& a) {
    return a.out_dtype == MLSTM_BF16 ? mm_launch<bf16>(a) : mm_launch<float>(a);
}

}  // namespace mlstm
