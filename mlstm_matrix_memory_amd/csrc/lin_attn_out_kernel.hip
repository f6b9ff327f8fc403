// Linear attention: outputs of a chunk from its entering state and its own rows; the gradients of
// q, k and v are the same form with other tensors in the places of a, y and z, forwards or
// backwards in time (lin_attn_common.h).
//
//   out_i = state_factor e^{g n_i} (state a_i) + row_factor sum_j e^{g|i-j|} (a_i . y_j) z_j
//
// A workgroup of four waves has 64 rows i, a wave 16 of them for all of the kernel (32 a wave leave room for half
// as many workgroups: a sixth slower at (1, 32768, 8 heads of 256)).  First it forms their products with all rows j of
// the chunk, transposed (j across the instruction's rows), so that a lane's results are already the
// operand of the next product: decayed and masked, in bf16 cut into two parts, they stay in
// registers.  Then, 64 columns of out at a time, the state's products with a, their decay, and
// the products with z.  y, the state and z pass through LDS in slabs of 64 x 64, one ahead (two at a time, with the products
// in one part: 231 us against 236).
//
// Bound by the slabs' way from HBM and L2: 235 to 240 us there for 0.72 GB read and 0.13 written, 3.6 TB/s; the waves wait 68%
// of their time, the matrix instructions take 13%.
//
// Rows of z later (backwards: earlier) than row i must not reach it, even where they are NaN or
// infinite and their factor is zero.  Only slabs on the diagonal have such rows: there a
// column's first such value is noted, and rows from it on become NaN (also where the sum would be infinite:
// the value's factors are gone by then).
#include "lin_attn_common.h"

namespace mlstm {
namespace {

constexpr int SLAB = 64, STRIDE = SLAB + 8;      // (a row is 36 banks: the reads of a row's pieces and of columns meet all banks)
constexpr int BLOCKS = LA_CHUNK / SLAB;
constexpr int MT = 1;                            // tiles of 16 rows a wave has
constexpr int BM = 64 * MT, RT = LA_CHUNK / BM;  // rows of a workgroup, workgroups of a chunk

struct OutShape {
    const void* a; long long a_stride; int da, a_per;
    const void* y; long long y_stride; int y_per;
    const void* z; long long z_stride; int dz, z_per;
    const void* kept; const float* log_decay;
    void* out; long long out_stride;
    int H, init;
    float state_factor, row_factor;
    Pieces chunk;
};

__device__ __forceinline__ void set_frag(Frag<bf16>& f, const Raw8<bf16>& r) { f.v = r.v; }
__device__ __forceinline__ void set_frag(Frag<float>& f, const Raw8<float>& r) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f.v[e] = r.get(e);
}

// the first or the second four of r
__device__ __forceinline__ void lds_put4(bf16* p, const Raw8<bf16>& r, int half) {
    *reinterpret_cast<bf16x4*>(p) = half ? __builtin_shufflevector(r.v, r.v, 4, 5, 6, 7) : __builtin_shufflevector(r.v, r.v, 0, 1, 2, 3);
}
__device__ __forceinline__ void lds_put4(float* p, const Raw8<float>& r, int half) { *reinterpret_cast<f32x4*>(p) = half ? r.b : r.a; }

// bit of the elements of r that are NaN or infinite
typedef unsigned short u16x8 __attribute__((ext_vector_type(8)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ unsigned strange(const Raw8<bf16>& r) {
    const u32x4 pairs = __builtin_bit_cast(u32x4, r.v) & 0x7f807f80u;
    unsigned any = 0;                            // an exponent of all ones carries into the bit above it
#pragma unroll
    for (int e = 0; e < 4; ++e) any |= (pairs[e] + 0x00800080u) & 0x80008000u;
    if (any == 0) return 0;
    const u16x8 bits = __builtin_bit_cast(u16x8, r.v);
    unsigned m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const unsigned short x = bits[e];
        if ((x & 0x7f80) == 0x7f80) m |= 1u << e;
    }
    return m;
}
__device__ __forceinline__ unsigned strange(const Raw8<float>& r) {
    unsigned m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float x = r.get(e);
        if ((__builtin_bit_cast(unsigned, x) & 0x7f800000u) == 0x7f800000u) m |= 1u << e;
    }
    return m;
}
__device__ __forceinline__ void clear(Raw8<bf16>& r, int e) { r.v[e] = (bf16)0.0f; }
__device__ __forceinline__ void clear(Raw8<float>& r, int e) { r.set(e, 0.0f); }

// HELD: 64-column slabs of a that stay in registers (0: read again where they are needed)
// COLS: the state's rows are a's columns; otherwise its rows are out's columns
template <typename T, typename OT, int HELD, bool BACK, bool COLS, bool WIDE>
__global__ __launch_bounds__(256, sizeof(T) == 4 || HELD > 4 ? 2 : HELD == 1 ? 4 : 3) void out_kernel(OutShape s, int groups)
{
    __shared__ __align__(16) T slab[2][SLAB * STRIDE];
    __shared__ int bad[3][SLAB];
    const int id = die_run(blockIdx.x, groups);
    const int rt = id % RT, h = id / RT % s.H, number = id / RT / s.H;
    if (number >= s.chunk.count()) return;
    const Pieces::At at = s.chunk.at(number);
    if (at.c == Pieces::NONE) return;
    const RowRange sq = s.chunk.sequence(at.b);
    if ((long long)at.c * LA_CHUNK + rt * BM >= sq.n) return;
    const int r0 = at.c * LA_CHUNK, n = min(LA_CHUNK, sq.n - r0);
    const int lane = threadIdx.x & 63, wave = wave_id(), lr = lane & 15, lg = lane >> 4;
    const int w0 = rt * BM + 16 * MT * wave;     // the wave's first row of the chunk
    const T* a = (const T*)s.a + (long long)(sq.lo + r0) * s.a_stride + (size_t)(h / s.a_per) * s.da;
    const T* y = (const T*)s.y + (long long)(sq.lo + r0) * s.y_stride + (size_t)(h / s.y_per) * s.da;
    const T* z = (const T*)s.z + (long long)(sq.lo + r0) * s.z_stride + (size_t)(h / s.z_per) * s.dz;
    OT* out = (OT*)s.out + (long long)(sq.lo + r0) * s.out_stride + (size_t)h * s.dz;
    const int ap = la_pad(s.da), zp = la_pad(s.dz), slabs = ap / SLAB;
    const T* state = (const T*)s.kept + ((size_t)(s.chunk.first(at.b, sq) + at.c) * s.H + h) * ap * zp;
    const bool entered = s.init || (BACK ? r0 + n < sq.n : at.c > 0);
    const int parts = zp / SLAB;
    // blocks of rows j that rows of this workgroup meet, and those where some pair is masked
    const int j0 = BACK ? rt * BM / SLAB : 0, j1 = BACK ? (n + SLAB - 1) / SLAB : min((rt + 1) * BM, n + SLAB - 1) / SLAB;
    const Decay decay(s.log_decay[h]);

    for (int i = threadIdx.x; i < 3 * SLAB; i += 256) bad[i / SLAB][i % SLAB] = BACK ? -1 : LA_CHUNK;

    // ---- slabs: thread t moves columns 8 (t % 8) .. + 7 of rows t / 8 and t / 8 + 32
    Raw8<T> moved[2];
    int left[2];                                 // elements of its row from there on
    const int tc = 8 * (threadIdx.x & 7), tr = threadIdx.x >> 3;
    auto fetch_rows = [&](const T* from, long long stride, int d, int block, int part) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = block * SLAB + tr + 32 * i;
            left[i] = r < n ? d - part * SLAB - tc : 0;
            moved[i] = load8<WIDE>(from + r * stride + part * SLAB + tc, left[i], from);
        }
    };
    // a block of the state: thread t moves 16 elements as they lie, columns 16 (t / 16 % 4) + 4 (t / 4 % 4) .. + 3 of
    // rows 16 (t / 64) + 4 (t % 4) .. + 3
    auto fetch_state = [&](int part, int k) {    // 64 columns of out, 64 of a
        const T* from = state + ((size_t)(COLS ? k : part) * ((COLS ? zp : ap) / SLAB) + (COLS ? part : k)) * (SLAB * SLAB) + 16 * threadIdx.x;
        moved[0].load(from);
        moved[1].load(from + 8);
    };
    const int sc = 16 * (threadIdx.x >> 4 & 3) + 4 * (threadIdx.x >> 2 & 3), sr = 16 * (threadIdx.x >> 6) + 4 * (threadIdx.x & 3);
    int turn = 0;
    auto put = [&](bool of_state, bool diagonal, int block) {
        if (!of_state) {
#pragma unroll
            for (int i = 0; i < 2; ++i) moved[i] = kept<WIDE>(moved[i], left[i]);
        }
        if (diagonal) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const unsigned m = strange(moved[i]);
                if (m) {
                    const int j = block * SLAB + tr + 32 * i;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (m >> e & 1) {
                            if (BACK) atomicMax(&bad[turn % 3][tc + e], j);
                            else atomicMin(&bad[turn % 3][tc + e], j);
                            clear(moved[i], e);
                        }
                }
            }
        }
        if (of_state) {
#pragma unroll
            for (int i = 0; i < 4; ++i) lds_put4(&slab[turn & 1][(sr + i) * STRIDE + sc], moved[i >> 1], i & 1);
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) lds_put(&slab[turn & 1][(tr + 32 * i) * STRIDE + tc], moved[i]);
        }
        __syncthreads();
        // the notes of the slab before are read: they serve the one after the next
        if (threadIdx.x < SLAB) bad[(turn + 2) % 3][threadIdx.x] = BACK ? -1 : LA_CHUNK;
    };
    __syncthreads();

    // ---- a's rows
    Frag<T> held[HELD ? MT : 1][HELD ? 2 * HELD : 1];
    auto a_frag = [&](int i, int k) {            // row 16 i + lr of the wave, columns 32 k + 8 lg ..
        Frag<T> f;
        const int r = w0 + 16 * i + lr;
        const int left = r < n ? s.da - 32 * k - 8 * lg : 0;
        set_frag(f, kept<WIDE>(load8<WIDE>(a + r * s.a_stride + 32 * k + 8 * lg, left, a), left));
        return f;
    };
    if (HELD) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int k = 0; k < 2 * HELD; ++k) held[HELD ? i : 0][HELD ? k : 0] = a_frag(i, k);
    }

    // ---- products with the rows of the chunk
    // powers inside a 16 x 16 tile: power[e] from column j = 4 lg + e of it to its edge next to the rows,
    // same[e] between row lr and column j of a tile on the diagonal, zero where j is masked
    float power[4], same[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int j = 4 * lg + e, d = BACK ? j - lr : lr - j;
        power[e] = decay(BACK ? j : 15 - j) * s.row_factor;
        same[e] = d >= 0 ? decay(max(d, 0)) * s.row_factor : 0.0f;
    }
    // rows j 32 k + {4 lg + e, 16 + 4 lg + e}, in bf16 as two parts: one rounding alone would be as large as the result's own
    constexpr int PARTS = sizeof(T) == 2 ? 2 : 1;
    Frag<T> p[PARTS][MT][2 * BLOCKS];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int k = 0; k < 2 * BLOCKS; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) p[0][i][k].v[e] = p[PARTS - 1][i][k].v[e] = (T)0.0f;
    // what follows a slab of y: the next of its block, the next block, or the first of the second part
    auto fetch_part = [&](int part) {
        if (entered) fetch_state(part, 0);
        else fetch_rows(z, s.z_stride, s.dz, j0, part);
    };
    fetch_rows(y, s.y_stride, s.da, j0, 0);
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b) {
        if (b < j0 || b >= j1) continue;
        f32x4 acc[MT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[i][t] = f32x4{0, 0, 0, 0};
        auto one = [&](int k) {
            Frag<T> mine[MT][2];
            if (!HELD) {
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c) mine[i][c] = a_frag(i, 2 * k + c);
            }
            put(false, false, 0);
            if (k + 1 < slabs) fetch_rows(y, s.y_stride, s.da, b, k + 1);
            else if (b + 1 < j1) fetch_rows(y, s.y_stride, s.da, b + 1, 0);
            else fetch_part(0);
            const T* from = slab[turn & 1];
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    Frag<T> fy;
                    frag_row(fy, &from[(16 * t + lr) * STRIDE + 32 * c + 8 * lg]);
#pragma unroll
                    for (int i = 0; i < MT; ++i) acc[i][t] = mma(fy, HELD ? held[HELD ? i : 0][HELD ? 2 * k + c : 0] : mine[i][c], acc[i][t]);
                }
            ++turn;
        };
        if (HELD) {
#pragma unroll
            for (int k = 0; k < (HELD ? HELD : 1); ++k)
                if (k < slabs) one(k);
        } else {
            for (int k = 0; k < slabs; ++k) one(k);
        }
        // decayed, masked
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int r = w0 + 16 * i, j = b * SLAB + 16 * t;
                const int d = BACK ? j - r - lr : r + lr - j - 15;   // from the tile's edge
                const float f = decay(max(d, 0));
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float w = r == j ? same[e] : f * power[e];
                    const bool in = BACK ? j >= r : j <= r;
                    const float v = r == j && (BACK ? 4 * lg + e < lr : 4 * lg + e > lr) ? 0.0f : acc[i][t][e] * w;
                    const float x = in ? v : 0.0f;
                    const T hi = (T)x;
                    p[0][i][2 * b + t / 2].v[4 * (t & 1) + e] = hi;
                    if (PARTS == 2) p[PARTS - 1][i][2 * b + t / 2].v[4 * (t & 1) + e] = (T)(x - (float)hi);
                }
            }
    }

    // ---- 64 columns of out at a time
    float carry[MT];                             // of the state to the wave's rows
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int r = w0 + 16 * i + lr;
        carry[i] = s.state_factor * decay(max(BACK ? n - 1 - r : r + 1, 0));
    }
    for (int q = 0; q < parts; ++q) {
        f32x4 acc[MT][4];                        // columns 64 q + 16 t + 4 lg + e of row w0 + 16 i + lr
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[i][t] = f32x4{0, 0, 0, 0};
        if (entered) {
            auto one = [&](int k) {
                Frag<T> mine[MT][2];
                if (!HELD) {
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int c = 0; c < 2; ++c) mine[i][c] = a_frag(i, 2 * k + c);
                }
                put(true, false, 0);
                if (k + 1 < slabs) fetch_state(q, k + 1);
                else fetch_rows(z, s.z_stride, s.dz, j0, q);
                const T* from = slab[turn & 1];
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        Frag<T> fs;
                        if (COLS) frag_col(fs, &from[16 * t], STRIDE, 32 * c + 8 * lg, 32 * c + 8 * lg + 4);
                        else frag_row(fs, &from[(16 * t + lr) * STRIDE + 32 * c + 8 * lg]);
#pragma unroll
                        for (int i = 0; i < MT; ++i) acc[i][t] = mma(fs, HELD ? held[HELD ? i : 0][HELD ? 2 * k + c : 0] : mine[i][c], acc[i][t]);
                    }
                ++turn;
            };
            if (HELD) {
#pragma unroll
                for (int k = 0; k < (HELD ? HELD : 1); ++k)
                    if (k < slabs) one(k);
            } else {
                for (int k = 0; k < slabs; ++k) one(k);
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][t][e] *= carry[i];
        }
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
            if (b < j0 || b >= j1) continue;
            // some row of the workgroup is before (backwards: behind) some row j of the block
            const bool diagonal = BACK ? b * SLAB < (rt + 1) * BM : (b + 1) * SLAB > rt * BM;
            put(false, diagonal, b);
            if (b + 1 < j1) fetch_rows(z, s.z_stride, s.dz, b + 1, q);
            else if (q + 1 < parts) fetch_part(q + 1);
            const T* from = slab[turn & 1];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                // rows j that are behind all of the wave's (backwards: before them) have no part
                const int j = b * SLAB + 32 * c;
                if (BACK ? j + 32 <= w0 : j >= w0 + 16 * MT) continue;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    Frag<T> fz;
                    frag_col(fz, &from[16 * t], STRIDE, 32 * c + 4 * lg, 32 * c + 16 + 4 * lg);
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int part = PARTS - 1; part >= 0; --part) acc[i][t] = mma(fz, p[part][i][2 * b + c], acc[i][t]);
                }
            }
            if (diagonal) {
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = bad[turn % 3][16 * t + 4 * lg + e];
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            const int r = w0 + 16 * i + lr;
                            if (BACK ? r <= j : r >= j) acc[i][t][e] = __builtin_nanf("");
                        }
                    }
            }
            ++turn;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int r = w0 + 16 * i + lr;
            if (r >= n) continue;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int c = q * SLAB + 16 * t + 4 * lg;
                Raw4<OT> o;
#pragma unroll
                for (int e = 0; e < 4; ++e) o.set(e, acc[i][t][e]);
                store_row4(out + r * s.out_stride + c, o, s.dz - c);
            }
        }
    }
}

template <typename T, typename OT, int HELD, bool BACK, bool COLS, bool WIDE>
hipError_t launch(const LaBatch& b, const OutShape& s) {
    const long long groups = ((long long)s.chunk.count() * s.H * RT + 7) / 8 * 8;
    if (!launchable(groups, 256)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((out_kernel<T, OT, HELD, BACK, COLS, WIDE>), dim3((unsigned)groups), dim3(256), 0, b.stream, s, (int)groups);
    return hipGetLastError();
}

template <typename T, typename OT, bool BACK, bool COLS>
hipError_t pick_held(const LaBatch& b, const OutShape& s) {
    // up to 6 of a's slabs are held: (4, 2048, 4 heads of 384) 82 us with 6 read again and again, 50 held.  Wider heads
    // read theirs for every slab (6 take 174 to 184 of 256 registers; more were not built)
    if (s.da % 8 || s.dz % 8) return launch<T, OT, 0, BACK, COLS, false>(b, s);
    if (s.da <= 64) return launch<T, OT, 1, BACK, COLS, true>(b, s);
    if (s.da <= 128) return launch<T, OT, 2, BACK, COLS, true>(b, s);
    if (s.da <= 256 && sizeof(T) == 2) return launch<T, OT, sizeof(T) == 2 ? 4 : 0, BACK, COLS, true>(b, s);
    if (s.da <= 384 && sizeof(T) == 2) return launch<T, OT, sizeof(T) == 2 ? 6 : 0, BACK, COLS, true>(b, s);
    return launch<T, OT, 0, BACK, COLS, true>(b, s);
}

template <typename T, typename OT>
hipError_t pick(const LaBatch& b, const OutShape& s, bool back, bool cols) {
    if (back) return cols ? pick_held<T, OT, true, true>(b, s) : pick_held<T, OT, true, false>(b, s);
    return cols ? pick_held<T, OT, false, true>(b, s) : pick_held<T, OT, false, false>(b, s);
}

// ---- heads that share q and k: their gradients summed --------------------------------
template <typename T>
__global__ __launch_bounds__(256) void sum_heads_kernel(const float* __restrict__ parts, int H, int G, int d, Pieces rows,
                                                        T* __restrict__ out, long long out_stride)
{
    // a wave per row: lanes over the row's G d elements
    const int row = blockIdx.x * 4 + wave_id(), lane = threadIdx.x & 63, per = H / G;
    if (row >= rows.rows || !rows.has(row)) return;
    const float* from = parts + (size_t)row * H * d;
    for (int i = lane; i < G * d; i += 64) {
        const int g = i / d, c = i - g * d;
        float sum = 0.0f;
        for (int k = 0; k < per; ++k) sum += from[(size_t)(g * per + k) * d + c];
        out[row * out_stride + i] = from_f32<T>(sum);
    }
}

}  // namespace

hipError_t launch_la_out(const LaBatch& b, const LaOut& o) {
    OutShape s = {};
    s.a = o.a.p; s.a_stride = o.a.stride; s.da = o.a.d; s.a_per = o.a.per;
    s.y = o.y.p; s.y_stride = o.y.stride; s.y_per = o.y.per;
    s.z = o.z.p; s.z_stride = o.z.stride; s.dz = o.z.d; s.z_per = o.z.per;
    s.kept = o.kept; s.log_decay = b.log_decay; s.out = o.out; s.out_stride = o.out_stride;
    s.H = b.H; s.init = o.init; s.state_factor = o.state_factor; s.row_factor = o.row_factor;
    s.chunk = make_pieces(b.seq_start, b.B, b.S, b.rows, LA_CHUNK);
    if (b.dtype == MLSTM_F32) return pick<float, float>(b, s, o.backwards, o.by_columns);
    // (only the gradients of q and k, which read states by columns, are ever wanted in fp32)
    if (o.out_f32) return o.backwards ? pick_held<bf16, float, true, true>(b, s) : pick_held<bf16, float, false, true>(b, s);
    return pick<bf16, bf16>(b, s, o.backwards, o.by_columns);
}

bool la_out_launchable(const LaBatch& b) {
    return launchable(((long long)la_chunks(b) * b.H * RT + 7) / 8 * 8, 256);
}
bool la_sum_heads_launchable(const LaBatch& b) { return launchable(((long long)b.rows + 3) / 4, 256); }

hipError_t launch_la_sum_heads(const LaBatch& b, const float* parts, int G, int d, void* out, long long out_stride) {
    const long long groups = ((long long)b.rows + 3) / 4;
    const Pieces rows = make_pieces(b.seq_start, b.B, b.S, b.rows, LA_CHUNK);
    if (b.dtype == MLSTM_BF16)
        hipLaunchKernelGGL(sum_heads_kernel<bf16>, dim3((unsigned)groups), dim3(256), 0, b.stream, parts, b.H, G, d, rows, (bf16*)out, out_stride);
    else
        hipLaunchKernelGGL(sum_heads_kernel<float>, dim3((unsigned)groups), dim3(256), 0, b.stream, parts, b.H, G, d, rows, (float*)out, out_stride);
    return hipGetLastError();
}

}  // namespace mlstm
