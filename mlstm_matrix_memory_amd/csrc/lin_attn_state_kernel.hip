// Linear attention: the states that enter chunks, or the gradients that leave them.
//
// A workgroup carries a tile of a head's state along a sequence (or a segment of it) in registers,
// WK x WV waves with 16 M x 16 M each, and writes it, rounded to the call's dtype, at every
// chunk: the output kernel needs it as an operand of that type only.  Rows pass through LDS in blocks
// of 32, one block ahead and the loads three; the contraction runs over rows, so both operands are
// read as columns.
//
// The state is held and returned in fp32, and its sums keep fp32's accuracy on bf16 instructions:
// the weighted rows w y (fp32) are cut into three bf16 parts, 8 bits each, whose sum they are
// exactly, and x is exact.  One part alone is 1.7e-3 off, two 2.7e-6.  Where only rounded states
// leave the call two parts are taken.  (An infinite y is cut into an infinity and NaN, and an infinite x meets parts
// that are zero: in bf16 both leave NaN where the sum is infinite.)
//
// Few tiles over long sequences are cut into segments: a first pass sums every segment from zero, a small
// kernel runs along these sums and leaves in their places the states that enter the segments (and
// the last one's end), and the second pass carries each segment from its own.  Only the first
// pass then has to be exact.  (Second pass with three parts, its segments joined by the readers: 186 us at
// (1, 32768, 8 heads of 256), now 129.)
//
// Bound there by the 64 turns between two barriers, 2 us each: without the parts' arithmetic 112 us of 122 (an earlier first
// pass; now 133), without the matrix instructions 90, with every block read again 125.  At 128 x 256 the passes spill
// up to 16 registers.  Kept as rows of dk, the states' stores of 32
// bytes made HBM read the lines first: 323 us against 230.
#include <type_traits>

#include "lin_attn_common.h"

namespace mlstm {
namespace {

constexpr int SB = 32;                           // rows per block

// w r as the sum of N bf16 rows: the top halves of the fp32 products, then of what is left (3 parts: all
// of it; the last of 2 is rounded)
template <int N>
__device__ __forceinline__ void cut(const Raw8<bf16>& r, float w, Raw8<bf16> (&part)[N]) {
    typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
    u32x4 out[N];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float x0 = w * r.get(2 * e), x1 = w * r.get(2 * e + 1);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if (N == 2 && k == 1) {
                typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
                out[k][e] = __builtin_bit_cast(unsigned, bf16x2{(bf16)x0, (bf16)x1});
            } else {
                const unsigned b0 = __builtin_bit_cast(unsigned, x0), b1 = __builtin_bit_cast(unsigned, x1);
                out[k][e] = __builtin_amdgcn_perm(b1, b0, 0x07060302);
                if (k + 1 < N) {
                    x0 -= __builtin_bit_cast(float, b0 & 0xffff0000u);
                    x1 -= __builtin_bit_cast(float, b1 & 0xffff0000u);
                }
            }
        }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) part[k].v = __builtin_bit_cast(bf16x8, out[k]);
}
template <int N>
__device__ __forceinline__ void cut(const Raw8<float>& r, float w, Raw8<float> (&part)[N]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) part[0].set(e, w * r.get(e));
}

template <typename T, int N, int M, int WK, int WV>
struct StateLds {
    static constexpr int EK = 16 * M * WK, EV = 16 * M * WV;
    static constexpr int PAD = sizeof(T) == 2 ? 16 : 4;
    static constexpr int YS = EK + PAD, XS = EV + PAD;   // row strides
    __align__(16) T y[2][N][SB * YS];            // weighted, in parts
    __align__(16) T x[2][SB * XS];
    float power[LA_CHUNK + 1];                   // e^{g n}
};

struct StateShape {
    const void* x; long long x_stride; int dv, x_per;
    const void* y; long long y_stride; int dk, y_per;
    const float* log_decay; const float* init; float* final; void* kept; float* parts;
    int H; float factor;
    Pieces segment, chunk;
    bool cut;                                    // sequences are cut into segments
};

// N parts of the weighted rows; FIRST: the pass over segments from zero
template <typename T, int N, int M, int WK, int WV, bool BACK, bool FIRST, bool WIDE>
__global__ __launch_bounds__(64 * WK * WV, 2) void state_kernel(StateShape s, int groups)
{
    typedef StateLds<T, N, M, WK, WV> Lds;
    constexpr int EK = Lds::EK, EV = Lds::EV, YS = Lds::YS, XS = Lds::XS, THREADS = 64 * WK * WV;
    constexpr int YT = SB * EK / 8 / THREADS, XT = SB * EV / 8 / THREADS;   // 8-element pieces a thread moves per block
    static_assert(YT * 8 * THREADS == SB * EK && XT * 8 * THREADS == SB * EV, "whole pieces");
    __shared__ Lds lds;
    const int tiles_k = (s.dk + EK - 1) / EK, tiles = tiles_k * ((s.dv + EV - 1) / EV);
    const int id = die_run(blockIdx.x, groups);
    const int tile = id % tiles, h = id / tiles % s.H, number = id / tiles / s.H;
    if (number >= s.segment.count()) return;
    const Pieces::At at = s.segment.at(number);
    if (at.c == Pieces::NONE) return;
    const RowRange sq = s.segment.sequence(at.b);
    const int length = s.segment.length;
    if (at.c > 0 && (long long)at.c * length >= sq.n) return;
    const int r0 = at.c * length, n = min(length, sq.n - r0), last = max((sq.n + length - 1) / length - 1, 0);
    // the last sum is read for the state behind it only
    if (FIRST && !s.final && at.c == (BACK ? 0 : last)) return;
    const int k0 = tile % tiles_k * EK, v0 = tile / tiles_k * EV;
    const int kp = la_pad(s.dk), vp = la_pad(s.dv);
    const int lane = threadIdx.x & 63, wave = wave_id(), lr = lane & 15, lg = lane >> 4;
    const int wk = 16 * M * (wave % WK), wv = 16 * M * (wave / WK), km = k0 + wk, vm = v0 + wv;  // the wave's part of the tile
    const Decay decay(s.log_decay[h]);
    const T* x = (const T*)s.x + (long long)sq.lo * s.x_stride + (size_t)(h / s.x_per) * s.dv;
    const T* y = (const T*)s.y + (long long)sq.lo * s.y_stride + (size_t)(h / s.y_per) * s.dk;

    // acc[i][j]: columns km + 16 i + 4 lg + e of dk, row vm + 16 j + lr of dv.  Of a state padded to multiples of
    // 64 a wave has all of its part or none.
    f32x4 acc[M][M];
    const bool mine = km < kp && vm < vp;
    const unsigned corner = (unsigned)(((vm / 64) * (kp / 64) + km / 64) * 4096 + (vm % 64 / 16 * 4 + km % 64 / 16) * 256 + 4 * lane);
    auto each = [&](auto f) {
#pragma unroll
        for (int j = 0; j < M; ++j)
#pragma unroll
            for (int i = 0; i < M; ++i) f(acc[i][j], km + 16 * i + 4 * lg, vm + 16 * j + lr);
    };
    auto each_padded = [&](auto f) {
        if (!mine) return;
#pragma unroll
        for (int j = 0; j < M; ++j)
#pragma unroll
            for (int i = 0; i < M; ++i) f(acc[i][j], corner + 1024 * j + 256 * i);
    };
    each([](f32x4& a, int, int) { a = f32x4{0, 0, 0, 0}; });
    const size_t state = (size_t)vp * kp;
    if (!FIRST) {
        if (s.cut) {
            const float* part = s.parts + ((size_t)(s.segment.first(at.b, sq) + at.c) * s.H + h) * state;
            each_padded([&](f32x4& a, unsigned at) { a = *reinterpret_cast<const f32x4*>(part + at); });
        } else if (s.init) {
            const float* init = s.init + ((size_t)at.b * s.H + h) * s.dv * s.dk;
            each([&](f32x4& a, int k, int v) {
                if (v < s.dv) a = load_row4(init + (size_t)v * s.dk + k, s.dk - k).v;
            });
        }
    }
    const int chunk0 = s.chunk.first(at.b, sq) + r0 / LA_CHUNK;
    const int chunks = (n + LA_CHUNK - 1) / LA_CHUNK;

    for (int i = threadIdx.x; i <= LA_CHUNK; i += THREADS) lds.power[i] = decay(i);

    // piece t + THREADS i of a block: columns 8 (piece % (E / 8)) .. + 7 of row piece / (E / 8)
    Raw8<T> xr[2][XT], yr[2][YT];                // of the next block and of the one behind it
    auto row_at = [](int i, int E) { return (int)(threadIdx.x + THREADS * i) / (E / 8); };
    auto col_at = [](int i, int E) { return 8 * ((int)(threadIdx.x + THREADS * i) % (E / 8)); };
    struct Block { int c, b, begin, len; };      // block b of the segment's c-th chunk in order, `len` rows from `begin`
    auto block_at = [&](int c) {
        const int cc = BACK ? chunks - 1 - c : c;
        return Block{c, 0, r0 + cc * LA_CHUNK, min(LA_CHUNK, n - cc * LA_CHUNK)};
    };
    auto next = [&](Block k) {
        if (SB * (k.b + 1) < k.len) return Block{k.c, k.b + 1, k.begin, k.len};
        return block_at(k.c + 1);                // (past the last chunk: not taken)
    };
    // elements that a piece's row has left from its column on, none for rows past the chunk's end
    auto left = [&](const Block& k, int r, int c, int d) { return SB * k.b + r < k.len ? d - c : 0; };
    auto load = [&](Block k, Raw8<T> (&xr)[XT], Raw8<T> (&yr)[YT]) {
        if (k.c >= chunks) k = Block{k.c, 0, r0, 0};
#pragma unroll
        for (int i = 0; i < XT; ++i) {
            const int r = row_at(i, EV), c = v0 + col_at(i, EV);
            xr[i] = load8<WIDE>(x + (k.begin + SB * k.b + r) * s.x_stride + c, left(k, r, c, s.dv), x + r0 * s.x_stride);
        }
#pragma unroll
        for (int i = 0; i < YT; ++i) {
            const int r = row_at(i, EK), c = k0 + col_at(i, EK);
            yr[i] = load8<WIDE>(y + (k.begin + SB * k.b + r) * s.y_stride + c, left(k, r, c, s.dk), y + r0 * s.y_stride);
        }
    };
    auto put = [&](const Block& k, const Raw8<T> (&xr)[XT], const Raw8<T> (&yr)[YT], int buf) {
#pragma unroll
        for (int i = 0; i < XT; ++i) {
            const int r = row_at(i, EV), c = col_at(i, EV);
            lds_put(&lds.x[buf][r * XS + c], kept<WIDE>(xr[i], left(k, r, v0 + c, s.dv)));
        }
#pragma unroll
        for (int i = 0; i < YT; ++i) {
            const int r = row_at(i, EK), c = col_at(i, EK), t = SB * k.b + r;
            const float w = BACK ? s.factor * lds.power[min(t + 1, LA_CHUNK)] : lds.power[min(max(k.len - 1 - t, 0), LA_CHUNK)];
            Raw8<T> part[N];
            cut<N>(kept<WIDE>(yr[i], left(k, r, k0 + c, s.dk)), w, part);
#pragma unroll
            for (int p = 0; p < N; ++p) lds_put(&lds.y[buf][p][r * YS + c], part[p]);
        }
    };
    const Factor whole(decay, LA_CHUNK);
    Block now = block_at(0), then = next(now), after = next(then);
    __syncthreads();                             // the powers
    if (chunks > 0) {
        load(now, xr[0], yr[0]);
        load(then, xr[1], yr[1]);
        put(now, xr[0], yr[0], 0);
        __builtin_amdgcn_sched_barrier(0);       // in the order in which they are waited for
        load(after, xr[0], yr[0]);
    }
    auto step = [&](auto odd) {
        constexpr int buf = odd, other = 1 - buf;
        __syncthreads();                         // this block is there, and the one before it read
        if (now.b == 0) {
            // the state that enters the chunk
            if (!FIRST && s.kept && (s.init || now.c > 0 || at.c != (BACK ? last : 0))) {
                const int cc = BACK ? chunks - 1 - now.c : now.c;
                T* kept = (T*)s.kept + ((size_t)(chunk0 + cc) * s.H + h) * state;
                each_padded([&](f32x4& a, unsigned at) {
                    Raw4<T> o;
#pragma unroll
                    for (int e = 0; e < 4; ++e) o.set(e, a[e]);
                    o.store(kept + at);
                });
            }
            const Factor f = now.len == LA_CHUNK ? whole : Factor(decay, now.len);
            each([&](f32x4& a, int, int) {
#pragma unroll
                for (int e = 0; e < 4; ++e) a[e] = f(a[e]);
            });
        }
        const int r = 4 * lg;                    // and 16 more: the four groups' reads then meet all banks
        Frag<T> fx[M];
#pragma unroll
        for (int j = 0; j < M; ++j) frag_col(fx[j], &lds.x[buf][wv + 16 * j], XS, r, r + 16);
#pragma unroll
        for (int p = 0; p < N; ++p)
#pragma unroll
            for (int i = 0; i < M; ++i) {
                Frag<T> fy;
                frag_col(fy, &lds.y[buf][p][wk + 16 * i], YS, r, r + 16);
#pragma unroll
                for (int j = 0; j < M; ++j) acc[i][j] = mma(fy, fx[j], acc[i][j]);
            }
        put(then, xr[other], yr[other], other);
        const Block last_loaded = next(after);
        load(last_loaded, xr[other], yr[other]);
        if (sizeof(T) == 2) {
            // vector instructions of the next block's parts between the matrix instructions of this one: both waves of a
            // SIMD are at the same place, so that one's vector instructions do not cover the other's
#pragma unroll
            for (int i = 0; i < N * M * M; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
            }
        }
        now = then;
        then = after;
        after = last_loaded;
    };
    while (now.c < chunks) {
        step(std::integral_constant<int, 0>{});
        if (now.c >= chunks) break;
        step(std::integral_constant<int, 1>{});
    }
    if (FIRST) {
        float* part = s.parts + ((size_t)(s.segment.first(at.b, sq) + at.c) * s.H + h) * state;
        each_padded([&](f32x4& a, unsigned at) { *reinterpret_cast<f32x4*>(part + at) = a; });
    } else if (s.final && !s.cut) {
        float* final = s.final + ((size_t)at.b * s.H + h) * s.dv * s.dk;
        each([&](f32x4& a, int k, int v) {
            if (v < s.dv) {
                Raw4<float> o;
                o.v = a;
                store_row4(final + (size_t)v * s.dk + k, o, s.dk - k);
            }
        });
    }
}

// Segments' sums in, the states that enter them out, in the same places; a thread has four neighbours of a
// state as the instruction's lanes hold them.
template <bool BACK>
__global__ __launch_bounds__(256) void join_kernel(StateShape s, int groups_per)
{
    const int bh = blockIdx.x / groups_per, b = bh / s.H, h = bh - b * s.H;
    const int kp = la_pad(s.dk), vp = la_pad(s.dv);
    const unsigned state = (unsigned)kp * vp, at = (blockIdx.x % groups_per * 256 + threadIdx.x) * 4;
    if (at >= state) return;
    const RowRange sq = s.segment.sequence(b);
    const int length = s.segment.length, segments = max((sq.n + length - 1) / length, 1), first = s.segment.first(b, sq);
    const unsigned block = at / 4096, tile = at % 4096 / 256, lane = at % 256 / 4;
    const int k = block % (kp / 64) * 64 + tile % 4 * 16 + lane / 16 * 4, v = block / (kp / 64) * 64 + tile / 4 * 16 + lane % 16;
    const size_t place = ((size_t)b * s.H + h) * s.dv * s.dk + (size_t)v * s.dk + k;
    const Decay decay(s.log_decay[h]);
    const Factor whole(decay, length);
    f32x4 x = {0, 0, 0, 0};
    if (s.init && v < s.dv) x = load_row4(s.init + place, s.dk - k).v;
    const size_t step = (size_t)s.H * state;
    float* part = s.parts + ((size_t)first * s.H + h) * state + at;
    auto pass = [&](int c, f32x4 sum) {
        *reinterpret_cast<f32x4*>(part + c * step) = x;
        const int rows = min(length, sq.n - c * length);
        const Factor f = rows == length ? whole : Factor(decay, rows);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = f(x[e]) + sum[e];
    };
    // four sums are read at a time, before the states take their places
    const int count = s.final ? segments : segments - 1;
    int i = 0;
    for (; i + 4 <= count; i += 4) {
        f32x4 sum[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) sum[u] = *reinterpret_cast<const f32x4*>(part + (BACK ? segments - 1 - i - u : i + u) * step);
#pragma unroll
        for (int u = 0; u < 4; ++u) pass(BACK ? segments - 1 - i - u : i + u, sum[u]);
    }
    for (; i < count; ++i) pass(BACK ? segments - 1 - i : i, *reinterpret_cast<const f32x4*>(part + (BACK ? segments - 1 - i : i) * step));
    if (!s.final) {
        *reinterpret_cast<f32x4*>(part + (BACK ? 0 : segments - 1) * step) = x;
    } else if (v < s.dv) {
        Raw4<float> o;
        o.v = x;
        store_row4(s.final + place, o, s.dk - k);
    }
}

struct Tile { int k, v; };
long long state_groups(const Tile& t, int dk, int dv, int H, const Pieces& segment) {
    return ((long long)((dk + t.k - 1) / t.k) * ((dv + t.v - 1) / t.v) * H * segment.count() + 7) / 8 * 8;
}

template <typename T, int N, int M, int WK, int WV, bool BACK, bool FIRST>
hipError_t launch(const LaBatch& b, const StateShape& s) {
    typedef StateLds<T, N, M, WK, WV> Lds;
    const long long groups = state_groups(Tile{Lds::EK, Lds::EV}, s.dk, s.dv, s.H, s.segment);
    if (!launchable(groups, 64 * WK * WV)) return hipErrorInvalidConfiguration;
    if (s.dk % 8 == 0 && s.dv % 8 == 0)
        hipLaunchKernelGGL((state_kernel<T, N, M, WK, WV, BACK, FIRST, true>), dim3((unsigned)groups), dim3(64 * WK * WV),
                           0, b.stream, s, (int)groups);
    else
        hipLaunchKernelGGL((state_kernel<T, N, M, WK, WV, BACK, FIRST, false>), dim3((unsigned)groups), dim3(64 * WK * WV),
                           0, b.stream, s, (int)groups);
    return hipGetLastError();
}

template <typename T, int M, int WK, int WV, bool BACK>
hipError_t passes(const LaBatch& b, const StateShape& s) {
    constexpr int WHOLE = sizeof(T) == 4 ? 1 : 3, ROUNDED = sizeof(T) == 4 ? 1 : 2;
    if (!s.cut) return s.final ? launch<T, WHOLE, M, WK, WV, BACK, false>(b, s) : launch<T, ROUNDED, M, WK, WV, BACK, false>(b, s);
    hipError_t e = s.final ? launch<T, WHOLE, M, WK, WV, BACK, true>(b, s) : launch<T, ROUNDED, M, WK, WV, BACK, true>(b, s);
    if (e != hipSuccess) return e;
    const int groups_per = la_pad(s.dk) * la_pad(s.dv) / 1024;
    hipLaunchKernelGGL(join_kernel<BACK>, dim3((unsigned)(b.B * b.H * groups_per)), dim3(256), 0, b.stream, s, groups_per);
    e = hipGetLastError();
    return e != hipSuccess || !s.kept ? e : launch<T, ROUNDED, M, WK, WV, BACK, false>(b, s);
}

Tile tile_of(const LaBatch& b, int dk, int dv) {
    if (b.dtype == MLSTM_F32 || (dk <= 64 && dv <= 64)) return Tile{64, 64};
    // 256 wide, the weighted rows are cut for twice the columns: 122 us against 142 a first pass at 256 x 256; where half of the
    // last tile would be empty (384) 65 against 49
    return (dv - 1) / 128 % 2 == 0 ? Tile{128, 128} : Tile{128, 256};
}

}  // namespace

// Sequences are cut where their tiles leave the chip idle, into segments of at least 2 chunks (2 against 4: 15 us a pass
// against 22 over 3158 rows of 8 heads of 96), from 8 chunks on: with 8, cut and whole take 60 and 80 us at 4 heads of 256, 46
// and 58 at 4 sequences of 6 heads of 96, the whole backward of the 3158 rows 125 and 137; with 6, 59 and 67, 47 and 48,
// but in fp32 70 and 61, backwards 178 and 157, and 75 and 63 over 3948 packed rows of 6 heads of 40 x 77.  A packed batch counts as
// B sequences of S rows: one long sequence among many short ones is not cut (8192 rows of 4 heads of 128 alone 54 us,
// with 63 sequences of 64 rows 342).
int la_segment_rows(const LaBatch& b, int dk, int dv) {
    const Tile t = tile_of(b, dk, dv);
    const long long tiles = (long long)((dk + t.k - 1) / t.k) * ((dv + t.v - 1) / t.v) * b.H * b.B;
    const int chunks = (b.S + LA_CHUNK - 1) / LA_CHUNK, room = t.v > 128 ? 256 : 512;   // workgroups that run at once
    if (tiles > room / 2 || chunks < 8) return 0;
    const int want = (int)(room / tiles), most = chunks / 2, cuts = want < most ? want : most;
    return (chunks + cuts - 1) / cuts * LA_CHUNK;
}

static Pieces la_segments(const LaBatch& b, int dk, int dv) {
    const int seg = la_segment_rows(b, dk, dv);
    return make_pieces(b.seq_start, b.B, b.S, b.rows, seg > 0 ? seg : (b.S + LA_CHUNK - 1) / LA_CHUNK * LA_CHUNK);
}

bool la_states_launchable(const LaBatch& b, int dk, int dv) {
    return launchable(state_groups(tile_of(b, dk, dv), dk, dv, b.H, la_segments(b, dk, dv)), 512) &&
           launchable((long long)b.B * b.H * (la_pad(dk) * la_pad(dv) / 1024), 256);
}

size_t la_state_parts_bytes(const LaBatch& b, int dk, int dv) {
    if (la_segment_rows(b, dk, dv) == 0) return 0;
    return (size_t)la_segments(b, dk, dv).count() * b.H * la_pad(dk) * la_pad(dv) * 4;
}

hipError_t launch_la_states(const LaBatch& b, const LaStates& a) {
    const int dk = a.y.d, dv = a.x.d;
    StateShape s = {};
    s.x = a.x.p; s.x_stride = a.x.stride; s.dv = dv; s.x_per = a.x.per;
    s.y = a.y.p; s.y_stride = a.y.stride; s.dk = dk; s.y_per = a.y.per;
    s.log_decay = b.log_decay; s.init = a.init; s.final = a.final; s.kept = a.kept; s.parts = a.parts;
    s.H = b.H; s.factor = a.factor; s.cut = la_segment_rows(b, dk, dv) > 0;
    s.segment = la_segments(b, dk, dv);
    s.chunk = make_pieces(b.seq_start, b.B, b.S, b.rows, LA_CHUNK);
    const Tile t = tile_of(b, dk, dv);
    if (b.dtype == MLSTM_F32) return a.backwards ? passes<float, 2, 2, 2, true>(b, s) : passes<float, 2, 2, 2, false>(b, s);
    if (t.k == 64) return a.backwards ? passes<bf16, 2, 2, 2, true>(b, s) : passes<bf16, 2, 2, 2, false>(b, s);
    if (t.v == 128) return a.backwards ? passes<bf16, 4, 2, 2, true>(b, s) : passes<bf16, 4, 2, 2, false>(b, s);
    return a.backwards ? passes<bf16, 4, 2, 4, true>(b, s) : passes<bf16, 4, 2, 4, false>(b, s);
}

}  // namespace mlstm
