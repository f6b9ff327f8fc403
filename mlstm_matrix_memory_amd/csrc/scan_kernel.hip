// Selective state space scan: forward over whole sequences and the one-row step.
//
// Per channel d (of group g) and state n, with s_t = softplus(dt_t + dt_bias):
//   h_t[n] = exp(s_t A[n]) h_{t-1}[n] + s_t x_t B_t[n]
//   o_t = sum_n C_t[n] h_t[n] + Dskip x_t,   y_t = o_t (or o_t z_t sigmoid(z_t))
// A decay of its own for every (channel, state) leaves no matrix product: per (row,
// channel, state) the scan takes a multiplication and an exponential for the decay,
// a multiplication and an addition for each of the update's and the read-out's
// products.  At N = 16 that arithmetic, not HBM, bounds it.
//
// A workgroup (scan_common.h) walks its rows in tiles of ROWS with two kinds of
// waves, one of each on a SIMD:
//   helpers   load x, dt and z of the tile after the next, put (s, s x) and (B, C) of the
//             next tile into LDS in fp32, and finish the tile before: add the waves' parts
//             of each row's sum over n, the skip and the gate, and store y;
//   scanners  run their states through the tile's rows.
// Both buffers in LDS are double, and one barrier per tile passes them on, so the scan,
// whose rows depend on each other, always has a second instruction stream beside it.
#include "scan_common.h"

namespace mlstm {
namespace {

// The channel of a tile at a place of its rows in LDS.  Threads stage four at a time; where the
// tile's count is no multiple of four the last four places hold its last four channels, some
// a second time, which are computed and stored twice with the same values.  (Guarding
// single channels instead made the waves run two paths: packed fp32 rows of 501 channels per
// group took 53 us against 48 us.)
__device__ __forceinline__ int scan_channel(int place, int count) {
    const int shared = count >= 4 && place >= count / 4 * 4 ? (4 - count % 4) % 4 : 0;
    return place - shared;
}

struct FwdParams {
    const void* x; const void* dt; const void* Bm; const void* Cm; const void* z;
    long long x_stride, dt_stride, B_stride, C_stride, z_stride, y_stride;
    const float* A; const float* Dskip; const float* dt_bias;
    const float* h_init;
    Pieces pieces;
    int D, G, N, softplus;
    void* y;
    float* h_final;
    float* piece_h;                      // [piece][NP][D]: end state of a piece that starts from zero
    float* piece_s;                      // [piece][D]: sum of its step sizes
};

// STATE: only the piece's end state from zero (no y); else the full scan from the true state.
// GATE: y is gated by z.
template <typename T, int NW, int NL, int ROWS, bool STATE, bool GATE>
__global__ __launch_bounds__(128 * NW) void scan_fwd_kernel(const FwdParams p)
{
    constexpr int NT = 64 * NW, NP = NW * NL;          // helper threads, padded states
    constexpr int PASS = ROWS * 16 / NT;          // rows a helper stages per tile, 4 channels each
    constexpr int BCN = ROWS * NP / NT;           // (B, C) pairs it stages
    __shared__ __align__(16) float2 du[2][ROWS][SCAN_TILE];
    __shared__ __align__(16) float bs[2][ROWS][NP], cs[2][ROWS][NP];
    __shared__ __align__(16) float part[STATE ? 1 : 2][STATE ? 1 : NW][ROWS][SCAN_TILE];

    const int tiles = scan_tiles(p.D, p.G);
    const int tile = blockIdx.x % tiles, number = blockIdx.x / tiles;
    const Pieces::At at = p.pieces.at(number);
    const int b = at.b, c = at.c;
    const RowRange sq = p.pieces.sequence(b);
    const long long t_first = (long long)c * p.pieces.length;
    if (t_first >= sq.n && c > 0) return;
    const bool last = t_first + p.pieces.length >= sq.n;       // the sequence ends in this piece
    if (STATE && last) return;                                 // no other piece starts from its end
    const int t_begin = (int)t_first;
    const int t_end = last ? sq.n : t_begin + p.pieces.length;
    const int turns = (t_end - t_begin + ROWS - 1) / ROWS;
    const ScanTile ch = scan_tile(tile, p.D, p.G);
    const int lane = threadIdx.x & 63, wave = wave_id();

    if (wave >= NW) {
        // helper: rows r0 + (NT / 16) i of a tile, channels c4 .. c4 + 3
        if (turns == 0) return;
        const int tid = threadIdx.x - NT, r0 = tid >> 4, c4 = (tid & 15) * 4;
        const int g4 = ch.count >= 4 ? min(c4, ch.count - 4) : c4;     // the first channel of LDS places c4 ..
        const int bt = tid / NP, bnn = tid % NP;
        const T* xp = (const T*)p.x + (long long)sq.lo * p.x_stride + ch.d0 + g4;
        const T* dtp = (const T*)p.dt + (long long)sq.lo * p.dt_stride + ch.d0 + g4;
        const T* zp = GATE ? (const T*)p.z + (long long)sq.lo * p.z_stride + ch.d0 + g4 : nullptr;
        T* yp = (T*)p.y + (long long)sq.lo * p.y_stride + ch.d0 + g4;
        const T* bp = (const T*)p.Bm + (long long)sq.lo * p.B_stride + ch.group * p.N + min(bnn, p.N - 1);
        const T* cp = (const T*)p.Cm + (long long)sq.lo * p.C_stride + ch.group * p.N + min(bnn, p.N - 1);
        float bias[4], skip[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            bias[e] = p.dt_bias && g4 + e < ch.count ? p.dt_bias[ch.d0 + g4 + e] : 0.0f;
            skip[e] = !STATE && p.Dskip && g4 + e < ch.count ? p.Dskip[ch.d0 + g4 + e] : 0.0f;
        }
        // Loads run two tiles ahead.  To know how many accesses lie between a load and its
        // use, and so wait for no later ones, the compiler needs every turn to issue the
        // same: rows past the end are read from the last row and masked when staged.
        auto work = [&](auto full_tag) {
            constexpr int FILL = full_tag;             // 2: 64 channels; 1: four to every thread; 0: fewer
            constexpr bool FULL = FILL > 0;
            const int nc = ch.count - c4;
            Raw4<T> xn[2][PASS], zn[2][PASS], dtn[2][PASS];
            T bn[2][BCN], cn[2][BCN];
            // x and z of the staged tile and the two before it
            Raw4<T> x0[PASS], z0[PASS], x1[PASS], z1[PASS], x2[PASS], z2[PASS];
            auto get = [&](const T* q) {
                Raw4<T> v;
                if (FULL) v.load(q);
                else v = load_row4(q, nc);
                return v;
            };
            auto load = [&](int turn, auto kc) {
                constexpr int k = kc;
                const int t0 = t_begin + min(turn, turns - 1) * ROWS;
#pragma unroll
                for (int i = 0; i < PASS; ++i) {
                    const long long t = min(t0 + r0 + (NT / 16) * i, t_end - 1);
                    xn[k][i] = get(xp + t * p.x_stride);
                    dtn[k][i] = get(dtp + t * p.dt_stride);
                    if (GATE) zn[k][i] = get(zp + t * p.z_stride);
                }
#pragma unroll
                for (int i = 0; i < BCN; ++i) {
                    const long long t = min(t0 + bt + (NT / NP) * i, t_end - 1);
                    bn[k][i] = bp[t * p.B_stride];
                    if (!STATE) cn[k][i] = cp[t * p.C_stride];
                }
            };
            auto stage = [&](int turn, auto kc) {
                constexpr int k = kc;
                const int t0 = t_begin + turn * ROWS, buf = turn & 1;
#pragma unroll
                for (int i = 0; i < PASS; ++i) {
                    const int r = r0 + (NT / 16) * i;
                    const bool row = t0 + r < t_end;   // past the end: decay 1, nothing added
                    float s[4], u[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[e] = dtn[k][i].get(e) + bias[e];
                    if (p.softplus)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[e] = softplus_hw(s[e]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        u[e] = row ? s[e] * xn[k][i].get(e) : 0.0f;
                        s[e] = row ? s[e] : 0.0f;
                    }
                    f32x4* to = reinterpret_cast<f32x4*>(&du[buf][r][c4]);
                    to[0] = f32x4{s[0], u[0], s[1], u[1]};
                    to[1] = f32x4{s[2], u[2], s[3], u[3]};
                    if (!STATE) {
                        x2[i] = x1[i]; x1[i] = x0[i]; x0[i] = xn[k][i];
                        if (GATE) { z2[i] = z1[i]; z1[i] = z0[i]; z0[i] = zn[k][i]; }
                    }
                }
#pragma unroll
                for (int i = 0; i < BCN; ++i) {
                    const int r = bt + (NT / NP) * i;
                    const bool live = t0 + r < t_end && bnn < p.N;
                    bs[buf][r][bnn] = live ? to_f32(bn[k][i]) : 0.0f;
                    if (!STATE) cs[buf][r][bnn] = live ? to_f32(cn[k][i]) : 0.0f;
                }
            };
            auto finish = [&](int turn, const Raw4<T>* x, const Raw4<T>* z) {
                const int t0 = t_begin + turn * ROWS, buf = turn & 1;
#pragma unroll
                for (int i = 0; i < PASS; ++i) {
                    const int r = r0 + (NT / 16) * i;
                    const long long t = t0 + r;
                    f32x4 y = *reinterpret_cast<const f32x4*>(&part[buf][0][r][c4]);
#pragma unroll
                    for (int w = 1; w < NW; ++w) y += *reinterpret_cast<const f32x4*>(&part[buf][w][r][c4]);
                    Raw4<T> o;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        y[e] = fmaf(skip[e], x[i].get(e), y[e]);
                        if (GATE) {
                            const float zv = z[i].get(e);
                            y[e] *= zv * sigmoid_hw(zv);
                        }
                        o.set(e, y[e]);
                    }
                    if (t < t_end && (FILL == 2 || c4 < ch.count)) {
                        if (FULL) o.store(yp + t * p.y_stride);
                        else store_row4(yp + t * p.y_stride, o, nc);
                    }
                }
            };
            typedef std::integral_constant<int, 0> Even;
            typedef std::integral_constant<int, 1> Odd;
            load(0, Even());
            load(1, Odd());
            stage(0, Even());
            load(2, Even());
            __syncthreads();
            // turn i: tile i is scanned, i + 1 staged and i - 1 finished
            auto turn = [&](int i, auto next) {
                if (i + 1 < turns) {
                    stage(i + 1, next);
                    if (!STATE && i > 0) finish(i - 1, x2, z2);
                } else if (!STATE && i > 0) {
                    finish(i - 1, x1, z1);
                }
                load(i + 3, next);
                __syncthreads();
            };
            for (int i = 0; i < turns; i += 2) {
                turn(i, Odd());
                if (i + 1 < turns) turn(i + 1, Even());
            }
            if (!STATE) finish(turns - 1, x0, z0);
        };
        if (ch.count == SCAN_TILE) work(std::integral_constant<int, 2>());
        else if (ch.count >= 4) work(std::integral_constant<int, 1>());
        else work(std::integral_constant<int, 0>());
        return;
    }

    // scanner: channel d, states n0 .. n0 + NL - 1
    const int d = ch.d0 + scan_channel(lane, ch.count), n0 = wave * NL;
    const bool own = lane < (ch.count + 3) / 4 * 4 && d < ch.d0 + ch.count;
    float a2[NL], h[NL];
#pragma unroll
    for (int j = 0; j < NL; ++j) {
        const bool live = own && n0 + j < p.N;
        a2[j] = live ? p.A[(size_t)d * p.N + n0 + j] * LOG2E : 0.0f;
        h[j] = !STATE && live && p.h_init ? p.h_init[((size_t)b * p.D + d) * p.N + n0 + j] : 0.0f;
    }
    if (!STATE && own) {
        // join: the states of the pieces before, each decayed by the sums of the step sizes behind it
#pragma unroll 4
        for (int e = number - c; e < number; ++e) {
            const float sum = p.piece_s[(size_t)e * p.D + d];
#pragma unroll
            for (int j = 0; j < NL; ++j)
                h[j] = fmaf(__builtin_amdgcn_exp2f(a2[j] * sum), h[j], p.piece_h[((size_t)e * NP + n0 + j) * p.D + d]);
        }
    }
    float sums = 0.0f;                                 // of step sizes (STATE)
    if (turns > 0) __syncthreads();
    for (int i = 0; i < turns; ++i) {
        const int buf = i & 1;
        // rows in groups of four, the next group's operands read from LDS before this one's run
        constexpr int GR = 4;
        float2 su[2][GR];
        float bv[2][GR], cv[2][GR][NL];
        auto read = [&](int k, int g) {
#pragma unroll
            for (int r = 0; r < GR; ++r) {
                su[k][r] = du[buf][g + r][lane];
                bv[k][r] = bs[buf][g + r][n0 + (lane & (NL - 1))];
                if (!STATE)
#pragma unroll
                    for (int j = 0; j < NL; j += 4)
                        *reinterpret_cast<f32x4*>(cv[k][r] + j) = *reinterpret_cast<const f32x4*>(&cs[buf][g + r][n0 + j]);
            }
        };
        read(0, 0);
#pragma unroll
        for (int g = 0; g < ROWS; g += GR) {
            const int k = g / GR & 1;
            if (g + GR < ROWS) read(k ^ 1, g + GR);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int r = 0; r < GR; ++r) {
                float y = 0.0f;
                for_each<NL>([&](auto jc) {
                    constexpr int j = jc;
                    const float a = __builtin_amdgcn_exp2f(su[k][r].x * a2[j]);
                    h[j] = fmaf(a, h[j], row_broadcast<j>(bv[k][r]) * su[k][r].y);
                    if (!STATE) y = j == 0 ? cv[k][r][0] * h[0] : fmaf(cv[k][r][j], h[j], y);
                });
                if (STATE) sums += su[k][r].x;
                else part[buf][wave][g + r][lane] = y;
            }
        }
        __syncthreads();
    }
    if (!own) return;
    if (STATE) {
#pragma unroll
        for (int j = 0; j < NL; ++j) p.piece_h[((size_t)number * NP + n0 + j) * p.D + d] = h[j];
        if (wave == 0) p.piece_s[(size_t)number * p.D + d] = sums;
    } else if (p.h_final && last) {
#pragma unroll
        for (int j = 0; j < NL; ++j)
            if (n0 + j < p.N) p.h_final[((size_t)b * p.D + d) * p.N + n0 + j] = h[j];
    }
}

// One row per sequence: a lane holds 4 states of a channel (one 16-byte access), LPC
// lanes a channel, of SEQS sequences.  Bound by the state's HBM traffic, 8 bytes per state:
// several sequences to a thread keep as many loads in flight, and read A once for them.
template <typename T, int LPC, int SEQS>
__global__ __launch_bounds__(256) void ssm_step_kernel(
    const T* __restrict__ x, long long x_stride, const T* __restrict__ dt, long long dt_stride,
    const float* __restrict__ A, const T* __restrict__ Bm, long long B_stride, const T* __restrict__ Cm,
    long long C_stride, const float* __restrict__ Dskip, const float* __restrict__ dt_bias,
    const T* __restrict__ z, long long z_stride, int B, int D, int G, int N, int softplus, float* __restrict__ h,
    T* __restrict__ y, long long y_stride)
{
    const int q = threadIdx.x % LPC, n = 4 * q;
    const int sets = (B + SEQS - 1) / SEQS;            // this thread's sequences: set, set + sets, ...
    const long long id = (long long)blockIdx.x * (256 / LPC) + threadIdx.x / LPC;
    const bool in = id < (long long)sets * D;          // a channel's lanes are in or not together
    const int set = in ? (int)(id / D) : 0, d = in ? (int)(id % D) : 0, g = d / (D / G);
    const int cnt = min(max(N - n, 0), 4);
    f32x4 hv[SEQS], av = {0, 0, 0, 0};
    Raw4<T> bv[SEQS], cv[SEQS];
    T xv[SEQS], dtv[SEQS], zv[SEQS];
    bool live[SEQS];
#pragma unroll
    for (int k = 0; k < SEQS; ++k) {
        const long long b = set + (long long)k * sets;
        live[k] = in && b < B;
        const long long r = live[k] ? b : 0;
        const float* hp = h + ((size_t)r * D + d) * N + n;
        if (cnt == 4) {
            hv[k] = *reinterpret_cast<const f32x4_u*>(hp);
        } else {
            hv[k] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (j < cnt) hv[k][j] = hp[j];
        }
        bv[k] = load_row4(Bm + r * B_stride + g * N + n, cnt);
        cv[k] = load_row4(Cm + r * C_stride + g * N + n, cnt);
        xv[k] = x[r * x_stride + d];
        dtv[k] = dt[r * dt_stride + d];
        if (z) zv[k] = z[r * z_stride + d];
    }
    {
        const Raw4<float> a = load_row4(A + (size_t)d * N + n, cnt);
#pragma unroll
        for (int j = 0; j < 4; ++j) av[j] = a.get(j) * LOG2E;
    }
    const float bias = dt_bias ? dt_bias[d] : 0.0f, skip = Dskip ? Dskip[d] : 0.0f;
#pragma unroll
    for (int k = 0; k < SEQS; ++k) {
        const long long b = set + (long long)k * sets;
        const float v = to_f32(dtv[k]) + bias, xf = to_f32(xv[k]);
        const float s = softplus ? softplus_hw(v) : v, u = s * xf;
        float o = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            hv[k][j] = fmaf(__builtin_amdgcn_exp2f(s * av[j]), hv[k][j], u * bv[k].get(j));
            o = fmaf(cv[k].get(j), hv[k][j], o);
        }
#pragma unroll
        for (int off = LPC / 2; off > 0; off >>= 1) o += __shfl_xor(o, off, 64);
        if (!live[k]) continue;
        float* hp = h + ((size_t)b * D + d) * N + n;
        if (cnt == 4) {
            *reinterpret_cast<f32x4_u*>(hp) = hv[k];
        } else {
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (j < cnt) hp[j] = hv[k][j];
        }
        if (q == 0) {
            o = fmaf(skip, xf, o);
            if (z) {
                const float zf = to_f32(zv[k]);
                o *= zf * sigmoid_hw(zf);
            }
            y[b * y_stride + d] = from_f32<T>(o);
        }
    }
}

// Rows per piece.  One piece to a sequence does the least work: where sequences are
// cut, the pieces' end states cost most of the scan a second time.  A workgroup alone on its
// compute unit takes about 70 ns a row; cut into some workgroups per compute unit the scan
// takes 7.2 ps per row and channel against 4.2 uncut.  So sequences are cut below 144
// workgroups: on one MI355X (2, 1024, 4096) (sequences, rows, channels; 128 workgroups) took
// 76 us uncut and 67 us in six pieces, (8, 2048, 1536) (192 workgroups) 148 us uncut and 173 us
// in eight; (1, 32768, 2048) 2512 us uncut, 646, 501, 483 and 499 us in 8, 16, 32 and 64 pieces.
// Up to 4 states, where a workgroup is two waves, cutting pays longer: (8, 1024, 2048), 256
// workgroups, took 117 us uncut and 69 us in four pieces at N = 4, 69 and 92 us at N = 8.
constexpr int CUT_BELOW = 144, CUT_BELOW_4 = 320, CUT_TO = 1024, SHORTEST_PIECE = 64;
int piece_rows(int S, int rows, int D, int G, int N) {
    // packed sequences count by the rows that there are
    const long long groups = ((long long)scan_tiles(D, G) * rows + S / 2) / S;
    const int whole = (S + 31) / 32 * 32;
    if (groups > (N <= 4 ? CUT_BELOW_4 : CUT_BELOW)) return whole;
    const long long n = groups > 0 ? (CUT_TO + groups - 1) / groups : CUT_TO;
    const int length = (int)(((S + n - 1) / n + 15) / 16 * 16);
    return length < SHORTEST_PIECE ? (SHORTEST_PIECE < whole ? SHORTEST_PIECE : whole) : length;
}

struct FwdPlan {
    Pieces pieces;
    size_t state;                        // floats of piece_h (piece_s lies behind them); 0: uncut
    size_t total;
};
FwdPlan plan(const int* seq_start, int B, int S, int rows, int D, int G, int N) {
    FwdPlan f = {};
    f.pieces = make_pieces(seq_start, B, S, rows, piece_rows(S, rows, D, G, N));
    if (f.pieces.length < S) {
        // as many as packed sequences may need, so that a workspace's size does not depend on seq_start
        const size_t count = (size_t)rows / f.pieces.length + B;
        f.state = count * scan_padded_states(N) * D;
        f.total = f.state + count * D;
    }
    return f;
}

template <typename T>
hipError_t fwd_t(const ScanArgs& a) {
    const FwdPlan f = plan(a.seq_start, a.B, a.S, a.rows, a.D, a.G, a.N);
    FwdParams p = {};
    p.x = a.x; p.dt = a.dt; p.Bm = a.Bm; p.Cm = a.Cm; p.z = a.z;
    p.x_stride = a.x_stride; p.dt_stride = a.dt_stride; p.B_stride = a.B_stride; p.C_stride = a.C_stride;
    p.z_stride = a.z_stride; p.y_stride = a.y_stride;
    p.A = a.A; p.Dskip = a.Dskip; p.dt_bias = a.dt_bias; p.h_init = a.h_init; p.pieces = f.pieces;
    p.D = a.D; p.G = a.G; p.N = a.N; p.softplus = a.softplus;
    p.y = a.y; p.h_final = a.h_final;
    p.piece_h = a.ws; p.piece_s = a.ws + f.state;
    const long long grid = (long long)scan_tiles(a.D, a.G) * f.pieces.count();
    // Tiles of 32 rows have half the barriers but at N = 16 take 104 KB of LDS, one workgroup to a
    // compute unit; of 16 rows two fit (by their 81 to 96 registers; by LDS three).  Uncut
    // sequences of at most 4 states and more than 64 rows always have more than 256 workgroups,
    // so the 32-row tiles of one wave run short ones only.  (4, 2048, 4096), 256 workgroups, uncut: 157 us against 177 us;
    // (16, 1024, 2048), 512 workgroups: 165 us against 139 us.
    const bool deep = !f.state && grid <= 256;
#define SCAN_LAUNCH(NW, NL, ROWS, STATE, GATE) \
    hipLaunchKernelGGL((scan_fwd_kernel<T, NW, NL, ROWS, STATE, GATE>), dim3((unsigned)grid), dim3(128 * NW), 0, a.stream, p)
#define SCAN_CALL(NW, NL)                                    \
    if (!launchable(grid, 128 * NW)) return hipErrorInvalidConfiguration; \
    if (f.state) SCAN_LAUNCH(NW, NL, 16, true, false);       \
    if (deep && a.z) SCAN_LAUNCH(NW, NL, 32, false, true);   \
    else if (deep) SCAN_LAUNCH(NW, NL, 32, false, false);    \
    else if (a.z) SCAN_LAUNCH(NW, NL, 16, false, true);      \
    else SCAN_LAUNCH(NW, NL, 16, false, false)
    SCAN_DISPATCH_N(a.N, SCAN_CALL)
#undef SCAN_CALL
#undef SCAN_LAUNCH
    return hipGetLastError();
}

constexpr long long STEP_SEQS_FROM = 1LL << 21;
template <typename T, int SEQS>
hipError_t step_launch(const ScanArgs& a) {
    const long long ch = (long long)((a.B + SEQS - 1) / SEQS) * a.D;
    if (!launchable((ch * (scan_padded_states(a.N) / 4) + 255) / 256, 256)) return hipErrorInvalidConfiguration;
#define STEP_CALL(LPC)                                                                                                 \
    hipLaunchKernelGGL((ssm_step_kernel<T, LPC, SEQS>), dim3((unsigned)((ch * LPC + 255) / 256)), dim3(256), 0,        \
                       a.stream, (const T*)a.x, a.x_stride, (const T*)a.dt, a.dt_stride, a.A, (const T*)a.Bm,          \
                       a.B_stride, (const T*)a.Cm, a.C_stride, a.Dskip, a.dt_bias, (const T*)a.z, a.z_stride, a.B,     \
                       a.D, a.G, a.N, a.softplus, a.h_final, (T*)a.y, a.y_stride)
    switch (scan_padded_states(a.N)) {
        case 4: STEP_CALL(1); break;
        case 8: STEP_CALL(2); break;
        case 16: STEP_CALL(4); break;
        case 32: STEP_CALL(8); break;
        default: STEP_CALL(16); break;
    }
#undef STEP_CALL
    return hipGetLastError();
}

template <typename T>
hipError_t step_t(const ScanArgs& a) {
    // (sequences, channels) at N = 16, bf16, one and two sequences to a thread: (256, 2048) 15.9 and 15.4 us,
    // (64, 2048) 5.9 and 5.5, (32, 2048) 4.3 and 4.3, (16, 2048) 3.5 and 3.8 (four: 15.5, 6.1, 5.1, 4.9)
    if ((long long)a.B * a.D * scan_padded_states(a.N) >= STEP_SEQS_FROM) return step_launch<T, 2>(a);
    return step_launch<T, 1>(a);
}

}  // namespace

size_t scan_fwd_workspace_bytes(int B, int S, int rows, int D, int G, int N) {
    return plan(nullptr, B, S, rows, D, G, N).total * sizeof(float);
}

hipError_t launch_scan_fwd(const ScanArgs& a) {
    return a.dtype == MLSTM_BF16 ? fwd_t<bf16>(a) : fwd_t<float>(a);
}
hipError_t launch_ssm_step(const ScanArgs& a) {
    return a.dtype == MLSTM_BF16 ? step_t<bf16>(a) : step_t<float>(a);
}

}  // namespace mlstm
