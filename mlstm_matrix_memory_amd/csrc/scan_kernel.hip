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
// A workgroup (scan_common.h) walks its rows in tiles of SCAN_ROWS.  Per tile
//   stage     all threads load x, dt and z as 16-byte pieces of rows and put (s, s x)
//             and (B, C) into LDS in fp32,
//   scan      each wave runs its states through the tile's rows and leaves its part of
//             each row's sum over n in LDS,
//   epilogue  all threads add the parts, the skip and the gate and store y.
// The next tile's loads are issued before the scan and arrive behind it.
#include "scan_common.h"

namespace mlstm {
namespace {

constexpr int SCAN_ROWS = 32;

struct FwdParams {
    const void* x; const void* dt; const void* Bm; const void* Cm; const void* z;
    long long x_stride, dt_stride, B_stride, C_stride, z_stride, y_stride;
    const float* A; const float* Dskip; const float* dt_bias;
    const int* seq_start; const float* h_init;
    int S, rows, D, G, N, softplus;
    int pieces, length;                  // pieces per sequence, rows per piece (a multiple of SCAN_ROWS)
    void* y;
    float* h_final;
    float* piece_h;                      // [B][pieces][NP][D]: end state of a piece that starts from zero
    float* piece_s;                      // [B][pieces][D]: sum of its step sizes
};

// STATE: only the piece's end state from zero (no y); else the full scan from the true state.
template <typename T, int NW, int NL, bool STATE>
__global__ __launch_bounds__(64 * NW) void scan_fwd_kernel(const FwdParams p)
{
    constexpr int NT = 64 * NW, NP = NW * NL;
    constexpr int PASS = SCAN_ROWS * 8 / NT;           // rows a thread stages per tile
    constexpr int BCN = SCAN_ROWS * NP / NT;           // (B, C) pairs it stages
    __shared__ __align__(16) float2 du[SCAN_ROWS][SCAN_TILE];
    __shared__ __align__(16) float2 bc[SCAN_ROWS][NP];
    __shared__ __align__(16) float part[STATE ? 1 : NW][SCAN_ROWS][SCAN_TILE];

    const int tiles = scan_tiles(p.D, p.G);
    const int pieces = STATE ? p.pieces - 1 : p.pieces;
    const int tile = blockIdx.x % tiles;
    const int c = (blockIdx.x / tiles) % pieces;
    const int b = blockIdx.x / tiles / pieces;
    const RowRange sq = sequence_rows(p.seq_start, b, p.S, p.rows);
    const long long t_first = (long long)c * p.length;
    if (t_first >= sq.n && c > 0) return;
    const int t_begin = (int)t_first;
    const int t_end = (int)min(t_first + p.length, (long long)sq.n);
    const ScanTile ch = scan_tile(tile, p.D, p.G);

    const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
    const int d = ch.d0 + lane, n0 = wave * NL;
    const bool own = lane < ch.count;

    float a2[NL], h[NL];
#pragma unroll
    for (int j = 0; j < NL; ++j) {
        const bool live = own && n0 + j < p.N;
        a2[j] = live ? p.A[(size_t)d * p.N + n0 + j] * LOG2E : 0.0f;
        h[j] = !STATE && live && p.h_init ? p.h_init[((size_t)b * p.D + d) * p.N + n0 + j] : 0.0f;
    }
    if (!STATE && own) {
        // join: the states of the pieces before, each decayed by the sums of the step sizes behind it
        for (int e = 0; e < c; ++e) {
            const size_t at = (size_t)b * p.pieces + e;
            const float sum = p.piece_s[at * p.D + d];
#pragma unroll
            for (int j = 0; j < NL; ++j)
                h[j] = fmaf(__builtin_amdgcn_exp2f(a2[j] * sum), h[j], p.piece_h[(at * NP + n0 + j) * p.D + d]);
        }
    }

    // staging: this thread's rows r0 + (NT / 8) i of a tile, channels c8 .. c8 + 7
    const int r0 = tid >> 3, c8 = (tid & 7) * 8;
    const T* xp = (const T*)p.x + sq.lo * p.x_stride + ch.d0 + c8;
    const T* dtp = (const T*)p.dt + sq.lo * p.dt_stride + ch.d0 + c8;
    const T* zp = (const T*)p.z + (p.z ? sq.lo * p.z_stride + ch.d0 + c8 : 0);
    T* yp = (T*)p.y + sq.lo * p.y_stride + ch.d0 + c8;
    const T* bp = (const T*)p.Bm + sq.lo * p.B_stride + ch.group * p.N;
    const T* cp = (const T*)p.Cm + sq.lo * p.C_stride + ch.group * p.N;
    float bias[8], skip[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        bias[e] = p.dt_bias && c8 + e < ch.count ? p.dt_bias[ch.d0 + c8 + e] : 0.0f;
        skip[e] = !STATE && p.Dskip && c8 + e < ch.count ? p.Dskip[ch.d0 + c8 + e] : 0.0f;
    }
    Raw8<T> xr[PASS], dtr[PASS], zr[PASS], xn[PASS], dtn[PASS], zn[PASS];
    T br[BCN], cr[BCN];
    auto load = [&](int t0) {
#pragma unroll
        for (int i = 0; i < PASS; ++i) {
            const int t = t0 + r0 + (NT / 8) * i;
            const int n = t < t_end ? ch.count - c8 : 0;
            xn[i] = load_row8(xp + t * p.x_stride, n);
            dtn[i] = load_row8(dtp + t * p.dt_stride, n);
            if (!STATE && p.z) zn[i] = load_row8(zp + t * p.z_stride, n);
        }
#pragma unroll
        for (int i = 0; i < BCN; ++i) {
            const int at = tid + NT * i, t = t0 + at / NP, n = at % NP;
            const bool live = t < t_end && n < p.N;
            br[i] = live ? bp[t * p.B_stride + n] : from_f32<T>(0.0f);
            if (!STATE) cr[i] = live ? cp[t * p.C_stride + n] : from_f32<T>(0.0f);
        }
    };

    float sums = 0.0f;                                 // of step sizes (STATE)
    load(t_begin);
    for (int t0 = t_begin; t0 < t_end; t0 += SCAN_ROWS) {
#pragma unroll
        for (int i = 0; i < PASS; ++i) {
            xr[i] = xn[i];
            dtr[i] = dtn[i];
            if (!STATE) zr[i] = zn[i];
            const int r = r0 + (NT / 8) * i;
            const bool row = t0 + r < t_end;           // past the end: decay 1, nothing added
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = dtr[i].get(e) + bias[e];
                const float s = row ? (p.softplus ? softplus_hw(v) : v) : 0.0f;
                du[r][c8 + e] = float2{s, s * xr[i].get(e)};
            }
        }
#pragma unroll
        for (int i = 0; i < BCN; ++i) {
            const int at = tid + NT * i;
            bc[at / NP][at % NP] = float2{to_f32(br[i]), STATE ? 0.0f : to_f32(cr[i])};
        }
        __syncthreads();
        if (t0 + SCAN_ROWS < t_end) load(t0 + SCAN_ROWS);
#pragma unroll 4
        for (int t = 0; t < SCAN_ROWS; ++t) {
            const float2 su = du[t][lane];
            const float2 bcv = bc[t][n0 + (lane & (NL - 1))];
            float y = 0.0f;
            for_each<NL>([&](auto jc) {
                constexpr int j = jc;
                const float a = __builtin_amdgcn_exp2f(su.x * a2[j]);
                h[j] = fmaf(a, h[j], row_broadcast<j>(bcv.x) * su.y);
                if (!STATE) y = fmaf(row_broadcast<j>(bcv.y), h[j], y);
            });
            if (STATE) sums += su.x;
            else part[wave][t][lane] = y;
        }
        __syncthreads();
        if (!STATE) {
#pragma unroll
            for (int i = 0; i < PASS; ++i) {
                const int r = r0 + (NT / 8) * i, t = t0 + r;
                Raw8<T> o;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float y = part[0][r][c8 + e];
#pragma unroll
                    for (int w = 1; w < NW; ++w) y += part[w][r][c8 + e];
                    y = fmaf(skip[e], xr[i].get(e), y);
                    if (p.z) {
                        const float z = zr[i].get(e);
                        y *= z * sigmoid_hw(z);
                    }
                    o.set(e, y);
                }
                store_row8(yp + t * p.y_stride, o, t < t_end ? ch.count - c8 : 0);
            }
        }
    }
    if (!own) return;
    if (STATE) {
        const size_t at = (size_t)b * p.pieces + c;
#pragma unroll
        for (int j = 0; j < NL; ++j) p.piece_h[(at * NP + n0 + j) * p.D + d] = h[j];
        if (wave == 0) p.piece_s[at * p.D + d] = sums;
    } else if (p.h_final && t_first + p.length >= sq.n) {      // the sequence ends in this piece
#pragma unroll
        for (int j = 0; j < NL; ++j)
            if (n0 + j < p.N) p.h_final[((size_t)b * p.D + d) * p.N + n0 + j] = h[j];
    }
}

// One row per sequence: a lane holds 4 states of a channel (one 16-byte access), LPC
// lanes a channel.  Bound by the state's HBM traffic, 8 bytes per state.
template <typename T, int LPC>
__global__ __launch_bounds__(256) void ssm_step_kernel(
    const T* __restrict__ x, long long x_stride, const T* __restrict__ dt, long long dt_stride,
    const float* __restrict__ A, const T* __restrict__ Bm, long long B_stride, const T* __restrict__ Cm,
    long long C_stride, const float* __restrict__ Dskip, const float* __restrict__ dt_bias,
    const T* __restrict__ z, long long z_stride, int B, int D, int G, int N, int softplus, float* __restrict__ h,
    T* __restrict__ y, long long y_stride)
{
    const int q = threadIdx.x % LPC, n = 4 * q;
    const long long ch = (long long)blockIdx.x * (256 / LPC) + threadIdx.x / LPC;
    const bool live = ch < (long long)B * D;           // a channel's lanes are live or not together
    const long long b = live ? ch / D : 0;
    const int d = live ? (int)(ch % D) : 0, g = d / (D / G);
    const int cnt = live ? min(max(N - n, 0), 4) : 0;
    const float v = to_f32(dt[b * dt_stride + d]) + (dt_bias ? dt_bias[d] : 0.0f);
    const float s = softplus ? softplus_hw(v) : v;
    const float xv = to_f32(x[b * x_stride + d]), u = s * xv;
    float* hp = h + ((size_t)b * D + d) * N + n;
    const float* ap = A + (size_t)d * N + n;
    const T* bp = Bm + b * B_stride + g * N + n;
    const T* cp = Cm + b * C_stride + g * N + n;
    f32x4 hv = {0, 0, 0, 0}, av = hv;
    if (cnt == 4) {
        hv = *reinterpret_cast<const f32x4_u*>(hp);
        av = *reinterpret_cast<const f32x4_u*>(ap);
    } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
            if (j < cnt) { hv[j] = hp[j]; av[j] = ap[j]; }
    }
    float o = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float bv = j < cnt ? to_f32(bp[j]) : 0.0f, cv = j < cnt ? to_f32(cp[j]) : 0.0f;
        hv[j] = fmaf(__builtin_amdgcn_exp2f(s * (av[j] * LOG2E)), hv[j], u * bv);
        o = fmaf(cv, hv[j], o);
    }
    if (cnt == 4) {
        *reinterpret_cast<f32x4_u*>(hp) = hv;
    } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
            if (j < cnt) hp[j] = hv[j];
    }
#pragma unroll
    for (int off = LPC / 2; off > 0; off >>= 1) o += __shfl_xor(o, off, 64);
    if (live && q == 0) {
        if (Dskip) o = fmaf(Dskip[d], xv, o);
        if (z) {
            const float zv = to_f32(z[b * z_stride + d]);
            o *= zv * sigmoid_hw(zv);
        }
        y[b * y_stride + d] = from_f32<T>(o);
    }
}

// Pieces of a sequence.  One piece does the least work (the pieces' end states cost
// most of the scan a second time), so a sequence is cut only where its workgroups
// leave compute units idle.
struct FwdPlan { int pieces, length; };
FwdPlan plan(int B, int S, int D, int G) {
    (void)B; (void)D; (void)G;
    return FwdPlan{1, (S + SCAN_ROWS - 1) / SCAN_ROWS * SCAN_ROWS};
}
size_t piece_h_elems(const FwdPlan& f, int B, int D, int N) {
    return (size_t)B * f.pieces * scan_padded_states(N) * D;
}

template <typename T>
hipError_t fwd_t(const ScanArgs& a) {
    const FwdPlan f = plan(a.B, a.S, a.D, a.G);
    FwdParams p = {};
    p.x = a.x; p.dt = a.dt; p.Bm = a.Bm; p.Cm = a.Cm; p.z = a.z;
    p.x_stride = a.x_stride; p.dt_stride = a.dt_stride; p.B_stride = a.B_stride; p.C_stride = a.C_stride;
    p.z_stride = a.z_stride; p.y_stride = a.y_stride;
    p.A = a.A; p.Dskip = a.Dskip; p.dt_bias = a.dt_bias; p.seq_start = a.seq_start; p.h_init = a.h_init;
    p.S = a.S; p.rows = a.rows; p.D = a.D; p.G = a.G; p.N = a.N; p.softplus = a.softplus;
    p.pieces = f.pieces; p.length = f.length;
    p.y = a.y; p.h_final = a.h_final;
    p.piece_h = a.ws; p.piece_s = a.ws + piece_h_elems(f, a.B, a.D, a.N);
    const unsigned per = (unsigned)scan_tiles(a.D, a.G) * a.B;
#define SCAN_CALL(NW, NL)                                                                                              \
    if (f.pieces > 1)                                                                                                  \
        hipLaunchKernelGGL((scan_fwd_kernel<T, NW, NL, true>), dim3(per * (f.pieces - 1)), dim3(64 * NW), 0, a.stream, \
                           p);                                                                                         \
    hipLaunchKernelGGL((scan_fwd_kernel<T, NW, NL, false>), dim3(per * f.pieces), dim3(64 * NW), 0, a.stream, p)
    SCAN_DISPATCH_N(a.N, SCAN_CALL)
#undef SCAN_CALL
    return hipGetLastError();
}

template <typename T>
hipError_t step_t(const ScanArgs& a) {
    const long long ch = (long long)a.B * a.D;
#define STEP_CALL(LPC)                                                                                                \
    hipLaunchKernelGGL((ssm_step_kernel<T, LPC>), dim3((unsigned)((ch * LPC + 255) / 256)), dim3(256), 0, a.stream,   \
                       (const T*)a.x, a.x_stride, (const T*)a.dt, a.dt_stride, a.A, (const T*)a.Bm, a.B_stride,       \
                       (const T*)a.Cm, a.C_stride, a.Dskip, a.dt_bias, (const T*)a.z, a.z_stride, a.B, a.D, a.G, a.N, \
                       a.softplus, a.h_final, (T*)a.y, a.y_stride)
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

}  // namespace

size_t scan_fwd_workspace_bytes(int B, int S, int D, int G, int N) {
    const FwdPlan f = plan(B, S, D, G);
    if (f.pieces == 1) return 0;
    return (piece_h_elems(f, B, D, N) + (size_t)B * f.pieces * D) * sizeof(float);
}

hipError_t launch_scan_fwd(const ScanArgs& a) {
    return a.dtype == MLSTM_BF16 ? fwd_t<bf16>(a) : fwd_t<float>(a);
}
hipError_t launch_ssm_step(const ScanArgs& a) {
    return a.dtype == MLSTM_BF16 ? step_t<bf16>(a) : step_t<float>(a);
}

}  // namespace mlstm
