// Backward of the selective state space scan.
//
// With s_t the step size, u_t = s_t x_t, a_t = exp(s_t A), ds_t the gradient of the
// read-out (dy_t, or dy_t z_t sigmoid(z_t)), per channel and state:
//   G_t = C_t ds_t + a_{t+1} G_{t+1}               (gradient of h_t)
//   dC_t = sum_d ds_t h_t        dB_t = sum_d G_t u_t
//   du_t = sum_n G_t B_t         w_t = G_t a_t h_{t-1}
//   ds'_t (of the step size) = x_t du_t + sum_n A w_t
//   dA = sum_t s_t w_t           dh_init = a_0 G_0
// The states are needed in reverse order.  A first kernel runs forward and keeps one
// state in every BWD_ROWS rows (4 bytes per state and BWD_ROWS rows through HBM, at N = 16 as
// much as one fp32 activation); the second goes back over tiles of BWD_ROWS rows,
// recomputes a tile's rows from the state in front of it and keeps their decays and
// states in registers.  Arithmetic bounds both: per (row, channel, state) an exponential
// and 3 vector instructions forward, twice, and about 11 back.
//
// The sums over channels (dB, dC) run across the lanes: each wave leaves the products
// of two rows in LDS and adds them with wide reads, one addition per product, which
// costs a fifth of a lane-exchange tree.  A tile of channels writes its sums to the
// workspace, and a last kernel adds the tiles (no atomics).
//
// A sequence that fills too little of the chip is cut into pieces.  The first kernel then
// starts every piece but a sequence's first from zero and also leaves the gradient
//   R = sum_t (prod_{r <= t} a_r) C_t ds_t
// that a piece passes to the rows before it, and sums of step sizes s: what enters a
// piece reaches the state k rows on by the factor exp(A (s_0 + ... + s_k)), so the second
// kernel adds it to the kept states, and joins the R of the pieces behind.
#include "scan_common.h"
#include <stdlib.h>

namespace mlstm {
namespace {

constexpr int BWD_ROWS = 16;

struct BwdParams {
    const void* x; const void* dt; const void* Bm; const void* Cm; const void* z; const void* dy;
    long long x_stride, dt_stride, B_stride, C_stride, z_stride, dy_stride;
    const float* A; const float* Dskip; const float* dt_bias;
    const float* h_init; const float* dh_final;
    Pieces pieces;                       // their length is a multiple of BWD_ROWS
    int D, G, N, softplus;
    void* dx; void* ddt; void* dz; void* dB; void* dC;
    long long dx_stride, ddt_stride, dz_stride, dB_stride, dC_stride;
    float* dA; float* dskip; float* dbias; float* dh_init;
    float* state;                        // [slot][NP][D]: the state in front of each tile of rows
    float* before;                       // [slot][D]: sum of the step sizes from the piece's start to there
    float* bc;                           // [channel tile][row][2 NP]: its dB and dC
    float* sums;                         // [piece][NP + 2][D]: dA, dskip, dbias
    float* piece_h; float* piece_g;      // [piece][NP][D]: end state and R
    float* piece_s;                      // [piece][D]: sum of the step sizes
};

// where a sequence's tiles of rows start among the slots of `state`: no two sequences share
// one, and rows / BWD_ROWS + B slots hold them all
__device__ __forceinline__ int first_slot(const RowRange& sq, int b) { return sq.lo / BWD_ROWS + b; }

// The piece, channel tile and rows of a workgroup, and its threads' part in staging
// a tile of rows: thread -> row tid / 16 (+ NT / 16 i), channels 4 (tid % 16) .. + 3.
template <typename T, int NW, int NL>
struct Work {
    static constexpr int NT = 64 * NW, NP = NW * NL;
    static constexpr int PASS = BWD_ROWS * 16 / NT;
    static constexpr int BCN = BWD_ROWS * NP / NT > 0 ? BWD_ROWS * NP / NT : 1;
    struct Lds {
        float2 su[BWD_ROWS][SCAN_TILE];                // step size, step size * x
        float ds[BWD_ROWS][SCAN_TILE];
        float2 bc[BWD_ROWS][NP];                       // B, C
    };

    const BwdParams& p;
    int b, c, number, tile, tid, lane, wave, d, n0, t_begin, t_end, r0, c4, slot;
    RowRange sq;
    ScanTile ch;
    bool own, live, last;
    const T *xp, *dtp, *zp, *dyp, *bp, *cp;
    float bias[4];
    Raw4<T> x[PASS], z[PASS], dy[PASS];                // the staged tile's
    float v[PASS][4];                                  // and its dt + bias
    Raw4<T> xn[PASS], vn[PASS], zn[PASS], dyn[PASS];   // the next tile's
    T bn[BCN], cn[BCN];

    __device__ __forceinline__ explicit Work(const BwdParams& p_) : p(p_) {
        const int tiles = scan_tiles(p.D, p.G);
        tile = blockIdx.x % tiles;
        number = blockIdx.x / tiles;
        const Pieces::At at = p.pieces.at(number);
        b = at.b;
        c = at.c;
        sq = p.pieces.sequence(b);
        const long long first = (long long)c * p.pieces.length;
        live = first < sq.n || c == 0;
        last = first + p.pieces.length >= sq.n;        // the sequence ends in this piece
        t_begin = live ? (int)first : 0;
        t_end = !live ? 0 : last ? sq.n : t_begin + p.pieces.length;
        ch = scan_tile(tile, p.D, p.G);
        tid = threadIdx.x;
        lane = tid & 63;
        wave = wave_id();
        d = ch.d0 + lane;
        n0 = wave * NL;
        own = lane < ch.count;
        slot = first_slot(sq, b);
        r0 = tid >> 4;
        c4 = (tid & 15) * 4;
        const long long lo = sq.lo;
        xp = (const T*)p.x + lo * p.x_stride + ch.d0 + c4;
        dtp = (const T*)p.dt + lo * p.dt_stride + ch.d0 + c4;
        zp = (const T*)p.z + (p.z ? lo * p.z_stride + ch.d0 + c4 : 0);
        dyp = (const T*)p.dy + lo * p.dy_stride + ch.d0 + c4;
        bp = (const T*)p.Bm + lo * p.B_stride + ch.group * p.N;
        cp = (const T*)p.Cm + lo * p.C_stride + ch.group * p.N;
#pragma unroll
        for (int e = 0; e < 4; ++e) bias[e] = p.dt_bias && c4 + e < ch.count ? p.dt_bias[ch.d0 + c4 + e] : 0.0f;
    }

    // issue the loads of the tile of rows at t0
    template <bool GRAD>
    __device__ __forceinline__ void load(int t0) {
#pragma unroll
        for (int i = 0; i < PASS; ++i) {
            const int t = t0 + r0 + (NT / 16) * i;
            const int n = t < t_end ? ch.count - c4 : 0;
            xn[i] = load_row4(xp + t * p.x_stride, n);
            vn[i] = load_row4(dtp + t * p.dt_stride, n);
            if (GRAD) {
                dyn[i] = load_row4(dyp + t * p.dy_stride, n);
                if (p.z) zn[i] = load_row4(zp + t * p.z_stride, n);
            }
        }
#pragma unroll
        for (int i = 0; i < BCN; ++i) {
            const int at = tid + NT * i, t = t0 + at / NP, n = at % NP;
            const bool ok = at < BWD_ROWS * NP && t < t_end && n < p.N;
            bn[i] = ok ? bp[t * p.B_stride + n] : from_f32<T>(0.0f);
            if (GRAD) cn[i] = ok ? cp[t * p.C_stride + n] : from_f32<T>(0.0f);
        }
    }

    // what has been loaded becomes the staged tile; rows past the end get step size 0
    // (decay 1) and no input or gradient
    template <bool GRAD>
    __device__ __forceinline__ void put(Lds& l, int t0) {
#pragma unroll
        for (int i = 0; i < PASS; ++i) {
            x[i] = xn[i];
            const int r = r0 + (NT / 16) * i;
            const bool row = t0 + r < t_end;
            if (GRAD) {
                dy[i] = dyn[i];
                if (p.z) z[i] = zn[i];
            }
            float sz[4], u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) sz[e] = v[i][e] = vn[i].get(e) + bias[e];
            if (p.softplus)
#pragma unroll
                for (int e = 0; e < 4; ++e) sz[e] = softplus_hw(sz[e]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                u[e] = row ? sz[e] * x[i].get(e) : 0.0f;
                sz[e] = row ? sz[e] : 0.0f;
            }
            f32x4* to = reinterpret_cast<f32x4*>(&l.su[r][c4]);
            to[0] = f32x4{sz[0], u[0], sz[1], u[1]};
            to[1] = f32x4{sz[2], u[2], sz[3], u[3]};
            if (GRAD) {
                f32x4 g;
#pragma unroll
                for (int e = 0; e < 4; ++e) g[e] = dy[i].get(e);
                if (p.z)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float zv = z[i].get(e);
                        g[e] *= zv * sigmoid_hw(zv);
                    }
                *reinterpret_cast<f32x4*>(&l.ds[r][c4]) = g;
            }
        }
#pragma unroll
        for (int i = 0; i < BCN; ++i) {
            const int at = tid + NT * i;
            if (at < BWD_ROWS * NP) l.bc[at / NP][at % NP] = float2{to_f32(bn[i]), GRAD ? to_f32(cn[i]) : 0.0f};
        }
    }
};

// Forward over a piece: the states in front of its tiles of rows.  CUT: sequences have several
// pieces; then also the sums of step sizes, the end state and R.
template <typename T, int NW, int NL, bool CUT>
__global__ __launch_bounds__(64 * NW) void scan_bwd_states_kernel(const BwdParams p)
{
    typedef Work<T, NW, NL> W;
    __shared__ __align__(16) typename W::Lds lds;
    W w(p);
    if (!w.live) return;
    float a2[NL], h[NL], prod[NL], R[NL], sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NL; ++j) {
        const bool live = w.own && w.n0 + j < p.N;
        a2[j] = live ? p.A[(size_t)w.d * p.N + w.n0 + j] * LOG2E : 0.0f;
        h[j] = live && w.c == 0 && p.h_init ? p.h_init[((size_t)w.b * p.D + w.d) * p.N + w.n0 + j] : 0.0f;
        R[j] = 0.0f;
        prod[j] = 1.0f;
    }
    if (w.t_begin < w.t_end) w.template load<CUT>(w.t_begin);
    for (int t0 = w.t_begin; t0 < w.t_end; t0 += BWD_ROWS) {
        if (w.own) {
            const size_t slot = w.slot + t0 / BWD_ROWS;
#pragma unroll
            for (int j = 0; j < NL; ++j) p.state[(slot * W::NP + w.n0 + j) * p.D + w.d] = h[j];
            if (CUT && w.wave == 0) p.before[slot * p.D + w.d] = sum;
        }
        if (!CUT && t0 + BWD_ROWS >= w.t_end) break;   // the last tile's end state is not needed
        w.template put<CUT>(lds, t0);
        __syncthreads();
        if (t0 + BWD_ROWS < w.t_end) w.template load<CUT>(t0 + BWD_ROWS);
#pragma unroll 4
        for (int t = 0; t < BWD_ROWS; ++t) {
            const float2 su = lds.su[t][w.lane];
            const float ds = CUT ? lds.ds[t][w.lane] : 0.0f;
            const float2 bcv = lds.bc[t][w.n0 + (w.lane & (NL - 1))];
            sum += su.x;
            for_each<NL>([&](auto jc) {
                constexpr int j = jc;
                const float a = __builtin_amdgcn_exp2f(su.x * a2[j]);
                h[j] = fmaf(a, h[j], row_broadcast<j>(bcv.x) * su.y);
                if (CUT) {
                    prod[j] *= a;
                    R[j] = fmaf(prod[j], row_broadcast<j>(bcv.y) * ds, R[j]);
                }
            });
        }
        __syncthreads();
    }
    if (!CUT || !w.own) return;
    const size_t at = w.number;
#pragma unroll
    for (int j = 0; j < NL; ++j) {
        p.piece_h[(at * W::NP + w.n0 + j) * p.D + w.d] = h[j];
        p.piece_g[(at * W::NP + w.n0 + j) * p.D + w.d] = R[j];
    }
    if (w.wave == 0) p.piece_s[at * p.D + w.d] = sum;
}

template <typename T, int NW, int NL, bool CUT>
__global__ __launch_bounds__(64 * NW, 2) void scan_bwd_kernel(const BwdParams p)
{
    typedef Work<T, NW, NL> W;
    constexpr int NT = W::NT, NP = W::NP, PASS = W::PASS;
    constexpr int RED = SCAN_TILE + 4;                 // padded row of the sums over channels
    __shared__ __align__(16) typename W::Lds lds;
    __shared__ __align__(16) float part[NW][3][BWD_ROWS][SCAN_TILE];   // o, du, sum_n A w by wave
    __shared__ __align__(16) float red[NW][8][RED];
    __shared__ __align__(16) float bcout[BWD_ROWS][2 * NP];
    W w(p);
    if (!w.live) return;
    const int lane = w.lane, d = w.d, n0 = w.n0;

    float a2[NL], G[NL], dA[NL], enter[NL];
    // the gradient that reaches the piece's last state, and the state that enters it (of a
    // sequence's first piece the kept states already have it)
#pragma unroll
    for (int j = 0; j < NL; ++j) {
        const bool live = w.own && n0 + j < p.N;
        a2[j] = live ? p.A[(size_t)d * p.N + n0 + j] * LOG2E : 0.0f;
        G[j] = live && p.dh_final ? p.dh_final[((size_t)w.b * p.D + d) * p.N + n0 + j] : 0.0f;
        dA[j] = enter[j] = 0.0f;
    }
    if (CUT && w.own) {
#pragma unroll 4
        for (int e = w.number - w.c; e < w.number; ++e) {
            const float sum = p.piece_s[(size_t)e * p.D + d];
#pragma unroll
            for (int j = 0; j < NL; ++j)
                enter[j] = fmaf(__builtin_amdgcn_exp2f(a2[j] * sum), enter[j], p.piece_h[((size_t)e * NP + n0 + j) * p.D + d]);
        }
#pragma unroll 4
        for (int e = w.number - w.c + (w.sq.n - 1) / p.pieces.length; e > w.number; --e) {
            const float sum = p.piece_s[(size_t)e * p.D + d];
#pragma unroll
            for (int j = 0; j < NL; ++j)
                G[j] = fmaf(__builtin_amdgcn_exp2f(a2[j] * sum), G[j], p.piece_g[((size_t)e * NP + n0 + j) * p.D + d]);
        }
    }

    float skip[4], dskip[4], dbias[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        skip[e] = p.Dskip && w.c4 + e < w.ch.count ? p.Dskip[w.ch.d0 + w.c4 + e] : 0.0f;
        dskip[e] = dbias[e] = 0.0f;
    }
    const long long lo = w.sq.lo;
    const int c0 = w.ch.d0 + w.c4;
    T* dxp = (T*)p.dx + lo * p.dx_stride + c0;
    T* ddtp = (T*)p.ddt + lo * p.ddt_stride + c0;
    T* dzp = (T*)p.dz + (p.z ? lo * p.dz_stride + c0 : 0);
    float* bcp = p.bc + ((size_t)w.tile * p.pieces.rows + lo) * (2 * NP);

    // back, tile by tile
    const int back = w.t_begin + (w.t_end - w.t_begin - 1) / BWD_ROWS * BWD_ROWS;
    if (w.t_begin < w.t_end) w.template load<true>(back);
    for (int t0 = back; t0 >= w.t_begin && w.t_begin < w.t_end; t0 -= BWD_ROWS) {
        // the state in front of the tile
        float h0[NL];
        const size_t slot = w.slot + t0 / BWD_ROWS;
        const float since = CUT && w.c > 0 && w.own ? p.before[slot * p.D + d] : 0.0f;
#pragma unroll
        for (int j = 0; j < NL; ++j) h0[j] = w.own ? p.state[(slot * NP + n0 + j) * p.D + d] : 0.0f;
        w.template put<true>(lds, t0);
        __syncthreads();
        if (t0 > w.t_begin) w.template load<true>(t0 - BWD_ROWS);
        for_each<NL / 4>([&](auto qc) {                // four states at a time
            constexpr int q = 4 * qc;
            float h[BWD_ROWS + 1][4], a[BWD_ROWS][4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                h[0][j] = CUT ? fmaf(__builtin_amdgcn_exp2f(a2[q + j] * since), enter[q + j], h0[q + j]) : h0[q + j];
#pragma unroll
            for (int t = 0; t < BWD_ROWS; ++t) {
                const float2 su = lds.su[t][lane];
                const float2 bcv = lds.bc[t][n0 + (lane & (NL - 1))];
                float o = 0.0f;
                for_each<4>([&](auto jc) {
                    constexpr int j = jc;
                    a[t][j] = __builtin_amdgcn_exp2f(su.x * a2[q + j]);
                    h[t + 1][j] = fmaf(a[t][j], h[t][j], row_broadcast<q + j>(bcv.x) * su.y);
                    o = fmaf(row_broadcast<q + j>(bcv.y), h[t + 1][j], o);
                });
                part[w.wave][0][t][lane] = q == 0 ? o : part[w.wave][0][t][lane] + o;
            }
#pragma unroll
            for (int t = BWD_ROWS - 1; t >= 0; --t) {
                const float2 su = lds.su[t][lane];
                const float ds = lds.ds[t][lane];
                const float2 bcv = lds.bc[t][n0 + (lane & (NL - 1))];
                float du = 0.0f, aw = 0.0f;
                for_each<4>([&](auto jc) {
                    constexpr int j = jc;
                    const float g = fmaf(row_broadcast<q + j>(bcv.y), ds, G[q + j]);
                    du = fmaf(row_broadcast<q + j>(bcv.x), g, du);
                    const float gw = g * (a[t][j] * h[t][j]);
                    aw = fmaf(a2[q + j], gw, aw);
                    dA[q + j] = fmaf(su.x, gw, dA[q + j]);
                    G[q + j] = a[t][j] * g;
                    red[w.wave][j][lane] = g * su.y;
                    red[w.wave][4 + j][lane] = ds * h[t + 1][j];
                });
                part[w.wave][1][t][lane] = q == 0 ? du : part[w.wave][1][t][lane] + du;
                part[w.wave][2][t][lane] = q == 0 ? aw : part[w.wave][2][t][lane] + aw;
                // 8 sums over 64 channels (dB, dC; 4 states): 8 lanes a sum
                __builtin_amdgcn_wave_barrier();
                const float* at = &red[w.wave][lane >> 3][(lane & 7) * 8];
                const f32x4 s4 = *reinterpret_cast<const f32x4*>(at) + *reinterpret_cast<const f32x4*>(at + 4);
                float s1 = (s4[0] + s4[1]) + (s4[2] + s4[3]);
                s1 += __shfl_xor(s1, 1, 64);
                s1 += __shfl_xor(s1, 2, 64);
                s1 += __shfl_xor(s1, 4, 64);
                if ((lane & 7) == 0) {
                    const int k = lane >> 3;           // dB or dC, state
                    bcout[t][(k >> 2) * NP + n0 + q + (k & 3)] = s1;
                }
                __builtin_amdgcn_wave_barrier();
            }
        });
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PASS; ++i) {
            const int r = w.r0 + (NT / 16) * i, t = t0 + r;
            const int n = t < w.t_end ? w.ch.count - w.c4 : 0;
            f32x4 sum[3];                              // o, du, sum_n A w
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                sum[q] = *reinterpret_cast<const f32x4*>(&part[0][q][r][w.c4]);
#pragma unroll
                for (int k = 1; k < NW; ++k) sum[q] += *reinterpret_cast<const f32x4*>(&part[k][q][r][w.c4]);
            }
            const f32x4 sa = *reinterpret_cast<const f32x4*>(&lds.su[r][w.c4]);
            const f32x4 sb = *reinterpret_cast<const f32x4*>(&lds.su[r][w.c4 + 2]);
            const f32x4 ds = *reinterpret_cast<const f32x4*>(&lds.ds[r][w.c4]);
            const float sz[4] = {sa[0], sa[2], sb[0], sb[2]};
            Raw4<T> dx, ddt, dz;
            float g[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                dx.set(e, fmaf(sz[e], sum[1][e], skip[e] * ds[e]));
                g[e] = fmaf(sum[2][e], LN2, w.x[i].get(e) * sum[1][e]);       // a2 carries log2(e)
            }
            if (p.softplus)
#pragma unroll
                for (int e = 0; e < 4; ++e) g[e] *= sigmoid_hw(w.v[i][e]);
            if (p.z)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float z = w.z[i].get(e), sg = sigmoid_hw(z);
                    dz.set(e, w.dy[i].get(e) * fmaf(skip[e], w.x[i].get(e), sum[0][e]) * (sg * (1.0f + z * (1.0f - sg))));
                }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                ddt.set(e, g[e]);
                if (e < n) {
                    dskip[e] = fmaf(ds[e], w.x[i].get(e), dskip[e]);
                    dbias[e] += g[e];
                }
            }
            store_row4(dxp + t * p.dx_stride, dx, n);
            store_row4(ddtp + t * p.ddt_stride, ddt, n);
            if (p.z) store_row4(dzp + t * p.dz_stride, dz, n);
        }
        for (int at = w.tid; at < BWD_ROWS * 2 * NP; at += NT) {
            const int r = at / (2 * NP);
            if (t0 + r < w.t_end) bcp[(size_t)(t0 + r) * (2 * NP) + at % (2 * NP)] = bcout[r][at % (2 * NP)];
        }
        __syncthreads();
    }

    // the piece's sums; those of dskip and dbias lie with the NT / 16 threads of a channel group
    float* so = p.sums + (size_t)w.number * (NP + 2) * p.D;
    if (w.own) {
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            so[(size_t)(n0 + j) * p.D + d] = dA[j];
            if (w.c == 0 && p.dh_init && n0 + j < p.N) p.dh_init[((size_t)w.b * p.D + d) * p.N + n0 + j] = G[j];
        }
    }
    float* sm = &part[0][0][0][0];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        sm[w.r0 * SCAN_TILE + w.c4 + e] = dskip[e];
        sm[(NT / 16 + w.r0) * SCAN_TILE + w.c4 + e] = dbias[e];
    }
    __syncthreads();
    if (w.tid < SCAN_TILE && w.own) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float s = 0.0f;
            for (int r = 0; r < NT / 16; ++r) s += sm[(k * (NT / 16) + r) * SCAN_TILE + lane];
            so[(size_t)(NP + k) * p.D + d] = s;
        }
    }
}

// dA, dskip and dbias: sums over the pieces, 64 channels of one of them per workgroup
__global__ __launch_bounds__(1024) void scan_bwd_sums_kernel(const BwdParams p, int NP)
{
    __shared__ float sm[16][SCAN_TILE];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int d = blockIdx.x * SCAN_TILE + lane, j = blockIdx.y < p.N ? blockIdx.y : NP + blockIdx.y - p.N;
    float s = 0.0f;
    const int count = p.pieces.count();
    for (int i = wave; i < count; i += 16) {
        const Pieces::At at = p.pieces.at(i);
        const bool there = at.c == 0 || (long long)at.c * p.pieces.length < p.pieces.sequence(at.b).n;
        if (there && d < p.D) s += p.sums[((size_t)i * (NP + 2) + j) * p.D + d];
    }
    sm[wave][lane] = s;
    __syncthreads();
    if (wave != 0 || d >= p.D) return;
#pragma unroll
    for (int w = 1; w < 16; ++w) s += sm[w][lane];
    if (j < p.N) p.dA[(size_t)d * p.N + j] = s;
    else if (j == NP) { if (p.dskip) p.dskip[d] = s; }
    else if (p.dbias) p.dbias[d] = s;
}

// dB, dC: sums over the channel tiles of a group, one thread per element
template <typename T>
__global__ __launch_bounds__(256) void scan_bwd_bc_kernel(const BwdParams p, int NP)
{
    const int b = blockIdx.y;
    const RowRange sq = p.pieces.sequence(b);
    const int width = 2 * p.G * p.N;
    const long long at = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long t = at / width;
    if (t >= sq.n) return;
    const int e = (int)(at % width), k = e / (p.G * p.N), g = e / p.N % p.G, n = e % p.N;
    const long long row = sq.lo + t;
    const int per = scan_tiles(p.D, p.G) / p.G;
    const float* src = p.bc + ((size_t)g * per * p.pieces.rows + row) * (2 * NP) + k * NP + n;
    float s = 0.0f;
    for (int i = 0; i < per; ++i) s += src[(size_t)i * p.pieces.rows * (2 * NP)];
    T* out = k == 0 ? (T*)p.dB + row * p.dB_stride : (T*)p.dC + row * p.dC_stride;
    out[g * p.N + n] = from_f32<T>(s);
}

int piece_rows(int S, int rows, int D, int G) {
    const long long groups = (long long)scan_tiles(D, G) * ((rows + S - 1) / S);
    const int whole = (S + BWD_ROWS - 1) / BWD_ROWS * BWD_ROWS;
    int n = 1; if (getenv("SCANBK")) n = atoi(getenv("SCANBK"));
    return (((S + n - 1) / n + 15) / 16 * 16);
}

struct BwdPlan {
    Pieces pieces;
    bool cut;
    size_t state, before, bc, sums, piece_h, piece_g, piece_s, total;      // offsets and size in floats
};
BwdPlan plan(const int* seq_start, int B, int S, int rows, int D, int G, int N) {
    const size_t NP = scan_padded_states(N);
    BwdPlan f = {};
    f.pieces = make_pieces(seq_start, B, S, rows, piece_rows(S, rows, D, G));
    f.cut = f.pieces.length < S;
    size_t at = 0;
    auto take = [&](size_t n) { const size_t o = at; at += (n + 63) / 64 * 64; return o; };
    // as many tiles of rows and pieces as packed sequences may need (also where they are not
    // packed: a workspace's size does not depend on seq_start)
    const size_t slots = (size_t)rows / BWD_ROWS + B, parts = (size_t)rows / f.pieces.length + B;
    f.state = take(slots * NP * D);
    f.bc = take((size_t)scan_tiles(D, G) * rows * 2 * NP);
    f.sums = take(parts * (NP + 2) * D);
    if (f.cut) {
        f.before = take(slots * D);
        f.piece_h = take(parts * NP * D);
        f.piece_g = take(parts * NP * D);
        f.piece_s = take(parts * D);
    }
    f.total = at;
    return f;
}

template <typename T>
hipError_t bwd_t(const ScanArgs& a) {
    const BwdPlan f = plan(a.seq_start, a.B, a.S, a.rows, a.D, a.G, a.N);
    const int NP = scan_padded_states(a.N);
    BwdParams p = {};
    p.x = a.x; p.dt = a.dt; p.Bm = a.Bm; p.Cm = a.Cm; p.z = a.z; p.dy = a.dy;
    p.x_stride = a.x_stride; p.dt_stride = a.dt_stride; p.B_stride = a.B_stride; p.C_stride = a.C_stride;
    p.z_stride = a.z_stride; p.dy_stride = a.dy_stride;
    p.A = a.A; p.Dskip = a.Dskip; p.dt_bias = a.dt_bias; p.h_init = a.h_init; p.dh_final = a.dh_final;
    p.pieces = f.pieces; p.D = a.D; p.G = a.G; p.N = a.N; p.softplus = a.softplus;
    p.dx = a.grad_x; p.ddt = a.grad_dt; p.dz = a.grad_z; p.dB = a.grad_B; p.dC = a.grad_C;
    p.dx_stride = a.grad_x_stride; p.ddt_stride = a.grad_dt_stride; p.dz_stride = a.grad_z_stride;
    p.dB_stride = a.grad_B_stride; p.dC_stride = a.grad_C_stride;
    p.dA = a.grad_A; p.dskip = a.grad_Dskip; p.dbias = a.grad_dt_bias; p.dh_init = a.grad_h;
    p.state = a.ws + f.state; p.before = a.ws + f.before; p.bc = a.ws + f.bc; p.sums = a.ws + f.sums;
    p.piece_h = a.ws + f.piece_h; p.piece_g = a.ws + f.piece_g; p.piece_s = a.ws + f.piece_s;
    const dim3 grid((unsigned)scan_tiles(a.D, a.G) * f.pieces.count());
#define SCAN_LAUNCH(NW, NL, CUT)                                                                               \
    hipLaunchKernelGGL((scan_bwd_states_kernel<T, NW, NL, CUT>), grid, dim3(64 * NW), 0, a.stream, p);         \
    hipLaunchKernelGGL((scan_bwd_kernel<T, NW, NL, CUT>), grid, dim3(64 * NW), 0, a.stream, p)
#define SCAN_CALL(NW, NL)                         \
    if (f.cut) { SCAN_LAUNCH(NW, NL, true); }     \
    else { SCAN_LAUNCH(NW, NL, false); }
    SCAN_DISPATCH_N(a.N, SCAN_CALL)
#undef SCAN_CALL
#undef SCAN_LAUNCH
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(scan_bwd_sums_kernel, dim3((a.D + 63) / 64, a.N + 2), dim3(1024), 0, a.stream, p, NP);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const long long elems = (long long)a.S * 2 * a.G * a.N;
    hipLaunchKernelGGL(scan_bwd_bc_kernel<T>, dim3((unsigned)((elems + 255) / 256), a.B), dim3(256), 0, a.stream, p, NP);
    return hipGetLastError();
}

}  // namespace

size_t scan_bwd_workspace_bytes(int B, int S, int rows, int D, int G, int N) {
    return plan(nullptr, B, S, rows, D, G, N).total * sizeof(float);
}

hipError_t launch_scan_bwd(const ScanArgs& a) {
    return a.dtype == MLSTM_BF16 ? bwd_t<bf16>(a) : bwd_t<float>(a);
}

}  // namespace mlstm
