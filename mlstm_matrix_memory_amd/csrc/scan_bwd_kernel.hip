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
// state in every KEEP = 8 rows (4 bytes per state and 8 rows through HBM, at N = 16 as much as
// two fp32 activations, written and read); the second goes back over tiles of BWD_ROWS = 16
// rows, recomputes every 8 rows from the state in front of them and keeps their decays
// and states in registers.  Arithmetic bounds both: per (row, channel, state) an exponential
// and 3 vector instructions forward, twice, and about 11 back.
//
// In the second kernel a lane holds 4 states (or several times 4, one after the other)
// of a channel, and LPC = NP / 4, at most 4, neighbouring lanes a channel.  The sums over
// a channel's states (read-out, du, sum_n A w) then take two additions with the DPP lane
// permutation, and the sums over the wave's channels (dB, dC) run as a
// halving exchange between lanes: the permlane swaps add two values in one addition.  Both
// stay in registers, free to overlap with the next rows' arithmetic; through LDS, with the
// states of a channel in four waves, the same kernel took 1.4 times as long, waiting for LDS.
// A tile of channels writes its sums to the workspace, and a last kernel adds the
// tiles (no atomics).
//
// A sequence that fills too little of the chip is cut into pieces.  The first kernel then
// starts every piece but a sequence's first from zero and also leaves the gradient
//   R = sum_t (prod_{r <= t} a_r) C_t ds_t
// that a piece passes to the rows before it, and sums of step sizes s: what enters a
// piece reaches the state k rows on by the factor exp(A (s_0 + ... + s_k)), so the second
// kernel adds it to the kept states, and joins the R of the pieces behind.
#include "scan_common.h"

namespace mlstm {
namespace {

constexpr int BWD_ROWS = 16;                     // rows staged at a time
constexpr int KEEP = 8;                          // rows between kept states

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
    float* state;                        // [slot][NP][D]: the state in front of every KEEP rows
    float* before;                       // [slot][D]: sum of the step sizes from the piece's start to there
    float* bc;                           // [channel tile][row][2 NP]: its dB and dC
    float* sums;                         // [piece][NP + 2][D]: dA, dskip, dbias
    float* piece_h; float* piece_g;      // [piece][NP][D]: end state and R
    float* piece_s;                      // [piece][D]: sum of the step sizes
};

// where a sequence's kept states start among the slots of `state`: no two sequences share a
// slot, and rows / KEEP + B slots hold them all
__device__ __forceinline__ int first_slot(const RowRange& sq, int b) { return sq.lo / KEEP + b; }

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
        float bs[BWD_ROWS][NP], cs[BWD_ROWS][NP];      // B, C
    };

    const BwdParams& p;
    int b, c, number, tile, tid, lane, wave, d, n0, t_begin, t_end, r0, c4, nc, slot;
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
        nc = min(ch.count - c4, 4);
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
            if (at < BWD_ROWS * NP) {
                l.bs[at / NP][at % NP] = to_f32(bn[i]);
                if (GRAD) l.cs[at / NP][at % NP] = to_f32(cn[i]);
            }
        }
    }
};

// Forward over a piece: the states in front of every KEEP rows.  CUT: sequences have several
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
        w.template put<CUT>(lds, t0);
        __syncthreads();
        if (t0 + BWD_ROWS < w.t_end) w.template load<CUT>(t0 + BWD_ROWS);
        for (int half = 0; half < BWD_ROWS; half += KEEP) {
            if (w.own && t0 + half < w.t_end) {
                const size_t slot = w.slot + (t0 + half) / KEEP;
#pragma unroll
                for (int j = 0; j < NL; ++j) p.state[(slot * W::NP + w.n0 + j) * p.D + w.d] = h[j];
                if (CUT && w.wave == 0) p.before[slot * p.D + w.d] = sum;
            }
#pragma unroll
            for (int t = 0; t < KEEP; ++t) {
                const float2 su = lds.su[half + t][w.lane];
                const float ds = CUT ? lds.ds[half + t][w.lane] : 0.0f;
                const int at = w.n0 + (w.lane & (NL - 1));
                const float bv = lds.bs[half + t][at], cv = CUT ? lds.cs[half + t][at] : 0.0f;
                sum += su.x;
                for_each<NL>([&](auto jc) {
                    constexpr int j = jc;
                    const float a = __builtin_amdgcn_exp2f(su.x * a2[j]);
                    h[j] = fmaf(a, h[j], row_broadcast<j>(bv) * su.y);
                    if (CUT) {
                        prod[j] *= a;
                        R[j] = fmaf(prod[j], row_broadcast<j>(cv) * ds, R[j]);
                    }
                });
            }
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

// x + x of lane ^ M (M = 1 or 2)
template <int M>
__device__ __forceinline__ float add_xor(float x) {
    constexpr int perm = M == 1 ? 0xB1 : 0x4E;         // quad_perm [1,0,3,2], [2,3,0,1]
    return x + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), perm, 0xF, 0xF, true));
}
// x + x of the lane R further on (in a ring) in its row of 16
template <int R>
__device__ __forceinline__ float add_ror(float x) {
    return x + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x120 + R, 0xF, 0xF, true));
}
// lanes 0..31: the sum of a over lanes l and l + 32; lanes 32..63: of b
__device__ __forceinline__ float add_halves(float a, float b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, a), __builtin_bit_cast(unsigned, b), false, false);
    return __builtin_bit_cast(float, (unsigned)r[0]) + __builtin_bit_cast(float, (unsigned)r[1]);
}
// even rows of 16 lanes: the sum of a over that row and the next; odd rows: of b over the one before and that
__device__ __forceinline__ float add_rows(float a, float b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, a), __builtin_bit_cast(unsigned, b), false, false);
    return __builtin_bit_cast(float, (unsigned)r[0]) + __builtin_bit_cast(float, (unsigned)r[1]);
}

template <typename T, int NW, int NL, bool CUT>
__global__ __launch_bounds__(64 * NW, NW == 4 && NL == 4 ? 2 : 1) void scan_bwd_kernel(const BwdParams p)
{
    typedef Work<T, NW, NL> W;
    constexpr int NT = W::NT, NP = W::NP, PASS = W::PASS;
    constexpr int LPC = NW, NB = NL / 4;               // lanes per channel, groups of 4 states per lane
    __shared__ __align__(16) typename W::Lds lds;
    __shared__ __align__(16) float part[4][BWD_ROWS][SCAN_TILE];       // o, du, sum_n A w, (unused)
    __shared__ __align__(16) float bcw[NW][BWD_ROWS][2 * NP];          // dB and dC of the wave's channels
    W w(p);
    float* so = p.sums + (size_t)w.number * (NP + 2) * p.D;    // the piece's sums
    if (!w.live) {
        // a number without a piece: its sums are zero
        if (w.own)
            for (int k = w.wave; k < NP + 2; k += NW) so[(size_t)k * p.D + w.d] = 0.0f;
        return;
    }
    const int lane = w.lane, ng = lane % LPC;
    const int chn = w.wave * (64 / LPC) + lane / LPC;  // the lane's channel in the tile
    const int d = w.ch.d0 + chn, n0 = 4 * ng;          // states n0 + 4 LPC k + j
    const bool own = chn < w.ch.count;

    float a2[NL], G[NL], dA[NL], enter[NL];
    // the gradient that reaches the piece's last state, and the state that enters it (of a
    // sequence's first piece the kept states already have it)
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int n = n0 + i / 4 * 4 * LPC + i % 4;
        const bool live = own && n < p.N;
        a2[i] = live ? p.A[(size_t)d * p.N + n] * LOG2E : 0.0f;
        G[i] = live && p.dh_final ? p.dh_final[((size_t)w.b * p.D + d) * p.N + n] : 0.0f;
        dA[i] = enter[i] = 0.0f;
    }
    if (CUT && own) {
#pragma unroll 4
        for (int e = w.number - w.c; e < w.number; ++e) {
            const float sum = p.piece_s[(size_t)e * p.D + d];
#pragma unroll
            for (int i = 0; i < NL; ++i)
                enter[i] = fmaf(__builtin_amdgcn_exp2f(a2[i] * sum), enter[i],
                                p.piece_h[((size_t)e * NP + n0 + i / 4 * 4 * LPC + i % 4) * p.D + d]);
        }
#pragma unroll 4
        for (int e = w.number - w.c + (w.sq.n - 1) / p.pieces.length; e > w.number; --e) {
            const float sum = p.piece_s[(size_t)e * p.D + d];
#pragma unroll
            for (int i = 0; i < NL; ++i)
                G[i] = fmaf(__builtin_amdgcn_exp2f(a2[i] * sum), G[i],
                            p.piece_g[((size_t)e * NP + n0 + i / 4 * 4 * LPC + i % 4) * p.D + d]);
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
        w.template put<true>(lds, t0);
        __syncthreads();
        if (t0 > w.t_begin) w.template load<true>(t0 - BWD_ROWS);
#pragma unroll 1
        for (int half = BWD_ROWS - KEEP; half >= 0; half -= KEEP)
        for_each<NB>([&](auto qc) {                    // KEEP rows and four states at a time
            constexpr int q = 4 * qc;
            const int n = n0 + q * LPC;
            float h[KEEP + 1][4], a[KEEP][4];
            // the state in front of the rows (rows past the end start from any)
            const size_t slot = w.slot + min(t0 + half, w.t_end - 1) / KEEP;
            const float since = CUT && w.c > 0 && own ? p.before[slot * p.D + d] : 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[0][j] = own ? p.state[(slot * NP + n + j) * p.D + d] : 0.0f;
                if (CUT) h[0][j] = fmaf(__builtin_amdgcn_exp2f(a2[q + j] * since), enter[q + j], h[0][j]);
            }
#pragma unroll
            for (int t = 0; t < KEEP; ++t) {
                const float2 su = lds.su[half + t][chn];
                const f32x4 bv = *reinterpret_cast<const f32x4*>(&lds.bs[half + t][n]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    a[t][j] = __builtin_amdgcn_exp2f(su.x * a2[q + j]);
                    h[t + 1][j] = fmaf(a[t][j], h[t][j], bv[j] * su.y);
                }
            }
#pragma unroll
            for (int t = KEEP - 1; t >= 0; --t) {
                const float2 su = lds.su[half + t][chn];
                const float ds = lds.ds[half + t][chn];
                const f32x4 bv = *reinterpret_cast<const f32x4*>(&lds.bs[half + t][n]);
                const f32x4 cv = *reinterpret_cast<const f32x4*>(&lds.cs[half + t][n]);
                float o = 0.0f, du = 0.0f, aw = 0.0f, v[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float g = fmaf(cv[j], ds, G[q + j]);
                    const float gw = g * (a[t][j] * h[t][j]);
                    o = j == 0 ? cv[0] * h[t + 1][0] : fmaf(cv[j], h[t + 1][j], o);
                    du = j == 0 ? bv[0] * g : fmaf(bv[j], g, du);
                    aw = j == 0 ? a2[q] * gw : fmaf(a2[q + j], gw, aw);
                    dA[q + j] = fmaf(su.x, gw, dA[q + j]);
                    G[q + j] = a[t][j] * g;
                    v[j] = g * su.y;
                    v[4 + j] = ds * h[t + 1][j];
                }
                // over the channel's states; lane ng of a channel stores the ng-th sum
                if (LPC > 1) { o = add_xor<1>(o); du = add_xor<1>(du); aw = add_xor<1>(aw); }
                if (LPC > 2) { o = add_xor<2>(o); du = add_xor<2>(du); aw = add_xor<2>(aw); }
                float* to = &part[0][half + t][chn];
                constexpr int PLANE = BWD_ROWS * SCAN_TILE;
                auto put = [&](int plane, float x) { to[plane * PLANE] = q == 0 ? x : to[plane * PLANE] + x; };
                if (LPC == 4) {
                    put(ng, ng == 0 ? o : ng == 1 ? du : aw);
                } else if (LPC == 2) {
                    put(ng, ng == 0 ? o : du);
                    put(2 + ng, aw);
                } else {
                    put(0, o);
                    put(1, du);
                    put(2, aw);
                }
                // over the wave's channels: value 4 bit5 + 2 bit4 + k of lane's r[k]
                float r[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    r[k] = add_rows(add_halves(v[k], v[4 + k]), add_halves(v[2 + k], v[6 + k]));
                    r[k] = add_ror<4>(add_ror<8>(r[k]));
                    if (LPC < 4) r[k] = add_ror<2>(r[k]);
                    if (LPC < 2) r[k] = add_ror<1>(r[k]);
                }
                const int k = lane >> 2 & 1, j = 2 * (lane >> 4 & 1) + k;
                // (lanes of one sum hold the same bits and store them to one address: no branch)
                bcw[w.wave][half + t][(lane >> 5) * NP + n + j] = k ? r[1] : r[0];
            }
        });
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PASS; ++i) {
            const int r = w.r0 + (NT / 16) * i, t = t0 + r;
            const int n = t < w.t_end ? w.nc : 0;
            f32x4 sum[3];                              // o, du, sum_n A w
#pragma unroll
            for (int q = 0; q < 3; ++q)
                sum[q] = *reinterpret_cast<const f32x4*>(&part[q][r][w.c4]);
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
            float v = bcw[0][r][at % (2 * NP)];
#pragma unroll
            for (int k = 1; k < NW; ++k) v += bcw[k][r][at % (2 * NP)];
            if (t0 + r < w.t_end) bcp[(size_t)(t0 + r) * (2 * NP) + at % (2 * NP)] = v;
        }
        __syncthreads();
    }

    // the piece's sums; those of dskip and dbias lie with the NT / 16 threads of a channel group
    if (own) {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int n = n0 + i / 4 * 4 * LPC + i % 4;
            so[(size_t)n * p.D + d] = dA[i];
            if (w.c == 0 && p.dh_init && n < p.N) p.dh_init[((size_t)w.b * p.D + d) * p.N + n] = G[i];
        }
    }
    float* sm = &part[0][0][0];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        sm[w.r0 * SCAN_TILE + w.c4 + e] = dskip[e];
        sm[(NT / 16 + w.r0) * SCAN_TILE + w.c4 + e] = dbias[e];
    }
    __syncthreads();
    if (w.tid < SCAN_TILE && w.own) {                  // (here a thread is its lane's channel again)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float s = 0.0f;
            for (int r = 0; r < NT / 16; ++r) s += sm[(k * (NT / 16) + r) * SCAN_TILE + lane];
            so[(size_t)(NP + k) * p.D + w.d] = s;
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
    if (d < p.D)
#pragma unroll 8
        for (int i = wave; i < count; i += 16) s += p.sums[((size_t)i * (NP + 2) + j) * p.D + d];
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
    const int width = 2 * p.G * p.N;
    const long long at = (long long)blockIdx.x * 256 + threadIdx.x, row = at / width;
    if (row >= p.pieces.rows || !p.pieces.has((int)row)) return;
    const int e = (int)(at % width), k = e / (p.G * p.N), g = e / p.N % p.G, n = e % p.N;
    const int per = scan_tiles(p.D, p.G) / p.G;
    const float* src = p.bc + ((size_t)g * per * p.pieces.rows + row) * (2 * NP) + k * NP + n;
    float s = 0.0f;
    for (int i = 0; i < per; ++i) s += src[(size_t)i * p.pieces.rows * (2 * NP)];
    T* out = k == 0 ? (T*)p.dB + row * p.dB_stride : (T*)p.dC + row * p.dC_stride;
    out[g * p.N + n] = from_f32<T>(s);
}

// Rows per piece.  Cutting costs the R and the sums of the first kernel (about a tenth of the
// whole), and pays where whole sequences would leave places unfilled, at N = 16 512 (two workgroups
// to a compute unit): (sequences, rows, channels) = (16, 1024, 2048), 512 workgroups, took
// 646 us whole and 719 us in four pieces; (4, 2048, 4096), 256 workgroups, 941 us whole, 775, 743
// and 732 us in 2, 4 and 8; (8, 2048, 1536) 917 us whole, 748, 594, 629 and 555 us in 2, 4, 6 and
// 8.  The 6 lose because their workgroups fill the places 2.25 times: so the number is taken that
// makes rounds * rows the least, with 24 rows for a piece's start, and among numbers within a
// twentieth of that the largest.
// The places by N: up to 4 states a workgroup is one wave, four to a compute unit ((1, 2048, 1536)
// at N = 4 took 111 us for 512 places and 76 us for 1024), above 16 registers leave room for
// one workgroup ((8, 1024, 2048) at N = 32 took 910 us in four pieces and 784 us whole).  For 5
// to 8 states, two waves whose registers leave room for two workgroups, neither count is the
// better one: at N = 8, as 1024 and as 512 places, (1, 2048, 1536) took 108 and 99 us, (16, 1024,
// 2048) 616 and 590, (2, 1024, 2048) 105 and 109, (24, 1024, 2048) 904 and 1017 us.
constexpr int SHORTEST_PIECE = 48, START_ROWS = 24;
int piece_rows(int S, int rows, int D, int G, int N) {
    const int places = N <= 8 ? 1024 : N <= 16 ? 512 : 256;
    // packed sequences count by the rows that there are
    const long long groups = ((long long)scan_tiles(D, G) * rows + S / 2) / S;
    const int whole = (S + BWD_ROWS - 1) / BWD_ROWS * BWD_ROWS;
    if (groups >= places - places / 8 || whole <= SHORTEST_PIECE) return whole;
    auto length = [&](int n) { return (int)(((S + n - 1) / n + BWD_ROWS - 1) / BWD_ROWS * BWD_ROWS); };
    auto cost = [&](int n) { return (groups * n + places - 1) / places * (length(n) + START_ROWS); };
    long long least = cost(1);
    const int most = (int)(4 * places / groups);
    for (int n = 2; n <= most && length(n) >= SHORTEST_PIECE; ++n)
        if (cost(n) < least) least = cost(n);
    int best = 1;
    for (int n = 2; n <= most && length(n) >= SHORTEST_PIECE; ++n)
        if (20 * cost(n) <= 21 * least) best = n;
    return length(best);
}

struct BwdPlan {
    Pieces pieces;
    bool cut;
    size_t state, before, bc, sums, piece_h, piece_g, piece_s, total;      // offsets and size in floats
};
BwdPlan plan(const int* seq_start, int B, int S, int rows, int D, int G, int N) {
    const size_t NP = scan_padded_states(N);
    BwdPlan f = {};
    f.pieces = make_pieces(seq_start, B, S, rows, piece_rows(S, rows, D, G, N));
    f.cut = f.pieces.length < S;
    size_t at = 0;
    auto take = [&](size_t n) { const size_t o = at; at += (n + 63) / 64 * 64; return o; };
    // as many kept states and pieces as packed sequences may need (also where they are not
    // packed: a workspace's size does not depend on seq_start)
    const size_t slots = (size_t)rows / KEEP + B, parts = (size_t)rows / f.pieces.length + B;
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
    const long long elems = (long long)a.rows * 2 * a.G * a.N, groups = (long long)scan_tiles(a.D, a.G) * f.pieces.count();
    if (!launchable((elems + 255) / 256, 256) || !launchable((long long)((a.D + 63) / 64) * (a.N + 2), 1024))
        return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)groups);
#define SCAN_LAUNCH(NW, NL, CUT)                                                                               \
    hipLaunchKernelGGL((scan_bwd_states_kernel<T, NW, NL, CUT>), grid, dim3(64 * NW), 0, a.stream, p);         \
    hipLaunchKernelGGL((scan_bwd_kernel<T, NW, NL, CUT>), grid, dim3(64 * NW), 0, a.stream, p)
#define SCAN_CALL(NW, NL)                         \
    if (!launchable(groups, 64 * NW)) return hipErrorInvalidConfiguration; \
    if (f.cut) { SCAN_LAUNCH(NW, NL, true); }     \
    else { SCAN_LAUNCH(NW, NL, false); }
    SCAN_DISPATCH_N(a.N, SCAN_CALL)
#undef SCAN_CALL
#undef SCAN_LAUNCH
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(scan_bwd_sums_kernel, dim3((a.D + 63) / 64, a.N + 2), dim3(1024), 0, a.stream, p, NP);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(scan_bwd_bc_kernel<T>, dim3((unsigned)((elems + 255) / 256)), dim3(256), 0, a.stream, p, NP);
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
