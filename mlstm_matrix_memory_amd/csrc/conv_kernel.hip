// Short causal depthwise convolution with an optional swish: forward, backward and
// the one-row step (the causal convolution that stands in front of a block's cell).
//
// Per channel, with W taps:
//   p_t = bias + sum_j w_j x_{t-W+1+j},  y_t = p_t or p_t sigmoid(p_t)
// Backward, with dp_t = dy_t act'(p_t) (0 outside the sequence):
//   dx_t = sum_j w_j dp_{t+W-1-j},  dw_j = sum_t dp_t x_{t-W+1+j},  dbias = sum_t dp_t
//
// A thread owns 8 neighbouring channels (one 16-byte access of a bf16 row) and a run of
// rows, fully unrolled: all of a run's loads are in flight together, and the W - 1 rows that
// neighbouring runs share come from the cache.  A workgroup is 32 threads of channels by
// 8 runs.  Bound by HBM.
//
// Where D is no multiple of 8 the last thread of a row takes the row's last 8 channels,
// some of them its neighbour's too: both compute and store the same values, and the
// wave has one path.  (With guarded accesses for the last channels it ran both paths one
// after the other: the backward at D = 1537 took 59 us against 33 us at 1536.)
#include <type_traits>

#include "block_internal.h"

namespace mlstm {
namespace {

constexpr int CONV_THREADS = 256;
constexpr int CONV_LANES = 32;                         // threads along the channels
constexpr int CONV_RUNS = CONV_THREADS / CONV_LANES;   // runs of a workgroup

// rows before the first of a sequence: row -m (1 <= m < W) is row W - 1 - m of its state
template <typename T, int W>
__device__ __forceinline__ Raw8<T> load_input(const T* x, long long stride, const T* state, int D, int t, int n) {
    if (t >= 0) return load_row8(x + t * stride, n);
    if (state) return load_row8(state + (size_t)(W - 1 + t) * D, n);
    Raw8<T> z;
    z.zero();
    return z;
}

// eight channels' taps w[j][e] and bias
template <int W>
__device__ __forceinline__ void load_taps(const float* weight, const float* bias, int c, int n, float (&w)[W][8],
                                          float (&bs)[8]) {
    if (n >= 8) {
        float v[8 * W];
#pragma unroll
        for (int k = 0; k < 2 * W; ++k)
            *reinterpret_cast<f32x4*>(v + 4 * k) = *reinterpret_cast<const f32x4_u*>(weight + (size_t)c * W + 4 * k);
        const Raw8<float> bv = load_row8(bias ? bias + c : weight, bias ? 8 : 0);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][e] = v[e * W + j];
            bs[e] = bv.get(e);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][e] = e < n ? weight[(size_t)(c + e) * W + j] : 0.0f;
            bs[e] = bias && e < n ? bias[c + e] : 0.0f;
        }
    }
}

template <typename T, int W, bool ACT, int RUN>
__global__ __launch_bounds__(CONV_THREADS) void conv_fwd_kernel(
    const T* __restrict__ x, long long x_stride, const float* __restrict__ weight, const float* __restrict__ bias,
    const T* __restrict__ state_init, const Pieces pieces, int D, T* __restrict__ y, long long y_stride,
    T* __restrict__ state_final)
{
    const int blocks = ((D + 7) / 8 + CONV_LANES - 1) / CONV_LANES;
    int c = ((blockIdx.x % blocks) * CONV_LANES + threadIdx.x % CONV_LANES) * 8;
    if (c >= D) return;
    if (D >= 8) c = min(c, D - 8);
    const int n = D - c;                               // below 8 only where D is
    const Pieces::At at = pieces.at(blockIdx.x / blocks);
    const RowRange sq = pieces.sequence(at.b);
    const long long first = (long long)at.c * pieces.length + threadIdx.x / CONV_LANES * RUN;
    if (first >= sq.n && first > 0) return;
    const int t0 = (int)first;
    const T* xs = x + sq.lo * x_stride + c;
    const T* st = state_init ? state_init + (size_t)at.b * (W - 1) * D + c : nullptr;
    if (t0 == 0 && state_final) {
        T* sf = state_final + (size_t)at.b * (W - 1) * D + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            store_row8(sf + (size_t)j * D, load_input<T, W>(xs, x_stride, st, D, sq.n - (W - 1) + j, n), n);
    }
    if (t0 >= sq.n) return;
    T* ys = y + sq.lo * y_stride + c;
    auto run = [&](auto full) {
        constexpr bool FULL = full;                    // all eight channels
        Raw8<T> in[RUN + W - 1];
#pragma unroll
        for (int i = 0; i < RUN; ++i) {                // rows past the end: the last, not stored
            const T* row = xs + (long long)min(t0 + i, sq.n - 1) * x_stride;
            if (FULL) in[W - 1 + i].load(row);
            else in[W - 1 + i] = load_row8(row, n);
        }
        if (t0 > 0) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                const T* row = xs + (long long)(t0 - (W - 1) + j) * x_stride;
                if (FULL) in[j].load(row);
                else in[j] = load_row8(row, n);
            }
        } else {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) in[j] = load_input<T, W>(xs, x_stride, st, D, j - (W - 1), n);
        }
        float w[W][8], bs[8];
        load_taps<W>(weight, bias, c, n, w, bs);
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
            Raw8<T> o;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float p = bs[e];
#pragma unroll
                for (int j = 0; j < W; ++j) p = fmaf(w[j][e], in[i + j].get(e), p);
                o.set(e, ACT ? p * sigmoid_hw(p) : p);
            }
            if (t0 + i < sq.n) {
                if (FULL) o.store(ys + (long long)(t0 + i) * y_stride);
                else store_row8(ys + (long long)(t0 + i) * y_stride, o, n);
            }
        }
    };
    if (n >= 8) run(std::true_type());
    else run(std::false_type());
}

template <typename T, int W, bool ACT>
__global__ __launch_bounds__(64) void conv_step_kernel(
    const T* __restrict__ x, long long x_stride, const float* __restrict__ weight, const float* __restrict__ bias,
    int B, int D, T* __restrict__ state, T* __restrict__ y, long long y_stride)
{
    const int groups = (D + 7) / 8;
    const long long id = (long long)blockIdx.x * 64 + threadIdx.x;
    const long long b = id / groups;
    if (b >= B) return;
    const int c = (int)(id % groups) * 8, n = D - c;
    T* st = state + (size_t)b * (W - 1) * D + c;
    Raw8<T> in[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) in[j] = load_row8(st + (size_t)j * D, n);
    in[W - 1] = load_row8(x + b * x_stride + c, n);
    float w[W][8], bs[8];
    load_taps<W>(weight, bias, c, n, w, bs);
    Raw8<T> o;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float p = bs[e];
#pragma unroll
        for (int j = 0; j < W; ++j) p = fmaf(w[j][e], in[j].get(e), p);
        o.set(e, ACT ? p * sigmoid_hw(p) : p);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_row8(st + (size_t)j * D, in[j + 1], n);
    store_row8(y + b * y_stride + c, o, n);
}

// A run of BWD_RUN rows: its dp give dw and dbias; dx of row t needs dp up to row t + W - 1, so
// a run reads W - 1 rows past its end.  The first run of a sequence also emits the gradient of
// the rows before it (its initial state).  A thread owns 4 channels here: taps, sums and
// windows of 8 took 396 registers, one wave to a SIMD.  The workgroup, 64 threads of channels
// by 4 runs, adds its runs' dw and dbias in LDS and writes one part of them.
// Rows of a run: with W = 4 29 make 8 blocks of 4.  13, 29 and 45 rows: (8, 2048, 1536) 50.4, 43.6
// and 46.7 us, packed rows of 1537 channels (6598 rows) 32.1, 28.3 and 45.7 us.
constexpr int BWD_RUN = 29;
constexpr int BWD_RUNS = CONV_THREADS / 64;
// FINAL: a gradient of the final state comes in.  (A template parameter because a load under a
// condition makes the compiler wait, where its value is used, for every load in flight: bf16
// rows of (8, 2048, 1536) took 52.6 us so and 43.6 us without it.)
template <typename T, int W, bool ACT, bool FINAL>
__global__ __launch_bounds__(CONV_THREADS) void conv_bwd_kernel(
    const T* __restrict__ x, long long x_stride, const float* __restrict__ weight, const float* __restrict__ bias,
    const T* __restrict__ state_init, const T* __restrict__ dy, long long dy_stride,
    const T* __restrict__ dstate_final, const Pieces pieces, int D, T* __restrict__ dx, long long dx_stride,
    T* __restrict__ grad_state, float* __restrict__ parts)
{
    __shared__ __align__(16) float red[BWD_RUNS][W + 1][256];
    const int blocks = (D + 255) / 256;
    const int lane = threadIdx.x & 63, turn = threadIdx.x >> 6;
    const int c0 = (blockIdx.x % blocks) * 256, own = D - (c0 + lane * 4);
    const int c = D >= 4 ? min(c0 + lane * 4, D - 4) : c0 + lane * 4;
    const int n = own > 0 ? D - c : 0;                 // below 4 only where D is, or no channel is left
    const int number = blockIdx.x / blocks;
    const Pieces::At at = pieces.at(number);
    const RowRange sq = pieces.sequence(at.b);
    const long long piece = (long long)at.c * pieces.length;
    const bool live = piece < sq.n || at.c == 0;       // (of others the part is zero)
    const long long first = piece + turn * BWD_RUN;
    float dw[W][4], db[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][e] = 0.0f;
        db[e] = 0.0f;
    }
    if (live && n > 0 && (first < sq.n || first == 0)) {
        const int t0 = (int)first, t1 = min(t0 + BWD_RUN, sq.n);
        const T* xs = x + sq.lo * x_stride + c;
        const T* gs = dy + sq.lo * dy_stride + c;
        const T* st = state_init ? state_init + (size_t)at.b * (W - 1) * D + c : nullptr;
        const T* df = FINAL ? dstate_final + (size_t)at.b * (W - 1) * D + c : nullptr;
        T* dxs = dx + sq.lo * dx_stride + c;
        T* gst = grad_state ? grad_state + (size_t)at.b * (W - 1) * D + c : nullptr;
        float w[W][4], bs[4], past[W - 1][4], dp[W][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][e] = e < n ? weight[(size_t)(c + e) * W + j] : 0.0f;
            bs[e] = bias && e < n ? bias[c + e] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int t = t0 - (W - 1) + j;
            Raw4<T> v;
            if (t >= 0) v = load_row4(xs + (long long)t * x_stride, n);
            else v = load_row4(st ? st + (size_t)(W - 1 + t) * D : xs, st ? n : 0);
#pragma unroll
            for (int e = 0; e < 4; ++e) past[j][e] = v.get(e);
        }
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) dp[j][e] = 0.0f;
        auto run = [&](auto full) {
            constexpr bool FULL = full;                // all four channels, and rows to read
            // blocks of BLOCK rows, the next block's loads in flight beside one's arithmetic
            constexpr int BLOCK = 4;
            Raw4<T> xv[BLOCK], gv[BLOCK], xn[BLOCK], gn[BLOCK];
            auto load = [&](int t) {
#pragma unroll
                for (int i = 0; i < BLOCK; ++i) {
                    if (FULL) {                        // rows past the end: the last, masked below
                        const long long r = min(t + i, sq.n - 1);
                        xn[i].load(xs + r * x_stride);
                        gn[i].load(gs + r * dy_stride);
                    } else {
                        const int m = t + i < sq.n ? n : 0;
                        xn[i] = load_row4(xs + (long long)(t + i) * x_stride, m);
                        gn[i] = load_row4(gs + (long long)(t + i) * dy_stride, m);
                    }
                }
            };
            load(t0);
            const int end = t1 + W - 1;                // rows from t1 on only complete gradients
            for (int tb = t0; tb < end; tb += BLOCK) {
#pragma unroll
                for (int i = 0; i < BLOCK; ++i) {
                    xv[i] = xn[i];
                    gv[i] = gn[i];
                }
                load(tb + BLOCK);
#pragma unroll
                for (int i = 0; i < BLOCK; ++i) {
                    const int t = tb + i;
                    const int s = t - (W - 1);                   // the row whose gradient is complete now
                    const int held = s - (sq.n - (W - 1));       // its place in the final state, if >= 0
                    Raw4<T> more, o;
                    more.zero();
                    if (FINAL && held >= 0 && held < W - 1) more = load_row4(df + (size_t)held * D, n);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float v = t < sq.n ? xv[i].get(e) : 0.0f;
                        float p = bs[e];
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) p = fmaf(w[j][e], past[j][e], p);
                        p = fmaf(w[W - 1][e], v, p);
                        float g = gv[i].get(e);
                        if (ACT) {
                            const float sg = sigmoid_hw(p);
                            g *= sg * (1.0f + p * (1.0f - sg));
                        }
                        g = t < sq.n ? g : 0.0f;
#pragma unroll
                        for (int j = 0; j + 1 < W; ++j) dp[j][e] = dp[j + 1][e];
                        dp[W - 1][e] = g;
                        const float gw = t < t1 ? g : 0.0f;
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) dw[j][e] = fmaf(gw, past[j][e], dw[j][e]);
                        dw[W - 1][e] = fmaf(gw, v, dw[W - 1][e]);
                        db[e] += gw;
                        // dx_s = sum_j w_j dp_{s + W - 1 - j};  dp[i] holds row s + i
                        float a = more.get(e);
#pragma unroll
                        for (int j = 0; j < W; ++j) a = fmaf(w[j][e], dp[W - 1 - j][e], a);
                        o.set(e, a);
#pragma unroll
                        for (int j = 0; j + 1 < W - 1; ++j) past[j][e] = past[j + 1][e];
                        past[W - 2][e] = v;
                    }
                    if (s >= t0 && s < t1) {
                        if (FULL) o.store(dxs + (long long)s * dx_stride);
                        else store_row4(dxs + (long long)s * dx_stride, o, n);
                    }
                    if (s < 0 && gst) store_row4(gst + (size_t)(W - 1 + s) * D, o, n);
                }
            }
        };
        if (n >= 4 && sq.n > 0) run(std::true_type());
        else run(std::false_type());
    }
    // of the channels it shares with its neighbour a thread adds none
    const int skip = own > 0 && own < 4 && D >= 4 ? 4 - own : 0;
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e >= skip) red[turn][j][lane * 4 + e - skip] = j < W ? dw[j < W ? j : 0][e] : db[e];
    __syncthreads();
    if (c0 + (int)threadIdx.x >= D) return;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        float v = red[0][j][threadIdx.x];
#pragma unroll
        for (int k = 1; k < BWD_RUNS; ++k) v += red[k][j][threadIdx.x];
        parts[((size_t)number * (W + 1) + j) * D + c0 + threadIdx.x] = v;
    }
}

// dweight[d][j], dbias[d] = sums of the parts: 64 channels of one tap per workgroup
template <int W>
__global__ __launch_bounds__(1024) void conv_sum_kernel(const float* __restrict__ parts, int count, int D,
                                                        float* __restrict__ dw, float* __restrict__ db)
{
    __shared__ float sm[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int d = blockIdx.x * 64 + lane, j = blockIdx.y;
    float s = 0.0f;
    if (d < D)
#pragma unroll 8
        for (int i = wave; i < count; i += 16) s += parts[((size_t)i * (W + 1) + j) * D + d];
    sm[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && d < D) {
#pragma unroll
        for (int w = 1; w < 16; ++w) s += sm[w][lane];
        if (j < W) dw[(size_t)d * W + j] = s;
        else if (db) db[d] = s;
    }
}

int conv_blocks(int D) { return ((D + 7) / 8 + CONV_LANES - 1) / CONV_LANES; }

template <typename T, int W, bool ACT, int RUN>
void fwd_run(const ConvArgs& a, const Pieces& pieces) {
    hipLaunchKernelGGL((conv_fwd_kernel<T, W, ACT, RUN>), dim3((unsigned)conv_blocks(a.D) * pieces.count()),
                       dim3(CONV_THREADS), 0, a.stream, (const T*)a.x, a.x_stride, a.weight, a.bias,
                       (const T*)a.state_init, pieces, a.D, (T*)a.y, a.y_stride, (T*)a.state_final);
}

template <typename T, int W, bool ACT>
hipError_t fwd_t(const ConvArgs& a) {
    // Long runs share the fewest rows, short ones fill the chip sooner.  bf16, rows of a half, runs of
    // 4, 8 and 16: (4, 2048, 4096) 30.5, 28.3 and 32.0 us, (8, 2048, 1536) 24.5, 23.3 and 22.1,
    // (1, 2048, 2048) 7.2, 7.2 and 8.9, (1, 512, 2048) 4.8, 5.8 and 7.6 us.
    const long long work = (long long)conv_blocks(a.D) * ((a.rows + 63) / 64);
    const int run = work >= 1024 ? 8 : 4;
    const Pieces pieces = make_pieces(a.seq_start, a.B, a.S, a.rows, run * CONV_RUNS);
    if (!launchable((long long)conv_blocks(a.D) * pieces.count(), CONV_THREADS)) return hipErrorInvalidConfiguration;
    if (run == 8) fwd_run<T, W, ACT, 8>(a, pieces);
    else fwd_run<T, W, ACT, 4>(a, pieces);
    return hipGetLastError();
}

template <typename T, int W, bool ACT>
hipError_t step_t(const ConvArgs& a) {
    const long long threads = (long long)a.B * ((a.D + 7) / 8);
    if (!launchable((threads + 63) / 64, 64)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((conv_step_kernel<T, W, ACT>), dim3((unsigned)((threads + 63) / 64)), dim3(64), 0, a.stream,
                       (const T*)a.x, a.x_stride, a.weight, a.bias, a.B, a.D, (T*)a.state_final, (T*)a.y, a.y_stride);
    return hipGetLastError();
}

Pieces bwd_pieces(const int* seq_start, int B, int S, int rows) {
    return make_pieces(seq_start, B, S, rows, BWD_RUN * BWD_RUNS);
}

template <typename T, int W, bool ACT, bool FINAL>
hipError_t bwd_run(const ConvArgs& a) {
    const Pieces pieces = bwd_pieces(a.seq_start, a.B, a.S, a.rows);
    if (!launchable((long long)((a.D + 255) / 256) * pieces.count(), CONV_THREADS)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((conv_bwd_kernel<T, W, ACT, FINAL>), dim3((unsigned)((a.D + 255) / 256) * pieces.count()),
                       dim3(CONV_THREADS), 0, a.stream, (const T*)a.x, a.x_stride, a.weight, a.bias,
                       (const T*)a.state_init, (const T*)a.dy, a.dy_stride, (const T*)a.dstate_final, pieces, a.D,
                       (T*)a.grad_x, a.grad_x_stride, (T*)a.grad_state, a.ws);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(conv_sum_kernel<W>, dim3((a.D + 63) / 64, W + 1), dim3(1024), 0, a.stream, a.ws, pieces.count(), a.D,
                       a.grad_weight, a.grad_bias);
    return hipGetLastError();
}

template <typename T, int W, bool ACT>
hipError_t bwd_t(const ConvArgs& a) {
    return a.dstate_final ? bwd_run<T, W, ACT, true>(a) : bwd_run<T, W, ACT, false>(a);
}

#define CONV_DISPATCH(F, a)                                                                   \
    const bool act = (a).act != 0;                                                            \
    if ((a).dtype == MLSTM_BF16) {                                                            \
        if ((a).width == 2) return act ? F<bf16, 2, true>(a) : F<bf16, 2, false>(a);          \
        if ((a).width == 3) return act ? F<bf16, 3, true>(a) : F<bf16, 3, false>(a);          \
        return act ? F<bf16, 4, true>(a) : F<bf16, 4, false>(a);                              \
    }                                                                                         \
    if ((a).width == 2) return act ? F<float, 2, true>(a) : F<float, 2, false>(a);            \
    if ((a).width == 3) return act ? F<float, 3, true>(a) : F<float, 3, false>(a);            \
    return act ? F<float, 4, true>(a) : F<float, 4, false>(a);

}  // namespace

hipError_t launch_conv_fwd(const ConvArgs& a) { CONV_DISPATCH(fwd_t, a) }
hipError_t launch_conv_step(const ConvArgs& a) { CONV_DISPATCH(step_t, a) }
hipError_t launch_conv_bwd(const ConvArgs& a) { CONV_DISPATCH(bwd_t, a) }

size_t conv_bwd_workspace_bytes(int B, int rows, int D, int width) {
    // as many pieces as packed sequences may need: the size does not depend on seq_start
    return ((size_t)rows / (BWD_RUN * BWD_RUNS) + B) * (width + 1) * D * sizeof(float);
}

}  // namespace mlstm
