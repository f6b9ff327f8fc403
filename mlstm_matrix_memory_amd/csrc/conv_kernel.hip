// Short causal depthwise convolution with an optional swish: forward, backward and
// the one-row step (the causal convolution that stands in front of a block's cell).
//
// Per channel, with W taps:
//   p_t = bias + sum_j w_j x_{t-W+1+j},  y_t = p_t or p_t sigmoid(p_t)
// Backward, with dp_t = dy_t act'(p_t) (0 outside the sequence):
//   dx_t = sum_j w_j dp_{t+W-1-j},  dw_j = sum_t dp_t x_{t-W+1+j},  dbias = sum_t dp_t
//
// A thread owns 8 neighbouring channels (one 16-byte access of a bf16 row) and walks
// a run of rows with the last W - 1 inputs in registers, so that each input is read
// once, but for the W - 1 rows at a run's start.  Threads are numbered through
// channels first: a wave's accesses are contiguous for any D.  Bound by HBM.
#include "block_internal.h"

namespace mlstm {
namespace {

constexpr int CONV_THREADS = 256;

// rows before the first of a sequence: row -m (1 <= m < W) is row W - 1 - m of its state
template <typename T, int W>
__device__ __forceinline__ Raw8<T> load_input(const T* x, long long stride, const T* state, int D, int t, int n) {
    if (t >= 0) return load_row8(x + t * stride, n);
    if (state) return load_row8(state + (size_t)(W - 1 + t) * D, n);
    Raw8<T> z;
    z.zero();
    return z;
}

template <typename T, int W, bool ACT>
__global__ __launch_bounds__(CONV_THREADS) void conv_fwd_kernel(
    const T* __restrict__ x, long long x_stride, const float* __restrict__ weight, const float* __restrict__ bias,
    const int* __restrict__ seq_start, const T* __restrict__ state_init, int S, int rows, int D, int run,
    T* __restrict__ y, long long y_stride, T* __restrict__ state_final)
{
    const int groups = (D + 7) / 8;
    const long long id = (long long)blockIdx.x * CONV_THREADS + threadIdx.x;
    const int c = (int)(id % groups) * 8;
    const long long t_first = id / groups * run;
    if (t_first >= S) return;
    const int b = blockIdx.y;
    const RowRange sq = sequence_rows(seq_start, b, S, rows);
    const int n = D - c;
    const T* xs = x + sq.lo * x_stride + c;
    const T* st = state_init ? state_init + (size_t)b * (W - 1) * D + c : nullptr;
    const int t0 = (int)t_first, t1 = min(t0 + run, sq.n);
    if (t0 == 0 && state_final) {
        T* sf = state_final + (size_t)b * (W - 1) * D + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            store_row8(sf + (size_t)j * D, load_input<T, W>(xs, x_stride, st, D, sq.n - (W - 1) + j, n), n);
    }
    if (t0 >= t1) return;
    float w[W][8], bs[8], past[W - 1][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][e] = e < n ? weight[(size_t)(c + e) * W + j] : 0.0f;
        bs[e] = bias && e < n ? bias[c + e] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const Raw8<T> v = load_input<T, W>(xs, x_stride, st, D, t0 - (W - 1) + j, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) past[j][e] = v.get(e);
    }
    T* ys = y + sq.lo * y_stride + c;
    for (int t = t0; t < t1; ++t) {
        const Raw8<T> v = load_row8(xs + t * x_stride, n);
        Raw8<T> o;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float p = bs[e];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) p = fmaf(w[j][e], past[j][e], p);
            p = fmaf(w[W - 1][e], v.get(e), p);
            o.set(e, ACT ? p * sigmoid_hw(p) : p);
#pragma unroll
            for (int j = 0; j + 1 < W - 1; ++j) past[j][e] = past[j + 1][e];
            past[W - 2][e] = v.get(e);
        }
        store_row8(ys + t * y_stride, o, n);
    }
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
    Raw8<T> o;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float p = bias && e < n ? bias[c + e] : 0.0f;
#pragma unroll
        for (int j = 0; j < W; ++j) p = fmaf(e < n ? weight[(size_t)(c + e) * W + j] : 0.0f, in[j].get(e), p);
        o.set(e, ACT ? p * sigmoid_hw(p) : p);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_row8(st + (size_t)j * D, in[j + 1], n);
    store_row8(y + b * y_stride + c, o, n);
}

// A run of rows [t0, t1): its dp give dw and dbias; dx of row t needs dp up to row
// t + W - 1, so the run reads W - 1 rows past its end.  The first run of a sequence
// also emits the gradient of the rows before it (its initial state).
template <typename T, int W, bool ACT>
__global__ __launch_bounds__(CONV_THREADS) void conv_bwd_kernel(
    const T* __restrict__ x, long long x_stride, const float* __restrict__ weight, const float* __restrict__ bias,
    const int* __restrict__ seq_start, const T* __restrict__ state_init,
    const T* __restrict__ dy, long long dy_stride, const T* __restrict__ dstate_final,
    int S, int rows, int D, int run, T* __restrict__ dx, long long dx_stride, T* __restrict__ grad_state,
    float* __restrict__ parts)
{
    const int groups = (D + 7) / 8;
    const long long id = (long long)blockIdx.x * CONV_THREADS + threadIdx.x;
    const int c = (int)(id % groups) * 8;
    const long long chunk = id / groups, t_first = chunk * run;
    if (t_first >= S) return;
    const int b = blockIdx.y;
    const RowRange sq = sequence_rows(seq_start, b, S, rows);
    const int n = D - c;
    const T* xs = x + sq.lo * x_stride + c;
    const T* gs = dy + sq.lo * dy_stride + c;
    const T* st = state_init ? state_init + (size_t)b * (W - 1) * D + c : nullptr;
    const T* df = dstate_final ? dstate_final + (size_t)b * (W - 1) * D + c : nullptr;
    T* dxs = dx + sq.lo * dx_stride + c;
    T* gst = grad_state ? grad_state + (size_t)b * (W - 1) * D + c : nullptr;
    const int t0 = (int)t_first, t1 = min(t0 + run, sq.n);
    float w[W][8], bs[8], past[W - 1][8], dp[W][8], dw[W][8], db[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
        for (int j = 0; j < W; ++j) {
            w[j][e] = e < n ? weight[(size_t)(c + e) * W + j] : 0.0f;
            dw[j][e] = 0.0f;
            dp[j][e] = 0.0f;
        }
        bs[e] = bias && e < n ? bias[c + e] : 0.0f;
        db[e] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const Raw8<T> v = load_input<T, W>(xs, x_stride, st, D, t0 - (W - 1) + j, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) past[j][e] = v.get(e);
    }
    // rows t1 .. t1 + W - 2 only complete the gradients of this run's rows
    const int end = t0 < t1 || t0 == 0 ? max(t1, t0) + W - 1 : t0;
    for (int t = t0; t < end; ++t) {
        Raw8<T> v, g;
        v.zero();
        g.zero();
        if (t < sq.n) {
            v = load_row8(xs + t * x_stride, n);
            g = load_row8(gs + t * dy_stride, n);
        }
        const int s = t - (W - 1);                       // the row whose gradient is complete now
        const int held = s - (sq.n - (W - 1));           // its place in the final state, if >= 0
        Raw8<T> more, o;
        more.zero();
        if (df && held >= 0 && held < W - 1) more = load_row8(df + (size_t)held * D, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float p = bs[e];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) p = fmaf(w[j][e], past[j][e], p);
            p = fmaf(w[W - 1][e], v.get(e), p);
            float d = g.get(e);
            if (ACT) {
                const float sg = sigmoid_hw(p);
                d *= sg * (1.0f + p * (1.0f - sg));
            }
#pragma unroll
            for (int j = 0; j + 1 < W; ++j) dp[j][e] = dp[j + 1][e];
            dp[W - 1][e] = d;
            if (t < t1) {
#pragma unroll
                for (int j = 0; j < W - 1; ++j) dw[j][e] = fmaf(d, past[j][e], dw[j][e]);
                dw[W - 1][e] = fmaf(d, v.get(e), dw[W - 1][e]);
                db[e] += d;
            }
            // dx_s = sum_j w_j dp_{s + W - 1 - j};  dp[i] holds row s + i
            float a = more.get(e);
#pragma unroll
            for (int j = 0; j < W; ++j) a = fmaf(w[j][e], dp[W - 1 - j][e], a);
            o.set(e, a);
#pragma unroll
            for (int j = 0; j + 1 < W - 1; ++j) past[j][e] = past[j + 1][e];
            past[W - 2][e] = v.get(e);
        }
        if (s >= t0 && s < t1) store_row8(dxs + s * dx_stride, o, n);
        if (s < 0 && gst) store_row8(gst + (size_t)(W - 1 + s) * D, o, n);
    }
    // parts [(b, run)][W + 1][D]
    const long long runs = (S + run - 1) / run;
    float* po = parts + (size_t)(b * runs + chunk) * (W + 1) * D + c;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        Raw8<float> o;
#pragma unroll
        for (int e = 0; e < 8; ++e) o.set(e, j < W ? dw[j < W ? j : 0][e] : db[e]);
        store_row8(po + (size_t)j * D, o, n);
    }
}

// dweight[d][j], dbias[d] = sums of the parts: 64 channels of one tap per workgroup
template <int W>
__global__ __launch_bounds__(1024) void conv_sum_kernel(const float* __restrict__ parts, long long n, int D,
                                                        float* __restrict__ dw, float* __restrict__ db)
{
    __shared__ float sm[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int d = blockIdx.x * 64 + lane, j = blockIdx.y;
    float s = 0.0f;
    if (d < D)
#pragma unroll 8
        for (long long p = wave; p < n; p += 16) s += parts[((size_t)p * (W + 1) + j) * D + d];
    sm[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && d < D) {
#pragma unroll
        for (int w = 1; w < 16; ++w) s += sm[w][lane];
        if (j < W) dw[(size_t)d * W + j] = s;
        else if (db) db[d] = s;
    }
}

// Rows per run of the forward: 16 where the sequence is long, fewer where that leaves
// the chip's 1024 SIMDs without two waves each.
int conv_run(int B, int S, int D, int longest) {
    const long long groups = (D + 7) / 8;
    int run = longest;
    while (run > 4 && (long long)B * groups * ((S + run - 1) / run) < 131072) run >>= 1;
    return run;
}
constexpr int CONV_FWD_RUN = 16;
constexpr int CONV_BWD_RUN = 128;

dim3 conv_grid(int B, int S, int D, int run) {
    const long long threads = (long long)((D + 7) / 8) * ((S + run - 1) / run);
    return dim3((unsigned)((threads + CONV_THREADS - 1) / CONV_THREADS), (unsigned)B);
}

template <typename T, int W, bool ACT>
hipError_t fwd_t(const ConvArgs& a) {
    const int run = conv_run(a.B, a.S, a.D, CONV_FWD_RUN);
    hipLaunchKernelGGL((conv_fwd_kernel<T, W, ACT>), conv_grid(a.B, a.S, a.D, run), dim3(CONV_THREADS), 0, a.stream,
                       (const T*)a.x, a.x_stride, a.weight, a.bias, a.seq_start, (const T*)a.state_init, a.S, a.rows,
                       a.D, run, (T*)a.y, a.y_stride, (T*)a.state_final);
    return hipGetLastError();
}

template <typename T, int W, bool ACT>
hipError_t step_t(const ConvArgs& a) {
    const long long threads = (long long)a.B * ((a.D + 7) / 8);
    hipLaunchKernelGGL((conv_step_kernel<T, W, ACT>), dim3((unsigned)((threads + 63) / 64)), dim3(64), 0, a.stream,
                       (const T*)a.x, a.x_stride, a.weight, a.bias, a.B, a.D, (T*)a.state_final, (T*)a.y, a.y_stride);
    return hipGetLastError();
}

template <typename T, int W, bool ACT>
hipError_t bwd_t(const ConvArgs& a) {
    const int run = conv_run(a.B, a.S, a.D, CONV_BWD_RUN);
    hipLaunchKernelGGL((conv_bwd_kernel<T, W, ACT>), conv_grid(a.B, a.S, a.D, run), dim3(CONV_THREADS), 0, a.stream,
                       (const T*)a.x, a.x_stride, a.weight, a.bias, a.seq_start, (const T*)a.state_init,
                       (const T*)a.dy, a.dy_stride, (const T*)a.dstate_final, a.S, a.rows, a.D, run,
                       (T*)a.grad_x, a.grad_x_stride, (T*)a.grad_state, a.ws);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const long long parts = (long long)a.B * ((a.S + run - 1) / run);
    hipLaunchKernelGGL(conv_sum_kernel<W>, dim3((a.D + 63) / 64, W + 1), dim3(1024), 0, a.stream, a.ws, parts, a.D,
                       a.grad_weight, a.grad_bias);
    return hipGetLastError();
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

size_t conv_bwd_workspace_bytes(int B, int S, int D, int width) {
    const int run = conv_run(B, S, D, CONV_BWD_RUN);
    return (size_t)B * ((S + run - 1) / run) * (width + 1) * D * sizeof(float);
}

}  // namespace mlstm
