// Residual addition and root-mean-square norm, in the inputs' type or in e4m3 with
// scales, and its backward (the norm that opens a block of the residual stack).
//
// Per row of d channels:
//   r = x + residual (rounded to its storage type),  k = 1 / sqrt(mean(r^2) + eps)
//   y = weight r k
//   e4m3: scale = max |y| / 448 over a group of columns,  q = round(y / scale)
// Backward, with v = weight dy:
//   dr = k (v - r k^2 mean(v r)) + dres,   dweight = sum over rows of dy r k
//
// One row per group of TPR threads (a wave, a workgroup of 256 or of 1024), which
// holds it in registers: each row is read once and written once.  Both sums of the
// backward need only r and dy, so k is not kept from the forward.  All sums are
// fp32.  The kernels are bound by HBM, at few rows by the launch.
#include "block_internal.h"

namespace mlstm {
namespace {

constexpr float E4M3_MAX = 448.0f;

// y / scale, scale = m / 448, for a group whose largest |y| is m, rounded as a division rounds it: y
// times the reciprocal, and the remainder of that times the reciprocal added.  (Without the
// remainder one value in some two million lands on the neighbouring e4m3 step; 8192 x 4096 in
// groups of 128 took 50 us without it, 51 us so and 55 us with the compiler's division.)  Small
// groups are scaled up, so that the remainder keeps its bits, and so does a scale below the
// smallest normal number; groups of zeros give zeros, and where scale is infinite finite values do.
struct Quotient {
    float up, scale, inv;
    __device__ __forceinline__ explicit Quotient(float m) {
        up = m < 0x1p-40f ? 0x1p100f : 1.0f;
        scale = m != 0.0f ? m * up / E4M3_MAX : 1.0f;
        inv = 1.0f / scale;
        if (inv == 0.0f) scale = 0.0f;
    }
    __device__ __forceinline__ float operator()(float y) const {
        y *= up;
        const float q = y * inv;
        return fmaf(fmaf(-q, scale, y), inv, q);
    }
};

// sum (or maximum) over the TPR threads of a row; red: one slot per wave of the workgroup
template <int TPR, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* red) {
    v = MAX ? wave_max(v) : wave_sum(v);
    if (TPR > 64) {
        __syncthreads();                         // an earlier reduction's slots are read
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int w = 1; w < TPR / 64; ++w) v = MAX ? fmaxf(v, red[w]) : v + red[w];
    }
    return v;
}

// Thread t of a row's TPR holds columns 8 (t + TPR c) .. + 7, c < CPT.
// QUANT: e4m3 output with scales.
template <typename T, typename RT, int TPR, int CPT, bool QUANT>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_fwd_kernel(
    const T* x, long long x_stride, const RT* residual, long long residual_stride,
    const float* __restrict__ weight, int rows, int d, float eps, int group,
    RT* residual_out, void* __restrict__ y_out, float* __restrict__ scale_out)
{
    constexpr int THREADS = TPR < 256 ? 256 : TPR;
    __shared__ float red[THREADS / 64];
    const int tl = threadIdx.x % TPR;
    const long long row = (long long)blockIdx.x * (THREADS / TPR) + threadIdx.x / TPR;
    const bool live = row < rows;                // a row's threads are live or not together
    const T* xr = x + (live ? row : 0) * x_stride;
    const RT* rr = residual + (residual && live ? row * residual_stride : 0);
    // all of the row's loads before its stores: residual_out may be x or residual, and
    // a thread then writes only elements that it has read
    Raw8<T> xv[CPT];
    Raw8<RT> rv[CPT];
    float r[CPT][8];
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
        const int col = 8 * (tl + TPR * c);
        const int n = live ? d - col : 0;
        xv[c] = load_row8(xr + col, n);
        rv[c].zero();
        if (residual) rv[c] = load_row8(rr + col, n);
    }
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
        const int col = 8 * (tl + TPR * c);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            rv[c].set(e, xv[c].get(e) + rv[c].get(e));   // rounded: the norm is of the stored sum
            r[c][e] = rv[c].get(e);
            sum += r[c][e] * r[c][e];
        }
        if (residual_out) store_row8(residual_out + (live ? row * d : 0) + col, rv[c], live ? d - col : 0);
    }
    const float k = 1.0f / sqrtf(row_reduce<TPR, false>(sum, red) / d + eps);
    float amax = 0.0f;
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
        const int col = 8 * (tl + TPR * c);
        const int n = live ? d - col : 0;
        const Raw8<float> w = load_row8(weight + col, d - col);
        if (!QUANT) {
            Raw8<T> yv;
#pragma unroll
            for (int e = 0; e < 8; ++e) yv.set(e, r[c][e] * k * w.get(e));
            store_row8((T*)y_out + (live ? row * d : 0) + col, yv, n);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                r[c][e] = r[c][e] * k * w.get(e);        // columns past d hold r = 0
                amax = fmaxf(amax, fabsf(r[c][e]));
            }
            if (group > 0) {
                // a group is 4, 8 or 16 consecutive threads of the wave
                float m = amax;
                amax = 0.0f;
                for (int off = 1; off < group / 8; off <<= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
                if (n > 0 && col % group == 0) scale_out[row * ((d + group - 1) / group) + col / group] = m / E4M3_MAX;
                const Quotient quotient(m);
#pragma unroll
                for (int e = 0; e < 8; ++e) r[c][e] = quotient(r[c][e]);
            }
        }
    }
    if (QUANT) {
        if (group == 0) {
            const float m = row_reduce<TPR, true>(amax, red);
            if (live && tl == 0) scale_out[row] = m / E4M3_MAX;
            const Quotient quotient(m);
#pragma unroll
            for (int c = 0; c < CPT; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e) r[c][e] = quotient(r[c][e]);
        }
        unsigned char* q = (unsigned char*)y_out + (live ? row * d : 0);
#pragma unroll
        for (int c = 0; c < CPT; ++c) {
            const int col = 8 * (tl + TPR * c);
            const int n = live ? d - col : 0;
            int lo = __builtin_amdgcn_cvt_pk_fp8_f32(r[c][0], r[c][1], 0, false);
            lo = __builtin_amdgcn_cvt_pk_fp8_f32(r[c][2], r[c][3], lo, true);
            int hi = __builtin_amdgcn_cvt_pk_fp8_f32(r[c][4], r[c][5], 0, false);
            hi = __builtin_amdgcn_cvt_pk_fp8_f32(r[c][6], r[c][7], hi, true);
            if (n >= 8) {
                typedef int int2_u __attribute__((ext_vector_type(2), aligned(1)));
                *reinterpret_cast<int2_u*>(q + col) = int2_u{lo, hi};
            } else {
#pragma unroll
                for (int e = 0; e < 7; ++e)
                    if (e < n) q[col + e] = (unsigned char)((e < 4 ? lo : hi) >> (8 * (e & 3)));
            }
        }
    }
}

// The workgroup's rows are blockIdx.x * RPW + (its row group), in steps of the grid; each
// row group sums dweight over its rows in registers, and the workgroup writes one part.
template <typename T, typename RT, int TPR, int CPT>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_bwd_kernel(
    const RT* __restrict__ r, long long r_stride, const float* __restrict__ weight,
    const T* __restrict__ dy, long long dy_stride, const RT* dres, int rows, int d, float eps,
    T* __restrict__ grad_x, RT* grad_residual, float* __restrict__ parts)
{
    constexpr int THREADS = TPR < 256 ? 256 : TPR;
    constexpr int RPW = THREADS / TPR;
    __shared__ float red[2][THREADS / 64];
    __shared__ __align__(16) float wsum[RPW > 1 ? RPW : 1][RPW > 1 ? TPR * CPT * 8 : 8];
    const int tl = threadIdx.x % TPR;
    float dw[CPT][8];
#pragma unroll
    for (int c = 0; c < CPT; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[c][e] = 0.0f;
    // every row group of the workgroup makes the same number of turns: barriers inside
    for (long long base = (long long)blockIdx.x * RPW; base < rows; base += (long long)gridDim.x * RPW) {
        const long long row = base + threadIdx.x / TPR;
        const bool live = row < rows;
        // all of the row's loads first: grad_residual may be dres
        Raw8<RT> a[CPT], add[CPT];
        Raw8<T> g[CPT];
#pragma unroll
        for (int c = 0; c < CPT; ++c) {
            const int col = 8 * (tl + TPR * c);
            const int n = live ? d - col : 0;
            a[c] = load_row8(r + (live ? row * r_stride : 0) + col, n);
            g[c] = load_row8(dy + (live ? row * dy_stride : 0) + col, n);
            add[c].zero();
            if (dres) add[c] = load_row8(dres + (live ? row * d : 0) + col, n);
        }
        float ss = 0.0f, sv = 0.0f;
#pragma unroll
        for (int c = 0; c < CPT; ++c) {
            const Raw8<float> w = load_row8(weight + 8 * (tl + TPR * c), d - 8 * (tl + TPR * c));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ss += a[c].get(e) * a[c].get(e);
                sv += a[c].get(e) * g[c].get(e) * w.get(e);
            }
        }
        ss = row_reduce<TPR, false>(ss, red[0]);
        sv = row_reduce<TPR, false>(sv, red[1]);
        const float k = 1.0f / sqrtf(ss / d + eps);
        const float t = k * k * (sv / d);
#pragma unroll
        for (int c = 0; c < CPT; ++c) {
            const int col = 8 * (tl + TPR * c);
            const int n = live ? d - col : 0;
            const Raw8<float> w = load_row8(weight + col, d - col);
            Raw8<T> gx;
            Raw8<RT> gr;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = k * (g[c].get(e) * w.get(e) - a[c].get(e) * t) + add[c].get(e);
                gx.set(e, v);
                gr.set(e, v);
                if (live) dw[c][e] += g[c].get(e) * a[c].get(e) * k;
            }
            if (grad_x) store_row8(grad_x + (live ? row * d : 0) + col, gx, n);
            if (grad_residual) store_row8(grad_residual + (live ? row * d : 0) + col, gr, n);
        }
    }
    if (RPW > 1) {
#pragma unroll
        for (int c = 0; c < CPT; ++c)
#pragma unroll
            for (int e = 0; e < 8; e += 4)
                *reinterpret_cast<f32x4*>(&wsum[threadIdx.x / TPR][8 * (tl + TPR * c) + e]) =
                    f32x4{dw[c][e], dw[c][e + 1], dw[c][e + 2], dw[c][e + 3]};
        __syncthreads();
        for (int col = threadIdx.x; col < d; col += THREADS) {
            float v = wsum[0][col];
#pragma unroll
            for (int k = 1; k < RPW; ++k) v += wsum[k][col];
            parts[(size_t)blockIdx.x * d + col] = v;
        }
    } else {
#pragma unroll
        for (int c = 0; c < CPT; ++c) {
            const int col = 8 * (tl + TPR * c);
            Raw8<float> o;
#pragma unroll
            for (int e = 0; e < 8; ++e) o.set(e, dw[c][e]);
            store_row8(parts + (size_t)blockIdx.x * d + col, o, d - col);
        }
    }
}

// out[c] = sum over parts of parts[p][c]: 64 columns per workgroup, the parts over its 16 waves
__global__ __launch_bounds__(1024) void sum_parts_kernel(const float* __restrict__ parts, int n, int width,
                                                         float* __restrict__ out)
{
    __shared__ float sm[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane;
    float s = 0.0f;
    if (c < width)
#pragma unroll 8
        for (int p = wave; p < n; p += 16) s += parts[(size_t)p * width + c];
    sm[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < width) {
#pragma unroll
        for (int w = 1; w < 16; ++w) s += sm[w][lane];
        out[c] = s;
    }
}

// rows per workgroup and threads per row by width (norm_variant below)
constexpr int norm_variant_rows(int v) { return v < 2 ? 4 : 1; }

// 0: a wave, d <= 512; 1: a wave, d <= 1024; 2: 256 threads, d <= 2048; 3: 256, d <= 4096;
// 4: 256, d <= 8192; 5: 1024 threads, d <= 16384
int norm_variant(int d) {
    return d <= 512 ? 0 : d <= 1024 ? 1 : d <= 2048 ? 2 : d <= 4096 ? 3 : d <= 8192 ? 4 : 5;
}

// Workgroups of the backward: two to a compute unit.  bf16 rows with an fp32 sum, 512, 1024 and
// 2048 workgroups: (rows, d) = (16384, 768) 47.5, 55.6 and 53.4 us, (8192, 2048) 55.4, 58.6 and
// 64.4 us; all bf16 (8192, 4096) 64.1, 72.2 and 70.3 us.
constexpr int NORM_BWD_GRID = 512;
int norm_bwd_grid(int rows, int d) {
    const int rpw = norm_variant_rows(norm_variant(d));
    const long long wanted = (rows + rpw - 1) / rpw;
    return (int)(wanted < NORM_BWD_GRID ? wanted : NORM_BWD_GRID);
}

#define NORM_DISPATCH(v, CALL)          \
    switch (v) {                        \
        case 0: CALL(64, 1); break;     \
        case 1: CALL(64, 2); break;     \
        case 2: CALL(256, 1); break;    \
        case 3: CALL(256, 2); break;    \
        case 4: CALL(256, 4); break;    \
        default: CALL(1024, 2); break;  \
    }

template <typename T, typename RT, bool QUANT>
hipError_t launch_fwd_t(const NormArgs& a) {
    const int v = norm_variant(a.d);
    const int rpw = norm_variant_rows(v);
    const dim3 grid((a.rows + rpw - 1) / rpw);
    if (!launchable(grid.x, v < 5 ? 256 : 1024)) return hipErrorInvalidConfiguration;
#define NORM_CALL(TPR, CPT)                                                                                     \
    hipLaunchKernelGGL((norm_fwd_kernel<T, RT, TPR, CPT, QUANT>), grid, dim3(TPR < 256 ? 256 : TPR), 0,        \
                       a.stream, (const T*)a.x, a.x_stride, (const RT*)a.residual, a.residual_stride, a.weight, \
                       a.rows, a.d, a.eps, a.group, (RT*)a.residual_out, a.y, a.scale)
    NORM_DISPATCH(v, NORM_CALL)
#undef NORM_CALL
    return hipGetLastError();
}

template <typename T, typename RT>
hipError_t launch_bwd_t(const NormArgs& a) {
    const int v = norm_variant(a.d);
    const dim3 grid(norm_bwd_grid(a.rows, a.d));
#define NORM_CALL(TPR, CPT)                                                                                     \
    hipLaunchKernelGGL((norm_bwd_kernel<T, RT, TPR, CPT>), grid, dim3(TPR < 256 ? 256 : TPR), 0, a.stream,     \
                       (const RT*)a.x, a.x_stride, a.weight, (const T*)a.dy, a.dy_stride, (const RT*)a.dres,    \
                       a.rows, a.d, a.eps, (T*)a.grad_x, (RT*)a.grad_residual, a.ws)
    NORM_DISPATCH(v, NORM_CALL)
#undef NORM_CALL
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(sum_parts_kernel, dim3((a.d + 63) / 64), dim3(1024), 0, a.stream, a.ws,
                       (int)grid.x, a.d, a.grad_weight);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_fwd(const NormArgs& a) {
    const bool b = a.dtype == MLSTM_BF16, rb = a.res_dtype == MLSTM_BF16;
    if (a.scale) {
        if (b) return rb ? launch_fwd_t<bf16, bf16, true>(a) : launch_fwd_t<bf16, float, true>(a);
        return rb ? launch_fwd_t<float, bf16, true>(a) : launch_fwd_t<float, float, true>(a);
    }
    if (b) return rb ? launch_fwd_t<bf16, bf16, false>(a) : launch_fwd_t<bf16, float, false>(a);
    return rb ? launch_fwd_t<float, bf16, false>(a) : launch_fwd_t<float, float, false>(a);
}

size_t norm_bwd_workspace_bytes(int rows, int d) {
    return (size_t)norm_bwd_grid(rows, d) * d * sizeof(float);
}

hipError_t launch_norm_bwd(const NormArgs& a) {
    const bool b = a.dtype == MLSTM_BF16, rb = a.res_dtype == MLSTM_BF16;
    if (b) return rb ? launch_bwd_t<bf16, bf16>(a) : launch_bwd_t<bf16, float>(a);
    return rb ? launch_bwd_t<float, bf16>(a) : launch_bwd_t<float, float>(a);
}

}  // namespace mlstm
