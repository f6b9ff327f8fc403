// Internal declarations of the block operators: the norm, the short convolution
// and the selective state space scan (gfx950 only).
#pragma once

#include "mlstm_internal.h"

namespace mlstm {

// ---- eight consecutive elements of a row ------------------------------------
// Rows may start at any element, so the vector types claim the alignment of one
// element only; the hardware takes a 16-byte access at any address.
typedef __bf16 bf16x8_u __attribute__((ext_vector_type(8), aligned(2)));
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));

template <typename T> struct Raw8;
template <> struct Raw8<bf16> {
    bf16x8 v;
    __device__ __forceinline__ float get(int e) const { return (float)v[e]; }
    __device__ __forceinline__ void set(int e, float x) { v[e] = (bf16)x; }
    __device__ __forceinline__ void load(const bf16* p) { v = *reinterpret_cast<const bf16x8_u*>(p); }
    __device__ __forceinline__ void store(bf16* p) const { *reinterpret_cast<bf16x8_u*>(p) = v; }
    __device__ __forceinline__ void zero() { v = bf16x8{0, 0, 0, 0, 0, 0, 0, 0}; }
};
template <> struct Raw8<float> {
    f32x4 a, b;
    __device__ __forceinline__ float get(int e) const { return e < 4 ? a[e & 3] : b[e & 3]; }
    __device__ __forceinline__ void set(int e, float x) { if (e < 4) a[e & 3] = x; else b[e & 3] = x; }
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const f32x4_u*>(p);
        b = *reinterpret_cast<const f32x4_u*>(p + 4);
    }
    __device__ __forceinline__ void store(float* p) const {
        *reinterpret_cast<f32x4_u*>(p) = a;
        *reinterpret_cast<f32x4_u*>(p + 4) = b;
    }
    __device__ __forceinline__ void zero() { a = f32x4{0, 0, 0, 0}; b = a; }
};

// the first n (<= 8, may be <= 0) of eight elements at p; the others are zero / not stored
template <typename T>
__device__ __forceinline__ Raw8<T> load_row8(const T* p, int n) {
    Raw8<T> r;
    if (n >= 8) {
        r.load(p);
    } else {
        r.zero();
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < n) r.set(e, to_f32(p[e]));
    }
    return r;
}
template <typename T>
__device__ __forceinline__ void store_row8(T* p, const Raw8<T>& r, int n) {
    if (n >= 8) {
        r.store(p);
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < n) p[e] = from_f32<T>(r.get(e));
    }
}

// four consecutive elements, likewise
typedef __bf16 bf16x4_u __attribute__((ext_vector_type(4), aligned(2)));
template <typename T> struct Raw4;
template <> struct Raw4<bf16> {
    bf16x4 v;
    __device__ __forceinline__ float get(int e) const { return (float)v[e]; }
    __device__ __forceinline__ void set(int e, float x) { v[e] = (bf16)x; }
    __device__ __forceinline__ void load(const bf16* p) { v = *reinterpret_cast<const bf16x4_u*>(p); }
    __device__ __forceinline__ void store(bf16* p) const { *reinterpret_cast<bf16x4_u*>(p) = v; }
    __device__ __forceinline__ void zero() { v = bf16x4{0, 0, 0, 0}; }
};
template <> struct Raw4<float> {
    f32x4 v;
    __device__ __forceinline__ float get(int e) const { return v[e]; }
    __device__ __forceinline__ void set(int e, float x) { v[e] = x; }
    __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const f32x4_u*>(p); }
    __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<f32x4_u*>(p) = v; }
    __device__ __forceinline__ void zero() { v = f32x4{0, 0, 0, 0}; }
};
template <typename T>
__device__ __forceinline__ Raw4<T> load_row4(const T* p, int n) {
    Raw4<T> r;
    if (n >= 4) {
        r.load(p);
    } else {
        r.zero();
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < n) r.set(e, to_f32(p[e]));
    }
    return r;
}
template <typename T>
__device__ __forceinline__ void store_row4(T* p, const Raw4<T>& r, int n) {
    if (n >= 4) {
        r.store(p);
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < n) p[e] = from_f32<T>(r.get(e));
    }
}

// ---- elementwise functions on the hardware exp, log and reciprocal -----------
// (each within about 1 ulp)
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

__device__ __forceinline__ float sigmoid_hw(float x) {
    // e^-x overflows to infinity below -88, where the reciprocal gives the limit 0
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-LOG2E * x));
}

// softplus(v) = log(1 + e^v), v itself above 20 (where the difference is below half
// a unit in the last place).  log(w) e / (w - 1) with w = 1 + e rounded keeps the
// relative accuracy of a small e, whose low bits w has lost: the rounding of w
// cancels between the logarithm and the difference (Kahan's log1p).
__device__ __forceinline__ float softplus_hw(float v) {
    const float e = __builtin_amdgcn_exp2f(LOG2E * v);
    const float w = 1.0f + e;
    const float l = __builtin_amdgcn_logf(w) * LN2 * e * __builtin_amdgcn_rcpf(w - 1.0f);
    // selects, not branches: a wave's elements then run through the pipeline together
    const float r = __builtin_unpredictable(w == 1.0f) ? e : l;
    return __builtin_unpredictable(v > 20.0f) ? v : r;
}

// ---- rows of a sequence --------------------------------------------------------
struct RowRange { int lo, n; };        // first row, number of rows

// Entries of seq_start come from device memory that no host check has seen: both
// ends are clamped into [0, rows] and the length to S.
__device__ __forceinline__ RowRange sequence_rows(const int* seq_start, int b, int S, int rows) {
    if (!seq_start) return RowRange{b * S, S};
    const int lo = min(max(seq_start[b], 0), rows);
    const int hi = min(max(seq_start[b + 1], lo), rows);
    return RowRange{lo, min(hi - lo, S)};
}

// A batch cut into pieces of `length` rows, numbered through all sequences: `per`
// pieces for each of equal length, or, packed, sequence b's pieces from number
// lo / length + b on, which leaves room for its last, shorter one (no two sequences
// share a number, and count() bounds them all by the rows that there are, however
// unequal the sequences).
struct Pieces {
    const int* seq_start;
    int B, S, rows, length, per;
    struct At { int b, c; };             // the c-th piece of sequence b
    // Numbers in front of the first sequence's own, where rows lie before it, are no piece: c is
    // then NONE, whose rows (c * length) are past every sequence's end, like those of numbers
    // between two sequences.
    static constexpr int NONE = 0x7fffffff;
    __host__ __device__ int count() const { return seq_start ? rows / length + B : B * per; }
    __device__ __forceinline__ int first(int b, const RowRange& sq) const {
        return seq_start ? sq.lo / length + b : b * per;
    }
    __device__ __forceinline__ At at(int number) const {
        if (!seq_start) return At{number / per, number % per};
        int b = 0, end = B;              // the last sequence whose first number is not above this one
        while (end - b > 1) {
            const int mid = (b + end) >> 1;
            if (min(max(seq_start[mid], 0), rows) / length + mid <= number) b = mid;
            else end = mid;
        }
        const int c = number - (min(max(seq_start[b], 0), rows) / length + b);
        return At{b, c < 0 ? NONE : c};
    }
    __device__ __forceinline__ RowRange sequence(int b) const { return sequence_rows(seq_start, b, S, rows); }
    // whether a sequence has the row
    __device__ __forceinline__ bool has(int row) const {
        if (!seq_start) return true;
        int b = 0, end = B;              // the last sequence that starts at the row or before it
        while (end - b > 1) {
            const int mid = (b + end) >> 1;
            if (seq_start[mid] <= row) b = mid;
            else end = mid;
        }
        const RowRange sq = sequence(b);
        return row >= sq.lo && row < sq.lo + sq.n;
    }
};
inline Pieces make_pieces(const int* seq_start, int B, int S, int rows, int length) {
    return Pieces{seq_start, B, S, rows, length, (S + length - 1) / length};
}

// ---- launchers -------------------------------------------------------------------
// One launch takes at most 2^32 - 1 threads; the launchers return
// hipErrorInvalidConfiguration, before any kernel of the call, where it would be more.
inline bool launchable(long long groups, int threads) { return groups <= 0xffffffffLL / threads; }

struct NormArgs {
    const void* x; long long x_stride;               // rows of the input (backward: r)
    const void* residual; long long residual_stride; // or null
    const float* weight;
    int rows, d;
    float eps;
    mlstm_dtype dtype, res_dtype;
    int group;                                       // columns per scale (quantised output)
    void* residual_out;                              // or null
    void* y;                                         // dtype, or e4m3 bytes where scale is given
    float* scale;                                    // null: y in dtype
    const void* dy; long long dy_stride;
    const void* dres;
    void* grad_x; void* grad_residual; float* grad_weight;
    float* ws;
    hipStream_t stream;
};
constexpr int NORM_MAX_D = 16384;
hipError_t launch_norm_fwd(const NormArgs& a);
size_t norm_bwd_workspace_bytes(int rows, int d);
hipError_t launch_norm_bwd(const NormArgs& a);

struct ConvArgs {
    const void* x; long long x_stride;
    const float* weight; const float* bias;          // bias or null
    const int* seq_start; const void* state_init;    // or null
    int B, S, rows, D, width;
    int act;                                         // 0 none, 1 swish
    mlstm_dtype dtype;
    void* y; long long y_stride;
    void* state_final;                               // or null (step: the state itself)
    const void* dy; long long dy_stride;
    const void* dstate_final;                        // or null
    void* grad_x; long long grad_x_stride;
    float* grad_weight; float* grad_bias;            // grad_bias or null
    void* grad_state;                                // or null
    float* ws;
    hipStream_t stream;
};
hipError_t launch_conv_fwd(const ConvArgs& a);
hipError_t launch_conv_step(const ConvArgs& a);
size_t conv_bwd_workspace_bytes(int B, int rows, int D, int width);
hipError_t launch_conv_bwd(const ConvArgs& a);

struct ScanArgs {
    const void* x; long long x_stride;
    const void* dt; long long dt_stride;
    const float* A;
    const void* Bm; long long B_stride;
    const void* Cm; long long C_stride;
    const float* Dskip; const float* dt_bias;        // or null
    const void* z; long long z_stride;               // or null
    const int* seq_start; const float* h_init;       // or null
    int B, S, rows, D, G, N;
    int softplus;
    mlstm_dtype dtype;
    void* y; long long y_stride;
    float* h_final;                                  // or null (step: the state itself)
    float* ws;
    hipStream_t stream;
    // backward
    const void* dy; long long dy_stride;
    const float* dh_final;                           // or null
    void* grad_x; long long grad_x_stride;
    void* grad_dt; long long grad_dt_stride;
    void* grad_z; long long grad_z_stride;           // null where z is
    void* grad_B; long long grad_B_stride;
    void* grad_C; long long grad_C_stride;
    float* grad_A; float* grad_Dskip; float* grad_dt_bias;
    float* grad_h;                                   // or null
};
constexpr int SCAN_MAX_N = 64;
size_t scan_fwd_workspace_bytes(int B, int S, int rows, int D, int G, int N);
hipError_t launch_scan_fwd(const ScanArgs& a);
hipError_t launch_ssm_step(const ScanArgs& a);
size_t scan_bwd_workspace_bytes(int B, int S, int rows, int D, int G, int N);
hipError_t launch_scan_bwd(const ScanArgs& a);

}  // namespace mlstm
