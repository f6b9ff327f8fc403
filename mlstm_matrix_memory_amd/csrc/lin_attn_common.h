// Linear attention with a decay for each head: what its kernels share.
//
// Per head, with a constant g <= 0 and states S [dv,dk]:
//   S_t = e^g S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t
// In chunks of LA_CHUNK rows, with S the state that enters a chunk and rows i, j = 0, 1, .. of it:
//   o_i = scale (e^{g(i+1)} S q_i + sum_{j<=i} e^{g(i-j)} (q_i . k_j) v_j)
// and, with T the gradient of the state that leaves the chunk of n rows:
//   dq_i = scale (e^{g(i+1)} S^T do_i + sum_{j<=i} e^{g(i-j)} (do_i . v_j) k_j)
//   dv_j = e^{g(n-1-j)} T k_j   + scale sum_{i>=j} e^{g(i-j)} (k_j . q_i) do_i
//   dk_j = e^{g(n-1-j)} T^T v_j + scale sum_{i>=j} e^{g(i-j)} (v_j . do_i) q_i
// All four are one form, o = state part + masked products of rows, forwards or backwards in time,
// and so one kernel (lin_attn_out_kernel.hip).  The states that enter chunks and the gradients that
// leave them are sums of weighted outer products, forwards or backwards, and another
// (lin_attn_state_kernel.hip).
#pragma once

#include "block_internal.h"

namespace mlstm {

constexpr int LA_CHUNK = 128;                    // rows between two kept states
__host__ __device__ inline int la_pad(int d) { return (d + 63) / 64 * 64; }   // widths of kept states

// e^{g n}.  g below -200 counts as -200, whose every power is zero in fp32, so that minus infinity
// (forget everything) is a decay like others; NaN stays.
struct Decay {
    double g2;                                   // g log2(e)
    __device__ __forceinline__ explicit Decay(float g) : g2((g < -200.0f ? -200.0f : g) * 1.4426950408889634) {}
    __device__ __forceinline__ float operator()(int n) const { return __builtin_amdgcn_exp2f((float)(n * g2)); }
};

// x e^{g n} with the factor kept in two parts: a state passes hundreds of chunks, and its factor's
// rounding would add up in one direction
struct Factor {
    float hi, lo;
    __device__ __forceinline__ Factor(const Decay& d, int n) {
        const double f = exp2(n * d.g2);
        hi = (float)f;
        lo = (float)(f - hi);
    }
    __device__ __forceinline__ float operator()(float x) const { return fmaf(x, hi, x * lo); }
};

// Eight elements of a row, of which n are left, at p; zero where n <= 0.  WIDE: rows are a multiple of eight wide, so
// that all are there or none.  The load is then made in any case, from `spare` where none are, and kept() puts the
// zeros in when the values are used: no branch, so the compiler counts the loads in flight and waits for
// the ones it needs only (with branches it waits for all).
template <bool WIDE, typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p, int n, const T* spare) {
    if (!WIDE) return load_row8(p, n);
    Raw8<T> r;
    r.load(n > 0 ? p : spare);
    return r;
}
template <bool WIDE>
__device__ __forceinline__ Raw8<bf16> kept(const Raw8<bf16>& r, int n) {
    typedef int i32x4 __attribute__((ext_vector_type(4)));
    if (!WIDE) return r;
    i32x4 v = __builtin_bit_cast(i32x4, r.v);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = n > 0 ? v[e] : 0;
    Raw8<bf16> o;
    o.v = __builtin_bit_cast(bf16x8, v);
    return o;
}
template <bool WIDE>
__device__ __forceinline__ Raw8<float> kept(const Raw8<float>& r, int n) {
    if (!WIDE) return r;
    Raw8<float> o;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        o.a[e] = n > 0 ? r.a[e] : 0.0f;
        o.b[e] = n > 0 ? r.b[e] : 0.0f;
    }
    return o;
}

// ---- operands of the matrix instructions ---------------------------------------
// A lane's eight elements of the contraction.  bf16: one 16 x 16 x 32 instruction; fp32: eight of
// 16 x 16 x 4, which take the same elements one by one.
template <typename T> struct Frag;
template <> struct Frag<bf16> { bf16x8 v; };
template <> struct Frag<float> { float v[8]; };

__device__ __forceinline__ f32x4 mma(const Frag<bf16>& a, const Frag<bf16>& b, f32x4 c) { return mfma(a.v, b.v, c); }
__device__ __forceinline__ f32x4 mma(const Frag<float>& a, const Frag<float>& b, f32x4 c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], c, 0, 0, 0);
    return c;
}

// eight neighbours of an LDS row
__device__ __forceinline__ void frag_row(Frag<bf16>& f, const bf16* p) { f.v = *reinterpret_cast<const bf16x8*>(p); }
__device__ __forceinline__ void frag_row(Frag<float>& f, const float* p) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) f.v[e] = a[e], f.v[4 + e] = b[e];
}
__device__ __forceinline__ void lds_put(bf16* p, const Raw8<bf16>& r) { *reinterpret_cast<bf16x8*>(p) = r.v; }
__device__ __forceinline__ void lds_put(float* p, const Raw8<float>& r) {
    *reinterpret_cast<f32x4*>(p) = r.a;
    *reinterpret_cast<f32x4*>(p + 4) = r.b;
}
// column l % 16 of the 16 columns at p, rows r .. r + 3 and s .. s + 3 (the same for the 16 lanes of a group)
__device__ __forceinline__ void frag_col(Frag<bf16>& f, const bf16* p, int stride, int r, int s) {
    const int j = threadIdx.x & 15;
    f.v = cat(lds_read_tr(p + (r + (j >> 2)) * stride + 4 * (j & 3)), lds_read_tr(p + (s + (j >> 2)) * stride + 4 * (j & 3)));
}
__device__ __forceinline__ void frag_col(Frag<float>& f, const float* p, int stride, int r, int s) {
    const int j = threadIdx.x & 15;
#pragma unroll
    for (int e = 0; e < 4; ++e) f.v[e] = p[(r + e) * stride + j], f.v[4 + e] = p[(s + e) * stride + j];
}

// ---- launches --------------------------------------------------------------------
// Rows of one tensor: element (row, head, i) at row * stride + head * d + i; `per` heads of the
// call's H read one of the tensor's.
struct LaRows { const void* p; long long stride; int d, per; };

struct LaBatch {
    const int* seq_start;
    int B, S, rows, H;
    const float* log_decay;
    mlstm_dtype dtype;
    hipStream_t stream;
};

// States [dv,dk] along the sequences: sums of w x_t y_t^T (x: dv wide, y: dk wide)
//   forwards   S <- e^{gn} S + sum_t e^{g(n-1-t)} x_t y_t^T             from init, to final
//   backwards  T <- e^{gn} T + factor sum_t e^{g(t+1)} x_t y_t^T        from init (of the last row), to final
// kept: [chunk][H] states in the call's dtype, the one that enters each chunk, or null; not written for the first
// chunk without init.  Each is la_pad(dv) x la_pad(dk) in blocks of 64 x 64 (those of one 64 rows of dv
// behind each other), and a block lies as the instruction's lanes hold it: 16 x 16 tiles [dv][dk], of which
// lane l has row l % 16, columns 4 (l / 16) .. + 3.  A tile is then one run of memory for the writer's
// wave, whole lines (as rows of dk they were 32 bytes each, and HBM read what it was about to write).
// In bf16 one part of a state is kept: results are then 2.1e-3 off, with two parts (hi and lo) 1.66e-3, their own rounding, but
// the call of (1, 32768, 8 heads of 256) takes 575 us for 454, the backward of (4, 2048, 4 heads of 384) 445 for 333.
struct LaStates {
    LaRows x, y;
    const float* init;                           // [B,H,dv,dk] or null
    float* final;                                // likewise
    void* kept;
    float* parts;                                // la_state_parts_bytes(...) bytes
    bool backwards;
    float factor;
};
int la_segment_rows(const LaBatch& b, int dk, int dv);                  // 0: sequences are not cut
size_t la_state_parts_bytes(const LaBatch& b, int dk, int dv);
bool la_states_launchable(const LaBatch& b, int dk, int dv);            // whether a launch takes that many threads
hipError_t launch_la_states(const LaBatch& b, const LaStates& s);

// out_i = state_factor e^{g n_i} (state a_i) + row_factor sum_j e^{g|i-j|} (a_i . y_j) z_j
//   forwards: j <= i, n_i = i + 1; backwards: j >= i, n_i = rows of the chunk - 1 - i
// The state is [z.d, a.d] (by_columns: [a.d, z.d]), as kept by launch_la_states; without
// init the first chunk (backwards: the last) has none.
struct LaOut {
    LaRows a, y, z;
    const void* kept;
    bool init, backwards, by_columns;
    float state_factor, row_factor;
    void* out; long long out_stride;             // like z with H heads, in the call's dtype, or fp32
    bool out_f32;
};
bool la_out_launchable(const LaBatch& b);
hipError_t launch_la_out(const LaBatch& b, const LaOut& o);

// out[row][g][i] = sum of parts[row][h][i] over the heads of group g, rows of sequences only
bool la_sum_heads_launchable(const LaBatch& b);
hipError_t launch_la_sum_heads(const LaBatch& b, const float* parts, int G, int d, void* out, long long out_stride);

struct LaStepArgs {
    LaRows q, k, v;
    const float* log_decay;
    int B, H;
    float scale;
    mlstm_dtype dtype;
    float* h;
    void* out; long long out_stride;
    hipStream_t stream;
};
hipError_t launch_la_step(const LaStepArgs& a);

inline int la_chunks(const LaBatch& b) { return make_pieces(b.seq_start, b.B, b.S, b.rows, LA_CHUNK).count(); }
inline size_t la_kept_bytes(const LaBatch& b, int dk, int dv) {
    return (size_t)la_chunks(b) * b.H * la_pad(dk) * la_pad(dv) * (b.dtype == MLSTM_BF16 ? 2 : 4);
}

// neighbouring workgroups go to different dies of eight: work item of a workgroup such that each die
// takes a run of them (items are at most `groups`, a multiple of 8)
__device__ __forceinline__ int die_run(int block, int groups) { return block % 8 * (groups / 8) + block / 8; }

}  // namespace mlstm
