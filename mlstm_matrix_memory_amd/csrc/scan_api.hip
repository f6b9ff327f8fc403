// Entry points of the selective state space scan (include/mlstm.h): argument
// validation and dispatch.
#include "block_checks.h"

namespace {

using namespace mlstm::checks;
using mlstm::fail;

mlstm_status check_scan(int B, int rows, int D, int G, int N) {
    if (G < 1 || D % G) return fail(MLSTM_ERR_INVALID_ARG, "D=%d is not a multiple of G=%d", D, G);
    if (N < 1 || N > mlstm::SCAN_MAX_N)
        return fail(MLSTM_ERR_INVALID_ARG, "N=%d must lie in [1, %d]", N, mlstm::SCAN_MAX_N);
    // workgroups: tiles of 64 channels times pieces, of which there are at most rows / 16 + B; 256
    // states each in the step; 256 elements of B and C each in the backward's sums
    const long long tiles = (long long)G * ((D / G + 63) / 64), bc = (long long)G * N;
    if (tiles * (rows / 16 + B) > MAX_GRID || bc > MAX_CHANNELS || rows * bc / 128 >= MAX_GRID ||
        (long long)B * D / 64 >= MAX_GRID)
        return fail(MLSTM_ERR_UNSUPPORTED, "batch too large");
    return MLSTM_OK;
}

struct Inputs {
    const void* x; long long x_stride; const void* dt; long long dt_stride; const float* A;
    const void* Bm; long long B_stride; const void* Cm; long long C_stride;
    const float* Dskip; const float* dt_bias; const void* z; long long z_stride;
    const int* seq_start; const float* h_init;
    int B, S, rows, D, G, N, softplus; mlstm_dtype dtype; void* stream;
};
constexpr int INPUTS = 10;

mlstm_status check_inputs(const Inputs& i, Region* r) {
    MLSTM_TRY(batch(i.B, i.S, i.rows, i.D, i.seq_start));
    MLSTM_TRY(check_scan(i.B, i.rows, i.D, i.G, i.N));
    if (i.softplus != 0 && i.softplus != 1)
        return fail(MLSTM_ERR_INVALID_ARG, "softplus=%d is neither 0 nor 1", i.softplus);
    MLSTM_TRY(dtype(i.dtype, "dtype"));
    const size_t el = elem(i.dtype), D = i.D, bc = (size_t)i.G * i.N;
    const Region in[INPUTS] = {
        strided(i.x, i.rows, D, i.x_stride, el, "x"),
        strided(i.dt, i.rows, D, i.dt_stride, el, "dt"),
        dense(i.A, D * i.N, 4, "A"),
        strided(i.Bm, i.rows, bc, i.B_stride, el, "Bm"),
        strided(i.Cm, i.rows, bc, i.C_stride, el, "Cm"),
        dense(i.Dskip, D, 4, "Dskip", false, true),
        dense(i.dt_bias, D, 4, "dt_bias", false, true),
        strided(i.z, i.rows, D, i.z ? i.z_stride : (long long)D, el, "z", false, true),
        dense(i.seq_start, i.B + 1, 4, "seq_start", false, true),
        dense(i.h_init, (size_t)i.B * D * i.N, 4, "h_init", false, true),
    };
    for (int k = 0; k < INPUTS; ++k) r[k] = in[k];
    return MLSTM_OK;
}

mlstm::ScanArgs make(const Inputs& i) {
    mlstm::ScanArgs a = {};
    a.x = i.x; a.x_stride = i.x_stride; a.dt = i.dt; a.dt_stride = i.dt_stride; a.A = i.A;
    a.Bm = i.Bm; a.B_stride = i.B_stride; a.Cm = i.Cm; a.C_stride = i.C_stride;
    a.Dskip = i.Dskip; a.dt_bias = i.dt_bias; a.z = i.z; a.z_stride = i.z_stride;
    a.seq_start = i.seq_start; a.h_init = i.h_init;
    a.B = i.B; a.S = i.S; a.rows = i.rows; a.D = i.D; a.G = i.G; a.N = i.N; a.softplus = i.softplus; a.dtype = i.dtype;
    a.stream = reinterpret_cast<hipStream_t>(i.stream);
    return a;
}

bool sizes_ok(int B, int S, int rows, int D, int G, int N) {
    return B >= 1 && S >= 1 && D >= 1 && B <= MAX_SEQUENCES && rows >= 1 && rows <= MAX_ROWS && S <= rows &&
           D <= MAX_CHANNELS &&
           check_scan(B, rows, D, G, N) == MLSTM_OK;
}

}  // namespace

extern "C" {

size_t ssm_scan_fwd_workspace_bytes(int B, int S, int rows, int D, int G, int N) {
    return sizes_ok(B, S, rows, D, G, N) ? mlstm::scan_fwd_workspace_bytes(B, S, rows, D, G, N) : 0;
}

mlstm_status ssm_scan_fwd(const void* x, long long x_stride, const void* dt, long long dt_stride,
                          const float* A, const void* Bm, long long B_stride, const void* Cm, long long C_stride,
                          const float* Dskip, const float* dt_bias, const void* z, long long z_stride,
                          const int* seq_start, const float* h_init,
                          int B, int S, int rows, int D, int G, int N, int softplus, mlstm_dtype dtype,
                          void* y_out, long long y_stride, float* h_final,
                          void* ws, size_t workspace_bytes, void* stream) {
    const Inputs in = {x, x_stride, dt, dt_stride, A, Bm, B_stride, Cm, C_stride, Dskip, dt_bias, z, z_stride,
                       seq_start, h_init, B, S, rows, D, G, N, softplus, dtype, stream};
    Region r[INPUTS + 3];
    MLSTM_TRY(check_inputs(in, r));
    const size_t need = mlstm::scan_fwd_workspace_bytes(B, S, rows, D, G, N);
    MLSTM_TRY(workspace(ws, workspace_bytes, need, 16));
    r[INPUTS] = strided(y_out, rows, D, y_stride, elem(dtype), "y_out", true);
    r[INPUTS + 1] = dense(h_final, (size_t)B * D * N, 4, "h_final", true, true);
    r[INPUTS + 2] = dense(need ? ws : nullptr, need, 1, "workspace", true, true);
    MLSTM_TRY(regions(r, INPUTS + 3));
    MLSTM_TRY(disjoint(r, INPUTS + 3));
    mlstm::ScanArgs a = make(in);
    a.y = y_out; a.y_stride = y_stride; a.h_final = h_final; a.ws = (float*)ws;
    return launched(mlstm::launch_scan_fwd(a));
}

mlstm_status ssm_step(const void* x, long long x_stride, const void* dt, long long dt_stride,
                      const float* A, const void* Bm, long long B_stride, const void* Cm, long long C_stride,
                      const float* Dskip, const float* dt_bias, const void* z, long long z_stride,
                      int B, int D, int G, int N, int softplus, mlstm_dtype dtype,
                      float* h, void* y_out, long long y_stride, void* stream) {
    const Inputs in = {x, x_stride, dt, dt_stride, A, Bm, B_stride, Cm, C_stride, Dskip, dt_bias, z, z_stride,
                       nullptr, nullptr, B, 1, B, D, G, N, softplus, dtype, stream};
    Region r[INPUTS + 2];
    MLSTM_TRY(check_inputs(in, r));
    r[INPUTS] = strided(y_out, B, D, y_stride, elem(dtype), "y_out", true);
    r[INPUTS + 1] = dense(h, (size_t)B * D * N, 4, "h", true);
    MLSTM_TRY(regions(r, INPUTS + 2));
    MLSTM_TRY(disjoint(r, INPUTS + 2));
    mlstm::ScanArgs a = make(in);
    a.y = y_out; a.y_stride = y_stride; a.h_final = h;
    return launched(mlstm::launch_ssm_step(a));
}

size_t ssm_scan_bwd_workspace_bytes(int B, int S, int rows, int D, int G, int N) {
    if (!sizes_ok(B, S, rows, D, G, N)) return 0;
    return mlstm::scan_bwd_workspace_bytes(B, S, rows, D, G, N);
}

mlstm_status ssm_scan_bwd(const void* x, long long x_stride, const void* dt, long long dt_stride,
                          const float* A, const void* Bm, long long B_stride, const void* Cm, long long C_stride,
                          const float* Dskip, const float* dt_bias, const void* z, long long z_stride,
                          const int* seq_start, const float* h_init,
                          const void* dy, long long dy_stride, const float* dh_final,
                          int B, int S, int rows, int D, int G, int N, int softplus, mlstm_dtype dtype,
                          void* grad_x, long long grad_x_stride, void* grad_dt, long long grad_dt_stride,
                          void* grad_z, long long grad_z_stride,
                          void* grad_B, long long grad_B_stride, void* grad_C, long long grad_C_stride,
                          float* grad_A, float* grad_Dskip, float* grad_dt_bias, float* grad_h_init,
                          void* ws, size_t workspace_bytes, void* stream) {
    const Inputs in = {x, x_stride, dt, dt_stride, A, Bm, B_stride, Cm, C_stride, Dskip, dt_bias, z, z_stride,
                       seq_start, h_init, B, S, rows, D, G, N, softplus, dtype, stream};
    constexpr int COUNT = INPUTS + 12;
    Region r[COUNT];
    MLSTM_TRY(check_inputs(in, r));
    const size_t need = mlstm::scan_bwd_workspace_bytes(B, S, rows, D, G, N);
    MLSTM_TRY(workspace(ws, workspace_bytes, need, 16));
    if (!z && grad_z) return fail(MLSTM_ERR_INVALID_ARG, "grad_z is given without z");
    if (!Dskip && grad_Dskip) return fail(MLSTM_ERR_INVALID_ARG, "grad_Dskip is given without Dskip");
    if (!dt_bias && grad_dt_bias) return fail(MLSTM_ERR_INVALID_ARG, "grad_dt_bias is given without dt_bias");
    const size_t el = elem(dtype), w = D, bc = (size_t)G * N, st = (size_t)B * D * N;
    const Region more[COUNT - INPUTS] = {
        strided(dy, rows, w, dy_stride, el, "dy"),
        dense(dh_final, st, 4, "dh_final", false, true),
        strided(grad_x, rows, w, grad_x_stride, el, "grad_x", true),
        strided(grad_dt, rows, w, grad_dt_stride, el, "grad_dt", true),
        strided(grad_z, rows, w, z ? grad_z_stride : (long long)D, el, "grad_z", true, !z),
        strided(grad_B, rows, bc, grad_B_stride, el, "grad_B", true),
        strided(grad_C, rows, bc, grad_C_stride, el, "grad_C", true),
        dense(grad_A, w * N, 4, "grad_A", true),
        dense(grad_Dskip, w, 4, "grad_Dskip", true, !Dskip),
        dense(grad_dt_bias, w, 4, "grad_dt_bias", true, !dt_bias),
        dense(grad_h_init, st, 4, "grad_h_init", true, true),
        dense(ws, need, 1, "workspace", true),
    };
    for (int k = 0; k < COUNT - INPUTS; ++k) r[INPUTS + k] = more[k];
    MLSTM_TRY(regions(r, COUNT));
    MLSTM_TRY(disjoint(r, COUNT));
    mlstm::ScanArgs a = make(in);
    a.dy = dy; a.dy_stride = dy_stride; a.dh_final = dh_final;
    a.grad_x = grad_x; a.grad_x_stride = grad_x_stride; a.grad_dt = grad_dt; a.grad_dt_stride = grad_dt_stride;
    a.grad_z = grad_z; a.grad_z_stride = grad_z_stride; a.grad_B = grad_B; a.grad_B_stride = grad_B_stride;
    a.grad_C = grad_C; a.grad_C_stride = grad_C_stride; a.grad_A = grad_A; a.grad_Dskip = grad_Dskip;
    a.grad_dt_bias = grad_dt_bias; a.grad_h = grad_h_init; a.ws = (float*)ws;
    return launched(mlstm::launch_scan_bwd(a));
}

}  // extern "C"
