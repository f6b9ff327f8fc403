// Entry points of the norm (include/mlstm.h): argument validation and dispatch.
#include "block_checks.h"

namespace {

using namespace mlstm::checks;
using mlstm::fail;

mlstm_status check_norm(int rows, int d, float eps, mlstm_dtype dt, mlstm_dtype res_dt) {
    if (rows < 1) return fail(MLSTM_ERR_INVALID_ARG, "rows=%d must be >= 1", rows);
    if (rows > MAX_ROWS) return fail(MLSTM_ERR_UNSUPPORTED, "rows=%d exceeds %d", rows, MAX_ROWS);
    if (d < 1 || d > mlstm::NORM_MAX_D)
        return fail(MLSTM_ERR_INVALID_ARG, "d=%d must lie in [1, %d]", d, mlstm::NORM_MAX_D);
    if (!(eps >= 0.0f) || eps > 3.0e38f) return fail(MLSTM_ERR_INVALID_ARG, "eps=%g must be finite and >= 0", eps);
    MLSTM_TRY(dtype(dt, "dtype"));
    return dtype(res_dt, "res_dtype");
}

mlstm_status norm_fwd(const void* x, long long x_stride, const void* residual, long long residual_stride,
                      const float* weight, int rows, int d, float eps, mlstm_dtype dt, mlstm_dtype res_dt, int group,
                      bool quant, void* residual_out, void* out, float* scale_out, void* stream) {
    MLSTM_TRY(check_norm(rows, d, eps, dt, res_dt));
    if (quant && group != 0 && group != 32 && group != 64 && group != 128)
        return fail(MLSTM_ERR_INVALID_ARG, "group=%d must be 0, 32, 64 or 128", group);
    const size_t n = (size_t)rows * d, per_row = group ? (d + group - 1) / group : 1;
    const Region r[] = {
        strided(x, rows, d, x_stride, elem(dt), "x"),
        strided(residual, rows, d, residual ? residual_stride : d, elem(res_dt), "residual", false, true),
        dense(weight, d, 4, "weight"),
        strided(residual_out, rows, d, d, elem(res_dt), "residual_out", true, true),
        dense(out, n, quant ? 1 : elem(dt), quant ? "q_out" : "y_out", true),
        dense(scale_out, quant ? rows * per_row : 1, 4, "scale_out", true, !quant),
    };
    const int count = (int)(sizeof(r) / sizeof(r[0]));
    MLSTM_TRY(regions(r, count));
    MLSTM_TRY(disjoint(r, count, [&](const Region& a, const Region& b) {
        return is(a, residual_out) && (is(b, residual) || (is(b, x) && dt == res_dt));
    }));
    mlstm::NormArgs a = {};
    a.x = x; a.x_stride = x_stride; a.residual = residual; a.residual_stride = residual_stride; a.weight = weight;
    a.rows = rows; a.d = d; a.eps = eps; a.dtype = dt; a.res_dtype = res_dt; a.group = group;
    a.residual_out = residual_out; a.y = out; a.scale = quant ? scale_out : nullptr;
    a.stream = reinterpret_cast<hipStream_t>(stream);
    return launched(mlstm::launch_norm_fwd(a));
}

}  // namespace

extern "C" {

mlstm_status mlstm_rms_norm_fwd(const void* x, long long x_stride, const void* residual, long long residual_stride,
                                const float* weight, int rows, int d, float eps, mlstm_dtype dt, mlstm_dtype res_dtype,
                                void* residual_out, void* y_out, void* stream) {
    return norm_fwd(x, x_stride, residual, residual_stride, weight, rows, d, eps, dt, res_dtype, 0, false,
                    residual_out, y_out, nullptr, stream);
}

mlstm_status mlstm_rms_norm_quant(const void* x, long long x_stride, const void* residual, long long residual_stride,
                                  const float* weight, int rows, int d, float eps, mlstm_dtype dt,
                                  mlstm_dtype res_dtype, int group, void* residual_out, void* q_out,
                                  float* scale_out, void* stream) {
    return norm_fwd(x, x_stride, residual, residual_stride, weight, rows, d, eps, dt, res_dtype, group, true,
                    residual_out, q_out, scale_out, stream);
}

size_t mlstm_rms_norm_bwd_workspace_bytes(int rows, int d) {
    if (check_norm(rows, d, 0.0f, MLSTM_F32, MLSTM_F32) != MLSTM_OK) return 0;
    return mlstm::norm_bwd_workspace_bytes(rows, d);
}

mlstm_status mlstm_rms_norm_bwd(const void* r, long long r_stride, const float* weight,
                                const void* dy, long long dy_stride, const void* dres,
                                int rows, int d, float eps, mlstm_dtype dt, mlstm_dtype res_dtype,
                                void* grad_x, void* grad_residual, float* grad_weight,
                                void* ws, size_t workspace_bytes, void* stream) {
    MLSTM_TRY(check_norm(rows, d, eps, dt, res_dtype));
    if (!grad_x && !grad_residual)
        return fail(MLSTM_ERR_INVALID_ARG, "grad_x and grad_residual are both NULL");
    const size_t need = mlstm::norm_bwd_workspace_bytes(rows, d);
    MLSTM_TRY(workspace(ws, workspace_bytes, need, 4));
    const Region t[] = {
        strided(r, rows, d, r_stride, elem(res_dtype), "r"),
        dense(weight, d, 4, "weight"),
        strided(dy, rows, d, dy_stride, elem(dt), "dy"),
        strided(dres, rows, d, d, elem(res_dtype), "dres", false, true),
        strided(grad_x, rows, d, d, elem(dt), "grad_x", true, true),
        strided(grad_residual, rows, d, d, elem(res_dtype), "grad_residual", true, true),
        dense(grad_weight, d, 4, "grad_weight", true),
        dense(ws, need, 1, "workspace", true),
    };
    const int count = (int)(sizeof(t) / sizeof(t[0]));
    MLSTM_TRY(regions(t, count));
    MLSTM_TRY(disjoint(t, count, [&](const Region& a, const Region& b) {
        return is(a, grad_residual) && is(b, dres);
    }));
    mlstm::NormArgs a = {};
    a.x = r; a.x_stride = r_stride; a.weight = weight; a.dy = dy; a.dy_stride = dy_stride; a.dres = dres;
    a.rows = rows; a.d = d; a.eps = eps; a.dtype = dt; a.res_dtype = res_dtype;
    a.grad_x = grad_x; a.grad_residual = grad_residual; a.grad_weight = grad_weight; a.ws = (float*)ws;
    a.stream = reinterpret_cast<hipStream_t>(stream);
    return launched(mlstm::launch_norm_bwd(a));
}

}  // extern "C"
