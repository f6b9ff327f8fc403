// Entry points of the short causal convolution (include/mlstm.h): argument validation
// and dispatch.
#include "block_checks.h"

namespace {

using namespace mlstm::checks;
using mlstm::fail;

mlstm_status check_conv(int width, ssm_act act, mlstm_dtype dt) {
    if (width < 2 || width > 4) return fail(MLSTM_ERR_INVALID_ARG, "width=%d must be 2, 3 or 4", width);
    if (act != SSM_ACT_NONE && act != SSM_ACT_SWISH)
        return fail(MLSTM_ERR_INVALID_ARG, "act=%d is neither SSM_ACT_NONE nor SSM_ACT_SWISH", (int)act);
    return dtype(dt, "dtype");
}

mlstm::ConvArgs args(const void* x, long long x_stride, const float* weight, const float* bias, int B, int S, int rows,
                     int D, int width, ssm_act act, mlstm_dtype dt, void* stream) {
    mlstm::ConvArgs a = {};
    a.x = x; a.x_stride = x_stride; a.weight = weight; a.bias = bias;
    a.B = B; a.S = S; a.rows = rows; a.D = D; a.width = width; a.act = act == SSM_ACT_SWISH; a.dtype = dt;
    a.stream = reinterpret_cast<hipStream_t>(stream);
    return a;
}

}  // namespace

extern "C" {

mlstm_status ssm_conv_fwd(const void* x, long long x_stride, const float* weight, const float* bias,
                          const int* seq_start, const void* state_init,
                          int B, int S, int rows, int D, int width, ssm_act act, mlstm_dtype dt,
                          void* y_out, long long y_stride, void* state_final, void* stream) {
    MLSTM_TRY(batch(B, S, rows, D, seq_start));
    MLSTM_TRY(check_conv(width, act, dt));
    const size_t el = elem(dt), st = (size_t)B * (width - 1) * D;
    const Region r[] = {
        strided(x, rows, D, x_stride, el, "x"),
        dense(weight, (size_t)D * width, 4, "weight"),
        dense(bias, D, 4, "bias", false, true),
        dense(seq_start, B + 1, 4, "seq_start", false, true),
        dense(state_init, st, el, "state_init", false, true),
        strided(y_out, rows, D, y_stride, el, "y_out", true),
        dense(state_final, st, el, "state_final", true, true),
    };
    MLSTM_TRY(regions(r, 7));
    MLSTM_TRY(disjoint(r, 7));
    mlstm::ConvArgs a = args(x, x_stride, weight, bias, B, S, rows, D, width, act, dt, stream);
    a.seq_start = seq_start; a.state_init = state_init; a.y = y_out; a.y_stride = y_stride; a.state_final = state_final;
    return launched(mlstm::launch_conv_fwd(a));
}

mlstm_status ssm_conv_step(const void* x, long long x_stride, const float* weight, const float* bias,
                           int B, int D, int width, ssm_act act, mlstm_dtype dt,
                           void* state, void* y_out, long long y_stride, void* stream) {
    MLSTM_TRY(batch(B, 1, B, D, nullptr));
    MLSTM_TRY(check_conv(width, act, dt));
    const size_t el = elem(dt);
    const Region r[] = {
        strided(x, B, D, x_stride, el, "x"),
        dense(weight, (size_t)D * width, 4, "weight"),
        dense(bias, D, 4, "bias", false, true),
        dense(state, (size_t)B * (width - 1) * D, el, "state", true),
        strided(y_out, B, D, y_stride, el, "y_out", true),
    };
    MLSTM_TRY(regions(r, 5));
    MLSTM_TRY(disjoint(r, 5));
    mlstm::ConvArgs a = args(x, x_stride, weight, bias, B, 1, B, D, width, act, dt, stream);
    a.y = y_out; a.y_stride = y_stride; a.state_final = state;
    return launched(mlstm::launch_conv_step(a));
}

size_t ssm_conv_bwd_workspace_bytes(int B, int rows, int D, int width) {
    if (B < 1 || rows < 1 || D < 1 || B > MAX_SEQUENCES || rows > MAX_ROWS || D > MAX_CHANNELS) return 0;
    if (check_conv(width, SSM_ACT_NONE, MLSTM_F32) != MLSTM_OK) return 0;
    return mlstm::conv_bwd_workspace_bytes(B, rows, D, width);
}

mlstm_status ssm_conv_bwd(const void* x, long long x_stride, const float* weight, const float* bias,
                          const int* seq_start, const void* state_init,
                          const void* dy, long long dy_stride, const void* dstate_final,
                          int B, int S, int rows, int D, int width, ssm_act act, mlstm_dtype dt,
                          void* grad_x, long long grad_x_stride, float* grad_weight, float* grad_bias,
                          void* grad_state_init, void* ws, size_t workspace_bytes, void* stream) {
    MLSTM_TRY(batch(B, S, rows, D, seq_start));
    MLSTM_TRY(check_conv(width, act, dt));
    const size_t need = mlstm::conv_bwd_workspace_bytes(B, rows, D, width);
    MLSTM_TRY(workspace(ws, workspace_bytes, need, 4));
    if (!bias && grad_bias) return fail(MLSTM_ERR_INVALID_ARG, "grad_bias is given without bias");
    const size_t el = elem(dt), st = (size_t)B * (width - 1) * D;
    const Region r[] = {
        strided(x, rows, D, x_stride, el, "x"),
        dense(weight, (size_t)D * width, 4, "weight"),
        dense(bias, D, 4, "bias", false, true),
        dense(seq_start, B + 1, 4, "seq_start", false, true),
        dense(state_init, st, el, "state_init", false, true),
        strided(dy, rows, D, dy_stride, el, "dy"),
        dense(dstate_final, st, el, "dstate_final", false, true),
        strided(grad_x, rows, D, grad_x_stride, el, "grad_x", true),
        dense(grad_weight, (size_t)D * width, 4, "grad_weight", true),
        dense(grad_bias, D, 4, "grad_bias", true, !bias),
        dense(grad_state_init, st, el, "grad_state_init", true, true),
        dense(ws, need, 1, "workspace", true),
    };
    MLSTM_TRY(regions(r, 12));
    MLSTM_TRY(disjoint(r, 12));
    mlstm::ConvArgs a = args(x, x_stride, weight, bias, B, S, rows, D, width, act, dt, stream);
    a.seq_start = seq_start; a.state_init = state_init; a.dy = dy; a.dy_stride = dy_stride;
    a.dstate_final = dstate_final; a.grad_x = grad_x; a.grad_x_stride = grad_x_stride;
    a.grad_weight = grad_weight; a.grad_bias = grad_bias; a.grad_state = grad_state_init; a.ws = (float*)ws;
    return launched(mlstm::launch_conv_bwd(a));
}

}  // extern "C"
