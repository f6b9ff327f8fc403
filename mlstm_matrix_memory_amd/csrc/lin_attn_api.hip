// Entry points of linear attention with a decay for each head (include/mlstm.h): argument
// validation and dispatch.
#include "block_checks.h"
#include "lin_attn_common.h"

namespace {

using namespace mlstm::checks;
using mlstm::fail;

constexpr int MAX_WIDTH = 1024;

mlstm_status check_heads(int H, int G, int dk, int dv) {
    if (H < 1 || G < 1 || H % G) return fail(MLSTM_ERR_INVALID_ARG, "H=%d is not a multiple of G=%d", H, G);
    if (dk < 1 || dk > MAX_WIDTH || dv < 1 || dv > MAX_WIDTH)
        return fail(MLSTM_ERR_INVALID_ARG, "dk=%d, dv=%d must lie in [1, %d]", dk, dv, MAX_WIDTH);
    if ((long long)H * (dk > dv ? dk : dv) > MAX_CHANNELS) return fail(MLSTM_ERR_UNSUPPORTED, "too many heads");
    return MLSTM_OK;
}

struct Inputs {
    const void* q; long long q_stride; const void* k; long long k_stride; const void* v; long long v_stride;
    const float* log_decay; const int* seq_start; const float* h_init;
    int B, S, rows, H, G, dk, dv; float scale; mlstm_dtype dtype; void* stream;
};
constexpr int INPUTS = 6;

mlstm_status check_inputs(const Inputs& i, Region* r) {
    MLSTM_TRY(check_heads(i.H, i.G, i.dk, i.dv));
    MLSTM_TRY(batch(i.B, i.S, i.rows, i.H * (i.dk > i.dv ? i.dk : i.dv), i.seq_start));
    if (!(i.scale > -3.0e38f && i.scale < 3.0e38f)) return fail(MLSTM_ERR_INVALID_ARG, "scale=%g must be finite", i.scale);
    MLSTM_TRY(dtype(i.dtype, "dtype"));
    const size_t el = elem(i.dtype), kw = (size_t)i.G * i.dk, vw = (size_t)i.H * i.dv;
    const Region in[INPUTS] = {
        strided(i.q, i.rows, kw, i.q_stride, el, "q"),
        strided(i.k, i.rows, kw, i.k_stride, el, "k"),
        strided(i.v, i.rows, vw, i.v_stride, el, "v"),
        dense(i.log_decay, i.H, 4, "log_decay"),
        dense(i.seq_start, i.B + 1, 4, "seq_start", false, true),
        dense(i.h_init, (size_t)i.B * i.H * i.dv * i.dk, 4, "h_init", false, true),
    };
    for (int n = 0; n < INPUTS; ++n) r[n] = in[n];
    return MLSTM_OK;
}

mlstm::LaBatch make(int B, int S, int rows, int H, mlstm_dtype dt, const int* seq_start) {
    mlstm::LaBatch b = {};
    b.seq_start = seq_start; b.B = B; b.S = S; b.rows = rows; b.H = H; b.dtype = dt;
    return b;
}
mlstm::LaBatch make(const Inputs& i) {
    mlstm::LaBatch b = make(i.B, i.S, i.rows, i.H, i.dtype, i.seq_start);
    b.log_decay = i.log_decay;
    b.stream = reinterpret_cast<hipStream_t>(i.stream);
    return b;
}

// every launch of a call fits before the first is made
mlstm_status check_launches(const mlstm::LaBatch& b, int dk, int dv, bool heads) {
    if (!mlstm::la_states_launchable(b, dk, dv) || !mlstm::la_out_launchable(b) || (heads && !mlstm::la_sum_heads_launchable(b)))
        return launched(hipErrorInvalidConfiguration);
    return MLSTM_OK;
}

size_t whole16(size_t n) { return (n + 15) / 16 * 16; }

// The kept states, then the segments' sums, then (backward, where heads share q and k) their gradients
// by head.  Packed batches have room for the chunks and segments that any seq_start makes.  Sequences of one chunk
// with no state at an end that needs one keep none.
bool keeps(int S, bool states) { return states || S > mlstm::LA_CHUNK; }

struct Workspace { size_t kept, parts, heads, all; };
Workspace workspace_of(const mlstm::LaBatch& b, int G, int dk, int dv, bool keep, bool backward) {
    Workspace w = {};
    w.kept = keep ? whole16(mlstm::la_kept_bytes(b, dk, dv)) : 0;
    w.parts = keep ? whole16(mlstm::la_state_parts_bytes(b, dk, dv)) : 0;
    w.heads = backward && G < b.H ? whole16((size_t)b.rows * b.H * dk * 4) : 0;
    w.all = w.kept + w.parts + w.heads;
    return w;
}

// of a call of these sizes; 0 for sizes that are refused
size_t call_bytes(int B, int S, int rows, int H, int G, int dk, int dv, mlstm_dtype dt, bool packed, bool states, bool backward) {
    if (check_heads(H, G, dk, dv) != MLSTM_OK || (dt != MLSTM_F32 && dt != MLSTM_BF16) || B < 1 || B > MAX_SEQUENCES ||
        S < 1 || rows < 1 || rows > MAX_ROWS || S > rows || (!packed && (long long)B * S != rows))
        return 0;
    const int any = 0;
    return workspace_of(make(B, S, rows, H, dt, packed ? &any : nullptr), G, dk, dv, keeps(S, states), backward).all;
}

size_t workspace_bytes_of(int B, int S, int rows, int H, int G, int dk, int dv, mlstm_dtype dt, bool backward) {
    // what a packed batch takes, or one of equal sequences, whose pieces are numbered otherwise
    const size_t packed = call_bytes(B, S, rows, H, G, dk, dv, dt, true, true, backward);
    const size_t equal = call_bytes(B, S, rows, H, G, dk, dv, dt, false, true, backward);
    return packed > equal ? packed : equal;
}

// the workspace as a tensor of the call, absent where it takes none
Region workspace_region(void* ws, size_t bytes) { return dense(bytes ? ws : nullptr, bytes, 1, "workspace", true, true); }

}  // namespace

extern "C" {

size_t lin_attn_fwd_workspace_bytes(int B, int S, int rows, int H, int G, int dk, int dv, mlstm_dtype dt) {
    return workspace_bytes_of(B, S, rows, H, G, dk, dv, dt, false);
}

size_t lin_attn_fwd_call_workspace_bytes(int B, int S, int rows, int H, int G, int dk, int dv, mlstm_dtype dt, int packed,
                                         int states) {
    return call_bytes(B, S, rows, H, G, dk, dv, dt, packed != 0, states != 0, false);
}

mlstm_status lin_attn_fwd(const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
                          long long v_stride, const float* log_decay, const int* seq_start, const float* h_init,
                          int B, int S, int rows, int H, int G, int dk, int dv, float scale, mlstm_dtype dt,
                          void* o_out, long long o_stride, float* h_final, void* ws, size_t workspace_bytes, void* stream) {
    const Inputs in = {q, q_stride, k, k_stride, v, v_stride, log_decay, seq_start, h_init, B, S, rows, H, G, dk, dv,
                       scale, dt, stream};
    Region r[INPUTS + 3];
    MLSTM_TRY(check_inputs(in, r));
    const mlstm::LaBatch b = make(in);
    MLSTM_TRY(check_launches(b, dk, dv, false));
    const bool keep = keeps(S, h_init != nullptr);
    const Workspace w = workspace_of(b, G, dk, dv, keep, false);
    MLSTM_TRY(workspace(ws, workspace_bytes, w.all, 16));
    r[INPUTS] = strided(o_out, rows, (size_t)H * dv, o_stride, elem(dt), "o_out", true);
    r[INPUTS + 1] = dense(h_final, (size_t)B * H * dv * dk, 4, "h_final", true, true);
    r[INPUTS + 2] = workspace_region(ws, w.all);
    MLSTM_TRY(regions(r, INPUTS + 3));
    MLSTM_TRY(disjoint(r, INPUTS + 3));
    const mlstm::LaRows qr = {q, q_stride, dk, H / G}, kr = {k, k_stride, dk, H / G}, vr = {v, v_stride, dv, 1};
    if (keep || h_final) {
        mlstm::LaStates s = {};
        s.x = vr; s.y = kr; s.init = h_init; s.final = h_final; s.kept = keep ? ws : nullptr; s.parts = (float*)((char*)ws + w.kept);
        MLSTM_TRY(launched(mlstm::launch_la_states(b, s)));
    }
    mlstm::LaOut o = {};
    o.a = qr; o.y = kr; o.z = vr; o.kept = ws; o.init = h_init != nullptr;
    o.state_factor = scale; o.row_factor = scale; o.out = o_out; o.out_stride = o_stride; o.out_f32 = dt == MLSTM_F32;
    return launched(mlstm::launch_la_out(b, o));
}

mlstm_status lin_attn_step(const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
                           long long v_stride, const float* log_decay, int B, int H, int G, int dk, int dv, float scale,
                           mlstm_dtype dt, float* h, void* o_out, long long o_stride, void* stream) {
    const Inputs in = {q, q_stride, k, k_stride, v, v_stride, log_decay, nullptr, nullptr, B, 1, B, H, G, dk, dv, scale, dt,
                       stream};
    Region r[INPUTS + 2];
    MLSTM_TRY(check_inputs(in, r));
    r[INPUTS] = strided(o_out, B, (size_t)H * dv, o_stride, elem(dt), "o_out", true);
    r[INPUTS + 1] = dense(h, (size_t)B * H * dv * dk, 4, "h", true);
    MLSTM_TRY(regions(r, INPUTS + 2));
    MLSTM_TRY(disjoint(r, INPUTS + 2));
    mlstm::LaStepArgs a = {};
    a.q = {q, q_stride, dk, H / G}; a.k = {k, k_stride, dk, H / G}; a.v = {v, v_stride, dv, 1};
    a.log_decay = log_decay; a.B = B; a.H = H; a.scale = scale; a.dtype = dt; a.h = h; a.out = o_out; a.out_stride = o_stride;
    a.stream = reinterpret_cast<hipStream_t>(stream);
    return launched(mlstm::launch_la_step(a));
}

size_t lin_attn_bwd_workspace_bytes(int B, int S, int rows, int H, int G, int dk, int dv, mlstm_dtype dt) {
    return workspace_bytes_of(B, S, rows, H, G, dk, dv, dt, true);
}

size_t lin_attn_bwd_call_workspace_bytes(int B, int S, int rows, int H, int G, int dk, int dv, mlstm_dtype dt, int packed,
                                         int states) {
    return call_bytes(B, S, rows, H, G, dk, dv, dt, packed != 0, states != 0, true);
}

mlstm_status lin_attn_bwd(const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
                          long long v_stride, const float* log_decay, const int* seq_start, const float* h_init,
                          const void* dout, long long do_stride, const float* dh_final,
                          int B, int S, int rows, int H, int G, int dk, int dv, float scale, mlstm_dtype dt,
                          void* grad_q, long long grad_q_stride, void* grad_k, long long grad_k_stride,
                          void* grad_v, long long grad_v_stride, float* grad_h_init,
                          void* ws, size_t workspace_bytes, void* stream) {
    const Inputs in = {q, q_stride, k, k_stride, v, v_stride, log_decay, seq_start, h_init, B, S, rows, H, G, dk, dv,
                       scale, dt, stream};
    constexpr int COUNT = INPUTS + 7;
    Region r[COUNT];
    MLSTM_TRY(check_inputs(in, r));
    const mlstm::LaBatch b = make(in);
    MLSTM_TRY(check_launches(b, dk, dv, G < H));
    const Workspace w = workspace_of(b, G, dk, dv, keeps(S, h_init || dh_final), true);
    MLSTM_TRY(workspace(ws, workspace_bytes, w.all, 16));
    const size_t el = elem(dt), kw = (size_t)G * dk, vw = (size_t)H * dv, state = (size_t)B * H * dv * dk;
    const Region more[COUNT - INPUTS] = {
        strided(dout, rows, vw, do_stride, el, "do"),
        dense(dh_final, state, 4, "dh_final", false, true),
        strided(grad_q, rows, kw, grad_q_stride, el, "grad_q", true),
        strided(grad_k, rows, kw, grad_k_stride, el, "grad_k", true),
        strided(grad_v, rows, vw, grad_v_stride, el, "grad_v", true),
        dense(grad_h_init, state, 4, "grad_h_init", true, true),
        workspace_region(ws, w.all),
    };
    for (int n = 0; n < COUNT - INPUTS; ++n) r[INPUTS + n] = more[n];
    MLSTM_TRY(regions(r, COUNT));
    MLSTM_TRY(disjoint(r, COUNT));
    const mlstm::LaRows qr = {q, q_stride, dk, H / G}, kr = {k, k_stride, dk, H / G}, vr = {v, v_stride, dv, 1},
                        dr = {dout, do_stride, dv, 1};
    float* parts = (float*)((char*)ws + w.kept);
    float* heads = (float*)((char*)ws + w.kept + w.parts);
    const bool shared = G < H, several = S > mlstm::LA_CHUNK;
    // out of q's and k's gradients: by head in fp32 first where heads share them
    auto by_head = [&](mlstm::LaOut& o, void* grad, long long stride) {
        o.out = shared ? (void*)heads : grad;
        o.out_stride = shared ? (long long)H * dk : stride;
        o.out_f32 = shared || dt == MLSTM_F32;
        mlstm_status st = launched(mlstm::launch_la_out(b, o));
        if (st != MLSTM_OK || !shared) return st;
        return launched(mlstm::launch_la_sum_heads(b, heads, G, dk, grad, stride));
    };
    // the states that enter chunks, for the gradient of q
    if (h_init || several) {
        mlstm::LaStates s = {};
        s.x = vr; s.y = kr; s.init = h_init; s.kept = ws; s.parts = parts;
        MLSTM_TRY(launched(mlstm::launch_la_states(b, s)));
    }
    mlstm::LaOut o = {};
    o.a = dr; o.y = vr; o.z = kr; o.kept = ws; o.init = h_init != nullptr; o.by_columns = true;
    o.state_factor = scale; o.row_factor = scale;
    MLSTM_TRY(by_head(o, grad_q, grad_q_stride));
    // the gradients of the states that leave them, in the same place, for the others
    if (dh_final || several || grad_h_init) {
        mlstm::LaStates s = {};
        s.x = dr; s.y = qr; s.init = dh_final; s.final = grad_h_init; s.kept = dh_final || several ? ws : nullptr; s.parts = parts;
        s.backwards = true; s.factor = scale;
        MLSTM_TRY(launched(mlstm::launch_la_states(b, s)));
    }
    o.backwards = true; o.init = dh_final != nullptr; o.state_factor = 1.0f;
    o.a = vr; o.y = dr; o.z = qr;
    MLSTM_TRY(by_head(o, grad_k, grad_k_stride));
    o.a = kr; o.y = qr; o.z = dr; o.by_columns = false;
    o.out = grad_v; o.out_stride = grad_v_stride; o.out_f32 = dt == MLSTM_F32;
    return launched(mlstm::launch_la_out(b, o));
}

}  // extern "C"
