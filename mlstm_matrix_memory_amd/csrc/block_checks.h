// Argument checks shared by the block operators' entry points.  Each returns MLSTM_OK
// or records the reason and returns the status to pass on.
#pragma once

#include "block_internal.h"

namespace mlstm {
namespace checks {

#define MLSTM_TRY(call)                                \
    do {                                               \
        const mlstm_status try_ = (call);              \
        if (try_ != MLSTM_OK) return try_;             \
    } while (0)

inline size_t elem(mlstm_dtype dt) { return dt == MLSTM_BF16 ? 2 : 4; }

inline mlstm_status dtype(mlstm_dtype dt, const char* name) {
    if (dt != MLSTM_F32 && dt != MLSTM_BF16)
        return fail(MLSTM_ERR_INVALID_ARG, "%s=%d is neither MLSTM_F32 nor MLSTM_BF16", name, (int)dt);
    return MLSTM_OK;
}

// A tensor of a call: rows of `width` bytes, `stride` bytes apart.
struct Region {
    const void* p;
    size_t rows, width, stride;
    const char* name;
    size_t align;              // of its elements
    bool out;                  // written by the call
    bool optional;
    long long given;           // the stride as given, in elements
};

inline Region dense(const void* p, size_t elems, size_t el, const char* name, bool out = false, bool optional = false) {
    return Region{p, 1, elems * el, elems * el, name, el, out, optional, (long long)elems};
}
inline Region strided(const void* p, size_t rows, size_t width, long long stride, size_t el, const char* name,
                      bool out = false, bool optional = false) {
    // a stride whose bytes could pass 64 bits counts as 0, which no row has
    const size_t bytes = stride < 0 || stride > (1LL << 50) ? 0 : (size_t)stride * el;
    return Region{p, rows, width * el, bytes, name, el, out, optional, stride};
}

// null pointers, element alignment, row strides
inline mlstm_status regions(const Region* r, int n) {
    for (int i = 0; i < n; ++i) {
        if (!r[i].p) {
            if (r[i].optional) continue;
            return fail(MLSTM_ERR_INVALID_ARG, "%s is NULL", r[i].name);
        }
        if (reinterpret_cast<uintptr_t>(r[i].p) % r[i].align)
            return fail(MLSTM_ERR_INVALID_ARG, "%s is not %zu-byte aligned", r[i].name, r[i].align);
        if (r[i].stride < r[i].width || r[i].stride > ((size_t)1 << 50) / (r[i].rows ? r[i].rows : 1))
            return fail(MLSTM_ERR_INVALID_ARG, "%s_stride=%lld is out of range for rows of %zu elements", r[i].name,
                        r[i].given, r[i].width / r[i].align);
    }
    return MLSTM_OK;
}

// Whether two tensors share a byte.  Rows of one stride are compared column by column;
// otherwise the spans from first to last byte are.
inline bool share(const Region& a, const Region& b) {
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    const uintptr_t ea = pa + (a.rows - 1) * a.stride + a.width, eb = pb + (b.rows - 1) * b.stride + b.width;
    if (pa >= eb || pb >= ea) return false;
    if (a.stride != b.stride || a.rows < 2 || b.rows < 2) return true;
    const size_t off = pb >= pa ? (pb - pa) % a.stride : (a.stride - (pa - pb) % a.stride) % a.stride;
    return off < a.width || off + b.width > a.stride;
}

// no output shares memory with another tensor; same(i, j) names pairs that may be one buffer
template <typename F>
mlstm_status disjoint(const Region* r, int n, F&& same) {
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < n; ++j) {
            if (i == j || !r[i].out || !r[i].p || !r[j].p || (r[j].out && j < i)) continue;
            if (r[i].p == r[j].p && r[i].rows == r[j].rows && r[i].stride == r[j].stride &&
                r[i].width == r[j].width && same(r[i], r[j]))
                continue;
            if (share(r[i], r[j])) return fail(MLSTM_ERR_INVALID_ARG, "%s overlaps %s", r[i].name, r[j].name);
        }
    return MLSTM_OK;
}
inline mlstm_status disjoint(const Region* r, int n) {
    return disjoint(r, n, [](const Region&, const Region&) { return false; });
}

inline bool is(const Region& r, const void* p) { return r.p == p; }

inline mlstm_status workspace(const void* ws, size_t given, size_t need, size_t align) {
    if (need == 0) return MLSTM_OK;
    if (!ws || given < need)
        return fail(MLSTM_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", ws ? given : (size_t)0, need);
    if (reinterpret_cast<uintptr_t>(ws) % align)
        return fail(MLSTM_ERR_INVALID_ARG, "workspace is not %zu-byte aligned", align);
    return MLSTM_OK;
}

// sizes of a batch of sequences over rows of D channels
constexpr int MAX_SEQUENCES = 65535, MAX_ROWS = 1 << 30, MAX_CHANNELS = 1 << 24;
constexpr long long MAX_GRID = 0x7fffffffLL;
inline mlstm_status batch(int B, int S, int rows, int D, const int* seq_start) {
    if (B < 1 || S < 1 || rows < 1 || D < 1)
        return fail(MLSTM_ERR_INVALID_ARG, "B=%d, S=%d, rows=%d, D=%d must all be >= 1", B, S, rows, D);
    if (B > MAX_SEQUENCES) return fail(MLSTM_ERR_UNSUPPORTED, "B=%d exceeds %d sequences", B, MAX_SEQUENCES);
    if (!seq_start && (long long)B * S != rows)
        return fail(MLSTM_ERR_INVALID_ARG, "rows=%d is not B*S=%lld", rows, (long long)B * S);
    if (S > rows) return fail(MLSTM_ERR_INVALID_ARG, "S=%d exceeds rows=%d", S, rows);
    // row and channel indexes, also rounded up to tiles, are 32-bit in the kernels, and so is the
    // number of workgroups: at most one per 64 channels and 16 rows (or sequence)
    if (rows > MAX_ROWS || D > MAX_CHANNELS || (long long)rows * D > (1LL << 40) ||
        (long long)((D + 63) / 64) * (rows / 16 + B) > MAX_GRID)
        return fail(MLSTM_ERR_UNSUPPORTED, "tensor too large");
    if (reinterpret_cast<uintptr_t>(seq_start) % 4)
        return fail(MLSTM_ERR_INVALID_ARG, "seq_start is not 4-byte aligned");
    return MLSTM_OK;
}

inline mlstm_status launched(hipError_t e) {
    if (e == hipErrorInvalidConfiguration)
        return fail(MLSTM_ERR_UNSUPPORTED, "batch too large: more threads than one launch takes");
    if (e != hipSuccess) return fail(MLSTM_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
    return ok();
}

}  // namespace checks
}  // namespace mlstm
