// Layout shared by the selective scan's kernels over sequences.
//
// A workgroup runs SCAN_TILE = 64 neighbouring channels of one group; its NW scanning waves
// split the NP = NW * NL (>= N, the states past N are zero) states.  In the forward and
// in the backward's first kernel a lane is a channel and a wave has NL of its states in
// registers, so the recurrence needs no exchange between lanes.  B_t[n] is then the
// same for all lanes of a wave: every 16 lanes hold NL of them, one per lane, and the
// products read them through the DPP row broadcast, which costs no instruction of its own;
// C_t[n] is read so in the backward's first kernel, and as vectors from LDS in the forward.
// The backward's main kernel lays its states out otherwise (described there).
#pragma once

#include <utility>

#include "block_internal.h"

namespace mlstm {

constexpr int SCAN_TILE = 64;                    // channels per workgroup

// value of lane J of each 16-lane row
template <int J>
__device__ __forceinline__ float row_broadcast(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x150 + J, 0xF, 0xF, true));
}

// f(std::integral_constant<int, 0>) ... f(std::integral_constant<int, N - 1>)
template <typename F, int... J>
__device__ __forceinline__ void for_each_j(F&& f, std::integer_sequence<int, J...>) {
    (f(std::integral_constant<int, J>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void for_each(F&& f) { for_each_j(f, std::make_integer_sequence<int, N>{}); }

// which channels a tile holds
struct ScanTile { int group, d0, count; };
__host__ __device__ inline int scan_tiles(int D, int G) { return G * ((D / G + SCAN_TILE - 1) / SCAN_TILE); }
__device__ __forceinline__ ScanTile scan_tile(int tile, int D, int G) {
    const int per = (D / G + SCAN_TILE - 1) / SCAN_TILE;
    const int g = tile / per, first = (tile % per) * SCAN_TILE;
    return ScanTile{g, g * (D / G) + first, min(SCAN_TILE, D / G - first)};
}

// waves and states per wave by N: NP = 4, 8, 16, 32 or 64
#define SCAN_DISPATCH_N(N, CALL)         \
    if ((N) <= 4) { CALL(1, 4); }        \
    else if ((N) <= 8) { CALL(2, 4); }   \
    else if ((N) <= 16) { CALL(4, 4); }  \
    else if ((N) <= 32) { CALL(4, 8); }  \
    else { CALL(4, 16); }
inline int scan_padded_states(int N) { return N <= 4 ? 4 : N <= 8 ? 8 : N <= 16 ? 16 : N <= 32 ? 32 : 64; }

}  // namespace mlstm
