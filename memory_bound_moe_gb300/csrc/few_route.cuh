// Routing of a few tokens (T <= 32) by every block on its own, in shared
// memory: at most tens of KB of logits from L2, so no block waits for another.
#pragma once

#include "moe_launch.h"
#include "route_device.cuh"

namespace moe {

constexpr int kMaxTokens = 32;                    // a token set is one 32-bit mask
constexpr int kMaxSlots = kMaxTokens * kMaxTopk;

// The batch's routing in shared memory.
struct FewRoute {
    float w[kMaxSlots];           // routing weight by slot t * k + j
    int32_t id[kMaxSlots];        // expert by slot
    uint32_t mask[1024];          // tokens of every expert; then the rank of a chosen expert
    uint32_t tokens[kMaxSlots];   // tokens of the d-th chosen expert, as a mask
    uint16_t expert[kMaxSlots];   // the d-th chosen expert, ascending
    uint16_t off[kMaxSlots];      // first activation row of the d-th chosen expert
    float row_w[kMaxSlots];       // routing weight by activation row
    uint8_t row_t[kMaxSlots];     // token by activation row
    int nd;                       // chosen experts
};

// What fc2 needs of it, left by fc1 in the workspace.
struct FewRouteCopy {
    uint32_t tokens[kMaxSlots];
    uint16_t expert[kMaxSlots];
    uint16_t off[kMaxSlots];
    uint8_t row_t[kMaxSlots];
    int nd;
};
static_assert(sizeof(FewRouteCopy) <= kFewRouteBytes, "workspace");

__device__ __forceinline__ void save_route(FewRouteCopy* to, const FewRoute& s, int S) {
    for (int i = threadIdx.x; i < S; i += int(blockDim.x)) {   // entries from nd on are not used
        to->tokens[i] = s.tokens[i];
        to->expert[i] = s.expert[i];
        to->off[i] = s.off[i];
        to->row_t[i] = s.row_t[i];
    }
    if (threadIdx.x == 0) to->nd = s.nd;
}

__device__ __forceinline__ void load_route(FewRoute& s, const FewRouteCopy* from, int S) {
    for (int i = threadIdx.x; i < S; i += int(blockDim.x)) {
        s.tokens[i] = from->tokens[i];
        s.expert[i] = from->expert[i];
        s.off[i] = from->off[i];
        s.row_t[i] = from->row_t[i];
    }
    if (threadIdx.x == 0) s.nd = from->nd;
    __syncthreads();
}

template <int EPL>
__device__ __noinline__ int route_token(const RouteArgs& a, int t) {
    const int lane = threadIdx.x % kWarp;
    uint32_t key[EPL];
    load_keys<32, EPL>(a, t, true, lane, key);
    return topk_select<32, EPL>(a, t, true, lane, key);
}

__device__ __forceinline__ void route_few(const LayerArgs& a, FewRoute& s, bool write_out) {
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    for (int e = threadIdx.x; e < a.E; e += int(blockDim.x)) s.mask[e] = 0u;
    __syncthreads();
    RouteArgs r = {};
    r.logits = a.logits;
    r.T = a.T; r.E = a.E; r.k = a.k; r.renorm = a.renorm;
    r.topk_ids = s.id;
    r.topk_weights = s.w;
    r.write_out = true;
    r.vec4 = a.E % 4 == 0 && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0;
    const int epl = (a.E + 31) / 32;
    for (int t = warp; t < a.T; t += int(blockDim.x) / kWarp) {
        const int e = epl <= 1 ? route_token<1>(r, t) : epl <= 2 ? route_token<2>(r, t) : epl <= 4 ? route_token<4>(r, t)
                    : epl <= 8 ? route_token<8>(r, t) : epl <= 16 ? route_token<16>(r, t) : route_token<32>(r, t);
        if (e >= 0) atomicOr(&s.mask[e], 1u << t);
    }
    __syncthreads();
    if (warp == 0) {   // the chosen experts in ascending order, and their activation rows
        int nd = 0, rows = 0;
        for (int e0 = 0; e0 < a.E; e0 += kWarp) {
            const int e = e0 + lane;
            const uint32_t m = e < a.E ? s.mask[e] : 0u;
            const unsigned have = __ballot_sync(kFull, m != 0u);
            int before = __popc(m);   // inclusive scan of the token counts
#pragma unroll
            for (int o = 1; o < kWarp; o <<= 1) {
                const int y = __shfl_up_sync(kFull, before, o);
                if (lane >= o) before += y;
            }
            if (m != 0u) {
                const int d = nd + __popc(have & ((1u << lane) - 1u));
                s.expert[d] = uint16_t(e);
                s.tokens[d] = m;
                s.off[d] = uint16_t(rows + before - __popc(m));
                s.mask[e] = uint32_t(d);
            }
            nd += __popc(have);
            rows += __shfl_sync(kFull, before, kWarp - 1);
        }
        if (lane == 0) s.nd = nd;
    }
    __syncthreads();
    const int S = a.T * a.k;
    for (int i = threadIdx.x; i < S; i += int(blockDim.x)) {
        const int t = i / a.k, d = int(s.mask[s.id[i]]);
        const int row = s.off[d] + __popc(s.tokens[d] & ((1u << t) - 1u));
        s.row_w[row] = s.w[i];
        s.row_t[row] = uint8_t(t);
        if (write_out) {
            if (a.topk_ids != nullptr) a.topk_ids[i] = s.id[i];
            if (a.topk_weights != nullptr) a.topk_weights[i] = s.w[i];
        }
    }
    __syncthreads();
}

}  // namespace moe
