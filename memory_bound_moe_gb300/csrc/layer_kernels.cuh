// Kernels of a whole MoE layer for a few tokens (T <= 32) in two kernels: routing and
// fc1 with SwiGLU, then fc2 with the weighted combine.
//
//   ids, w = top-k of softmax(logits)   (as moe_route)
//   a[t, j, i]  = bf16( w[t, j] * silu(W1g[e] x_t)_i * (W1u[e] x_t)_i ),  e = ids[t, j]
//   out[t, h]   = bf16( sum_j (W2[e_j] a[t, j])_h )
//
// At a few tokens the layer is bound by the bytes of the chosen experts'
// weights, each read once. The routing weight goes into the activation before
// its one rounding (tensor cores take bfloat16 operands), so the combine is a
// plain sum over the concatenated k of all chosen experts, in float32.
//
// Routing is redundant: every block routes the whole batch in shared memory
// (tens of KB of logits at most), so no block waits for another.
//   fc1: an item is 8 R columns of one expert's activation. A tile's 16 A rows
//   are 8 gate rows and the same 8 up rows, so one lane's accumulators hold
//   both halves of a SwiGLU. The block's warps split k; blocks sweep the items
//   grid-stride. The activation is stored compactly, expert-sorted (row
//   off[d] + rank of the token among the expert's), for the tokens routed.
//   fc2: a cluster of C blocks takes 16 R output columns; its warps split the
//   (expert, k) units of all chosen experts. B columns are the tokens
//   themselves, zero where a token is not routed to the expert.
// All sums are taken in a fixed order: results do not depend on timing.
#pragma once

#include "few_device.cuh"
#include "moe_launch.h"
#include "route_device.cuh"
#include "rows_common.cuh"

namespace moe {
namespace {

constexpr int kNw = 8;
constexpr int kNt = kNw * kWarp;
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
    int nd;                       // chosen experts
};

template <int EPL>
__device__ __noinline__ int route_token(const RouteArgs& a, int t) {
    const int lane = threadIdx.x % kWarp;
    uint32_t key[EPL];
    load_keys<32, EPL>(a, t, true, lane, key);
    return topk_select<32, EPL>(a, t, true, lane, key);
}

__device__ __forceinline__ void route_few(const LayerArgs& a, FewRoute& s, bool write_out) {
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    for (int e = threadIdx.x; e < a.E; e += kNt) s.mask[e] = 0u;
    __syncthreads();
    RouteArgs r = {};
    r.logits = a.logits;
    r.T = a.T; r.E = a.E; r.k = a.k; r.renorm = a.renorm;
    r.topk_ids = s.id;
    r.topk_weights = s.w;
    r.write_out = true;
    r.vec4 = a.E % 4 == 0 && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0;
    const int epl = (a.E + 31) / 32;
    for (int t = warp; t < a.T; t += kNw) {
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
    for (int i = threadIdx.x; i < S; i += kNt) {
        const int t = i / a.k, d = int(s.mask[s.id[i]]);
        s.row_w[s.off[d] + __popc(s.tokens[d] & ((1u << t) - 1u))] = s.w[i];
        if (write_out) {
            if (a.topk_ids != nullptr) a.topk_ids[i] = s.id[i];
            if (a.topk_weights != nullptr) a.topk_weights[i] = s.w[i];
        }
    }
    __syncthreads();
}

__device__ __forceinline__ float silu(float v) { return v / (1.0f + expf(-v)); }

// The c-th set bit of m (c < popc(m)).
__device__ __forceinline__ int nth_token(uint32_t m, int c) {
    for (int i = 0; i < c; ++i) m &= m - 1u;
    return __ffs(m) - 1;
}

template <int F, int R, int NG, int U>
__global__ void __launch_bounds__(kNt, 2) fc1_kernel(LayerArgs a) {
    extern __shared__ float s_red[];             // [kNw][8 NG][16 R]
    __shared__ FewRoute s;
    constexpr int kOut = 8 * NG * 16 * R;
    pdl_wait_and_release();
    route_few(a, s, blockIdx.x == 0);
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp, g = lane / 4, q = lane % 4;
    const uint32_t K = uint32_t(a.H), I = uint32_t(a.I);
    const uint32_t rb = row_bytes<F>(K), rs = row_scales<F>(K);
    const uint32_t tiles = (I + 8 * R - 1) / (8 * R);
    const uint32_t units = ((rb + 63) / 64 + U - 1) / U;
    const uint32_t items = uint32_t(s.nd) * tiles;
    for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
        const uint32_t d = item / tiles, j0 = (item - d * tiles) * (8 * R);
        const uint32_t e = s.expert[d], tokens = s.tokens[d];
        const int m = __popc(tokens), groups = (m + 7) / 8;
        const uint16_t* xrow[NG];
#pragma unroll
        for (int n = 0; n < NG; ++n)
            xrow[n] = n * 8 + g < m ? a.x + uint64_t(nth_token(tokens, n * 8 + g)) * K : nullptr;
        const uint64_t first = uint64_t(e) * 2 * I;
        float acc[R][NG][4] = {};
        for (uint32_t u = warp; u < units; u += kNw) {
            AGran<F> w[U][R];
#pragma unroll
            for (int i = 0; i < U; ++i)
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t j = j0 + r * 8 + g;
                        const uint64_t row = first + uint64_t(h) * I + j;
                        const WRow p = {static_cast<const uint8_t*>(a.w13) + row * rb, a.w13_scales + row * rs};
                        load_gran<F>(w[i][r], h, p, j < I, u * U + i, q, rb);
                    }
#pragma unroll
            for (int i = 0; i < U; ++i)
                mma_step<F, R, NG>(acc, w[i], (1u << groups) - 1u, 1.0f, [&](int n, BGran<F>& b) {
                    load_x<F>(b, xrow[n], xrow[n] != nullptr, u * U + i, q, K);
                });
        }
        store_partial<R, NG>(s_red + warp * kOut, acc);
        __syncthreads();
        float scale = 1.0f;
        if constexpr (F == kWNvfp4) scale = 1.0f / a.w13_global[e];
        // thread -> (token of the expert, column); the two halves lie 8 rows apart
        for (int o = threadIdx.x; o < m * 8 * R; o += kNt) {
            const int c = o / (8 * R), i = o % (8 * R);
            const int at = c * (16 * R) + (i / 8) * 16 + i % 8;
            float gate = 0.0f, up = 0.0f;
#pragma unroll
            for (int w = 0; w < kNw; ++w) {
                gate += s_red[w * kOut + at];
                up += s_red[w * kOut + at + 8];
            }
            gate *= scale;
            up *= scale;
            const uint32_t row = s.off[d] + c;
            if (j0 + i < I) a.act[uint64_t(row) * I + j0 + i] = uint16_t(pack_bf16x2(s.row_w[row] * (silu(gate) * up), 0.0f));
        }
        __syncthreads();
    }
}

template <int F, int R, int NG, int U>
__global__ void __launch_bounds__(kNt, 2) fc2_kernel(LayerArgs a, uint32_t C) {
    extern __shared__ float s_red[];
    __shared__ FewRoute s;
    constexpr int kOut = 8 * NG * 16 * R;
    pdl_wait_and_release();
    route_few(a, s, false);
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp, g = lane / 4, q = lane % 4;
    const uint32_t K = uint32_t(a.I), H = uint32_t(a.H);
    const uint32_t rb = row_bytes<F>(K), rs = row_scales<F>(K);
    const uint32_t rank = blockIdx.x % C, row0 = blockIdx.x / C * (16 * R);
    const uint32_t units = ((rb + 63) / 64 + U - 1) / U;   // per expert
    const uint32_t total = uint32_t(s.nd) * units;
    // kCompact: B columns are the expert's own tokens, 8 to a group, and its
    // sums are added to the warp's part of s_red when the warp leaves the expert
    constexpr bool kCompact = WInfo<F>::kFp4 && NG > 1;
    float* s_warp = s_red + warp * kOut;
    if constexpr (kCompact) {
        for (int o = lane; o < kOut; o += kWarp) s_warp[o] = 0.0f;
        __syncwarp();
    }
    float acc[R][NG][4] = {};
    const uint32_t first = rank * kNw + warp, stride = C * kNw;
    for (uint32_t v = first; v < total; v += stride) {
        const uint32_t d = v / units, u = v - d * units;
        const uint32_t e = s.expert[d], tokens = s.tokens[d], off = s.off[d];
        const int m = __popc(tokens);
        AGran<F> w[U][R];
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t j = row0 + r * 16 + h * 8 + g;
                    const uint64_t row = uint64_t(e) * H + j;
                    const WRow p = {static_cast<const uint8_t*>(a.w2) + row * rb, a.w2_scales + row * rs};
                    load_gran<F>(w[i][r], h, p, j < H, u * U + i, q, rb);
                }
        float scale = 1.0f;
        if constexpr (F == kWNvfp4) scale = 1.0f / a.w2_global[e];
        uint32_t live = 0;   // groups with a token of this expert: warp-uniform
#pragma unroll
        for (int n = 0; n < NG; ++n)
            live |= uint32_t(kCompact ? n * 8 < m : ((tokens >> (8 * n)) & 0xffu) != 0u) << n;
#pragma unroll
        for (int i = 0; i < U; ++i)
            mma_step<F, R, NG>(acc, w[i], live, scale, [&](int n, BGran<F>& b) {
                const uint32_t c = n * 8 + g;   // column: the expert's c-th token, or token c
                const bool mine = kCompact ? int(c) < m : ((tokens >> c) & 1u) != 0u;
                const uint32_t row = off + (kCompact ? c : uint32_t(__popc(tokens & ((1u << c) - 1u))));
                load_x<F>(b, a.act + uint64_t(row) * K, mine, u * U + i, q, K);
            });
        if constexpr (kCompact) {
            if (v + stride >= total || (v + stride) / units != d) {
#pragma unroll
                for (int n = 0; n < NG; ++n) {
                    if (!((live >> n) & 1u)) continue;
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const int c = n * 8 + 2 * q + z;
                        if (c < m) {
                            float* col = s_warp + nth_token(tokens, c) * (16 * R) + g;
#pragma unroll
                            for (int r = 0; r < R; ++r) {
                                col[r * 16] += acc[r][n][z];
                                col[r * 16 + 8] += acc[r][n][z + 2];
                            }
                        }
                    }
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int z = 0; z < 4; ++z) acc[r][n][z] = 0.0f;
                }
                __syncwarp();
            }
        }
    }
    if constexpr (!kCompact) store_partial<R, NG>(s_warp, acc);
    __syncthreads();
    if (C > 1) {
        for (int o = threadIdx.x; o < kOut; o += kNt) {
            float v = s_red[o];
#pragma unroll
            for (int w = 1; w < kNw; ++w) v += s_red[w * kOut + o];
            s_red[o] = v;   // this thread alone reads and writes column o
        }
        cluster_sync();
    }
    for (int o = threadIdx.x + (C > 1 ? int(rank) * kNt : 0); o < kOut; o += kNt * int(C)) {
        float v;
        if (C > 1) {
            v = ld_cluster(s_red + o, 0);
            for (uint32_t c = 1; c < C; ++c) v += ld_cluster(s_red + o, c);
        } else {
            v = s_red[o];
#pragma unroll
            for (int w = 1; w < kNw; ++w) v += s_red[w * kOut + o];
        }
        const uint32_t t = uint32_t(o) / (16 * R), row = row0 + uint32_t(o) % (16 * R);
        if (t < uint32_t(a.T) && row < H) a.out[uint64_t(t) * H + row] = uint16_t(pack_bf16x2(v, 0.0f));
    }
    if (C > 1) cluster_sync();   // the others may still read this block's sums
}

template <int F, int NG>
cudaError_t launch_ng(const LayerArgs& a, int num_sms, cudaStream_t stream) {
    constexpr int R = WInfo<F>::kFp4 ? 2 : 1, U = WInfo<F>::kFp4 ? 2 : 4;
    constexpr size_t smem = sizeof(float) * kNw * 8 * NG * 16 * R;
    auto fc1 = fc1_kernel<F, R, NG, U>;
    auto fc2 = fc2_kernel<F, R, NG, U>;
    const uint64_t nd = std::min<uint64_t>(a.E, uint64_t(a.T) * a.k);   // most experts that can be chosen
    const uint64_t items = nd * ((uint64_t(a.I) + 8 * R - 1) / (8 * R));
    const uint32_t grid = uint32_t(std::min<uint64_t>(items, 2ull * num_sms));
    cudaError_t err = launch_pdl(fc1, dim3(grid), dim3(kNt), smem, stream, a);
    if (err != cudaSuccess) return err;
    const uint32_t tiles = (uint32_t(a.H) + 16 * R - 1) / (16 * R);
    uint32_t C = 1;
    while (C < 8 && tiles * C < 2u * uint32_t(num_sms)) C *= 2;
    return launch_cluster(fc2, dim3(tiles * C), dim3(kNt), C, smem, stream, a, C);
}

template <int F>
cudaError_t launch_layer_f(const LayerArgs& a, int num_sms, cudaStream_t stream) {
    if (a.T <= 8) return launch_ng<F, 1>(a, num_sms, stream);
    if (a.T <= 16) return launch_ng<F, 2>(a, num_sms, stream);
    return launch_ng<F, 4>(a, num_sms, stream);
}

}  // namespace

}  // namespace moe
