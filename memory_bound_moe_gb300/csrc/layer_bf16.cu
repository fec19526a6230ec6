// A whole MoE layer for a few tokens (T <= 32), bfloat16 weights, in two
// kernels: routing and fc1 with SwiGLU, then fc2 with the weighted combine.
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
// Routing is redundant in fc1: every block routes the whole batch in shared
// memory (tens of KB of logits at most), so no block waits for another; one
// leaves it to fc2 in the workspace. A warp takes tiles of 16 weight rows
// (few_device.cuh); the KS splits of k of a block sum in shared memory.
//   fc1: a tile is 8 gate rows and the same 8 up rows, so 8 columns of one
//        expert's activation; a block takes an even share of all tiles. B
//        columns are the expert's own tokens. The activation is stored
//        compactly, expert-sorted (row off[d] + rank of the token).
//   fc2: a cluster of C blocks takes 16 output columns per row group; its
//        blocks and their KS splits share the (expert, chunk) list evenly. B
//        columns are the tokens themselves, zero where a token is not routed to
//        the expert, so the sums stay in registers to the end.
// All sums are taken in a fixed order: results do not depend on timing.
//
// Measured on GB300 in graphs: T=16, E=256, k=8, H=7168, I=2048 1.25-1.34 ms
// (by the experts that the tokens choose; fc1 two thirds of it), the copy rate;
// T=1, E=128, k=8, H=2048, I=768 26.4 us where the bytes take 11.3 (latency:
// launches, routing, short rows, and fc2's weights asked for after fc1's end).
#include "few_device.cuh"
#include "few_route.cuh"
#include "moe_launch.h"
#include "rows_common.cuh"

namespace moe {
namespace {

constexpr int kNw = 8;             // warps per block
constexpr int kNt = kNw * kWarp;
constexpr uint32_t kChunk = 128;   // k per chunk

// The products of half a chunk (64 k) with one group of tokens.
__device__ __forceinline__ void mma_half(float (&c)[4], const Bits<32>& w0, const Bits<32>& w1, const uint4& x0, const uint4& x1) {
    const uint32_t b[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(w0.w[2 * j]), "r"(w1.w[2 * j]), "r"(w0.w[2 * j + 1]), "r"(w1.w[2 * j + 1]), "r"(b[2 * j]), "r"(b[2 * j + 1]));
}

// Half of a lane's 64 bytes of x in chunk c (NULL: zeros).
__device__ __forceinline__ void load_x(uint4 (&x)[2], const uint16_t* row, uint32_t K, uint32_t c, int half) {
    const uint32_t k0 = c * kChunk + (threadIdx.x % 4) * 32u + half * 16u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (row != nullptr && k0 + i * 8u < K) x[i] = __ldg(reinterpret_cast<const uint4*>(row + k0) + i);
    }
}

// Where a lane's rows lie: its 64 bytes of row g in chunk 0, the distance to
// row g + 8, and which of the two exist.
struct Rows {
    const uint8_t* w;
    uint64_t half_w;
    uint32_t rows;
};

// The chunks c0 .. c1 - 1 of one tile of rows of K values, against the groups of
// 8 tokens set in `live` (the same for the whole warp); x[n]: this lane's
// token's row of group n, or NULL. The next chunk's loads go out as soon as
// half of the registers is used up.
template <int NG>
__device__ __forceinline__ void bf16_tile(float (&acc)[NG][4], Rows p, uint32_t K, bool wide, uint32_t c0, uint32_t c1,
                                          const uint16_t* const (&x)[NG], uint32_t live) {
    if (c0 >= c1) return;
    const uint32_t rb = 2 * K, whole = wide && __all_sync(kFull, p.rows == 3u) ? rb / 256u : 0u;   // chunks below it are whole
    Bits<32> w[2][2];
    p.w += c0 * 256u;
    load_rows(w, 0, p.w, p.half_w, c0 < whole, p.rows, row_granules(rb, c0), wide);
    load_rows(w, 1, p.w, p.half_w, c0 < whole, p.rows, row_granules(rb, c0), wide);
#pragma unroll 1
    for (uint32_t c = c0; c < c1; ++c) {
        p.w += 256;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                if (NG > 1 && !((live >> n) & 1u)) continue;
                uint4 b[2];
                load_x(b, x[n], K, c, half);
                mma_half(acc[n], w[0][half], w[1][half], b[0], b[1]);
            }
            if (c + 1 < c1) load_rows(w, half, p.w, p.half_w, c + 1 < whole, p.rows, row_granules(rb, c + 1), wide);
        }
    }
}

__device__ __forceinline__ bool rows_wide(uint32_t K, const void* w) {
    return K % 16 == 0 && reinterpret_cast<uintptr_t>(w) % 32 == 0;
}

template <int NG>
__global__ void __launch_bounds__(kNt, NG == 4 ? 2 : 3) fc1_kernel(LayerArgs a, int KS) {
    __shared__ FewRoute s;
    __shared__ float s_part[kNw * 128];          // [warp][8 tokens][16 rows]
    pdl_wait_and_release();
    route_few(a, s, blockIdx.x == 0);
    if (blockIdx.x == 0) save_route(static_cast<FewRouteCopy*>(a.route), s, a.T * a.k);
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp, g = lane / 4, q = lane % 4;
    const int RG = kNw / KS, rg = warp / KS, ks = warp % KS;
    const uint32_t H = uint32_t(a.H), I = uint32_t(a.I), tiles = I / 8, chunks = (H + kChunk - 1) / kChunk;
    const uint32_t total = uint32_t(s.nd) * tiles, k0 = chunks * ks / KS, k1 = chunks * (ks + 1) / KS;
    const uint32_t begin = uint32_t(uint64_t(total) * blockIdx.x / gridDim.x), end = uint32_t(uint64_t(total) * (blockIdx.x + 1) / gridDim.x);
    const bool wide = rows_wide(H, a.w13);
    for (uint32_t t = begin + rg; t < end; t += RG) {
        const uint32_t d = t / tiles, j0 = (t - d * tiles) * 8;
        const int m = __popc(s.tokens[d]), groups = (m + 7) / 8;
        const uint16_t* x[NG];
#pragma unroll
        for (int n = 0; n < NG; ++n) x[n] = n * 8 + g < m ? a.x + uint64_t(s.row_t[s.off[d] + n * 8 + g]) * H : nullptr;
        const Rows p = {static_cast<const uint8_t*>(a.w13) + (uint64_t(s.expert[d]) * 2 * I + j0 + g) * (2 * H) + q * 64,
                        uint64_t(I) * (2 * H), 3u};
        float acc[NG][4] = {};
        bf16_tile<NG>(acc, p, H, wide, k0, k1, x, (1u << groups) - 1u);
        for (int n = 0; n < groups; ++n) {
            group_sync(rg, KS);
            store_group<NG>(s_part + warp * 128, acc, n);
            group_sync(rg, KS);
            // (token, column): gate and up rows lie 8 apart
            for (int o = threadIdx.x % (KS * kWarp); o < 64; o += KS * kWarp) {
                const int c = o / 8;
                if (n * 8 + c >= m) continue;
                const uint32_t row = s.off[d] + n * 8 + c;
                const float gate = sum_splits(s_part, rg, KS, 128, c * 16 + o % 8), up = sum_splits(s_part, rg, KS, 128, c * 16 + o % 8 + 8);
                a.act[uint64_t(row) * I + j0 + o % 8] = uint16_t(pack_bf16x2(s.row_w[row] * (silu(gate) * up), 0.0f));
            }
        }
    }
}

template <int NG>
__global__ void __launch_bounds__(kNt, NG == 4 ? 2 : 3) fc2_kernel(LayerArgs a, int KS, uint32_t C) {
    __shared__ FewRoute s;
    __shared__ float s_part[kNw * 128];
    __shared__ float s_sum[kMaxTokens * kNw * 16];   // [T][rows]
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp, g = lane / 4, q = lane % 4;
    const int RG = kNw / KS, rg = warp / KS, ks = warp % KS, rows = RG * 16;
    const uint32_t H = uint32_t(a.H), I = uint32_t(a.I), chunks = (I + kChunk - 1) / kChunk;
    const uint32_t rank = blockIdx.x % C, row0 = blockIdx.x / C * rows, mine = row0 + rg * 16 + g;
    pdl_wait_and_release();
    load_route(s, static_cast<const FewRouteCopy*>(a.route), a.T * a.k);
    const bool wide = rows_wide(I, a.w2);
    const uint32_t rows_ok = uint32_t(mine < H) | uint32_t(mine + 8 < H) << 1;
    // this warp's part of the (expert, chunk) list
    const uint64_t all = uint64_t(s.nd) * chunks, slot = rank * KS + ks, slots = uint64_t(C) * KS;
    const uint32_t stop = uint32_t(all * (slot + 1) / slots);
    float acc[NG][4] = {};
    for (uint32_t c = uint32_t(all * slot / slots); c < stop;) {
        const uint32_t d = c / chunks, k0 = c - d * chunks, k1 = min(chunks, k0 + (stop - c)), m = s.tokens[d];
        const uint16_t* x[NG];
        uint32_t live = 0;
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            const uint32_t t = n * 8 + g;
            x[n] = (m >> t) & 1u ? a.act + uint64_t(s.off[d] + __popc(m & ((1u << t) - 1u))) * I : nullptr;
            live |= uint32_t(((m >> (8 * n)) & 0xffu) != 0u) << n;
        }
        const Rows p = {static_cast<const uint8_t*>(a.w2) + (uint64_t(s.expert[d]) * H + mine) * (2 * I) + q * 64, 8ull * (2 * I), rows_ok};
        float before[NG][4];
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
            for (int z = 0; z < 4; ++z) before[n][z] = acc[n][z];
        bf16_tile<NG>(acc, p, I, wide, k0, k1, x, live);
        // zeros times a non-finite weight are NaN: the columns of tokens that did not choose the expert stay as they
        // were (T=16: 1329 us, 1326 without)
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
            for (int z = 0; z < 4; ++z) acc[n][z] = (m >> (n * 8 + 2 * q + (z & 1))) & 1u ? acc[n][z] : before[n][z];
        c += k1 - k0;
    }
    for (int n = 0; n < (a.T + 7) / 8; ++n) {
        __syncthreads();
        store_group<NG>(s_part + warp * 128, acc, n);
        __syncthreads();
        for (int o = threadIdx.x; o < 8 * rows; o += kNt)
            if (n * 8 + o / rows < a.T) s_sum[(n * 8 + o / rows) * rows + o % rows] = sum_splits(s_part, o % rows / 16, KS, 128, o / rows * 16 + o % 16);
    }
    cluster_store(s_sum, a.T * rows, rows, rank, C, [&](int t, int i, float v) {
        if (row0 + i < H) a.out[uint64_t(t) * H + row0 + i] = uint16_t(pack_bf16x2(v, 0.0f));
    });
}

template <int NG>
cudaError_t launch_ng(const LayerArgs& a, int num_sms, cudaStream_t stream) {
    auto fc1 = fc1_kernel<NG>;
    auto fc2 = fc2_kernel<NG>;
    constexpr uint32_t kPerSm = NG == 4 ? 2 : 3;   // what the registers allow; T=16 with 2: 1.55 ms, with 3: 1.25
    static ClusterSlots clusters;
    const uint32_t slots1 = kPerSm * uint32_t(num_sms);
    uint32_t slots[9];
    cudaError_t err = clusters.get(fc2, kNt, 0, int(slots1), slots);
    if (err != cudaSuccess) return err;
    // the experts that a batch of independent tokens is expected to choose
    double miss = 1.0;
    for (int t = 0; t < a.T; ++t) miss *= 1.0 - double(a.k) / a.E;
    const double nd = std::max<double>(a.k, a.E * (1.0 - miss));
    // fc1: splits of k until every warp has about three pieces (the last then costs little; one, three and six
    // pieces are within 0.4%)
    const uint32_t chunks1 = (uint32_t(a.H) + kChunk - 1) / kChunk;
    const uint64_t tiles1 = uint64_t(nd * (a.I / 8)), most = std::min<uint64_t>(a.E, uint64_t(a.T) * a.k) * uint64_t(a.I / 8);
    uint32_t ks = 1;
    while (ks < uint32_t(kNw) && 4 * ks <= chunks1 && tiles1 * ks < 3ull * kNw * slots1) ks *= 2;
    const uint32_t grid = uint32_t(std::min<uint64_t>((most * ks + kNw - 1) / kNw, slots1));
    err = launch_pdl(fc1, dim3(grid), dim3(kNt), 0, stream, a, int(ks));
    if (err != cudaSuccess) return err;
    // fc2: of the splits (KS in a block, C blocks) the one with the fullest waves, then the fewest (one token, H=2048,
    // I=768: 26.4 us, 27.2 without clusters)
    const uint32_t chunks2 = uint32_t(nd * ((uint32_t(a.I) + kChunk - 1) / kChunk));
    uint32_t KS = 1, C = 1;
    double full = -1.0;
    for (uint32_t k = 1; k <= uint32_t(kNw); k *= 2) {
        const uint32_t tiles = (uint32_t(a.H) + kNw / k * 16 - 1) / (kNw / k * 16);
        for (uint32_t c = 1; c <= 8 && (c * k == 1 || 4 * c * k <= chunks2); ++c) {
            const uint32_t waves = (tiles + slots[c] - 1) / slots[c];
            const double f = double(tiles) * c / (double(waves) * slots1) - 0.03 * (waves - 1) - (c > 1 ? 0.02 : 0.0);
            if (f > full + 0.02) { full = f; KS = k; C = c; }
        }
    }
    const uint32_t tiles = (uint32_t(a.H) + kNw / KS * 16 - 1) / (kNw / KS * 16);
    return launch_cluster(fc2, dim3(tiles * C), dim3(kNt), C, 0, stream, a, int(KS), C);
}

}  // namespace

cudaError_t launch_layer_bf16(const LayerArgs& a, int num_sms, cudaStream_t stream) {
    if (a.T <= 8) return launch_ng<1>(a, num_sms, stream);
    if (a.T <= 16) return launch_ng<2>(a, num_sms, stream);
    return launch_ng<4>(a, num_sms, stream);
}

}  // namespace moe
