// Kernels of the MoE layer for a few tokens with 4-bit weights, on the inner
// loop of few_fp4.cuh. See layer_bf16.cu for what fc1 and fc2 compute and how
// the batch is routed; the activation is f16 with exponents of its own here, and
// with NVFP4 already divided by the tensor scale of the expert's w2. Up to 8
// tokens the B columns are the tokens themselves; above, they are the expert's
// own tokens, 8 to a group and two groups to a pass: an expert with more than 16
// of at most 32 tokens takes a second pass over its weights (from L2 or not). Two
// more groups' accumulators in every warp would cost every batch. (MXFP4, T=8:
// 117 us in the first form, 151 in the second.)
//   fc1: a tile is 8 gate rows and the same 8 up rows, so 8 columns of one
//        expert's activation; a block takes an even share of all tiles, RG at a
//        time. Up to 8 tokens one converted x serves every expert, and if it
//        fits shared memory at once the row groups run on their own.
//   fc2: a cluster of C blocks takes 16 output columns per row group and shares
//        the (expert, chunk) list evenly, slice by slice. Up to 8 tokens slices
//        run across experts and the sums stay in registers; above, a slice
//        stays within an expert, and the sums are added to the warp's own
//        [T][16] in shared memory behind it.
//
// Measured on GB300 in graphs: MXFP4, T=8, E=32, k=4, H=I=2880 118 us (fc1 three
// fifths of it; the bytes take 41.5), NVFP4, T=32, E=8, k=2, H=4096, I=14336 252
// us (fc1 as much; 119). Bound by latency: DRAM is 25% to 47% busy, issue 35%
// to 53%, no pipe above 36%, with 3 or 4 warps per scheduler whose registers
// hold all the bytes in flight.
#pragma once

#include "few_fp4.cuh"
#include "few_route.cuh"
#include "rows_common.cuh"

namespace moe {
namespace {

template <int F, int NG>
__global__ void __launch_bounds__(Fp4Block<F, NG>::kMaxThreads, 1) fc1_fp4_kernel(LayerArgs a, int KS) {
    constexpr bool kCompact = NG > 1;   // B columns are the expert's own tokens
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ FewRoute s;
    if (threadIdx.x == 0) XRange::init(smem);
    pdl_wait_and_release();
    route_few(a, s, blockIdx.x == 0);
    if (blockIdx.x == 0) save_route(static_cast<FewRouteCopy*>(a.route), s, a.T * a.k);
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp, g = lane / 4, q = lane % 4, W = blockDim.x / kWarp;
    const int RG = W / KS, rg = warp / KS, ks = warp % KS;
    const uint32_t H = uint32_t(a.H), I = uint32_t(a.I), tiles = I / 8, chunks = (H + kChunkK - 1) / kChunkK;
    const uint32_t total = uint32_t(s.nd) * tiles;
    const uint32_t begin = uint32_t(uint64_t(total) * blockIdx.x / gridDim.x), end = uint32_t(uint64_t(total) * (blockIdx.x + 1) / gridDim.x);
    const Shape4 sh = fp4_shape<F>(I, H, a.w13);
    const uint32_t rs = row_scales<F>(H);
    float* s_part = reinterpret_cast<float*>(smem + kPartAt);
    uint32_t staged = ~0u;   // what x shared memory holds
    uint32_t stop, first = 0;   // first: the pass's first token of the expert
    for (uint32_t t0 = begin; t0 < end;) {
        // the row groups' tiles t0 .. t0 + RG - 1, of one expert if kCompact
        const uint32_t x = kCompact ? t0 / tiles : 0u;
        stop = kCompact ? min(end, (x + 1) * tiles) : end;
        const int left = kCompact ? __popc(s.tokens[x]) - int(first) : 8, groups = min(NG, (left + 7) / 8);
        const uint32_t t = t0 + rg, d = min(t, stop - 1u) / tiles, j0 = (t - d * tiles) * 8, e = s.expert[d], m = s.tokens[d];
        const uint64_t row = uint64_t(e) * 2 * I + j0 + g;
        const Place4 p = {static_cast<const uint8_t*>(a.w13) + row * sh.rb + q * 64,
                          a.w13_scales + row * rs + q * (128 / WInfo<F>::kBlock), 3u};
        const float g13 = F == kWNvfp4 ? a.w13_global[e] : 1.0f, g2 = F == kWNvfp4 ? a.w2_global[e] : 1.0f;
        const uint32_t slice = kUnits / 4 / groups;
        float acc[NG][4] = {};
        for (uint32_t s0 = 0; s0 < chunks; s0 += slice) {
            const uint32_t n = min(slice, chunks - s0), per = n * 4;
            if (staged != (x * 4u + first / 8u) * 4096u + s0) {   // s0 < 2048
                __syncthreads();
                stage_units<F>(smem, per * groups, H, [&](uint32_t u, uint32_t& chunk) -> const uint16_t* {
                    const uint32_t gr = u / per, c = gr * 8 + g;
                    chunk = s0 + (u - gr * per) / 4;
                    if (kCompact) return int(c) < left ? a.x + uint64_t(s.row_t[s.off[x] + first + c]) * H : nullptr;
                    return int(c) < a.T ? a.x + uint64_t(c) * H : nullptr;
                });
                __syncthreads();
                staged = (x * 4u + first / 8u) * 4096u + s0;
            }
            const uint32_t k0 = n * ks / KS, k1 = n * (ks + 1) / KS;
            if (t < stop) fp4_tile<F, NG>(acc, p, sh, s0 + k0, s0 + k1, smem, k0 * 4, per, groups);
        }
        // a pass over the block's tiles of the expert, then the next 8 NG tokens or the next expert
        const uint32_t tokens0 = first;
        t0 = min(t0 + RG, stop);
        if (kCompact && t0 == stop) {
            first = left > 8 * NG ? first + 8 * NG : 0u;
            if (first > 0u) t0 = max(begin, x * tiles);
        }
        if (t >= stop) continue;   // the whole row group
        for (int n = 0; n < groups; ++n) {
            group_sync(rg, KS);
            store_group<NG>(s_part + warp * 128, acc, n);
            group_sync(rg, KS);
            // (token, column): gate and up rows lie 8 apart
            for (int o = threadIdx.x % (KS * kWarp); o < 64; o += KS * kWarp) {
                const int c = o / 8, col = int(tokens0) + n * 8 + c;
                if (kCompact ? col >= __popc(m) : !((m >> col) & 1u)) continue;
                const uint32_t to = s.off[d] + (kCompact ? col : __popc(m & ((1u << col) - 1u)));
                float gate = sum_splits(s_part, rg, KS, 128, c * 16 + o % 8), up = sum_splits(s_part, rg, KS, 128, c * 16 + o % 8 + 8);
                if constexpr (F == kWNvfp4) {
                    gate /= g13;
                    up /= g13;
                }
                float v = s.row_w[to] * (silu(gate) * up);
                if constexpr (F == kWNvfp4) v /= g2;   // fc2 sums over experts of different scales
                const uint64_t at = uint64_t(to) * I + j0;
                uint32_t exponent;
                a.act[at + o % 8] = act_to_f16(v, exponent);   // a token's 8 columns: 8 lanes, all here or none
                if (o % 8 == 0) a.act_exps[at / 8] = uint8_t(exponent);
            }
        }
    }
}

template <int F, int NG>
__global__ void __launch_bounds__(Fp4Block<F, NG>::kMaxThreads, 1) fc2_fp4_kernel(LayerArgs a, int KS, uint32_t C) {
    constexpr bool kCompact = NG > 1;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ FewRoute s;
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp, g = lane / 4, q = lane % 4, W = blockDim.x / kWarp;
    const int RG = W / KS, rg = warp / KS, ks = warp % KS, rows = RG * 16, part = (a.T + 7) / 8 * 128;
    const uint32_t H = uint32_t(a.H), I = uint32_t(a.I), chunks = (I + kChunkK - 1) / kChunkK, rs = row_scales<F>(I);
    const uint32_t rank = blockIdx.x % C, row0 = blockIdx.x / C * rows, mine = row0 + rg * 16 + g;
    float* s_sum = reinterpret_cast<float*>(smem);              // [T][rows], in the place of x at the end
    float* s_part = reinterpret_cast<float*>(smem + kPartAt);   // [warp][T rounded up to 8][16]
    float* s_mine = s_part + warp * part;
    if (kCompact)
        for (int o = lane; o < part; o += kWarp) s_mine[o] = 0.0f;
    if (threadIdx.x == 0) XRange::init(smem);
    pdl_wait_and_release();
    load_route(s, static_cast<const FewRouteCopy*>(a.route), a.T * a.k);
    const Shape4 sh = fp4_shape<F>(8, I, a.w2);
    const uint32_t rows_ok = uint32_t(mine < H) | uint32_t(mine + 8 < H) << 1;
    const uint64_t all = uint64_t(s.nd) * chunks;
    const uint32_t c1 = uint32_t(all * (rank + 1) / C);
    float acc[NG][4] = {};
    uint32_t n = 0, first = 0;   // first: the pass's first token of the expert
    for (uint32_t c0 = uint32_t(all * rank / C); c0 < c1;) {
        // the slice: chunks c0 .. c0 + n - 1 of the list, for 8 NG tokens of the expert if kCompact; its first pass,
        // which has the most groups, says how long it is, and every pass covers the same chunks
        const uint32_t d0 = c0 / chunks;
        const int left = kCompact ? __popc(s.tokens[d0]) - int(first) : 8, groups = min(NG, (left + 7) / 8);
        if (first == 0u) n = min(kUnits / 4 / groups, (kCompact ? min(c1, (d0 + 1) * chunks) : c1) - c0);
        const uint32_t per = n * 4;
        __syncthreads();
        stage_units<F>(smem, per * groups, I, [&](uint32_t u, uint32_t& chunk) -> const uint16_t* {
            const uint32_t gr = u / per, c = c0 + (u - gr * per) / 4, d = c / chunks, col = gr * 8 + g, m = s.tokens[d];
            chunk = c - d * chunks;
            if (kCompact ? int(col) >= left : !((m >> col) & 1u)) return nullptr;
            return a.act + uint64_t(s.off[d] + (kCompact ? first + col : uint32_t(__popc(m & ((1u << col) - 1u))))) * I;
        }, a.act, a.act_exps);
        __syncthreads();
        // this warp's share, expert by expert
        const uint32_t k1 = c0 + n * (ks + 1) / KS;
        for (uint32_t c = c0 + n * ks / KS; c < k1;) {
            const uint32_t d = c / chunks, from = c - d * chunks, to = min(chunks, from + (k1 - c)), e = s.expert[d];
            const uint64_t row = uint64_t(e) * H + mine;
            const Place4 p = {static_cast<const uint8_t*>(a.w2) + row * sh.rb + q * 64,
                              a.w2_scales + row * rs + q * (128 / WInfo<F>::kBlock), rows_ok};
            float before[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) before[z] = acc[0][z];
            fp4_tile<F, NG>(acc, p, sh, from, to, smem, (c - c0) * 4, per, groups);
            if constexpr (!kCompact) {   // zeros times a NaN weight are NaN: other tokens' columns stay as they were
#pragma unroll
                for (int z = 0; z < 4; ++z) acc[0][z] = (s.tokens[d] >> (2 * q + (z & 1))) & 1u ? acc[0][z] : before[z];
            }
            c += to - from;
        }
        if constexpr (kCompact) {   // to the tokens' own columns
#pragma unroll
            for (int k = 0; k < NG; ++k) {
                if (k >= groups) break;
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const int col = k * 8 + 2 * q + (z & 1);
                    if (col < left) s_mine[s.row_t[s.off[d0] + first + col] * 16 + g + (z >> 1) * 8] += acc[k][z];
                    acc[k][z] = 0.0f;
                }
            }
            __syncwarp();
        }
        // the slice's next tokens, or the next slice
        first = left > 8 * NG ? first + 8 * NG : 0u;
        if (first == 0u) c0 += n;
    }
    if constexpr (!kCompact) store_group<NG>(s_mine, acc, 0);
    __syncthreads();
    for (int o = threadIdx.x; o < a.T * rows; o += blockDim.x)
        s_sum[o] = sum_splits(s_part, o % rows / 16, KS, part, o / rows * 16 + o % 16);
    cluster_store(s_sum, a.T * rows, rows, rank, C, [&](int t, int i, float v) {
        if (row0 + i < H) a.out[uint64_t(t) * H + row0 + i] = uint16_t(pack_bf16x2(v, 0.0f));
    });
}

template <int F, int NG>
cudaError_t launch_ng(const LayerArgs& a, int num_sms, cudaStream_t stream) {
    auto fc1 = fc1_fp4_kernel<F, NG>;
    auto fc2 = fc2_fp4_kernel<F, NG>;
    using B = Fp4Block<F, NG>;
    static SmemGrant grant1, grant2;
    static ClusterSlots clusters;
    uint32_t slots[9];
    cudaError_t err = grant1.ensure(fc1);
    if (err == cudaSuccess) err = grant2.ensure(fc2);
    if (err == cudaSuccess) err = clusters.get(fc2, B::kMaxThreads, B::kSmem, num_sms, slots);
    if (err != cudaSuccess) return err;
    constexpr uint32_t kMax = B::kMaxWarps;
    const uint32_t sms = uint32_t(num_sms), chunks1 = (uint32_t(a.H) + kChunkK - 1) / kChunkK, chunks2 = (uint32_t(a.I) + kChunkK - 1) / kChunkK;
    // the experts that a batch of independent tokens is expected to choose
    double miss = 1.0;
    for (int t = 0; t < a.T; ++t) miss *= 1.0 - double(a.k) / a.E;
    const double nd = std::max<double>(a.k, a.E * (1.0 - miss));
    // fc1: splits of k until every warp has about three pieces (the last then costs little; NVFP4, T=32: 251 us, the
    // same with one piece, 268 with six)
    const uint64_t tiles1 = uint64_t(nd * (a.I / 8));
    uint32_t ks = 1;
    for (uint32_t k = 2; k <= kMax && k <= chunks1 && tiles1 * ks < 3ull * kMax * sms; ++k)
        if (kMax % k == 0) ks = k;
    // fewer warps where there is less than a piece for each
    uint32_t w = kMax;
    while (w >= 2 * ks && w % 2 == 0 && (w / 2) % ks == 0 && tiles1 * ks < uint64_t(w) / 2 * sms) w /= 2;
    const uint64_t most = std::min<uint64_t>(a.E, uint64_t(a.T) * a.k) * uint64_t(a.I / 8);
    const uint32_t grid = uint32_t(std::min<uint64_t>((most * ks + w - 1) / w, sms));
    err = launch_pdl(fc1, dim3(grid), dim3(w * kWarp), B::kSmem, stream, a, int(ks));
    if (err != cudaSuccess) return err;
    const Fp4Split sp = fp4_split((uint64_t(a.H) + 15) / 16, uint32_t(nd * chunks2), NG == 1 ? 1.0 : std::max(1.0, 0.4 + a.T * a.k / (8.0 * nd)),
                                  (uint32_t(a.T) + 7) / 8, kMax, slots);
    const uint32_t rows = sp.w / sp.ks * 16, tiles = (uint32_t(a.H) + rows - 1) / rows;
    return launch_cluster(fc2, dim3(tiles * sp.c), dim3(sp.w * kWarp), sp.c, B::kSmem, stream, a,
                          int(sp.ks), sp.c);
}

template <int F>
cudaError_t launch_layer_fp4(const LayerArgs& a, int num_sms, cudaStream_t stream) {
    return a.T <= 8 ? launch_ng<F, 1>(a, num_sms, stream) : launch_ng<F, 2>(a, num_sms, stream);
}

}  // namespace
}  // namespace moe
