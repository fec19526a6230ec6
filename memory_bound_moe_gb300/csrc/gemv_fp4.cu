// Products of a few tokens with a 4-bit weight matrix:
//   y[t, n] = sum_k x[t, k] W[n, k],   1 <= t <= 32,
// W in the library's MXFP4 or NVFP4 layout (codes [N, K/2], scales
// [N, K/block]). Bound by the weights' bytes (0.53 or 0.56 per value).
//
// A block takes 16 rows per row group; its row groups share x, its KS splits
// and the C blocks of its cluster share k (few_fp4.cuh). The partial sums meet
// in shared memory, then through distributed shared memory, always in the same
// order: results do not depend on timing.
//
// Measured on GB300 in graphs: T=7, N=28672, K=4096 NVFP4 19.5 us (3.4 TB/s of
// weights, half the copy rate: 13.5 us of it are the loop over k, the rest x to
// f16, sums and the last wave); T=16, N=4096, K=7168 NVFP4 12.8 us, T=32, N=5760,
// K=2880 MXFP4 14.8 us, T=1, N=2048, K=768 MXFP4 4.0 us (latency: launch, x to
// f16, one or two chunks per warp, sums, one after the other).
#include "few_fp4.cuh"
#include "moe_launch.h"
#include "rows_common.cuh"

namespace moe {
namespace {

struct GemvArgs {
    const uint16_t* x;
    const uint8_t* codes;
    const uint8_t* scales;
    void* y;
    uint32_t T, N, K;
    uint32_t chunks;   // of k in all
    float g;           // tensor scale (NVFP4)
    int y_f32;
};

// k is taken slice by slice (what shared memory holds of x; usually all of the
// block's share), each converted by the whole block first.
template <int F, int NG>
__global__ void __launch_bounds__(Fp4Block<F, NG>::kMaxThreads, 1) gemv_kernel(GemvArgs a, int KS, uint32_t C) {
    extern __shared__ __align__(16) uint8_t smem[];
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp, g = lane / 4, q = lane % 4;
    const int W = blockDim.x / kWarp, rg = warp / KS, ks = warp % KS, rows = W / KS * 16, T = int(a.T), groups = (T + 7) / 8;
    const uint32_t rank = blockIdx.x % C, row0 = blockIdx.x / C * rows, mine = row0 + rg * 16 + g;
    const uint32_t c0 = a.chunks * rank / C, c1 = a.chunks * (rank + 1) / C;
    float* s_part = reinterpret_cast<float*>(smem + kPartAt);
    float* s_sum = reinterpret_cast<float*>(smem);   // [T][rows], in the place of x at the end
    const Shape4 sh = fp4_shape<F>(8, a.K, a.codes);
    const Place4 p = {a.codes + uint64_t(mine) * sh.rb + q * 64,
                      a.scales + uint64_t(mine) * row_scales<F>(a.K) + q * (128 / WInfo<F>::kBlock),
                      uint32_t(mine < a.N) | uint32_t(mine + 8 < a.N) << 1};
    if (threadIdx.x == 0) XRange::init(smem);
    __syncthreads();
    pdl_wait_and_release();
    float acc[NG][4] = {};
    const uint32_t slice = kUnits / 4 / groups;
    for (uint32_t s0 = c0; s0 < c1; s0 += slice) {
        const uint32_t n = min(slice, c1 - s0), per = n * 4;
        if (s0 > c0) __syncthreads();
        stage_units<F>(smem, per * groups, a.K, [&](uint32_t u, uint32_t& chunk) -> const uint16_t* {
            const uint32_t gr = u / per, r = gr * 8 + g;
            chunk = s0 + (u - gr * per) / 4;
            return r < a.T ? a.x + uint64_t(r) * a.K : nullptr;
        });
        __syncthreads();
        const uint32_t k0 = n * ks / KS, k1 = n * (ks + 1) / KS;
        fp4_tile<F, NG>(acc, p, sh, s0 + k0, s0 + k1, smem, k0 * 4, per, groups);
    }
    for (int n = 0; n < groups; ++n) {
        __syncthreads();
        store_group<NG>(s_part + warp * 128, acc, n);
        __syncthreads();
        for (int o = threadIdx.x; o < 8 * rows; o += blockDim.x) {
            const int c = o / rows, i = o % rows;
            if (n * 8 + c < T) s_sum[(n * 8 + c) * rows + i] = sum_splits(s_part, i / 16, KS, 128, c * 16 + i % 16);
        }
    }
    cluster_store(s_sum, T * rows, rows, rank, C, [&](int t, int i, float v) {
        const uint32_t row = row0 + i;
        if (row < a.N) {
            if constexpr (F == kWNvfp4) v /= a.g;   // 1 / g would round once more, and is infinite for a subnormal g
            const uint64_t to = uint64_t(t) * a.N + row;
            if (a.y_f32) static_cast<float*>(a.y)[to] = v;
            else static_cast<uint16_t*>(a.y)[to] = uint16_t(pack_bf16x2(v, 0.0f));
        }
    });
}

template <int F, int NG>
cudaError_t launch_ng(GemvArgs a, int num_sms, cudaStream_t stream) {
    auto kernel = gemv_kernel<F, NG>;
    using B = Fp4Block<F, NG>;
    static SmemGrant grant;
    static ClusterSlots clusters;
    uint32_t slots[9];
    cudaError_t err = grant.ensure(kernel);
    if (err == cudaSuccess) err = clusters.get(kernel, B::kMaxThreads, B::kSmem, num_sms, slots);
    if (err != cudaSuccess) return err;
    a.chunks = (a.K + kChunkK - 1) / kChunkK;
    const Fp4Split sp = fp4_split((uint64_t(a.N) + 15) / 16, a.chunks, (a.T + 7) / 8, (a.T + 7) / 8, B::kMaxWarps, slots);
    const uint32_t rows = sp.w / sp.ks * 16, tiles = (a.N + rows - 1) / rows;
    return launch_cluster(kernel, dim3(tiles * sp.c), dim3(sp.w * kWarp), sp.c, B::kSmem, stream, a,
                          int(sp.ks), sp.c);
}

template <int F>
cudaError_t launch_f(const GemvArgs& a, int num_sms, cudaStream_t stream) {
    if (a.T <= 8) return launch_ng<F, 1>(a, num_sms, stream);
    if (a.T <= 16) return launch_ng<F, 2>(a, num_sms, stream);
    return launch_ng<F, 4>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_gemv_fp4(const uint16_t* x, int T, int K, const uint8_t* codes, const uint8_t* scales, int N,
                            bool nvfp4, float g, void* y, bool y_f32, int num_sms, cudaStream_t stream) {
    GemvArgs a = {};
    a.x = x;
    a.codes = codes;
    a.scales = scales;
    a.y = y;
    a.T = uint32_t(T); a.N = uint32_t(N); a.K = uint32_t(K);
    a.g = g;
    a.y_f32 = y_f32 ? 1 : 0;
    return nvfp4 ? launch_f<kWNvfp4>(a, num_sms, stream) : launch_f<kWMxfp4>(a, num_sms, stream);
}

}  // namespace moe
