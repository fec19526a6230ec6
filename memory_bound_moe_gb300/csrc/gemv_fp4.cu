// Products of a few tokens with a 4-bit weight matrix:
//   y[t, n] = sum_k x[t, k] W[n, k],   1 <= t <= 32,
// W in the library's MXFP4 or NVFP4 layout (codes [N, K/2], scales
// [N, K/block]). Bound by the weights' bytes (0.53 or 0.56 per value).
//
// A block takes 16 R rows; its 8 warps, and the C blocks of its cluster, split
// k in units of U steps (few_device.cuh). The partial sums meet in shared
// memory, then through distributed shared memory, always in the same order:
// results do not depend on timing.
#include "few_device.cuh"
#include "moe_launch.h"
#include "rows_common.cuh"

namespace moe {
namespace {

constexpr int kNw = 8;             // warps per block
constexpr int kNt = kNw * kWarp;

struct GemvArgs {
    const uint16_t* x;
    const uint8_t* codes;
    const uint8_t* scales;
    void* y;
    uint32_t T, N, K;
    uint32_t units;    // units of U steps along k
    float inv_g;       // 1 / tensor scale (1 for MXFP4)
    int y_f32;
};

template <int F, int R, int NG, int U>
__global__ void __launch_bounds__(kNt, 2) gemv_kernel(GemvArgs a, uint32_t C) {
    extern __shared__ float s_red[];             // [kNw][8 NG][16 R]
    constexpr int kOut = 8 * NG * 16 * R;
    pdl_wait_and_release();
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp, g = lane / 4, q = lane % 4;
    const uint32_t rank = blockIdx.x % C, row0 = blockIdx.x / C * (16 * R);
    const uint32_t rb = row_bytes<F>(a.K), rs = row_scales<F>(a.K);
    float acc[R][NG][4] = {};
    for (uint32_t u = rank * kNw + warp; u < a.units; u += C * kNw) {
        AGran<F> w[U][R];
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t row = row0 + r * 16 + h * 8 + g;
                    const WRow p = {a.codes + uint64_t(row) * rb, a.scales + uint64_t(row) * rs};
                    load_gran<F>(w[i][r], h, p, row < a.N, u * U + i, q, rb);
                }
#pragma unroll
        for (int i = 0; i < U; ++i)
            mma_step<F, R, NG>(acc, w[i], ~0u, 1.0f, [&](int n, BGran<F>& b) {
                load_x<F>(b, a.x + uint64_t(n * 8 + g) * a.K, n * 8 + g < a.T, u * U + i, q, a.K);
            });
    }
    store_partial<R, NG>(s_red + warp * kOut, acc);
    __syncthreads();
    if (C > 1) {
        for (int o = threadIdx.x; o < kOut; o += kNt) {
            float s = s_red[o];
#pragma unroll
            for (int w = 1; w < kNw; ++w) s += s_red[w * kOut + o];
            s_red[o] = s;   // this thread alone reads and writes column o
        }
        cluster_sync();
    }
    for (int o = threadIdx.x + (C > 1 ? int(rank) * kNt : 0); o < kOut; o += kNt * int(C)) {
        float s;
        if (C > 1) {
            s = ld_cluster(s_red + o, 0);
            for (uint32_t c = 1; c < C; ++c) s += ld_cluster(s_red + o, c);
        } else {
            s = s_red[o];
#pragma unroll
            for (int w = 1; w < kNw; ++w) s += s_red[w * kOut + o];
        }
        const uint32_t t = uint32_t(o) / (16 * R), row = row0 + uint32_t(o) % (16 * R);
        if (t < a.T && row < a.N) {
            s *= a.inv_g;
            const uint64_t at = uint64_t(t) * a.N + row;
            if (a.y_f32) static_cast<float*>(a.y)[at] = s;
            else static_cast<uint16_t*>(a.y)[at] = uint16_t(pack_bf16x2(s, 0.0f));
        }
    }
    if (C > 1) cluster_sync();   // the others may still read this block's sums
}

template <int F, int R, int NG>
cudaError_t launch_r(GemvArgs a, int num_sms, cudaStream_t stream) {
    constexpr int U = 2;
    auto kernel = gemv_kernel<F, R, NG, U>;
    constexpr size_t smem = sizeof(float) * kNw * 8 * NG * 16 * R;
    const uint32_t steps = (row_bytes<F>(a.K) + 63) / 64;
    a.units = (steps + U - 1) / U;
    const uint32_t tiles = (a.N + 16 * R - 1) / (16 * R);
    // split k over a cluster until two blocks per SM are busy and while every warp still has a unit
    uint32_t C = 1;
    while (C < 8 && tiles * C < 2u * uint32_t(num_sms) && a.units >= 2 * C * kNw) C *= 2;
    return launch_cluster(kernel, dim3(tiles * C), dim3(kNt), C, smem, stream, a, C);
}

template <int F>
cudaError_t launch_f(const GemvArgs& a, int num_sms, cudaStream_t stream) {
    const bool wide = a.N >= 32u * 2u * uint32_t(num_sms);
    if (a.T <= 8) return wide ? launch_r<F, 2, 1>(a, num_sms, stream) : launch_r<F, 1, 1>(a, num_sms, stream);
    if (a.T <= 16) return wide ? launch_r<F, 2, 2>(a, num_sms, stream) : launch_r<F, 1, 2>(a, num_sms, stream);
    return wide ? launch_r<F, 2, 4>(a, num_sms, stream) : launch_r<F, 1, 4>(a, num_sms, stream);
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
    a.inv_g = nvfp4 ? 1.0f / g : 1.0f;
    a.y_f32 = y_f32 ? 1 : 0;
    return nvfp4 ? launch_f<kWNvfp4>(a, num_sms, stream) : launch_f<kWMxfp4>(a, num_sms, stream);
}

}  // namespace moe
