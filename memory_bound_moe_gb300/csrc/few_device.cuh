// Device-side pieces shared by the products for a few tokens (few_fp4.cuh,
// layer_bf16.cu): weights streamed once from HBM into tensor-core fragments.
//
// One m16n8k16 product takes 16 weight rows as A and up to 8 tokens as B, in
// float32. Lane (g, q) = (lane / 4, lane % 4) holds rows g and g + 8 of A,
// token g of B, and tokens 2 q and 2 q + 1 of rows g and g + 8 of C. The order
// of k inside a product is free as long as A and B agree, so a lane takes 64
// contiguous bytes of each of its rows (4 lanes: 256 bytes of a row, a "chunk")
// in 32-byte loads and the same k of its token, and feeds them to the products
// without any exchange between lanes. Nothing is staged: registers hold the
// loads in flight. (A ring of 16-byte cp.async copies in shared memory moved
// twice the bytes between L2 and SM: 101 MB for 50 MB of weights.)
#pragma once

#include "moe_device.cuh"
#include "rows_common.cuh"

#include <cstdint>

namespace moe {

// 16-byte granules of a lane's 64 bytes of chunk c that lie in a row of rb bytes.
__device__ __forceinline__ uint32_t row_granules(uint32_t rb, uint32_t c) {
    const uint32_t at = c * 256u + (threadIdx.x % 4) * 64u;
    return at < rb ? min((rb - at) / 16u, 4u) : 0u;
}

// Half `half` (32 bytes) of a lane's 64 bytes of its two rows, at w and w +
// half_w; the words of row h at out[h]. `whole`: all of it lies in the matrix
// and may be read in 32-byte pieces. Else `rows` says which rows exist (bit h),
// n how many granules of the 64 bytes, and `wide` whether 32-byte pieces are
// aligned; the rest reads as zero.
__device__ __forceinline__ void load_rows(Bits<32> (&out)[2][2], int half, const uint8_t* w, uint64_t half_w, bool whole,
                                          uint32_t rows, uint32_t n, bool wide) {
    if (whole) {
        ld_stream(out[0][half], w + half * 32);
        ld_stream(out[1][half], w + half_w + half * 32);
        return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t m = (rows >> h) & 1u ? n : 0u;
        const uint8_t* p = w + h * half_w + half * 32;
#pragma unroll
        for (int z = 0; z < 8; ++z) out[h][half].w[z] = 0u;
        if (wide && m >= uint32_t(2 * half + 2)) {
            ld_stream(out[h][half], p);
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (uint32_t(2 * half + i) < m) {
                    Bits<16> v;
                    ld_stream(v, p + i * 16);
#pragma unroll
                    for (int z = 0; z < 4; ++z) out[h][half].w[4 * i + z] = v.w[z];
                }
        }
    }
}

// Barrier of the KS warps of row group rg.
__device__ __forceinline__ void group_sync(int rg, int KS) {
    if (KS == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(rg + 1), "r"(KS * kWarp) : "memory");
}

// One group's accumulators -> [token][row], 16 rows.
template <int NG>
__device__ __forceinline__ void store_group(float* p, const float (&acc)[NG][4], int n) {
    const int lane = threadIdx.x % kWarp, g = lane / 4, q = lane % 4;
#pragma unroll
    for (int k = 0; k < NG; ++k)
        if (k == n) {
#pragma unroll
            for (int z = 0; z < 4; ++z) p[(2 * q + (z & 1)) * 16 + g + (z >> 1) * 8] = acc[k][z];
        }
}

// Sum over the KS splits of k (warps rg KS ..) of element i of their `stride`
// floats.
__device__ __forceinline__ float sum_splits(const float* s_part, int rg, int KS, int stride, int i) {
    const float* p = s_part + rg * KS * stride + i;
    float v = p[0];
    for (int k = 1; k < KS; ++k) v += p[k * stride];
    return v;
}

// ---------------------------------------------------------------------------
// Thread-block clusters: barrier, a float of another block's shared memory, and
// the sum of s_sum[T][rows] over the C blocks, in rank order, to store(t, row,
// value).
// ---------------------------------------------------------------------------

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ float ld_cluster(const float* p, uint32_t rank) {
    const uint32_t a = uint32_t(__cvta_generic_to_shared(p));
    uint32_t r;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(r) : "memory");
    return v;
}

template <typename Store>
__device__ __forceinline__ void cluster_store(const float* s_sum, int total, int rows, uint32_t rank, uint32_t C, Store&& store) {
    if (C > 1) cluster_sync();
    else __syncthreads();
    for (int o = int(threadIdx.x + rank * blockDim.x); o < total; o += int(blockDim.x * C)) {
        float v;
        if (C > 1) {
            v = ld_cluster(s_sum + o, 0);
            for (uint32_t c = 1; c < C; ++c) v += ld_cluster(s_sum + o, c);
        } else {
            v = s_sum[o];
        }
        store(o / rows, o % rows, v);
    }
    if (C > 1) cluster_sync();   // the others may still read this block's sums
}

__device__ __forceinline__ float silu(float v) { return v / (1.0f + expf(-v)); }

}  // namespace moe
