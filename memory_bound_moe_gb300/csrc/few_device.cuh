// Device-side pieces of the products for a few tokens (gemv_fp4.cu, layer.cu):
// weights streamed once from HBM into tensor-core fragments, bfloat16 or
// 4-bit with block scales.
//
// One m16n8k16 product takes 16 weight rows as A and up to 8 tokens as B, in
// float32. Lane (g, q) = (lane / 4, lane % 4) holds rows g and g + 8 of A and
// token g of B. The order of k inside a product is free as long as A and B
// agree, so a lane takes one contiguous 16-byte granule of each of its rows
// (4 lanes = 64 consecutive bytes of a row, a "step") and the same k of its
// token, and feeds them to the products without any exchange between lanes:
//   bfloat16: 8 values per granule, 32 k per step, 2 products per 16 rows;
//   4 bits:  32 values per granule, 128 k per step, 8 products per 16 rows (f16).
// Nothing is staged: at a few tokens per weight the kernels are bound by the
// weights' bytes, and registers hold as many loads in flight as a
// shared-memory ring would.
#pragma once

#include "moe_device.cuh"

#include <cstdint>

namespace moe {

enum WFmt { kWBf16 = 0, kWNvfp4 = 1, kWMxfp4 = 2 };

template <int F>
struct WInfo {
    static constexpr bool kFp4 = F != kWBf16;
    static constexpr int kStepK = kFp4 ? 128 : 32;              // k per step
    static constexpr int kXVec = kFp4 ? 4 : 1;                  // 16-byte vectors of x per lane and step
    static constexpr int kBlock = F == kWNvfp4 ? 16 : 32;       // values per scale
};

// Bytes of a weight row of K values, and its scales.
template <int F>
__host__ __device__ constexpr uint32_t row_bytes(uint32_t K) { return WInfo<F>::kFp4 ? K / 2 : K * 2; }
template <int F>
__host__ __device__ constexpr uint32_t row_scales(uint32_t K) { return K / WInfo<F>::kBlock; }

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The 8 E2M1 codes of w times scale (an f16 in both halves) as f16 pairs
// (codes 2 i, 2 i + 1). Exact: 2 significant bits times at most 4.
__device__ __forceinline__ void e2m1_to_f16(uint32_t w, uint32_t scale, uint32_t (&p)[4]) {
    asm("{.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t"
        "mul.rn.f16x2 %0, %0, %5;\n\tmul.rn.f16x2 %1, %1, %5;\n\t"
        "mul.rn.f16x2 %2, %2, %5;\n\tmul.rn.f16x2 %3, %3, %5;}"
        : "=&r"(p[0]), "=&r"(p[1]), "=&r"(p[2]), "=&r"(p[3])
        : "r"(w), "r"(scale));
}

// One lane's granules of two weight rows at one step, with their scales.
template <int F>
struct AGran {
    Bits<16> w[2];
    uint32_t s[WInfo<F>::kFp4 ? 2 : 1];
};

// A row of weights: its first byte and its first scale.
struct WRow {
    const uint8_t* w;
    const uint8_t* s;
};

template <int F>
__device__ __forceinline__ void load_gran(AGran<F>& a, int half, const WRow& row, bool valid, uint32_t step,
                                          int q, uint32_t rb) {
    const uint32_t off = step * 64u + q * 16u;
    if (valid && off < rb) {
        ld_stream(a.w[half], row.w + off);
        if constexpr (F == kWNvfp4) a.s[half] = __ldg(reinterpret_cast<const uint16_t*>(row.s) + (off >> 4));
        if constexpr (F == kWMxfp4) a.s[half] = __ldg(row.s + (off >> 4));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) a.w[half].w[i] = 0u;
        if constexpr (WInfo<F>::kFp4) a.s[half] = 0u;
    }
}

// One lane's values of its token at one step.
template <int F>
struct BGran {
    uint4 x[WInfo<F>::kXVec];
};

template <int F>
__device__ __forceinline__ void load_x(BGran<F>& b, const uint16_t* xrow, bool valid, uint32_t step, int q, uint32_t K) {
    const uint32_t k0 = step * WInfo<F>::kStepK + q * (WInfo<F>::kStepK / 4);
    if (valid && k0 < K) {
        const uint4* p = reinterpret_cast<const uint4*>(xrow + k0);
#pragma unroll
        for (int i = 0; i < WInfo<F>::kXVec; ++i) b.x[i] = __ldg(p + i);
    } else {
#pragma unroll
        for (int i = 0; i < WInfo<F>::kXVec; ++i) b.x[i] = make_uint4(0u, 0u, 0u, 0u);
    }
}

// ---------------------------------------------------------------------------
// 4-bit weights go through f16 products. E2M1 converts to f16 in hardware (one
// instruction per two codes; there is none to bfloat16, where placing the bits
// by shifts and masks costs four), and a weight times its scale is exact in
// f16. That leaves bfloat16's range to be carried beside the f16 values:
//  - x: each token's values of one step (128 k) are multiplied by the power of
//    two that brings their largest into [2^14, 2^15), and the step's float32
//    sums by its inverse. A value 2^-32 of the step's largest still keeps its 8
//    bits; what smaller ones lose is under 2^-39 of the largest.
//  - MXFP4: an E8M0 scale enters as 2^(X - Xmax + 13), Xmax the largest of the
//    warp's blocks in the step, and 2^(Xmax - 13) multiplies the sums. Blocks
//    more than 2^27 below the largest take another turn with their own Xmax.
//  - NVFP4: E4M3 scales and their products with E2M1 are within f16's range.
// ---------------------------------------------------------------------------

constexpr int kXPairs = 16;   // f16 pairs of one lane's x in a step of 4-bit weights

// One lane's 32 values of its token as f16, times a power of two shared by the
// token's four lanes; returns the inverse of that power. Infinities and NaN
// stay what they are.
__device__ __forceinline__ float x_to_f16(const uint4 (&x)[4], uint32_t (&h)[kXPairs]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) { h[4 * i] = x[i].x; h[4 * i + 1] = x[i].y; h[4 * i + 2] = x[i].z; h[4 * i + 3] = x[i].w; }
    uint32_t m = 0;   // |largest| of each half: max of magnitudes, NaN ignored, sign to be dropped
#pragma unroll
    for (int i = 0; i < kXPairs; ++i) asm("max.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(h[i]));
    m &= 0x7fff7fffu;
    m = max(m >> 16, m & 0xffffu);
    m = max(m, __shfl_xor_sync(kFull, m, 1));
    m = max(m, __shfl_xor_sync(kFull, m, 2));
    const uint32_t e = min(max(m >> 7, 15u), 254u);                  // biased exponent of the largest
    const float scale = __uint_as_float((268u - e) << 23);           // 2^(14 - (e - 127))
#pragma unroll
    for (int i = 0; i < kXPairs; ++i) {
        float lo, hi;
        f2_split(mul2(bf16x2_to_f2(h[i]), f2(scale, scale)), lo, hi);
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h[i]) : "f"(hi), "f"(lo));
    }
    return __uint_as_float((e - 14u) << 23);                         // 2^(e - 127 - 14)
}

// Products of one step: R tiles of 16 rows against `groups` groups of 8 tokens
// (those set in `live`, a bit each, the same for the whole warp). load(n, b)
// fetches the x of group n; f multiplies the sums of 4-bit weights. With
// 4-bit weights a further group decodes the weights again: keeping the decoded
// step (32 registers a tile) or several groups' x (16 each) beside the loads
// in flight costs more in occupancy than it saves, and an expert seldom has
// more than 8 of at most 32 tokens.
template <int F, int R, int NG, typename Load>
__device__ __forceinline__ void mma_step(float (&acc)[R][NG][4], const AGran<F> (&a)[R], uint32_t live, float f,
                                         Load&& load) {
#pragma unroll
    for (int n = 0; n < NG; ++n) {
        if (NG > 1 && !((live >> n) & 1u)) continue;
        BGran<F> b;
        load(n, b);
        if constexpr (F == kWBf16) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                mma_bf16(acc[r][n], a[r].w[0].w[0], a[r].w[1].w[0], a[r].w[0].w[1], a[r].w[1].w[1], b.x[0].x, b.x[0].y);
                mma_bf16(acc[r][n], a[r].w[0].w[2], a[r].w[1].w[2], a[r].w[0].w[3], a[r].w[1].w[3], b.x[0].z, b.x[0].w);
            }
        } else {
            const int q = threadIdx.x % 4;
            uint32_t h[kXPairs];
            const float inv = x_to_f16(b.x, h) * f;
            // of this lane's two tokens in C, 2 q and 2 q + 1
            const float f0 = __shfl_sync(kFull, inv, 8 * q), f1 = __shfl_sync(kFull, inv, 8 * q + 4);
            uint32_t todo = ~0u;    // MXFP4: the blocks (bit 2 r + half) still to be added
            while (true) {
                float g0 = f0, g1 = f1;
                uint32_t top = 0;
                if constexpr (F == kWMxfp4) {
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            if (((todo >> (2 * r + k)) & 1u) && a[r].s[k] != 255u) top = max(top, a[r].s[k]);
                    top = __reduce_max_sync(kFull, top);
                    // 2^(top - 127 - 13), a subnormal float for top < 14
                    const float fx = top >= 14u ? __uint_as_float((top - 13u) << 23) : __uint_as_float(1u << (top + 9u));
                    g0 *= fx;
                    g1 *= fx;
                }
                uint32_t far = 0;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    uint32_t s[2][2];   // the scales of k 0..15 and 16..31 of the granule, in both halves
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if constexpr (F == kWNvfp4) {
                            uint32_t v;
                            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(v) : "h"(uint16_t(a[r].s[k])));
                            s[k][0] = __byte_perm(v, v, 0x1010);
                            s[k][1] = __byte_perm(v, v, 0x3232);
                        } else {
                            const uint32_t x = a[r].s[k];
                            const int d = int(x) - int(top) + 28;      // biased f16 exponent
                            const bool mine = (todo >> (2 * r + k)) & 1u;
                            uint32_t v = d >= 1 ? uint32_t(d) * 0x04000400u : 0u;
                            if (x == 255u) v = 0x7e007e00u;            // NaN
                            s[k][0] = s[k][1] = mine ? v : 0u;
                            far |= uint32_t(mine && d < 1) << (2 * r + k);
                        }
                    }
                    float c[4] = {};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t p0[4], p1[4];
                        e2m1_to_f16(a[r].w[0].w[j], s[0][j / 2], p0);
                        e2m1_to_f16(a[r].w[1].w[j], s[1][j / 2], p1);
                        mma_f16(c, p0[0], p1[0], p0[1], p1[1], h[4 * j], h[4 * j + 1]);
                        mma_f16(c, p0[2], p1[2], p0[3], p1[3], h[4 * j + 2], h[4 * j + 3]);
                    }
                    acc[r][n][0] = fmaf(c[0], g0, acc[r][n][0]);
                    acc[r][n][1] = fmaf(c[1], g1, acc[r][n][1]);
                    acc[r][n][2] = fmaf(c[2], g0, acc[r][n][2]);
                    acc[r][n][3] = fmaf(c[3], g1, acc[r][n][3]);
                }
                if constexpr (F == kWNvfp4) break;
                if (!__any_sync(kFull, far != 0u)) break;
                // blocks far below the largest: another turn, unless all their codes are zero
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const Bits<16>& w = a[r].w[k];
                        if (((w.w[0] | w.w[1] | w.w[2] | w.w[3]) & 0x77777777u) == 0u) far &= ~(1u << (2 * r + k));
                    }
                todo = far;
                if (!__any_sync(kFull, todo != 0u)) break;
            }
        }
    }
}

// A warp's accumulators -> its part of the block's partial sums
// s_red[warp][token][row], rows 0..16 R - 1 (C fragment: lane (g, q) holds
// rows g, g + 8 of tokens 2 q, 2 q + 1).
template <int R, int NG>
__device__ __forceinline__ void store_partial(float* s_warp, const float (&acc)[R][NG][4]) {
    const int lane = threadIdx.x % kWarp, g = lane / 4, q = lane % 4;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                s_warp[(n * 8 + 2 * q + (i & 1)) * (16 * R) + r * 16 + g + (i >> 1) * 8] = acc[r][n][i];
}

// ---------------------------------------------------------------------------
// Thread-block clusters: barrier and a float of another block's shared memory.
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

}  // namespace moe
