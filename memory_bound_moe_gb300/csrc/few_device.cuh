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
//   4 bits:  32 values per granule, 128 k per step, 8 products per 16 rows.
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

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// The 8 E2M1 codes of w times scale (a bfloat16 in both halves) as bfloat16
// pairs p[i] = (code i, code i + 4). A code's exponent and mantissa bits
// placed at bits 8..6 of a bfloat16 read as its value times 2^-126 (code 0x1
// as a subnormal), so two products give value * scale; both are exact: the
// value has 2 significant bits and the scale at most 4.
__device__ __forceinline__ void e2m1_to_bf16(uint32_t w, uint32_t scale, uint32_t (&p)[4]) {
    constexpr uint32_t kSign = 0x80008000u, kMag = 0x01c001c0u, kTwo126 = 0x7e807e80u;
    p[0] = ((w << 12) & kSign) | ((w << 6) & kMag);
    p[1] = ((w << 8) & kSign) | ((w << 2) & kMag);
    p[2] = ((w << 4) & kSign) | ((w >> 2) & kMag);
    p[3] = (w & kSign) | ((w >> 6) & kMag);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = mul_bf16x2(mul_bf16x2(p[i], kTwo126), scale);
}

// An E8M0 byte as a bfloat16 in both halves: 2^(b - 127), NaN for 255.
__device__ __forceinline__ uint32_t e8m0_bf16x2(uint32_t b) {
    const uint32_t v = b == 0 ? 0x0040u : b == 255 ? 0x7fc0u : b << 7;
    return v * 0x00010001u;
}

// The E4M3 bytes of a 16-bit pair as bfloat16 values, each in both halves of
// its result (exact: 4 significant bits).
__device__ __forceinline__ void e4m3_bf16x2(uint32_t pair, uint32_t& s0, uint32_t& s1) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(pair)));
    float lo, hi;
    asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(lo), "=f"(hi) : "r"(h));
    s0 = pack_bf16x2(lo, lo);
    s1 = pack_bf16x2(hi, hi);
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

// The products of one step: R tiles of 16 rows against NG groups of 8 tokens
// (the first `groups` of them, the same for the whole warp).
template <int F, int R, int NG>
__device__ __forceinline__ void mma_step(float (&acc)[R][NG][4], const AGran<F> (&a)[R], const BGran<F> (&b)[NG],
                                         int groups) {
    if constexpr (F == kWBf16) {
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            if (NG > 1 && n >= groups) break;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                mma_bf16(acc[r][n], a[r].w[0].w[0], a[r].w[1].w[0], a[r].w[0].w[1], a[r].w[1].w[1], b[n].x[0].x, b[n].x[0].y);
                mma_bf16(acc[r][n], a[r].w[0].w[2], a[r].w[1].w[2], a[r].w[0].w[3], a[r].w[1].w[3], b[n].x[0].z, b[n].x[0].w);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {   // word j of the granule: k = 8 j .. 8 j + 7
            uint32_t bp[NG][4];         // x pairs (i, i + 4), as the codes' pairs
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                const uint4 x = b[n].x[j];
                bp[n][0] = __byte_perm(x.x, x.z, 0x5410);
                bp[n][1] = __byte_perm(x.x, x.z, 0x7632);
                bp[n][2] = __byte_perm(x.y, x.w, 0x5410);
                bp[n][3] = __byte_perm(x.y, x.w, 0x7632);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                uint32_t p[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t s;
                    if constexpr (F == kWMxfp4) {
                        s = e8m0_bf16x2(a[r].s[h]);
                    } else {
                        uint32_t s0, s1;
                        e4m3_bf16x2(a[r].s[h], s0, s1);
                        s = j < 2 ? s0 : s1;
                    }
                    e2m1_to_bf16(a[r].w[h].w[j], s, p[h]);
                }
#pragma unroll
                for (int n = 0; n < NG; ++n) {
                    if (NG > 1 && n >= groups) break;
                    mma_bf16(acc[r][n], p[0][0], p[1][0], p[0][1], p[1][1], bp[n][0], bp[n][1]);
                    mma_bf16(acc[r][n], p[0][2], p[1][2], p[0][3], p[1][3], bp[n][2], bp[n][3]);
                }
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
