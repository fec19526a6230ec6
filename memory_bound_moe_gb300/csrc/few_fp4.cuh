// Products of a few tokens with 4-bit weights: the streaming core of
// moe_gemv_fp4 and of both kernels of moe_layer_fp4.
//
// Numbers. E2M1 converts to f16 in hardware (one instruction per two codes;
// there is none to bfloat16, where placing the bits by shifts and masks costs
// four), and a weight times its scale is exact in f16, so the products are
// m16n8k16 f16 with float32 sums. bfloat16's range is carried beside the f16
// values:
//  - x: each token's values of one step (128 k) are multiplied by the power of
//    two that brings their largest into [2^14, 2^15), and the step's sums by
//    its inverse. A value 2^-31 of the step's largest still keeps its 8 bits: it
//    is 2^-17 or more, and f16's last step is 2^-24. What smaller ones lose is at
//    most 2^-39 of the largest.
//  - a, the layer's activation: fc1 leaves it as f16 with an exponent per 8
//    columns, its largest in [2^14, 2^15) as well; fc2 takes a step's values to
//    the largest exponent among them. That keeps 11 bits in 2.1 bytes. bfloat16
//    would leave 8, a second rounding as large as the result's own; float32 has
//    twice the bytes. (T=32, E=8, k=2, H=4096, I=14336: NVFP4 252 us, MXFP4 358;
//    249 and 356 in bfloat16, 263 and 370 in float32.)
//  - MXFP4: an E8M0 scale enters as 2^(X - Xmax + 13), Xmax the largest of the
//    warp's blocks in a chunk of 512 k, and 2^(Xmax - 13) multiplies the sums. Where
//    blocks lie more than 2^27 apart they take turns, each with its own Xmax; so
//    they do where the powers of two for x and for the weights have a product
//    that is no float32.
//  - NVFP4: E4M3 scales and their products with E2M1 are within f16's range.
//
// Work. Next to the loads what bounds it is the arithmetic logic pipe: 16 lanes
// a clock, 4 conversions per 8 weights and lane, and every further integer
// operation at the same price (the matrix instructions and the scale products
// have pipes of their own). So the loop over k holds little else:
//  - a warp takes a tile of 16 rows; a lane takes 64 contiguous bytes (128 k) of
//    each of its two rows, a "chunk" of 512 k per warp, in two 256-bit loads,
//    their scales in one. A chunk is four steps of 128 k, granule i of every
//    lane making step i. The next chunk's loads go out as soon as half of the
//    registers is used up; the other warps of the SM hide the rest.
//  - MXFP4 chunks whose blocks need turns are only noted, and added by a second
//    look at the tile behind the loop: what they need stays out of its registers.
//  - x is converted once per block, into shared memory, in the order the B
//    fragments are read: all distances in the loop are constants. (With the
//    same data in global memory behind run-time strides the loop took 24
//    instructions per matrix instruction instead of 13.)
// Measured on GB300 with the inner loop alone (57344 x 4096 weights, 132 MB,
// one wave): loads without products 24.6 us, products without loads 22.9 us;
// together 26.9 us with 24 warps of 80 registers, 30.9 us with 16 of 128, and
// 34.1 us with two tiles per warp and 16 warps.
#pragma once

#include "few_device.cuh"

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

namespace moe {

enum WFmt { kWNvfp4 = 1, kWMxfp4 = 2 };

template <int F>
struct WInfo {
    static constexpr int kBlock = F == kWNvfp4 ? 16 : 32;   // values per scale
};

// Scales of a weight row of K values.
template <int F>
__host__ __device__ constexpr uint32_t row_scales(uint32_t K) { return K / WInfo<F>::kBlock; }

constexpr int kXPairs = 16;         // f16 pairs of one lane's x in a step
constexpr uint32_t kChunkK = 512;   // k per chunk

// Blocks are one per SM, of up to kMaxWarps warps (what the registers allow: 96
// each with 20 warps, 128 with 16), in RG row groups x KS splits of k. With one
// group of tokens 20 warps are the better for NVFP4; for MXFP4 they spill: the
// layer of T=8, E=32, k=4, H=I=2880 takes 135 us with 20 and 117 with 16.
constexpr uint32_t kUnits = 88;                       // (group, step) units of x that shared memory holds
constexpr uint32_t kUnit = 2048;                      // one unit: 8 tokens x 128 k, f16
constexpr uint32_t kInvAt = kUnits * kUnit;           // the units' inverse powers of two, 8 each
constexpr uint32_t kRangeAt = kInvAt + kUnits * 32u;  // bits of the least and the largest of them, as XRange
constexpr uint32_t kPartAt = kRangeAt + 16u;          // partial sums: [warp][tokens][16 rows]

template <int F, int NG>
struct Fp4Block {
    static constexpr int kMaxWarps = NG == 1 && F == kWNvfp4 ? 20 : 16;
    static constexpr int kMaxThreads = kMaxWarps * kWarp;
    // partial sums of up to 32 tokens (8 if NG == 1)
    static constexpr uint32_t kSmem = kPartAt + kMaxWarps * (NG == 1 ? 512u : 2048u);
};

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
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;}"
        : "=r"(p[0]), "=r"(p[1]), "=r"(p[2]), "=r"(p[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(p[i]) : "r"(scale));
}

// One lane's 32 values of its token as f16, times a power of two shared by the
// token's four lanes; returns the inverse of that power (1 if all are zero).
// Infinities and NaN stay what they are.
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
    const uint32_t e = m == 0u ? 141u : min(max(m >> 7, 15u), 254u);   // biased exponent of the largest
    const float scale = __uint_as_float((268u - e) << 23);           // 2^(14 - (e - 127))
#pragma unroll
    for (int i = 0; i < kXPairs; ++i) {
        float lo, hi;
        f2_split(mul2(bf16x2_to_f2(h[i]), f2(scale, scale)), lo, hi);
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h[i]) : "f"(hi), "f"(lo));
    }
    return __uint_as_float((e - 14u) << 23);                         // 2^(e - 127 - 14)
}

// A column's activation v as fc1 leaves it: f16, times the power of two that
// brings the largest of its 8 columns, in this and its 7 neighbouring lanes, into
// [2^14, 2^15); exponent: that largest's, biased, or 0 where all are zero or NaN.
__device__ __forceinline__ uint16_t act_to_f16(float v, uint32_t& exponent) {
    float most = fabsf(v);
#pragma unroll
    for (int i = 1; i < 8; i <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffu << (threadIdx.x & 24), most, i));
    exponent = most > 0.0f ? min(max(__float_as_uint(most) >> 23, 15u), 254u) : 0u;
    uint16_t r;
    asm("cvt.rn.f16.f32 %0, %1;" : "=h"(r) : "f"(exponent > 0u ? v * __uint_as_float((268u - exponent) << 23) : v));
    return r;
}

// Four f16 pairs times 2^-d, d <= 14.
__device__ __forceinline__ void scale_f16(uint32_t* h, uint32_t d) {
    const uint32_t m = 0x3c003c00u - d * 0x04000400u;
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h[i]) : "r"(m));
}

// x_to_f16 of 32 activations as act_to_f16 left them, the 8 of x[z] with the
// exponent in byte z of exps: all to the largest exponent of the four lanes.
__device__ __forceinline__ float a_to_f16(const uint4 (&x)[4], uint32_t exps, uint32_t (&h)[kXPairs]) {
    uint32_t d[4], top = 0, far = 0;
#pragma unroll
    for (int z = 0; z < 4; ++z) {
        d[z] = __byte_perm(exps, 0, 0x4440 + z);
        top = max(top, d[z]);
    }
    top = max(top, __shfl_xor_sync(kFull, top, 1));
    top = max(top, __shfl_xor_sync(kFull, top, 2));
#pragma unroll
    for (int z = 0; z < 4; ++z) {
        d[z] = top - d[z];
        far = max(far, d[z]);
        h[4 * z] = x[z].x; h[4 * z + 1] = x[z].y; h[4 * z + 2] = x[z].z; h[4 * z + 3] = x[z].w;
        scale_f16(h + 4 * z, min(d[z], 14u));
    }
#pragma unroll 1
    for (uint32_t s = 14; s < min(far, 42u); s += 14)   // rare; below 2^-42 nothing is left of f16
#pragma unroll
        for (int z = 0; z < 4; ++z) scale_f16(h + 4 * z, min(d[z] - min(d[z], s), 14u));
    return top == 0u ? 1.0f : __uint_as_float((top - 14u) << 23);
}

// Whether a product of two powers of two is one, not 0 or infinity.
__device__ __forceinline__ bool in_range(float p) { return p > 0.0f && p < __int_as_float(0x7f800000); }

// 2^(x - 127 - 13), a subnormal float for x < 14.
__device__ __forceinline__ float mxfp4_unit(uint32_t x) {
    return x >= 14u ? __uint_as_float((x - 13u) << 23) : __uint_as_float(1u << (x + 9u));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// The least and the largest inverse power of two among all units that the block
// has staged so far: with these bits an MXFP4 chunk knows whether a product of
// the factors for its weights and for x could leave float32. init by one thread,
// before a barrier before the first stage_units.
struct XRange {
    uint32_t lo, hi;
    __device__ __forceinline__ static XRange* at(uint8_t* smem) { return reinterpret_cast<XRange*>(smem + kRangeAt); }
    __device__ __forceinline__ static void init(uint8_t* smem) {
        at(smem)->lo = at(smem)->hi = __float_as_uint(1.0f);
    }
};

// Units of x into shared memory, by all warps of the block: unit u is step u %
// 4 of 8 rows; where(u, chunk) gives the lane group's row (NULL gives zeros)
// and the chunk of k. For j = 0..3 a unit holds the 16 bytes that every lane
// reads for word j of its granule. Two units' loads are in flight per warp.
// The rows are bfloat16, or activations (act and exps: the whole arrays).
template <int F, typename Where>
__device__ __forceinline__ void stage_units(uint8_t* smem, uint32_t units, uint32_t K, Where&& where, const uint16_t* act = nullptr,
                                            const uint8_t* exps = nullptr) {
    const int lane = threadIdx.x % kWarp, g = lane / 4, q = lane % 4;
    const uint32_t W = blockDim.x / kWarp;
    uint32_t lo = __float_as_uint(1.0f), hi = lo;
#pragma unroll 1
    for (uint32_t u0 = threadIdx.x / kWarp; u0 < units; u0 += 2 * W) {
        uint4 x[2][4] = {};
        uint32_t ex[2] = {};
#pragma unroll
        for (uint32_t k = 0; k < 2; ++k) {
            const uint32_t u = u0 + k * W;
            if (u >= units) break;
            uint32_t chunk;
            const uint16_t* row = where(u, chunk);
            const uint32_t k0 = chunk * kChunkK + q * 128u + u % 4 * 32u;
            if (row != nullptr && k0 < K) {
#pragma unroll
                for (int z = 0; z < 4; ++z) x[k][z] = __ldg(reinterpret_cast<const uint4*>(row + k0) + z);
                if (exps != nullptr) ex[k] = __ldg(reinterpret_cast<const uint32_t*>(exps + uint64_t(row + k0 - act) / 8));
            }
        }
#pragma unroll
        for (uint32_t k = 0; k < 2; ++k) {
            const uint32_t u = u0 + k * W;
            if (u >= units) break;
            uint32_t h[kXPairs];
            const float inv = exps != nullptr ? a_to_f16(x[k], ex[k], h) : x_to_f16(x[k], h);
            uint4* p = reinterpret_cast<uint4*>(smem + u * kUnit) + lane;
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j * 32] = make_uint4(h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3]);
            if (q == 0) reinterpret_cast<float*>(smem + kInvAt)[u * 8 + g] = inv;
            lo = min(lo, __float_as_uint(inv));
            hi = max(hi, __float_as_uint(inv));
        }
    }
    if constexpr (F == kWMxfp4) {
        lo = __reduce_min_sync(kFull, lo);
        hi = __reduce_max_sync(kFull, hi);
        if (lane == 0) {
            atomicMin(&XRange::at(smem)->lo, lo);
            atomicMax(&XRange::at(smem)->hi, hi);
        }
    }
}

// One lane's weights of a chunk: 64 bytes of its rows g and g + 8 of a tile,
// and their scales as loaded: two parts of two granules each (nothing is put
// together before it is used, as that would wait for the load).
template <int F>
struct WChunk4 {
    Bits<32> w[2][2];        // [row half][half of the 64 bytes]
    uint32_t s[2][2];        // [row half][part]: 2 E8M0 or 4 E4M3 bytes
};

// Where a lane's rows lie: its 64 bytes of row g in chunk 0, their scales, and
// the distances to row g + 8.
struct Place4 {
    const uint8_t* w;
    const uint8_t* s;
    uint32_t rows;       // bit h: row g + 8 h exists
};
struct Shape4 {
    uint64_t half_w, half_s;
    uint32_t rb;         // bytes of a row
    uint32_t whole;      // chunks that lie wholly in a row, if rows may be read in 32-byte pieces (else 0)
    int scale_align;     // bytes: at most 8
};

template <int F>
__device__ __forceinline__ Shape4 fp4_shape(uint64_t half_rows, uint32_t K, const void* w) {
    const uint32_t rb = K / 2, rs = row_scales<F>(K);
    const uint32_t al = rs & (0u - rs);   // largest power of two that divides a row's scales
    const bool wide = rb % 32u == 0u && reinterpret_cast<uintptr_t>(w) % 32u == 0u;
    return {half_rows * rb, half_rows * rs, rb, wide ? rb / 256u : 0u, int(min(al, 8u))};
}

template <int F>
__device__ __forceinline__ void load_scales(WChunk4<F>& a, const Place4& at, const Shape4& sh, uint32_t c, bool whole) {
    constexpr int kPart = F == kWNvfp4 ? 4 : 2;   // bytes of a part
    const uint32_t n = whole ? 4u : row_granules(sh.rb, c);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint8_t* p = at.s + h * sh.half_s;
        const uint32_t m = whole || ((at.rows >> h) & 1u) ? n : 0u;
        if (sh.scale_align >= kPart) {
            if (whole && F == kWNvfp4 && sh.scale_align == 2 * kPart) {
                const uint2 t = __ldg(reinterpret_cast<const uint2*>(p));
                a.s[h][0] = t.x;
                a.s[h][1] = t.y;
            } else {
#pragma unroll
                for (uint32_t i = 0; i < 2; ++i) {
                    a.s[h][i] = 0u;
                    if (m >= 2 * i + 2) {
                        if constexpr (F == kWNvfp4) a.s[h][i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
                        else a.s[h][i] = __ldg(reinterpret_cast<const uint16_t*>(p) + i);
                    } else if (m == 2 * i + 1) {
                        if constexpr (F == kWNvfp4) a.s[h][i] = __ldg(reinterpret_cast<const uint16_t*>(p) + 2 * i);
                        else a.s[h][i] = __ldg(p + 2 * i);
                    }
                }
            }
        } else {   // rows of scales at odd places: granule by granule
#pragma unroll
            for (uint32_t i = 0; i < 2; ++i) {
                a.s[h][i] = 0u;
#pragma unroll
                for (uint32_t k = 0; k < 2; ++k)
                    if (2 * i + k < m) {
                        if constexpr (F == kWNvfp4) a.s[h][i] |= uint32_t(__ldg(reinterpret_cast<const uint16_t*>(p) + 2 * i + k)) << (16 * k);
                        else a.s[h][i] |= uint32_t(__ldg(p + 2 * i + k)) << (8 * k);
                    }
            }
        }
    }
}

// MXFP4 blocks further apart than one window, with a NaN scale, or with factors
// whose product is no float32: turn by turn, each with the largest scale among
// the blocks not yet added. Adds one group's products of a chunk (its B
// fragments at xb, its inverse powers of two at inv) to acc.
__device__ __forceinline__ void mxfp4_apart(float (&acc)[4], const WChunk4<kWMxfp4>& a, uint32_t xb, const float* inv) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float f0 = inv[i * 8], f1 = inv[i * 8 + 1];
        uint32_t todo = 3u, sc[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) sc[k] = (a.s[k][i / 2] >> (8 * (i % 2))) & 255u;
#pragma unroll 1
        while (__any_sync(kFull, todo != 0u)) {
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (((todo >> k) & 1u) && sc[k] != 255u) top = max(top, sc[k]);
            top = __reduce_max_sync(kFull, top);
            const float fx = mxfp4_unit(top);
            uint32_t s[2], left = 0;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t(&v)[8] = a.w[k][i / 2].w;
                const uint32_t codes = v[i % 2 * 4] | v[i % 2 * 4 + 1] | v[i % 2 * 4 + 2] | v[i % 2 * 4 + 3];
                const int d = int(sc[k]) - int(top) + 28;   // biased f16 exponent
                s[k] = 0;
                if ((todo >> k) & 1u) {
                    if (sc[k] == 255u) s[k] = 0x7e007e00u;     // NaN
                    else if (d >= 1) s[k] = uint32_t(d) * 0x04000400u;
                    else if ((codes & 0x77777777u) != 0u) left |= 1u << k;
                }
            }
            float c[4] = {};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t p0[4], p1[4];
                e2m1_to_f16(a.w[0][i / 2].w[i % 2 * 4 + j], s[0], p0);
                e2m1_to_f16(a.w[1][i / 2].w[i % 2 * 4 + j], s[1], p1);
                const uint4 b = lds128(xb + i * kUnit + j * 512u);
                mma_f16(c, p0[0], p1[0], p0[1], p1[1], b.x, b.y);
                mma_f16(c, p0[2], p1[2], p0[3], p1[3], b.z, b.w);
            }
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const float fz = z & 1 ? f1 : f0, p = fz * fx;
                // where the factors' product leaves float32 both are small or both large: one at a time, no step of
                // c leaves it before the result does
                acc[z] = in_range(p) ? fmaf(c[z], p, acc[z]) : acc[z] + (c[z] * fz) * fx;
            }
            todo = left;
        }
    }
}

// MXFP4: the scales lo .. lo + n whose factors 2^(top - 140) have a float32
// product with every factor 2^(i - 127) of x: -149 <= i + top - 267 <= 127.
struct TopRange {
    uint32_t lo, n;
    __device__ __forceinline__ static TopRange of(uint8_t* smem) {
        const uint32_t i0 = XRange::at(smem)->lo >> 23, i1 = XRange::at(smem)->hi >> 23;   // i0 <= 127 <= i1
        const uint32_t lo = i0 < 118u ? 118u - i0 : 0u;
        return {lo, min(254u, 394u - i1) - lo};
    }
};

// MXFP4: the largest scale of chunk c's blocks over the warp, and whether they
// need turns. Granules that are cut off (their codes are zero) take the largest
// scale for theirs, but not NaN (255), which would make them NaN as well.
__device__ __forceinline__ uint32_t mxfp4_top(WChunk4<kWMxfp4>& a, bool& apart, const Place4& p, const Shape4& sh, uint32_t c, bool whole,
                                              TopRange ok) {
    uint32_t top = 0, low = 255u;
    if (!whole) {
        const uint32_t n = row_granules(sh.rb, c);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) top = max(top, (a.s[h][i / 2] >> (8 * (i % 2))) & 255u);
        top = min(__reduce_max_sync(kFull, top), 254u);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t m = (p.rows >> h) & 1u ? n : 0u;
#pragma unroll
            for (uint32_t i = 0; i < 2; ++i)
                a.s[h][i] |= m >= 2 * i + 2 ? 0u : m == 2 * i + 1 ? top << 8 : top * 0x0101u;
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = __byte_perm(a.s[h][i / 2], 0, 0x4440 + i % 2);
            top = max(top, x);
            low = min(low, x);
        }
    top = __reduce_max_sync(kFull, top);
    apart = __any_sync(kFull, low + 28u <= top) || top - ok.lo > ok.n;
    return top;
}

// Adds the chunks c0 .. c1 - 1 of a tile that need turns, and only those, to one
// group's sums; x of chunk c0 begins at unit u0.
__device__ __forceinline__ void mxfp4_apart_chunks(float* sums, const Place4* place, const Shape4* shape, uint32_t c0, uint32_t c1,
                                                   uint8_t* smem, uint32_t u0) {
    const int lane = threadIdx.x % kWarp, q = lane % 4;
    const TopRange ok = TopRange::of(smem);
    const Shape4 sh = *shape;
    Place4 p = *place;
    float acc[4] = {sums[0], sums[1], sums[2], sums[3]};
    const uint32_t whole = __all_sync(kFull, p.rows == 3u) ? sh.whole : 0u;
    p.w += c0 * 256u;
    p.s += c0 * (kChunkK / WInfo<kWMxfp4>::kBlock);
#pragma unroll 1
    for (uint32_t c = c0; c < c1; ++c) {
        WChunk4<kWMxfp4> a;
        bool apart;
        load_scales(a, p, sh, c, c < whole);
        mxfp4_top(a, apart, p, sh, c, c < whole, ok);
        if (apart) {
            const uint32_t n = row_granules(sh.rb, c), u = u0 + (c - c0) * 4;
            load_rows(a.w, 0, p.w, sh.half_w, c < whole, p.rows, n, sh.whole > 0u);
            load_rows(a.w, 1, p.w, sh.half_w, c < whole, p.rows, n, sh.whole > 0u);
            mxfp4_apart(acc, a, uint32_t(__cvta_generic_to_shared(smem)) + u * kUnit + lane * 16u,
                        reinterpret_cast<const float*>(smem + kInvAt) + u * 8 + 2 * q);
        }
        p.w += 256;
        p.s += kChunkK / WInfo<kWMxfp4>::kBlock;
    }
#pragma unroll
    for (int z = 0; z < 4; ++z) sums[z] = acc[z];
}

// The products of step i of a chunk with the first `groups` groups of 8 tokens.
// xb[n]: this lane's B fragments of group n in the chunk's first unit, inv[n]:
// that unit's inverse powers of two of the lane's two tokens in C, 2 q and 2 q
// + 1; top as of mxfp4_top.
template <int F, int NG>
__device__ __forceinline__ void fp4_step(float (&acc)[NG][4], const WChunk4<F>& a, const uint32_t (&sc)[2][2],
                                         int i, const uint32_t (&xb)[NG], const float* (&inv)[NG], int groups,
                                         uint32_t top) {
    float f = 1.0f;     // multiplies the sums
    uint32_t s[2][2];   // f16 scale in both halves: [row g or g + 8][k 0..15 or 16..31 of the granule]
    if constexpr (F == kWNvfp4) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t v;
            asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l;}"
                : "=r"(v) : "r"(i % 2 ? sc[k][i / 2] >> 16 : sc[k][i / 2]));
            s[k][0] = __byte_perm(v, v, 0x1010);
            s[k][1] = __byte_perm(v, v, 0x3232);
        }
    } else {
        f = mxfp4_unit(top);
        const uint32_t shift = (28u - top) * 0x04000400u;   // biased f16 exponent X - top + 28, in both halves
#pragma unroll
        for (int k = 0; k < 2; ++k) s[k][0] = s[k][1] = __byte_perm(sc[k][i / 2], 0, 0x4440 + i % 2) * 0x04000400u + shift;
    }
    float c[NG][4] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t p[2][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) e2m1_to_f16(a.w[k][i / 2].w[(i % 2) * 4 + j], s[k][j / 2], p[k]);
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            if (NG > 1 && n >= groups) break;
            const uint4 b = lds128(xb[n] + i * kUnit + j * 512u);
            mma_f16(c[n], p[0][0], p[1][0], p[0][1], p[1][1], b.x, b.y);
            mma_f16(c[n], p[0][2], p[1][2], p[0][3], p[1][3], b.z, b.w);
        }
    }
#pragma unroll
    for (int n = 0; n < NG; ++n) {
        if (NG > 1 && n >= groups) break;
        const float2 v = *reinterpret_cast<const float2*>(inv[n] + i * 8);
        const float f0 = v.x * f, f1 = v.y * f;
        acc[n][0] = fmaf(c[n][0], f0, acc[n][0]);
        acc[n][1] = fmaf(c[n][1], f1, acc[n][1]);
        acc[n][2] = fmaf(c[n][2], f0, acc[n][2]);
        acc[n][3] = fmaf(c[n][3], f1, acc[n][3]);
    }
}

// The chunks c0 .. c1 - 1 of one tile; x of chunk c0 begins at unit u0 of
// shared memory, each group's `group_units` behind the one before.
template <int F, int NG>
__device__ __forceinline__ void fp4_tile(float (&acc)[NG][4], const Place4& p0, const Shape4& sh, uint32_t c0, uint32_t c1,
                                         uint8_t* smem, uint32_t u0, uint32_t group_units, int groups) {
    if (c0 >= c1) return;
    const int lane = threadIdx.x % kWarp, q = lane % 4;
    uint32_t xb[NG];
    const float* inv[NG];
#pragma unroll
    for (int n = 0; n < NG; ++n) {
        const uint32_t u = u0 + n * group_units;
        xb[n] = uint32_t(__cvta_generic_to_shared(smem)) + u * kUnit + lane * 16u;
        inv[n] = reinterpret_cast<const float*>(smem + kInvAt) + u * 8 + 2 * q;
    }
    const uint32_t whole = __all_sync(kFull, p0.rows == 3u) ? sh.whole : 0u;   // chunks below it are whole
    bool some = false;   // MXFP4: whether chunks were left out, whose blocks need turns
    TopRange ok = {};
    if constexpr (F == kWMxfp4) ok = TopRange::of(smem);
    Place4 p = p0;
    p.w += c0 * 256u;
    p.s += c0 * (kChunkK / WInfo<F>::kBlock);
    WChunk4<F> a;
    load_rows(a.w, 0, p.w, sh.half_w, c0 < whole, p.rows, row_granules(sh.rb, c0), sh.whole > 0u);
    load_rows(a.w, 1, p.w, sh.half_w, c0 < whole, p.rows, row_granules(sh.rb, c0), sh.whole > 0u);
    load_scales(a, p, sh, c0, c0 < whole);
#pragma unroll 1
    for (uint32_t c = c0; c < c1; ++c) {
        uint32_t top = 0;
        bool apart = false;
        if constexpr (F == kWMxfp4) top = mxfp4_top(a, apart, p, sh, c, c < whole, ok);
        uint32_t sc[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int z = 0; z < 2; ++z) sc[h][z] = a.s[h][z];
        const bool more = c + 1 < c1;
        p.w += 256;
        p.s += kChunkK / WInfo<F>::kBlock;
        if (more) load_scales(a, p, sh, c + 1, c + 1 < whole);
        some |= apart;
        if (!apart) {
            fp4_step<F, NG>(acc, a, sc, 0, xb, inv, groups, top);
            fp4_step<F, NG>(acc, a, sc, 1, xb, inv, groups, top);
        }
        if (more) load_rows(a.w, 0, p.w, sh.half_w, c + 1 < whole, p.rows, row_granules(sh.rb, c + 1), sh.whole > 0u);
        if (!apart) {
            fp4_step<F, NG>(acc, a, sc, 2, xb, inv, groups, top);
            fp4_step<F, NG>(acc, a, sc, 3, xb, inv, groups, top);
        }
        if (more) load_rows(a.w, 1, p.w, sh.half_w, c + 1 < whole, p.rows, row_granules(sh.rb, c + 1), sh.whole > 0u);
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            xb[n] += 4 * kUnit;
            inv[n] += 32;
        }
    }
    if constexpr (F == kWMxfp4) {
        if (some) {   // rare: a second look at the tile, for the chunks left out
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                if (NG > 1 && n >= groups) break;
                float v[4] = {acc[n][0], acc[n][1], acc[n][2], acc[n][3]};
                const Place4 place = p0;
                const Shape4 shape = sh;
                mxfp4_apart_chunks(v, &place, &shape, c0, c1, smem, u0 + n * group_units);
#pragma unroll
                for (int z = 0; z < 4; ++z) acc[n][z] = v[z];
            }
        }
    }
}

// How a kernel of one block per SM over `tiles` row tiles divides its work: W
// warps per block, KS splits of k in a block, C blocks of a cluster, that share
// the `chunks` of a tile, each for `groups` groups of 8 tokens (on average), of
// `outs` that the results have. The least of an estimate in microseconds, its
// constants fitted to 60 measured divisions of the workloads' shapes: a wave of
// blocks pays 2 for launch and sums (1 more for a cluster) and 0.15 for every
// tile and group it adds up, 0.6 per unit of x that a warp converts, 1.5 for
// every further filling of shared memory, and per chunk 0.25 for every warp of
// a scheduler and as much per group, but no less than a load's latency, 1.0.
// The least is also what measured best, e.g. T=32, N=5760, K=2880: 15.4 us with
// (16, 2, 3), 19.8 with (16, 1, 6); T=7, N=28672, K=4096: 19.2 with (12, 1, 1),
// 20.8 with (16, 1, 1).
struct Fp4Split {
    uint32_t w, ks, c;
};
inline Fp4Split fp4_split(uint64_t tiles, uint32_t chunks, double groups, uint32_t outs, uint32_t max_warps, const uint32_t (&slots)[9]) {
    Fp4Split best = {max_warps, 1, 1};
    const uint32_t room = std::max(1u, kUnits / 4 / uint32_t(groups + 0.999));   // chunks of x in shared memory
    double least = 1e30;
    for (uint32_t w = 4; w <= max_warps; w += 4)
        for (uint32_t ks = 1; ks <= w && ks <= chunks; ++ks) {
            if (w % ks != 0) continue;
            for (uint32_t c = 1; c <= 8 && (c == 1 || c * ks <= chunks); ++c) {
                const uint32_t rg = w / ks, share = (chunks + c - 1) / c;
                const uint64_t waves = ((tiles + rg - 1) / rg + slots[c] - 1) / slots[c];
                const uint32_t fills = (share + room - 1) / room, per_fill = (share + fills - 1) / fills;
                const double chunk = std::max(1.0, 0.125 * w * (0.5 + 0.5 * groups));
                const double convert = 0.6 * std::ceil(share * 4 * groups / w);
                const double t = double(waves) * (2.0 + (c > 1 ? 1.0 : 0.0) + 0.15 * outs * rg + convert + 1.5 * (fills - 1) +
                                                  chunk * fills * ((per_fill + ks - 1) / ks));
                if (t < least * 0.99) {
                    least = t;
                    best = {w, ks, c};
                }
            }
        }
    return best;
}

}  // namespace moe
