// Device-side block quantization shared by the kernels that store E4M3 or E2M1
// codes (quant.cu, rmsnorm.cu): the element conversions, the shared exponent,
// and the quantization of one lane's values with its block's scale. The
// formats are defined at the top of quant.cu.
#pragma once

#include "moe_device.cuh"

#include <cstdint>

namespace moe {

// Two floats -> two E4M3 bytes (the first argument in the low byte).
__device__ __forceinline__ uint16_t pack_e4m3x2(float lo, float hi) {
    uint16_t d;
    asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n\tmov.b16 %0, t;\n\t}"
        : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// Two floats -> one byte of two E2M1 codes (the first argument in the low
// nibble).
__device__ __forceinline__ uint32_t pack_e2m1x2(float lo, float hi) {
    uint16_t d;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u16.u8 %0, t;\n\t}"
        : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// The value of a non-negative E4M3 byte (4 exponent bits with bias 7, 3
// fraction bits), exactly.
__device__ __forceinline__ float e4m3_value(uint32_t b) {
    const uint32_t e = (b >> 3) & 0xfu, m = b & 7u;
    if (e == 0) return float(m) * __uint_as_float(uint32_t(127 - 9) << 23);
    return float(8u + m) * __uint_as_float((e - 10u + 127u) << 23);
}

// Shared exponent of a block from its largest magnitude (amax >= 0, a
// bfloat16 value): floor(log2 amax) is the float's exponent field minus 127
// for normal values; EMAX is the element format's largest exponent (8 for
// E4M3, 2 for E2M1); amax below 2^-119 (zero and subnormal included) clamps
// to X = -127.
template <int EMAX>
__device__ __forceinline__ int mx_exponent(float amax) {
    const int ef = int((__float_as_uint(amax) >> 23) & 0xffu);
    if (ef == 0) return -127;
    return max(min(ef - 127 - EMAX, 127), -127);
}

// 2^-x for x in [-127, 126] as an exact float.
__device__ __forceinline__ float exp2_neg(int x) {
    return __uint_as_float(uint32_t(127 - x) << 23);
}

enum Fmt { kMxfp8 = 0, kMxfp4 = 1, kNvfp4 = 2 };

template <int F>
struct FmtInfo {
    static constexpr int kBlock = F == kNvfp4 ? 16 : 32;   // values per scale
    static constexpr int kBits = F == kMxfp8 ? 8 : 4;      // bits per code
};

// EPT consecutive values of one row (EPT = 16 or 8) -> codes, and the scale
// byte of their block; a block spans kBlock / EPT consecutive lanes (aligned),
// reduced with xor shuffles. All lanes of the warp must call; `valid` lanes
// contribute their values. g: the NVFP4 tensor scale.
template <int F, int EPT>
struct QChunk {
    static constexpr int kWords = EPT * FmtInfo<F>::kBits / 32;
    uint32_t codes[kWords];
    uint32_t scale;
};

// NVFP4: the multiplier fl(g / s) of every non-negative E4M3 scale byte
// (value s; 0 for s = 0), one IEEE division each, computed once per block
// before the dependency wait. Scale bytes of absolute maxima are at most
// 0x7E (448, saturated).
constexpr int kScaleTable = 128;

constexpr int kMaxTopK = 16;   // MOE_MAX_TOPK

__device__ __forceinline__ void fill_nvfp4_table(float* s_q, float g) {
    for (int i = threadIdx.x; i < kScaleTable; i += blockDim.x) {
        const float sv = e4m3_value(uint32_t(i));
        s_q[i] = sv > 0.0f ? __fdiv_rn(g, sv) : 0.0f;
    }
}

// fl(x / 6) for x >= 0 without a division: q0 = fl(x * fl(1/6)) corrected
// by one fused multiply-add of its residual (Markstein's method). Checked
// against the IEEE quotient for every finite float32: identical wherever the
// quotient is a normal float; below 2^-126 both lie far under half the
// smallest E4M3 step (2^-10), so the scale byte they round to is 0 either
// way. Overflowed (infinite) x passes through.
__device__ __forceinline__ float div6(float x) {
    constexpr float kSixth = 1.0f / 6.0f;
    const float q0 = __fmul_rn(x, kSixth);
    const float r = __fmaf_rn(-q0, 6.0f, x);
    return x < __int_as_float(0x7f800000) ? __fmaf_rn(r, kSixth, q0) : x;
}

template <int F, int EPT>
__device__ __forceinline__ QChunk<F, EPT> quantize_chunk(const float (&v)[EPT], bool valid, float g,
                                                         const float* s_q) {
    constexpr int kLanes = FmtInfo<F>::kBlock / EPT;
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < EPT; ++i) amax = fmaxf(amax, fabsf(v[i]));
    if (!valid) amax = 0.0f;
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
    QChunk<F, EPT> c;
    float m;   // the values' multiplier before the element conversion
    if constexpr (F == kNvfp4) {
        c.scale = pack_e4m3x2(div6(__fmul_rn(g, amax)), 0.0f) & 0xffu;
        m = s_q[c.scale & (kScaleTable - 1)];
    } else {
        const int x = mx_exponent<F == kMxfp8 ? 8 : 2>(amax);
        c.scale = uint32_t(x + 127);
        m = exp2_neg(min(x, 126));   // exact: a power of two
    }
    float p[EPT];   // the values the element conversion rounds: fl(v * m), as pairs
#pragma unroll
    for (int i = 0; i < EPT; i += 2) f2_split(mul2(f2(v[i], v[i + 1]), f2(m, m)), p[i], p[i + 1]);
    if constexpr (F == kMxfp8) {
#pragma unroll
        for (int q = 0; q < EPT / 4; ++q)
            c.codes[q] = uint32_t(pack_e4m3x2(p[4 * q], p[4 * q + 1])) |
                         (uint32_t(pack_e4m3x2(p[4 * q + 2], p[4 * q + 3])) << 16);
    } else {
#pragma unroll
        for (int q = 0; q < EPT / 8; ++q)
            c.codes[q] = pack_e2m1x2(p[8 * q], p[8 * q + 1]) | (pack_e2m1x2(p[8 * q + 2], p[8 * q + 3]) << 8) |
                         (pack_e2m1x2(p[8 * q + 4], p[8 * q + 5]) << 16) |
                         (pack_e2m1x2(p[8 * q + 6], p[8 * q + 7]) << 24);
    }
    return c;
}

template <int W>
__device__ __forceinline__ void store_words(uint8_t* p, const uint32_t (&w)[W]) {
    if constexpr (W == 4) {
        asm volatile("st.global.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]) : "memory");
    } else if constexpr (W == 2) {
        asm volatile("st.global.v2.u32 [%0], {%1,%2};" ::"l"(p), "r"(w[0]), "r"(w[1]) : "memory");
    } else {
        asm volatile("st.global.u32 [%0], %1;" ::"l"(p), "r"(w[0]) : "memory");
    }
}

// Byte offset of value column col of a row in the code buffer.
template <int F>
__device__ __forceinline__ uint64_t code_offset(uint64_t row, uint32_t n, uint32_t col) {
    return (row * n + col) * FmtInfo<F>::kBits / 8;
}

}  // namespace moe
