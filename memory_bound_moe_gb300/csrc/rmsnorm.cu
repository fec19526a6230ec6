// RMS normalisation of token rows with the residual's addition, bfloat16 or
// MXFP8 output: the norm in front of a router and its experts.
//
//   h = x + residual (float32),  residual_out = bf16(h),
//   y = bf16( (w + bias) * (h * r) ),  r = 1 / sqrt(sum(h^2) / H + eps)
//
// The norm is taken of the float32 sum, not of the rounded residual: the sum
// is in registers anyway, and this way y is rounded once. The MXFP8 form
// quantizes the bfloat16 values of y (32 per scale, as moe_expand_mxfp8 would
// quantize them), so a consumer of y and a consumer of the codes see the same
// rows; y itself is then optional.
//
// One pass over memory: WPR warps hold one row in registers (NV vectors of VB
// bytes per thread), add, reduce the sum of squares by shuffles and one
// shared-memory exchange, scale and store. Rows of more than kMaxWarps * 32 *
// 4 vectors take the two-pass form, which reads x and the residual again
// (from L2) for the second half of the work. The largest one-pass form (four
// 32-byte vectors a thread, 64 registers: H above 32768) spills about 300 bytes a
// thread and is still the faster one: T=512, H=65536 58.5 us, MXFP8 55.5, where
// two passes over 16-byte vectors take 65.8 and 62.4.
//
// Bound by bytes: 8 per value (6 + 1 1/32 with MXFP8 alone). Measured on GB300
// in graphs: T=8192, H=4096 40.4 us, 6.65 TB/s (99% of a copy); with MXFP8 and
// bfloat16 out T=4096, H=2048 11.4 us (99%); T=16, H=7168 2.4 us, a launch.
#include "moe_device.cuh"
#include "moe_launch.h"
#include "quant_device.cuh"
#include "rows_common.cuh"

namespace moe {
namespace {

constexpr int kMaxWarps = 32;

struct NormArgs {
    const uint8_t* x;
    const uint8_t* residual;   // NULL: h = x
    const uint8_t* weight;
    uint8_t* out;              // NULL: not stored
    uint8_t* residual_out;     // NULL: not stored; may be `residual`
    uint8_t* codes;            // MXFP8 form only
    uint8_t* scales;
    uint32_t rows;
    uint32_t nvec;             // vectors per row
    uint32_t wpr;              // warps per row
    float bias, eps, inv_h;
};

// h of one vector; the residual may be rewritten in place by this kernel, so
// it is read through the coherent path.
template <int VB>
__device__ __forceinline__ void load_sum(const NormArgs& a, uint64_t off, float (&h)[VB / 2]) {
    Bits<VB> xv;
    ld_stream(xv, a.x + off);
    if (a.residual != nullptr) {
        Bits<VB> rv;
        ld_coherent(rv, a.residual + off);
#pragma unroll
        for (int i = 0; i < VB / 4; ++i) {
            h[2 * i] = bf16_lo(xv.w[i]) + bf16_lo(rv.w[i]);
            h[2 * i + 1] = bf16_hi(xv.w[i]) + bf16_hi(rv.w[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VB / 4; ++i) {
            h[2 * i] = bf16_lo(xv.w[i]);
            h[2 * i + 1] = bf16_hi(xv.w[i]);
        }
    }
}

// Stores of one vector: the residual, and y as bfloat16 and/or MXFP8. Every
// lane of the warp calls (the MXFP8 scale is shared by neighbouring lanes);
// lanes without a vector pass valid = false.
template <int VB, bool MX>
__device__ __forceinline__ void finish_vector(const NormArgs& a, uint32_t row, uint32_t v, bool valid, float r,
                                              const float (&h)[VB / 2]) {
    constexpr int EPT = VB / 2;
    const uint64_t off = (uint64_t(row) * a.nvec + v) * VB;
    Bits<VB> wv;
    if (valid) {
        const uint4* wp = reinterpret_cast<const uint4*>(a.weight + uint64_t(v) * VB);
#pragma unroll
        for (int i = 0; i < VB / 16; ++i) {
            const uint4 q = __ldg(wp + i);   // the same for every row: kept in L1
            wv.w[4 * i] = q.x; wv.w[4 * i + 1] = q.y; wv.w[4 * i + 2] = q.z; wv.w[4 * i + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VB / 4; ++i) wv.w[i] = 0u;
    }
    Bits<VB> y;
#pragma unroll
    for (int i = 0; i < VB / 4; ++i)
        y.w[i] = pack_bf16x2((bf16_lo(wv.w[i]) + a.bias) * (h[2 * i] * r), (bf16_hi(wv.w[i]) + a.bias) * (h[2 * i + 1] * r));
    if (valid && a.residual_out != nullptr) {
        Bits<VB> o;
#pragma unroll
        for (int i = 0; i < VB / 4; ++i) o.w[i] = pack_bf16x2(h[2 * i], h[2 * i + 1]);
        st_global(a.residual_out + off, o);
    }
    if (valid && a.out != nullptr) st_global(a.out + off, y);
    if constexpr (MX) {
        float e[EPT];
#pragma unroll
        for (int i = 0; i < VB / 4; ++i) {
            e[2 * i] = valid ? bf16_lo(y.w[i]) : 0.0f;
            e[2 * i + 1] = valid ? bf16_hi(y.w[i]) : 0.0f;
        }
        const QChunk<kMxfp8, EPT> q = quantize_chunk<kMxfp8, EPT>(e, valid, 0.0f, nullptr);
        if (valid) {
            store_words(a.codes + off / 2, q.codes);
            if (v % (32 / EPT) == 0) a.scales[off / 64] = uint8_t(q.scale);
        }
    }
}

// Sum of s over the row's warps (whole warps per row; a.wpr of them). Every
// thread of the block calls.
__device__ __forceinline__ float row_sum(float s, uint32_t wpr) {
    __shared__ float s_part[kMaxWarps];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
    if (wpr == 1) return s;
    const uint32_t warp = threadIdx.x / kWarp;
    if (threadIdx.x % kWarp == 0) s_part[warp] = s;
    __syncthreads();
    const uint32_t lane = threadIdx.x % kWarp;
    s = lane < wpr ? s_part[warp / wpr * wpr + lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
    return s;
}

template <int VB, int NV, bool MX>
__global__ void __launch_bounds__(kMaxWarps * kWarp) add_rmsnorm_kernel(NormArgs a) {
    pdl_wait_and_release();
    const uint32_t tpr = a.wpr * kWarp;                       // threads per row
    const uint32_t row = blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
    const uint32_t i0 = threadIdx.x % tpr;
    const bool live = row < a.rows;
    float h[NV][VB / 2];
    float ss = 0.0f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const uint32_t v = i0 + n * tpr;
        if (live && v < a.nvec) {
            load_sum<VB>(a, (uint64_t(row) * a.nvec + v) * VB, h[n]);
        } else {
#pragma unroll
            for (int i = 0; i < VB / 2; ++i) h[n][i] = 0.0f;
        }
    }
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int i = 0; i < VB / 2; ++i) ss = fmaf(h[n][i], h[n][i], ss);
    const float r = rsqrtf(row_sum(ss, a.wpr) * a.inv_h + a.eps);
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const uint32_t v = i0 + n * tpr;
        finish_vector<VB, MX>(a, row, v, live && v < a.nvec, r, h[n]);
    }
}

// Rows too long for the registers of one block: one block per row, x and the
// residual read twice. A thread rewrites only residual vectors that it alone
// reads, after it has read them.
template <bool MX>
__global__ void __launch_bounds__(kMaxWarps * kWarp) add_rmsnorm_long_kernel(NormArgs a) {
    constexpr int VB = 16;
    pdl_wait_and_release();
    const uint32_t row = blockIdx.x;
    float ss = 0.0f;
    for (uint32_t v = threadIdx.x; v < a.nvec; v += blockDim.x) {
        float h[VB / 2];
        load_sum<VB>(a, (uint64_t(row) * a.nvec + v) * VB, h);
#pragma unroll
        for (int i = 0; i < VB / 2; ++i) ss = fmaf(h[i], h[i], ss);
    }
    const float r = rsqrtf(row_sum(ss, a.wpr) * a.inv_h + a.eps);
    // warp-uniform loop: the MXFP8 scale needs whole warps
    for (uint32_t base = threadIdx.x / kWarp * kWarp; base < a.nvec; base += blockDim.x) {
        const uint32_t v = base + threadIdx.x % kWarp;
        const bool valid = v < a.nvec;
        float h[VB / 2];
        if (valid) {
            load_sum<VB>(a, (uint64_t(row) * a.nvec + v) * VB, h);
        } else {
#pragma unroll
            for (int i = 0; i < VB / 2; ++i) h[i] = 0.0f;
        }
        finish_vector<VB, MX>(a, row, v, valid, r, h);
    }
}

// Vectors per thread and warps per row: as few vectors as keep the row within
// one block (T=4096, H=2048, MXFP8 and bfloat16 out: 11.4 us with one, 13.9 with
// two; T=8192, H=4096: 40.4 and 42.1). Rows per block: about 128 threads (11.4
// us; 11.8 with 256, 12.9 with 512).
template <int VB, bool MX>
cudaError_t launch_vb(NormArgs a, int64_t T, uint32_t H, cudaStream_t stream) {
    a.nvec = H / (VB / 2);
    uint32_t nv = 1;
    while (nv <= 4 && a.nvec > nv * kMaxWarps * kWarp) nv *= 2;
    const bool is_long = nv > 4;
    a.wpr = is_long ? kMaxWarps : (a.nvec + nv * kWarp - 1) / (nv * kWarp);
    const uint32_t rpb = a.wpr >= 4 ? 1 : 4 / a.wpr;   // rows per block
    const int64_t rows_per_launch = std::max<int64_t>(1, int64_t(kMaxItemsPerLaunch / a.nvec));
    const uint8_t *x = a.x, *res = a.residual;
    for (int64_t t0 = 0; t0 < T; t0 += rows_per_launch) {
        const int64_t n = std::min(rows_per_launch, T - t0);
        const uint64_t off = uint64_t(t0) * 2 * H;
        NormArgs b = a;
        b.x = x + off;
        b.residual = res ? res + off : nullptr;
        b.out = a.out ? a.out + off : nullptr;
        b.residual_out = a.residual_out ? a.residual_out + off : nullptr;
        if (MX) {
            b.codes = a.codes + off / 2;
            b.scales = a.scales + off / 64;
        }
        b.rows = uint32_t(n);
        const dim3 grid(uint32_t((n + rpb - 1) / rpb)), block(a.wpr * rpb * kWarp);
        cudaError_t err;
        if (is_long) {
            if constexpr (VB == 16)
                err = launch_pdl(add_rmsnorm_long_kernel<MX>, dim3(uint32_t(n)), block, 0, stream, b);
            else
                err = cudaErrorInvalidConfiguration;
        }
        else if (nv == 1) err = launch_pdl(add_rmsnorm_kernel<VB, 1, MX>, grid, block, 0, stream, b);
        else if (nv == 2) err = launch_pdl(add_rmsnorm_kernel<VB, 2, MX>, grid, block, 0, stream, b);
        else err = launch_pdl(add_rmsnorm_kernel<VB, 4, MX>, grid, block, 0, stream, b);
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_add_rmsnorm(const uint16_t* x, const uint16_t* residual, int64_t T, int H, const uint16_t* weight,
                               float bias, float eps, uint16_t* out, uint16_t* residual_out, uint8_t* codes,
                               uint8_t* scales, cudaStream_t stream) {
    NormArgs a = {};
    a.x = reinterpret_cast<const uint8_t*>(x);
    a.residual = reinterpret_cast<const uint8_t*>(residual);
    a.weight = reinterpret_cast<const uint8_t*>(weight);
    a.out = reinterpret_cast<uint8_t*>(out);
    a.residual_out = reinterpret_cast<uint8_t*>(residual_out);
    a.codes = codes;
    a.scales = scales;
    a.bias = bias;
    a.eps = eps;
    a.inv_h = 1.0f / float(H);
    // the 32-byte form holds up to 4 * 1024 vectors of 16 values (T=8192, H=4096: 40.4 us; 44.3 in 16-byte pieces)
    const bool wide = can_use_32b(uint64_t(2) * H, {x, residual, weight, out, residual_out}) && H <= 65536;
    if (codes != nullptr)
        return wide ? launch_vb<32, true>(a, T, uint32_t(H), stream) : launch_vb<16, true>(a, T, uint32_t(H), stream);
    return wide ? launch_vb<32, false>(a, T, uint32_t(H), stream) : launch_vb<16, false>(a, T, uint32_t(H), stream);
}

}  // namespace moe
