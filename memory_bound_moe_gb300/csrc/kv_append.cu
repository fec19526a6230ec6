// Rotary embedding of q and k with the write of k and v into a paged cache:
// memory-bound, every value read once and written once.
//
// A "piece" is 16 columns of a head, two 16-byte vectors: columns i .. i + 7
// and rot/2 + i .. rot/2 + i + 7 in the half form, 16 contiguous columns in the
// pair form and behind rot. A lane keeps one piece of one token, whose cosines
// and sines it loads once, and goes over the token's heads (q, then k, then v),
// kU heads' loads in flight, the first of them before the slot is known.
#include "moe_device.cuh"
#include "moe_launch.h"
#include "quant_device.cuh"
#include "rows_common.cuh"

namespace moe {
namespace {

constexpr int kNt = 128;
// Two heads' loads in flight and 28 warps per SM: more of either costs the other through its
// registers (GB300, 8192 tokens of 32 + 4 heads of 128: 30.0 us; 4 heads and 16 warps 32.2 us,
// 2 heads and 32 warps 31.2 us, 1 head and 32 warps 32.2 us).
constexpr int kU = 2;
constexpr int kBlocks = 7;   // of an SM

__device__ __forceinline__ void unpack(const Bits<16>& b, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(b.w[i]);
        x[2 * i + 1] = bf16_hi(b.w[i]);
    }
}

// x in bfloat16, or the bits it came from where it is the same value.
__device__ __forceinline__ void store(void* p, const Bits<16>& from, const float (&x)[8], bool same) {
    Bits<16> b;
#pragma unroll
    for (int i = 0; i < 4; ++i) b.w[i] = same ? from.w[i] : pack_bf16x2(x[2 * i], x[2 * i + 1]);
    st_global(p, b);
}

__device__ __forceinline__ void store_e4m3(void* p, const float (&x)[8], float inv) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = uint32_t(pack_e4m3x2(x[4 * i] * inv, x[4 * i + 1] * inv)) |
               (uint32_t(pack_e4m3x2(x[4 * i + 2] * inv, x[4 * i + 3] * inv)) << 16);
    asm volatile("st.global.v2.u32 [%0], {%1,%2};" ::"l"(p), "r"(w[0]), "r"(w[1]) : "memory");
}

// Warps of a token: `parts` of them share its heads.
template <int D, bool E4M3, bool PAIRS>
__global__ void __launch_bounds__(kNt, kBlocks) kv_append_kernel(const AppendArgs a, int parts) {
    constexpr int kPieces = D / 16, kHeads = kWarp / kPieces;   // heads a warp covers at once
    pdl_wait_and_release();
    const int lane = threadIdx.x % kWarp;
    const int64_t warp = int64_t(blockIdx.x) * (kNt / kWarp) + threadIdx.x / kWarp;
    const int64_t t = warp / parts;
    if (t >= a.N) return;
    const int64_t slot = a.slots[t];
    const int64_t pos = a.rot > 0 ? a.positions[t] : 0;

    // columns of this lane's two vectors
    const int piece = lane % kPieces, half = a.rot / 2;
    const bool turned = piece * 16 < a.rot;
    const int c0 = turned && !PAIRS ? piece * 8 : piece * 16;
    const int c1 = turned && !PAIRS ? half + piece * 8 : c0 + 8;
    const int kh = a.cache.heads, all = a.q_heads + 2 * kh, step = kHeads * parts;
    Bits<16> lo[kU], hi[kU];
    const auto load = [&](int base) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int h = base + u * step + lane / kPieces;
            if (h < all) {
                const uint16_t* src = h < a.q_heads ? a.q + t * a.q_stride + h * D
                                      : h < a.q_heads + kh ? a.k + t * a.k_stride + (h - a.q_heads) * D
                                                           : a.v + t * a.v_stride + (h - a.q_heads - kh) * D;
                ld_coherent(lo[u], src + c0);   // q and k may be written in place
                ld_coherent(hi[u], src + c1);
            }
        }
    };
    const int first = int(warp % parts) * kHeads;
    load(first);   // on their way while the slot and the angles come
    if (slot < 0 || (slot >> a.cache.page_shift) >= a.cache.num_pages) return;
    if (a.rot > 0 && (pos < 0 || pos >= a.max_positions)) return;
    const int64_t page = slot >> a.cache.page_shift, row = slot & ((int64_t(1) << a.cache.page_shift) - 1);
    uint8_t* const kc = a.cache.k + page * a.cache.k_page + row * a.cache.k_token;
    uint8_t* const vc = a.cache.v + page * a.cache.v_page + row * a.cache.v_token;
    const float k_inv = 1.0f / a.cache.k_scale, v_inv = 1.0f / a.cache.v_scale;

    float cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        cs[i] = 1.0f;
        sn[i] = 0.0f;
    }
    if (turned) {
        const float4* p = reinterpret_cast<const float4*>(a.cos_sin + pos * a.rot + piece * 8);
        const float4* q = reinterpret_cast<const float4*>(a.cos_sin + pos * a.rot + half + piece * 8);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 x = p[i], y = q[i];
            cs[4 * i] = x.x; cs[4 * i + 1] = x.y; cs[4 * i + 2] = x.z; cs[4 * i + 3] = x.w;
            sn[4 * i] = y.x; sn[4 * i + 1] = y.y; sn[4 * i + 2] = y.z; sn[4 * i + 3] = y.w;
        }
    }

    for (int base = first; base < all; base += step * kU) {
        if (base != first) load(base);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int h = base + u * step + lane / kPieces;
            if (h >= all) continue;
            float x[8], y[8];
            unpack(lo[u], x);
            unpack(hi[u], y);
            const bool value = h >= a.q_heads + kh, same = value || !turned;
            if (!same) {
                if (PAIRS) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float p = x[2 * i], q = y[2 * i];
                        x[2 * i] = p * cs[i] - x[2 * i + 1] * sn[i];
                        x[2 * i + 1] = x[2 * i + 1] * cs[i] + p * sn[i];
                        y[2 * i] = q * cs[4 + i] - y[2 * i + 1] * sn[4 + i];
                        y[2 * i + 1] = y[2 * i + 1] * cs[4 + i] + q * sn[4 + i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float p = x[i];
                        x[i] = p * cs[i] - y[i] * sn[i];
                        y[i] = y[i] * cs[i] + p * sn[i];
                    }
                }
            }
            if (h < a.q_heads) {
                uint16_t* dst = a.q_out + t * a.q_out_stride + h * D;
                store(dst + c0, lo[u], x, same);
                store(dst + c1, hi[u], y, same);
                continue;
            }
            const int kv = value ? h - a.q_heads - kh : h - a.q_heads;
            uint8_t* dst = value ? vc + kv * a.cache.v_head : kc + kv * a.cache.k_head;
            if constexpr (E4M3) {
                const float inv = value ? v_inv : k_inv;
                store_e4m3(dst + c0, x, inv);
                store_e4m3(dst + c1, y, inv);
            } else {
                store(dst + 2 * c0, lo[u], x, same);
                store(dst + 2 * c1, hi[u], y, same);
            }
            if (!value && a.k_out != nullptr) {
                uint16_t* ko = a.k_out + t * a.k_out_stride + kv * D;
                store(ko + c0, lo[u], x, same);
                store(ko + c1, hi[u], y, same);
            }
        }
    }
}

template <int D>
cudaError_t launch_d(const AppendArgs& a, int num_sms, cudaStream_t stream) {
    constexpr int kHeads = kWarp / (D / 16);
    const int rounds = (a.q_heads + 2 * a.cache.heads + kHeads - 1) / kHeads;   // of one warp, a head row each
    // a token's rounds on several warps where tokens alone leave SMs without: up to 16 or more warps
    // an SM (1023 tokens of 16 + 2 heads of 256 into E4M3: 5.4 us; up to 32: 8.0 us)
    int parts = 1;
    while (parts < rounds && int64_t(a.N) * parts < int64_t(num_sms) * 16) parts *= 2;
    parts = std::min(parts, rounds);
    const int64_t warps = int64_t(a.N) * parts;
    const int64_t grid = (warps + kNt / kWarp - 1) / (kNt / kWarp);
    auto kernel = a.cache.e4m3 ? (a.interleaved ? kv_append_kernel<D, true, true> : kv_append_kernel<D, true, false>)
                               : (a.interleaved ? kv_append_kernel<D, false, true> : kv_append_kernel<D, false, false>);
    return launch_pdl(kernel, dim3(unsigned(grid)), dim3(kNt), 0, stream, a, parts);
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, int num_sms, cudaStream_t stream) {
    switch (a.cache.head_dim) {
        case 64: return launch_d<64>(a, num_sms, stream);
        case 128: return launch_d<128>(a, num_sms, stream);
        case 256: return launch_d<256>(a, num_sms, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace moe
