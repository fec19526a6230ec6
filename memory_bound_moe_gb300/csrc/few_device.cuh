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
//
// Each warp streams its weights through a ring of its own in shared memory:
// a lane copies its granules in with cp.async and reads the same 16 bytes
// back, so the ring needs no barrier, costs no registers, and D chunks (4 KB
// each) stay in flight per warp while another is being multiplied.
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

// One lane's granules of two weight rows (g and g + 8 of a tile) at one step.
struct AGran {
    Bits<16> w[2];
};

// Where a chunk lies: US steps from `step` on, of the rows g (+ 8) of R tiles.
struct WChunk {
    const uint8_t* w;      // this lane's granule of its first row at step 0
    const uint8_t* s;      // that row's first scale
    uint32_t rows;         // bit 2 r + h: row exists (all clear: nothing to fetch)
    uint32_t step;
};

// Distances in bytes between a lane's rows: from tile to tile, and from row g
// to row g + 8 of a tile; of the weights and of the scales.
struct WStride {
    uint64_t tile_w, half_w, tile_s, half_s;
};

// A warp's ring of D chunks in shared memory.
template <int F, int R, int US, int D>
struct WRing {
    static constexpr uint32_t kChunk = US * R * 2 * 512;   // bytes
    static constexpr uint32_t kBytes = kChunk * D;
    uint32_t base;                                         // this lane's first granule
    uint32_t slot;                                         // byte offset of the next chunk to read (and refill)

    __device__ __forceinline__ void init(uint8_t* smem) {
        base = uint32_t(__cvta_generic_to_shared(smem)) + (threadIdx.x % kWarp) * 16u;
        slot = 0;
    }

    // Start copying a chunk into the slot at byte offset `at`. Granules outside
    // the matrix are zero-filled and nothing is read for them; chunks that lie
    // wholly inside (nearly all) skip those tests.
    __device__ __forceinline__ void fetch(uint32_t at, const WChunk& c, const WStride& st, const uint8_t* any,
                                          uint32_t rb) {
        const bool inside = c.rows == (1u << (2 * R)) - 1u && (c.step + US) * 64u <= rb;
        if (__all_sync(kFull, inside)) {
            const uint8_t* p = c.w + c.step * 64u;
#pragma unroll
            for (int i = 0; i < US; ++i)
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(base + at + ((i * R + r) * 2 + h) * 512u),
                                     "l"(p + r * st.tile_w + h * st.half_w + i * 64)
                                     : "memory");
            return;
        }
        const uint32_t q16 = (threadIdx.x % 4) * 16u;
#pragma unroll 1
        for (int i = 0; i < US; ++i) {
            const uint32_t off = (c.step + i) * 64u;
#pragma unroll 1
            for (int r = 0; r < R; ++r)
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    const bool ok = off + q16 < rb && ((c.rows >> (2 * r + h)) & 1u);
                    const uint8_t* p = ok ? c.w + r * st.tile_w + h * st.half_w + off : any;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(base + at + ((i * R + r) * 2 + h) * 512u),
                                 "l"(p), "r"(ok ? 16 : 0)
                                 : "memory");
                }
        }
    }
    __device__ __forceinline__ static void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

    // Nothing may be in flight when the block ends.
    __device__ __forceinline__ static void drain() { asm volatile("cp.async.wait_all;" ::: "memory"); }

    // Wait for the oldest chunk: all but the D - 1 newest groups are complete.
    __device__ __forceinline__ static void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory"); }

    // This lane's granules of tile r at step i of that chunk.
    __device__ __forceinline__ void read(AGran& a, int i, int r) const {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(a.w[h].w[0]), "=r"(a.w[h].w[1]), "=r"(a.w[h].w[2]), "=r"(a.w[h].w[3])
                         : "r"(base + slot + uint32_t((i * R + r) * 2 + h) * 512u)
                         : "memory");
    }
    __device__ __forceinline__ void next() { slot = slot + kChunk == kBytes ? 0u : slot + kChunk; }
};

// The scales of a chunk's granules (4-bit weights): read ahead by one chunk,
// 32 bytes of a row's scales serve 4 to 8 steps from L1.
template <int F, int R, int US>
struct WScales {
    uint32_t s[WInfo<F>::kFp4 ? US : 1][R][2];

    __device__ __forceinline__ void load(const WChunk& c, const WStride& st, uint32_t rb) {
        if constexpr (WInfo<F>::kFp4) {
            const int q = threadIdx.x % 4;
            const uint32_t bytes = F == kWNvfp4 ? 2 : 1;   // per granule
            const bool inside = c.rows == (1u << (2 * R)) - 1u && (c.step + US) * 64u <= rb;
            const uint8_t* p = c.s + (c.step * 4u + q) * bytes;
            if (__all_sync(kFull, inside)) {
#pragma unroll
                for (int i = 0; i < US; ++i)
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int h = 0; h < 2; ++h) s[i][r][h] = one(p + r * st.tile_s + h * st.half_s + i * 4 * bytes);
            } else {
#pragma unroll
                for (int i = 0; i < US; ++i)
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const bool ok = (c.step + i) * 64u + q * 16u < rb && ((c.rows >> (2 * r + h)) & 1u);
                            s[i][r][h] = ok ? one(p + r * st.tile_s + h * st.half_s + i * 4 * bytes) : 0u;
                        }
            }
        }
    }

private:
    __device__ __forceinline__ static uint32_t one(const uint8_t* p) {
        if constexpr (F == kWNvfp4) return __ldg(reinterpret_cast<const uint16_t*>(p));
        else return __ldg(p);
    }
};

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

// Products of one step, bfloat16 weights: R tiles of 16 rows against the
// groups of 8 tokens set in `live` (a bit each, the same for the whole warp).
// tile(a, r) reads a tile's granules, load(n, b) the x of group n.
template <int R, int NG, typename Tile, typename Load>
__device__ __forceinline__ void bf16_step(float (&acc)[R][NG][4], uint32_t live, Tile&& tile, Load&& load) {
    BGran<kWBf16> b[NG];
#pragma unroll
    for (int n = 0; n < NG; ++n)
        if (NG == 1 || ((live >> n) & 1u)) load(n, b[n]);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        AGran a;
        tile(a, r);
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            if (NG > 1 && !((live >> n) & 1u)) continue;
            mma_bf16(acc[r][n], a.w[0].w[0], a.w[1].w[0], a.w[0].w[1], a.w[1].w[1], b[n].x[0].x, b[n].x[0].y);
            mma_bf16(acc[r][n], a.w[0].w[2], a.w[1].w[2], a.w[0].w[3], a.w[1].w[3], b[n].x[0].z, b[n].x[0].w);
        }
    }
}

// A warp's accumulators -> its part of the block's partial sums
// s_red[warp][token][row], rows 0..16 R - 1 of the first `cols` tokens (C
// fragment: lane (g, q) holds rows g, g + 8 of tokens 2 q, 2 q + 1).
template <int R, int NG>
__device__ __forceinline__ void store_partial(float* s_warp, const float (&acc)[R][NG][4], int cols) {
    const int lane = threadIdx.x % kWarp, g = lane / 4, q = lane % 4;
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const int c = n * 8 + 2 * q + z;
            if (c < cols) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    s_warp[c * (16 * R) + r * 16 + g] = acc[r][n][z];
                    s_warp[c * (16 * R) + r * 16 + g + 8] = acc[r][n][z + 2];
                }
            }
        }
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
