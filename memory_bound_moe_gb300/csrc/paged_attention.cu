// Attention of one new token per sequence over a paged key-value cache.
//
// The G = num_q_heads / num_heads query heads that share a key head make up to
// 16 rows of an m16n8k16 product (more than 16: several groups), so a cached
// element is read once for all of them and costs 4 G operations for 4 bytes: at
// G = 16 that is 16 operations a byte, where this GPU has 280. Reading the
// cache bounds it, and mma.sync keeps up with HBM at a quarter of its rate; a
// 128-row tcgen05 tile would be empty to seven eighths or more.
//
// Split. A unit of work is (sequence, key head, group of 16 heads); its tiles
// are 64 tokens. All units' tiles, one after another, are cut into equal runs,
// one per resident block: whatever the lengths are, every SM reads the same
// number of bytes (the lengths are on the GPU, so every block adds them up for
// itself). A unit inside one run is finished there; what a run has of a unit
// that goes on in another run goes to the workspace (at most two per run), and
// a second kernel joins those in order of the runs.
//
// A block's 4 warps take 16 tokens of a tile each and never meet inside a unit:
// each has its own ring of kStages steps in shared memory, filled by 16-byte
// cp.async, and its own running maximum, sum and output (online softmax); the
// four are joined when the run leaves the unit.
#include "few_device.cuh"
#include "moe_launch.h"

namespace moe {
namespace {

constexpr int kWarps = 4;
constexpr int kNt = kWarps * kWarp;
constexpr int kRows = 16;            // query heads of a unit
constexpr int kStep = 16;            // tokens of a warp's step
constexpr int kTile = kWarps * kStep;
constexpr int kStages = 3;
constexpr int kMaxBlocks = 640;      // runs the workspace holds the ends of
constexpr int kMinTiles = 2;         // tiles of a run, at least
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// ---------------------------------------------------------------------------
// Workspace: for every run two partial results (a unit that began in an earlier
// run, a unit that goes on in a later one), then a note per run of the unit that
// begins in it and is split.
// ---------------------------------------------------------------------------

struct Note {
    int32_t b, unit, last, pad;   // b < 0: none; last: the unit's last run
};

struct Partials {
    float* o;      // [2 blocks][rows][D], weighted by 2^(x - m)
    float* m;      // [2 blocks][rows], log2 units
    float* l;      // [2 blocks][rows]
    Note* notes;   // [blocks]
};

__host__ __device__ inline int unit_rows(int group) { return group < kRows ? group : kRows; }

__host__ __device__ inline Partials partials(void* ws, int blocks, int rows, int D) {
    Partials p;
    p.o = static_cast<float*>(ws);
    p.m = p.o + int64_t(2) * blocks * rows * D;
    p.l = p.m + int64_t(2) * blocks * kRows;
    p.notes = reinterpret_cast<Note*>(p.l + int64_t(2) * blocks * kRows);
    return p;
}

// ---------------------------------------------------------------------------
// PTX
// ---------------------------------------------------------------------------

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
    const int n = valid ? 16 : 0;   // 0: zeros, nothing is read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(p) : "memory");
}

__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(p) : "memory");
}

template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Two E4M3 bytes (the low 16 bits of w) -> two f16, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
    uint32_t d;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(d) : "r"(w));
    return d;
}

// ---------------------------------------------------------------------------
// The tokens of a sequence, and where a run begins
// ---------------------------------------------------------------------------

struct Span {
    int first, len, tiles;   // tokens first .. len - 1; tiles counted from first / kTile
    __device__ __forceinline__ int tile0() const { return first / kTile; }
};

__device__ __forceinline__ Span span_of(const AttentionArgs& a, int b) {
    Span s;
    const int64_t most = int64_t(a.max_pages) << a.cache.page_shift;
    s.len = int(min(int64_t(max(a.lengths[b], 0)), most));
    s.first = a.window > 0 && s.len > a.window ? s.len - a.window : 0;
    s.tiles = s.len == 0 ? 0 : (s.len - 1) / kTile + 1 - s.tile0();
    return s;
}

struct Place {
    int64_t run;      // tiles of a run
    int64_t total;    // tiles of all units
    int64_t base;     // tiles before sequence b's units
    int b;            // the sequence in which this block's run begins
};

// Every block adds up the sequences' tiles for itself. A thread's sequences
// are a run of them, so that the thread in whose range this block's run begins
// can walk to its sequence.
__device__ __forceinline__ Place find_run(const AttentionArgs& a, int units) {
    __shared__ int64_t s_warp[kWarps];
    __shared__ int64_t s_base;
    __shared__ int s_b;
    const int per = (a.B + kNt - 1) / kNt, b0 = min(a.B, int(threadIdx.x) * per), b1 = min(a.B, b0 + per);
    int64_t sum = 0;
#pragma unroll 4
    for (int b = b0; b < b1; ++b) sum += span_of(a, b).tiles;
    sum *= units;
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    int64_t x = sum;
#pragma unroll
    for (int o = 1; o < kWarp; o <<= 1) {
        const int64_t y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
    }
    if (lane == kWarp - 1) s_warp[warp] = x;
    __syncthreads();
    int64_t total = 0, before = x - sum;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_warp[w];
        total += s_warp[w];
    }
    Place p;
    p.total = total;
    p.run = max(int64_t(kMinTiles), (total + gridDim.x - 1) / gridDim.x);
    const int64_t start = p.run * blockIdx.x;
    if (before <= start && start < before + sum) {
        int b = b0;
        int64_t n = int64_t(span_of(a, b).tiles) * units;
        while (before + n <= start) {
            before += n;
            n = int64_t(span_of(a, ++b).tiles) * units;
        }
        s_base = before;
        s_b = b;
    }
    __syncthreads();
    p.base = s_base;
    p.b = s_b;
    return p;
}

// ---------------------------------------------------------------------------
// Main kernel
// ---------------------------------------------------------------------------

template <int D, bool E4M3>
struct Tile {
    static constexpr int kBytes = D * (E4M3 ? 1 : 2);      // of a token's head
    static constexpr int kVecs = kBytes / 16;
    static constexpr int kSide = kStep * kBytes;           // keys or values of a step
    static constexpr int kRing = kStages * 2 * kSide;      // of a warp
    static constexpr int kPitch = D + 8;                   // floats between output rows: no bank conflicts
    static constexpr int kSmem = kWarps * kRing;
    static_assert(kRows * kPitch * 4 <= kRing, "a warp's output takes the place of its ring");
    // 16-byte vector v of row r lies at v ^ swz(r): 8 rows at the same vector hit 8 different banks of 16 bytes
    static __device__ __forceinline__ int swz(int r) { return kVecs >= 8 ? r & 7 : (r >> 1) & 3; }
    static __device__ __forceinline__ uint32_t at(int r, int v) { return uint32_t(r * kBytes + ((v ^ swz(r)) << 4)); }
};

// One side (keys or values) of a step into shared memory: row r from src + its
// page's and token's offset.
template <int D, bool E4M3>
__device__ __forceinline__ void load_side(uint32_t dst, const uint8_t* src, int page_shift, int64_t page_stride, int64_t token_stride,
                                          int page, int t0, uint32_t mask) {
    using T = Tile<D, E4M3>;
    constexpr int kPer = kWarp / T::kVecs > 0 ? kWarp / T::kVecs : 1;   // rows per instruction
    const int lane = threadIdx.x % kWarp, v = lane % T::kVecs;
    const int in_page = (1 << page_shift) - 1;
#pragma unroll
    for (int i = 0; i < kStep / kPer; ++i) {
        const int r = i * kPer + lane / T::kVecs;
        const int pg = page_shift >= 4 ? page : __shfl_sync(kFull, page, r);
        const bool valid = (mask >> r) & 1u;
        const uint8_t* p = src + (valid ? int64_t(pg) * page_stride + int64_t((t0 + r) & in_page) * token_stride + v * 16 : 0);
        cp_async16(dst + T::at(r, v), p, valid);
    }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kNt) attention_kernel(const AttentionArgs a, int groups) {
    using T = Tile<D, E4M3>;
    constexpr int kD16 = D / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
    pdl_wait_and_release();
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp, g = lane / 4, quad = lane % 4;
    const int heads = a.cache.heads, group = a.q_heads / heads, units = heads * groups;
    const Partials ws = partials(a.workspace, gridDim.x, unit_rows(group), D);
    uint8_t* const ring = smem + warp * T::kRing;
    const uint32_t ring_at = uint32_t(__cvta_generic_to_shared(ring));

    // sequences without tokens
    for (int b = blockIdx.x; b < a.B; b += gridDim.x)
        if (span_of(a, b).tiles == 0) {
            uint4* o = reinterpret_cast<uint4*>(a.out + int64_t(b) * a.q_heads * D);
            for (int i = threadIdx.x; i < a.q_heads * D / 8; i += kNt) o[i] = make_uint4(0, 0, 0, 0);
            if (a.lse != nullptr)
                for (int i = threadIdx.x; i < a.q_heads; i += kNt) a.lse[int64_t(b) * a.q_heads + i] = -INFINITY;
        }

    const Place place = find_run(a, units);
    int64_t pos = place.run * blockIdx.x;
    const int64_t end = min(place.total, pos + place.run);
    Note note = {-1, 0, 0, 0};
    int b = place.b;
    Span s = {};
    int unit = 0, local = 0;
    if (pos < end) {
        s = span_of(a, b);
        unit = int((pos - place.base) / s.tiles);
        local = int((pos - place.base) % s.tiles);
    }
    while (pos < end) {
        const int seg = int(min(int64_t(s.tiles - local), end - pos));
        const int head = unit / groups, chunk = unit % groups;
        const int rows = min(kRows, group - chunk * kRows);
        const int h0 = head * group + chunk * kRows;

        // q, as A: row g (and g + 8) is head h0 + g. For E4M3 the order of the 16 columns of a
        // product is that in which the keys' bytes come out of ldmatrix: 4 quad .. 4 quad + 3.
        uint32_t aq[kD16][4];
        float c[2];   // what a row's scores are multiplied by, with log2 e
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = g + 8 * h;
            const uint16_t* q = a.q + int64_t(b) * a.q_stride + int64_t(h0 + r) * D;
            c[h] = a.scale * a.cache.k_scale * kLog2e;
            if constexpr (!E4M3) {
#pragma unroll
                for (int k = 0; k < kD16; ++k) {
                    aq[k][h] = r < rows ? *reinterpret_cast<const uint32_t*>(q + k * 16 + quad * 2) : 0u;
                    aq[k][h + 2] = r < rows ? *reinterpret_cast<const uint32_t*>(q + k * 16 + quad * 2 + 8) : 0u;
                }
            } else {
                uint2 w[kD16];
                float most = 0.0f;
#pragma unroll
                for (int k = 0; k < kD16; ++k) {
                    w[k] = r < rows ? *reinterpret_cast<const uint2*>(q + k * 16 + quad * 4) : make_uint2(0u, 0u);
                    most = fmaxf(fmaxf(most, fmaxf(fabsf(bf16_lo(w[k].x)), fabsf(bf16_hi(w[k].x)))),
                                 fmaxf(fabsf(bf16_lo(w[k].y)), fabsf(bf16_hi(w[k].y))));
                }
                most = fmaxf(most, __shfl_xor_sync(kFull, most, 1));
                most = fmaxf(most, __shfl_xor_sync(kFull, most, 2));
                // f16 holds q times 2^(14 - e), e the exponent of the row's largest (1 for a row of zeros or with an infinity)
                const int e = most > 0.0f && most < INFINITY ? max(int(__float_as_uint(most) >> 23) - 127, -112) : 14;
                const float up = __uint_as_float(uint32_t(127 + 14 - e) << 23);
                c[h] *= __uint_as_float(uint32_t(127 - 14 + e) << 23);
#pragma unroll
                for (int k = 0; k < kD16; ++k) {
                    aq[k][h] = pack_f16x2(bf16_lo(w[k].x) * up, bf16_hi(w[k].x) * up);
                    aq[k][h + 2] = pack_f16x2(bf16_lo(w[k].y) * up, bf16_hi(w[k].y) * up);
                }
            }
        }

        float o[D / 8][4] = {};
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
        {
            // this warp's steps: tokens t_at(j) .. t_at(j) + 15
            const int begin = (s.tile0() + local) * kTile;
            const int from = max(begin, s.first & ~(kStep - 1)), to = min(s.len, begin + seg * kTile);
            const int steps_all = (to - from + kStep - 1) / kStep;
            const int steps = (steps_all - warp + kWarps - 1) / kWarps;
            const auto t_at = [&](int j) { return from + (j * kWarps + warp) * kStep; };
            const int32_t* table = a.block_table + int64_t(b) * a.max_pages;
            const uint8_t* kp = a.cache.k + head * a.cache.k_head;
            const uint8_t* vp = a.cache.v + head * a.cache.v_head;
            // the page of token t_at(j) + lane % 16; -1 where there is none
            const auto page_of = [&](int j) {
                if (j >= steps) return -1;
                const int t = t_at(j) + lane % kStep;
                if (t < s.first || t >= s.len) return -1;
                const int pg = table[t >> a.cache.page_shift];
                return pg < a.cache.num_pages ? pg : -1;
            };
            const auto issue = [&](int j, int page) -> uint32_t {
                const uint32_t mask = __ballot_sync(kFull, page >= 0) & 0xffffu;
                if (j < steps) {
                    const uint32_t dst = ring_at + (j % kStages) * 2 * T::kSide;
                    int pg = page;
                    if (a.cache.page_shift >= 4) pg = __shfl_sync(kFull, page, mask != 0 ? __ffs(mask) - 1 : 0);
                    load_side<D, E4M3>(dst, kp, a.cache.page_shift, a.cache.k_page, a.cache.k_token, pg, t_at(j), mask);
                    load_side<D, E4M3>(dst + T::kSide, vp, a.cache.page_shift, a.cache.v_page, a.cache.v_token, pg, t_at(j), mask);
                }
                cp_commit();
                return mask;
            };
            uint32_t masks[kStages];
            int pages[kStages];
#pragma unroll
            for (int i = 0; i < kStages; ++i) pages[i] = page_of(i);
#pragma unroll
            for (int i = 0; i + 1 < kStages; ++i) masks[i] = issue(i, pages[i]);
            int page = pages[kStages - 1];
            for (int j = 0; j < steps; ++j) {
                cp_wait<kStages - 2>();
                __syncwarp();
                masks[kStages - 1] = issue(j + kStages - 1, page);
                page = page_of(j + kStages);
                const uint32_t ks = ring_at + (j % kStages) * 2 * T::kSide, vs = ks + T::kSide;
                const uint32_t mask = masks[0];
#pragma unroll
                for (int i = 0; i + 1 < kStages; ++i) masks[i] = masks[i + 1];

                float x[2][4] = {};   // [8 tokens][row g: tokens 2 quad, 2 quad + 1; row g + 8: the same]
                if constexpr (!E4M3) {
                    const int row = lane % 8 + (lane & 16) / 2, v = (lane >> 3) & 1;
#pragma unroll
                    for (int k = 0; k < kD16; ++k) {
                        uint32_t r[4];
                        ldsm(r, ks + T::at(row, 2 * k + v));
                        mma<false>(x[0], aq[k], r[0], r[1]);
                        mma<false>(x[1], aq[k], r[2], r[3]);
                    }
                } else {
                    const int row = lane % 16, v = lane >> 4;
#pragma unroll
                    for (int k = 0; k < kD16; k += 2) {
                        uint32_t r[4];
                        ldsm(r, ks + T::at(row, k + v));
#pragma unroll
                        for (int z = 0; z < 4; ++z)
                            mma<true>(x[z & 1], aq[k + z / 2], e4m3x2_to_f16x2(r[z]), e4m3x2_to_f16x2(r[z] >> 16));
                    }
                }
                float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const bool seen = (mask >> (n * 8 + quad * 2 + (z & 1))) & 1u;
                        x[n][z] = seen ? x[n][z] * c[z >> 1] : -INFINITY;
                        top[z >> 1] = fmaxf(top[z >> 1], x[n][z]);
                    }
                bool more = false;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    top[h] = fmaxf(top[h], __shfl_xor_sync(kFull, top[h], 1));
                    top[h] = fmaxf(top[h], __shfl_xor_sync(kFull, top[h], 2));
                    more |= top[h] > m[h];
                }
                if (__any_sync(kFull, more)) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float now = fmaxf(m[h], top[h]);
                        const float f = now == -INFINITY ? 1.0f : ex2_approx(m[h] - now);
                        m[h] = now;
                        l[h] *= f;
#pragma unroll
                        for (int d = 0; d < D / 8; ++d) {
                            o[d][2 * h] *= f;
                            o[d][2 * h + 1] *= f;
                        }
                    }
                }
                // weights 2^(x - m); for f16 times 2^15, so that those down to 2^-39 of the largest count
                float base[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) base[h] = (m[h] == -INFINITY ? 0.0f : m[h]) - (E4M3 ? 15.0f : 0.0f);
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        x[n][z] = ex2_approx(x[n][z] - base[z >> 1]);
                        l[z >> 1] += x[n][z];
                    }
                if constexpr (!E4M3) {
                    // two bfloat16 terms: the upper half of the float, and what it leaves. (One alone
                    // would cost as much as the output's own rounding.) The rest is never 0, so that
                    // an infinite value does not become NaN by it.
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float p0 = x[i >> 1][2 * (i & 1)], p1 = x[i >> 1][2 * (i & 1) + 1];
                        const uint32_t u0 = __float_as_uint(p0) & 0xffff0000u, u1 = __float_as_uint(p1) & 0xffff0000u;
                        hi[i] = (u0 >> 16) | u1;
                        lo[i] = pack_bf16x2(fmaxf(p0 - __uint_as_float(u0), 1.2e-38f), fmaxf(p1 - __uint_as_float(u1), 1.2e-38f));
                    }
                    const int row = lane % 16, v = lane >> 4;
#pragma unroll
                    for (int d = 0; d < kD16; ++d) {
                        uint32_t r[4];
                        ldsm_t(r, vs + T::at(row, 2 * d + v));
                        mma<false>(o[2 * d], hi, r[0], r[1]);
                        mma<false>(o[2 * d + 1], hi, r[2], r[3]);
                        mma<false>(o[2 * d], lo, r[0], r[1]);
                        mma<false>(o[2 * d + 1], lo, r[2], r[3]);
                    }
                } else {
                    uint32_t p[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) p[i] = pack_f16x2(x[i >> 1][2 * (i & 1)], x[i >> 1][2 * (i & 1) + 1]);
                    // A transposed 16-bit unit is two columns' bytes: even columns make one product, odd ones another.
                    const int row = lane % 16, v = lane >> 4;
#pragma unroll
                    for (int d = 0; d < kD16; d += 2) {
                        uint32_t r[4];
                        ldsm_t(r, vs + T::at(row, d + v));
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            const uint32_t r0 = r[2 * z], r1 = r[2 * z + 1];
                            mma<true>(o[2 * (d + z)], p, e4m3x2_to_f16x2(__byte_perm(r0, 0, 0x4420)), e4m3x2_to_f16x2(__byte_perm(r1, 0, 0x4420)));
                            mma<true>(o[2 * (d + z) + 1], p, e4m3x2_to_f16x2(__byte_perm(r0, 0, 0x4431)), e4m3x2_to_f16x2(__byte_perm(r1, 0, 0x4431)));
                        }
                    }
                }
            }
            cp_wait<0>();
            __syncwarp();
        }

        // this warp's result where its ring was
        float* const mine = reinterpret_cast<float*>(ring);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(kFull, l[h], 1);
            l[h] += __shfl_xor_sync(kFull, l[h], 2);
            const int r = g + 8 * h;
            if (r < rows) {
                if (quad == 0) {
                    s_m[warp][r] = m[h];
                    s_l[warp][r] = l[h];
                }
#pragma unroll
                for (int d = 0; d < kD16; ++d) {
                    if constexpr (!E4M3) {
                        *reinterpret_cast<float2*>(mine + r * T::kPitch + d * 16 + quad * 2) = make_float2(o[2 * d][2 * h], o[2 * d][2 * h + 1]);
                        *reinterpret_cast<float2*>(mine + r * T::kPitch + d * 16 + 8 + quad * 2) =
                            make_float2(o[2 * d + 1][2 * h], o[2 * d + 1][2 * h + 1]);
                    } else {
                        *reinterpret_cast<float4*>(mine + r * T::kPitch + d * 16 + quad * 4) =
                            make_float4(o[2 * d][2 * h], o[2 * d + 1][2 * h], o[2 * d][2 * h + 1], o[2 * d + 1][2 * h + 1]);
                    }
                }
            }
        }
        __syncthreads();
        const bool begins = local == 0, ends = local + seg == s.tiles;
        const int64_t slot = 2 * int64_t(blockIdx.x) + (begins ? 1 : 0);
        for (int i = threadIdx.x; i < rows * (D / 4); i += kNt) {
            const int r = i / (D / 4), d = i % (D / 4) * 4;
            float most = s_m[0][r];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) most = fmaxf(most, s_m[w][r]);
            const float base = most == -INFINITY ? 0.0f : most;
            float sum = 0.0f;
            float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2_approx(s_m[w][r] - base);
                const float4 z = *reinterpret_cast<const float4*>(smem + w * T::kRing + (r * T::kPitch + d) * 4);
                sum += f * s_l[w][r];
                y.x += f * z.x;
                y.y += f * z.y;
                y.z += f * z.z;
                y.w += f * z.w;
            }
            if (begins && ends) {
                const int64_t row = int64_t(b) * a.q_heads + h0 + r;
                const float f = sum == 0.0f ? 0.0f : a.cache.v_scale / sum;
                *reinterpret_cast<uint2*>(a.out + row * D + d) = make_uint2(pack_bf16x2(y.x * f, y.y * f), pack_bf16x2(y.z * f, y.w * f));
                if (a.lse != nullptr && d == 0) a.lse[row] = (most + log2f(sum) - (E4M3 ? 15.0f : 0.0f)) * kLn2;
            } else {
                *reinterpret_cast<float4*>(ws.o + (slot * unit_rows(group) + r) * D + d) = y;
                if (d == 0) {
                    ws.m[slot * kRows + r] = most;
                    ws.l[slot * kRows + r] = sum;
                }
            }
        }
        if (begins && !ends) note = {b, unit, int((pos + s.tiles - 1) / place.run), 0};
        __syncthreads();   // the rings may be filled again

        pos += seg;
        local = 0;
        if (++unit == units && pos < end) {
            unit = 0;
            do s = span_of(a, ++b);
            while (s.tiles == 0);
        }
    }
    if (threadIdx.x == 0) ws.notes[blockIdx.x] = note;
}

// ---------------------------------------------------------------------------
// Join of the units that several runs share: block x looks at the note of run
// x, block y takes every gridDim.y-th row.
// ---------------------------------------------------------------------------

template <int D, bool E4M3>
__global__ void __launch_bounds__(kNt) join_kernel(const AttentionArgs a, int groups, int blocks) {
    constexpr int kCols = D / 4, kParts = kNt / kCols;   // float4 columns; parts added side by side
    __shared__ float s_f[kMaxBlocks];
    __shared__ float s_red[2][kWarps];
    __shared__ float4 s_o[kParts][kCols];
    pdl_wait_and_release();
    const int heads = a.cache.heads, group = a.q_heads / heads, run = blockIdx.x;
    const Partials ws = partials(a.workspace, blocks, unit_rows(group), D);
    const Note note = ws.notes[run];
    if (note.b < 0) return;
    const int head = note.unit / groups, chunk = note.unit % groups;
    const int rows = min(kRows, group - chunk * kRows), h0 = head * group + chunk * kRows;
    const int parts = note.last - run + 1, warp = threadIdx.x / kWarp;
    const auto slot_of = [&](int i) { return i == 0 ? 2 * int64_t(run) + 1 : 2 * int64_t(run + i); };
    for (int r = blockIdx.y; r < rows; r += gridDim.y) {
        float most = -INFINITY;
        for (int i = threadIdx.x; i < parts; i += kNt) most = fmaxf(most, ws.m[slot_of(i) * kRows + r]);
#pragma unroll
        for (int o = kWarp / 2; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(kFull, most, o));
        if (threadIdx.x % kWarp == 0) s_red[0][warp] = most;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) most = fmaxf(most, s_red[0][w]);
        const float base = most == -INFINITY ? 0.0f : most;
        float sum = 0.0f;
        for (int i = threadIdx.x; i < parts; i += kNt) {
            const float f = ex2_approx(ws.m[slot_of(i) * kRows + r] - base);
            s_f[i] = f;
            sum += f * ws.l[slot_of(i) * kRows + r];
        }
#pragma unroll
        for (int o = kWarp / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
        if (threadIdx.x % kWarp == 0) s_red[1][warp] = sum;
        __syncthreads();
        sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += s_red[1][w];
        const int d = threadIdx.x % kCols, p0 = threadIdx.x / kCols;
        float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
        for (int i = p0; i < parts; i += kParts) {
            const float f = s_f[i];
            const float4 z = *reinterpret_cast<const float4*>(ws.o + (slot_of(i) * unit_rows(group) + r) * D + d * 4);
            y.x += f * z.x;
            y.y += f * z.y;
            y.z += f * z.z;
            y.w += f * z.w;
        }
        s_o[p0][d] = y;
        __syncthreads();
        if (p0 == 0) {
            for (int i = 1; i < kParts; ++i) {
                y.x += s_o[i][d].x;
                y.y += s_o[i][d].y;
                y.z += s_o[i][d].z;
                y.w += s_o[i][d].w;
            }
            const int64_t row = int64_t(note.b) * a.q_heads + h0 + r;
            const float f = sum == 0.0f ? 0.0f : a.cache.v_scale / sum;
            *reinterpret_cast<uint2*>(a.out + row * D + d * 4) = make_uint2(pack_bf16x2(y.x * f, y.y * f), pack_bf16x2(y.z * f, y.w * f));
            if (a.lse != nullptr && d == 0) a.lse[row] = (most + log2f(sum) - (E4M3 ? 15.0f : 0.0f)) * kLn2;
        }
        __syncthreads();   // s_f, s_red and s_o are used again
    }
}

template <int D, bool E4M3>
cudaError_t launch_d(const AttentionArgs& a, int num_sms, cudaStream_t stream) {
    static SmemGrant grant;
    auto kernel = attention_kernel<D, E4M3>;
    constexpr int smem = Tile<D, E4M3>::kSmem;
    cudaError_t err = grant.ensure(kernel);
    if (err != cudaSuccess) return err;
    static const int occ = [&] {
        int n = 0;
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kNt, smem) == cudaSuccess && n > 0 ? n : 1;
    }();
    const int group = a.q_heads / a.cache.heads, groups = (group + kRows - 1) / kRows;
    // no more blocks than the most tiles that these tables can hold need
    const int64_t most = (((int64_t(a.max_pages) << a.cache.page_shift) + kTile - 1) / kTile + 1) * a.cache.heads * groups * a.B;
    const int blocks = int(std::max<int64_t>(1, std::min<int64_t>({int64_t(num_sms) * occ, kMaxBlocks, (most + kMinTiles - 1) / kMinTiles})));
    err = launch_pdl(kernel, dim3(blocks), dim3(kNt), smem, stream, a, groups);
    if (err != cudaSuccess) return err;
    // few units: each is split many times, so its rows are joined by a block each
    const int64_t all = int64_t(a.B) * a.cache.heads * groups;
    const int y = all * 4 <= blocks ? unit_rows(group) : 1;
    return launch_pdl(join_kernel<D, E4M3>, dim3(blocks, y), dim3(kNt), 0, stream, a, groups, blocks);
}

}  // namespace

size_t paged_attention_workspace(int64_t, int q_heads, int heads, int head_dim) {
    const size_t rows = size_t(unit_rows(q_heads / heads));
    return size_t(2 * kMaxBlocks) * (rows * head_dim + 2 * kRows) * sizeof(float) + kMaxBlocks * sizeof(Note);
}

cudaError_t launch_paged_attention(const AttentionArgs& a, int num_sms, cudaStream_t stream) {
    switch (a.cache.head_dim) {
        case 64: return a.cache.e4m3 ? launch_d<64, true>(a, num_sms, stream) : launch_d<64, false>(a, num_sms, stream);
        case 128: return a.cache.e4m3 ? launch_d<128, true>(a, num_sms, stream) : launch_d<128, false>(a, num_sms, stream);
        case 256: return a.cache.e4m3 ? launch_d<256, true>(a, num_sms, stream) : launch_d<256, false>(a, num_sms, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace moe
