// Attention of one new token per sequence over a paged key-value cache.
//
// The G = num_q_heads / num_heads query heads that share a key head make up to
// 16 rows of an m16n8k16 product (more than 16: several groups), so a cached
// element is read once for all of them and costs 4 G operations for 4 bytes (8
// bits: 2): at G = 16 that is 16 (32) operations a byte, where this GPU has 280.
// Reading the cache bounds it, and mma.sync keeps up with HBM at a quarter of its
// rate (a third with 8 bits); a 128-row tcgen05 tile would be empty to seven
// eighths or more.
//
// Split. A unit of work is (sequence, up to 4 key heads, or groups of 16 query
// heads of one, side by side). All units' tiles, one after another, are cut into equal runs, one per
// resident block, whatever the lengths are (they are on the GPU, so every block adds them up for itself;
// to enter a unit counts as two tiles, so a run of many short units reads less). A unit inside one run is finished there; what a run has of a unit that goes on
// in another run goes to the workspace (at most two per run), and a second
// kernel joins those in order of the runs. Units that are few and short go to a
// cluster of blocks each instead, which joins them in its shared memory.
//
// A block's 4 warps read up to 4 key heads of the same tokens, or steps (16 or
// 32 tokens) in turn of fewer heads, and never meet inside a unit: each has its
// own ring of kStages steps in shared memory, filled by 16-byte cp.async, and
// its own running maximum, sum and output (online softmax); warps of the same
// head are joined when the run leaves the unit. The ring goes on over the units:
// the next ones' first steps are on their way while one is finished, in the
// stage that was read last.
//
// The output is held transposed, 16 columns as a product's rows and 8 heads as
// its columns: the weights leave the scores' product in just the layout that the
// next one takes them in, up to 8 heads need half the products, and the values
// come through ldmatrix.trans.
//
// Measured on GB300 (6.77 TB/s copy): 1.07 GB of keys and values at 6.6 TB/s (two
// sequences of 131072 tokens), 6.4 (256 of up to 4096), 6.3 (8 bits); 269 MB at
// 5.3. DRAM is 74% busy in 270 MB, the warps issue 25% of the time (48% with 8
// bits, whose conversions take the ALU pipe to 45%). Runs cost about 11 us beside
// the reading: 4 to the first step's arrival, 2 as SMs differ in speed, 1 to leave
// the last unit, 4 for the second kernel.
#include "few_device.cuh"
#include "moe_launch.h"

#include <algorithm>
#include <cmath>

namespace moe {
namespace {

constexpr int kWarps = 4;
constexpr int kNt = kWarps * kWarp;
constexpr int kRows = 16;            // query heads of a unit, at most
constexpr int kMaxBlocks = 640;      // runs the workspace holds the ends of
constexpr int kMinTiles = 3;         // tiles of a run, at least
// Tiles that entering and leaving a unit counts in a run: about 2 us, in which a warp's ring runs dry
// (GB300, the decode batch of 16 sequences of 1 to 8192 tokens: 53.9 us at 0, 52.4 at 1, 52.2 at 2).
constexpr int kUnitCost = 2;
static_assert(kMinTiles > kUnitCost, "a run goes on");
constexpr double kLog2e = 1.44269504088896340736;
constexpr float kLn2 = 0.69314718055994530942f;

// ---------------------------------------------------------------------------
// Workspace: for every run two partial results (a unit that began in an earlier
// run, a unit that goes on in a later one), then a note per run of the unit that
// begins in it and is split.
// ---------------------------------------------------------------------------

struct Note {
    int32_t b, unit, last, run;   // b < 0: none; the unit's last and first run
};

struct Partials {
    float* o;      // [2 blocks][heads at once][rows][D], weighted by 2^(x - m)
    float* m;      // [2 blocks][heads at once][kRows], log2 units
    float* l;      // the same
    Note* notes;   // [blocks]
};

// Key heads (or groups of 16 query heads of one) that a block's warps read side
// by side: a token's heads lie beside each other in most caches, so its bytes
// are asked for together, groups of a head find theirs in L2, and such warps have
// nothing to join. all: key heads times groups.
inline int heads_at_once(int all) { return all % 4 == 0 ? 4 : all % 2 == 0 ? 2 : 1; }

__host__ __device__ inline int unit_rows(int group) { return group < kRows ? group : kRows; }

__host__ __device__ inline Partials partials(void* ws, int results, int rows, int D) {   // results: blocks times heads at once
    Partials p;
    p.o = static_cast<float*>(ws);
    p.m = p.o + int64_t(2) * results * rows * D;
    p.l = p.m + int64_t(2) * results * kRows;
    p.notes = reinterpret_cast<Note*>(p.l + int64_t(2) * results * kRows);
    return p;
}

// ---------------------------------------------------------------------------
// PTX
// ---------------------------------------------------------------------------

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

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

// |x|, or 0 for an infinity or NaN.
__device__ __forceinline__ float finite_size(float x) {
    const float a = fabsf(x);
    return a < INFINITY ? a : 0.0f;
}

// The means of four columns' values into the output. The values' scale comes after the division by the
// weights' sum: the sum is up to 2^45, and a scale near 2^-126 divided by it would be 0.
__device__ __forceinline__ uint2 pack_out(const float4& y, float v_scale) {
    return make_uint2(pack_bf16x2(y.x * v_scale, y.y * v_scale), pack_bf16x2(y.z * v_scale, y.w * v_scale));
}

// ---------------------------------------------------------------------------
// The tokens of a sequence, and where a run begins
// ---------------------------------------------------------------------------

// A tile is 2^ts tokens; they are counted from the one that holds `first`.
struct Span {
    int first, len, tiles;   // tokens first .. len - 1
};

__device__ __forceinline__ Span span_of(const AttentionArgs& a, int b, int ts) {
    Span s;
    const int64_t most = int64_t(a.max_pages) << a.cache.page_shift;
    s.len = int(min(int64_t(max(a.lengths[b], 0)), most));
    s.first = a.window > 0 && s.len > a.window ? s.len - a.window : 0;
    s.tiles = s.len == 0 ? 0 : ((s.len - 1) >> ts) + 1 - (s.first >> ts);
    return s;
}

// A place in a run: it goes on with `left` tiles (and the cost of other units)
// from tile `local` of unit `unit` of sequence b on.
struct Cursor {
    int64_t left;
    int b, unit, local;
    Span s;
    __device__ __forceinline__ int tiles() const { return int(min(int64_t(s.tiles - local), left)); }   // of this unit
    __device__ __forceinline__ void next_unit(const AttentionArgs& a, int units, int ts) {
        left -= tiles();
        local = 0;
        left = max(int64_t(0), left - kUnitCost);
        if (++unit == units && left > 0) {
            unit = 0;
            do s = span_of(a, ++b, ts);
            while (s.tiles == 0);
        }
    }
};

// a / b of non-negative numbers: a 64-bit division takes four times as long.
__device__ __forceinline__ int64_t divide(int64_t a, uint32_t b) {
    return a >> 32 == 0 ? int64_t(uint32_t(a) / b) : a / b;
}

// This block's run. Every block adds up the sequences' tiles for itself. A
// thread's sequences are a run of them, so that the thread in whose range this
// block's run begins can walk to its sequence. A unit counts its tiles and, in
// front of them, kUnitCost. `run`: the length of a run.
__device__ __forceinline__ Cursor find_run(const AttentionArgs& a, int units, int ts, int64_t& run) {
    __shared__ int64_t s_warp[kWarps];
    __shared__ int64_t s_base;
    __shared__ int s_b;
    const int per = (a.B + kNt - 1) / kNt, b0 = min(a.B, int(threadIdx.x) * per), b1 = min(a.B, b0 + per);
    const auto count = [&](int b) {
        const int tiles = span_of(a, b, ts).tiles;
        return tiles > 0 ? tiles + kUnitCost : 0;
    };
    int64_t sum = 0;
#pragma unroll 4
    for (int b = b0; b < b1; ++b) sum += count(b);
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
    run = max(int64_t(kMinTiles), divide(total + gridDim.x - 1, gridDim.x));
    const int64_t start = run * blockIdx.x;
    if (before <= start && start < before + sum) {
        int b = b0;
        int64_t n = int64_t(count(b)) * units;
        while (before + n <= start) {
            before += n;
            n = int64_t(count(++b)) * units;
        }
        s_base = before;
        s_b = b;
    }
    __syncthreads();
    Cursor c = {};
    c.left = max(int64_t(0), min(run, total - start));
    if (c.left > 0) {
        c.b = s_b;
        c.s = span_of(a, c.b, ts);
        const int n = c.s.tiles + kUnitCost;
        c.unit = int(divide(start - s_base, n));
        const int at = int(start - s_base - int64_t(c.unit) * n);
        c.local = max(0, at - kUnitCost);
        c.left = max(int64_t(0), c.left - max(0, kUnitCost - at));
    }
    return c;
}

// ---------------------------------------------------------------------------
// Main kernel: NH groups of 8 query heads. ranks = 0: this block's run of all
// units; else clusters of `ranks` blocks, a unit each (side is then 1).
// ---------------------------------------------------------------------------

template <int D, bool E4M3, int NH>
struct Tile {
    static constexpr int kStepLog2 = (E4M3 && D < 256) || D == 64 ? 5 : 4;
    static constexpr int kStep = 1 << kStepLog2;              // tokens of a warp's step
    static constexpr int kBytes = D * (E4M3 ? 1 : 2);         // of a token's head
    static constexpr int kVecs = kBytes / 16;
    static constexpr int kPer = kWarp / kVecs;                // rows that a warp copies with one instruction
    static constexpr int kSide = kStep * kBytes;              // keys or values of a step
    static constexpr int kStage = 2 * kSide;
    // Of an SM; the rings fill its shared memory, and the registers allow no more. When these were
    // chosen: 256 ragged sequences of bfloat16 heads of 128 172 us with 2 blocks of 3 stages, 179 with 3
    // of 2; 394 MB of 8-bit heads of 64 77.2 us with 3 blocks of 3 stages, 79.2 with 4, 83.3 with 3 of 2.
    // D = 256 spills in three of its four kernels, 160 to 216 bytes a thread of 255 registers (8 bits with up
    // to 8 heads fit): its output, q and a step's scores and weights are more than a thread may have. 8-bit
    // heads of 128 with 9 to 16 query heads spill 12 bytes.
    static constexpr int kBlocks = D == 256 ? (E4M3 ? 2 : 1) : D == 128 && (!E4M3 || NH == 2) ? 2 : 3;
    static constexpr int kStages = kBlocks < 3 || kStage == 4096 ? 3 : 2;
    static constexpr int kRing = kStages * kStage;            // of a warp
    static constexpr int kSmem = kWarps * kRing;
    static constexpr int kRounds = NH * 8 * D * 4 <= kStage ? 1 : NH;   // a warp's output takes the place of a stage
    static_assert(NH * 8 * D * 4 <= kStage * kRounds, "a stage holds a round's rows");
    // 16-byte vector v of row r lies at v ^ swz(r): 8 rows at the same vector hit 8 different banks of 16 bytes
    static __device__ __forceinline__ int swz(int r) { return kVecs >= 8 ? r & 7 : (r >> 1) & 3; }
    static __device__ __forceinline__ uint32_t at(int r, int v) { return uint32_t(r * kBytes + ((v ^ swz(r)) << 4)); }
    // float d of output row r, in a stage
    static __device__ __forceinline__ int out_at(int r, int d) { return r * D + (d ^ (((r >> 1) & 3) * 8)); }
};

__device__ __forceinline__ int64_t shfl64(int64_t v, int lane) {
    return (int64_t(__shfl_sync(kFull, int(v >> 32), lane)) << 32) | uint32_t(__shfl_sync(kFull, int(v), lane));
}

// A step's keys and values into a stage. page: that of token t0 + lane %
// kStep; mask: the tokens to be read, the others become zeros.
template <typename T>
__device__ __forceinline__ void load_step(uint32_t dst, const CacheView& c, const uint8_t* k, const uint8_t* v, int t0, int page,
                                          uint32_t mask) {
    const int lane = threadIdx.x % kWarp, vec = lane % T::kVecs, row = lane / T::kVecs;
    const int in_page = (1 << c.page_shift) - 1;
    constexpr uint32_t kAll = T::kStep == 32 ? 0xffffffffu : 0xffffu;
    if (mask == kAll && c.page_shift >= 4) {
        // 16 tokens in a row are one page's
#pragma unroll
        for (int r0 = 0; r0 < T::kStep; r0 += 16) {
            const int64_t pg = __shfl_sync(kFull, page, r0);
            const int t = ((t0 + r0) & in_page) + row;
            const uint8_t* kp = k + pg * c.k_page + t * c.k_token + vec * 16;
            const uint8_t* vp = v + pg * c.v_page + t * c.v_token + vec * 16;
#pragma unroll
            for (int i = 0; i < 16; i += T::kPer) {
                cp_async16(dst + T::at(r0 + i + row, vec), kp + i * c.k_token);
                cp_async16(dst + T::kSide + T::at(r0 + i + row, vec), vp + i * c.v_token);
            }
        }
        return;
    }
    // Each lane has its row's offsets (its token's, where there is one) and the rows' lanes ask for them.
    const int64_t pg = page, t = (t0 + lane % T::kStep) & in_page;
    const int64_t ko = pg * c.k_page + t * c.k_token, vo = pg * c.v_page + t * c.v_token;
    k += vec * 16;
    v += vec * 16;
    if (mask == kAll) {
        const bool alike = c.k_page == c.v_page && c.k_token == c.v_token;
#pragma unroll
        for (int i = 0; i < T::kStep; i += T::kPer) {
            const int64_t kr = shfl64(ko, i + row);
            cp_async16(dst + T::at(i + row, vec), k + kr);
            if (alike) cp_async16(dst + T::kSide + T::at(i + row, vec), v + kr);
        }
        if (!alike)
#pragma unroll
            for (int i = 0; i < T::kStep; i += T::kPer) cp_async16(dst + T::kSide + T::at(i + row, vec), v + shfl64(vo, i + row));
        return;
    }
#pragma unroll
    for (int i = 0; i < T::kStep; i += T::kPer) {
        const int r = i + row;
        const bool valid = (mask >> r) & 1u;
        const int64_t kr = shfl64(ko, r), vr = shfl64(vo, r);
        cp_async16(dst + T::at(r, vec), k + (valid ? kr : 0), valid);
        cp_async16(dst + T::kSide + T::at(r, vec), v + (valid ? vr : 0), valid);
    }
}

constexpr int kMaxRanks = 8;   // blocks of a cluster: the portable limit

__device__ __forceinline__ float4 ld_cluster4(const float* p, uint32_t rank) {
    const uint32_t a = uint32_t(__cvta_generic_to_shared(p));
    uint32_t r;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(r) : "memory");
    return v;
}

template <int D, bool E4M3, int NH>
__global__ void __launch_bounds__(kNt, Tile<D, E4M3, NH>::kBlocks)
    attention_kernel(const AttentionArgs a, int groups, int side, int ranks) {
    using T = Tile<D, E4M3, NH>;
    constexpr int kD16 = D / 16, kStep = T::kStep, kTiles8 = kStep / 8, kStages = T::kStages;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows], s_f[kWarps][kRows];
    __shared__ const float* s_out[kWarps];
    __shared__ float s_cm[kRows], s_cl[kRows];   // this block's share of a cluster's unit
    pdl_wait_and_release();
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp, g = lane / 4, quad = lane % 4;
    const int heads = a.cache.heads, group = a.q_heads / heads, units = heads * groups / side;
    const int mine_head = warp % side, phase = warp / side, phases = kWarps / side;
    const int ts = __ffs(kStep * phases) - 1;
    const Partials ws = partials(a.workspace, gridDim.x * side, unit_rows(group), D);
    uint8_t* const ring = smem + warp * T::kRing;
    float* const s_co = reinterpret_cast<float*>(smem + T::kSmem);   // [rows][D], for clusters alone
    const uint32_t ring_at = uint32_t(__cvta_generic_to_shared(ring));

    int64_t run = 0;
    Cursor c = {};
    const int rank = ranks > 0 ? blockIdx.x % ranks : 0;
    if (ranks > 0) {
        // a cluster's unit, its tiles in equal shares
        const int u = blockIdx.x / ranks;
        c.b = u / units;
        c.unit = u % units;
        c.s = span_of(a, c.b, ts);
        const int share = (c.s.tiles + ranks - 1) / ranks;
        c.local = min(rank * share, c.s.tiles);
        c.left = min(share, c.s.tiles - c.local);
        if (threadIdx.x < kRows) {
            s_cm[threadIdx.x] = -INFINITY;
            s_cl[threadIdx.x] = 0.0f;
        }
        __syncthreads();
    } else {
        c = find_run(a, units, ts, run);
    }
    // this warp's steps of a cursor's unit: tokens from + (j phases + phase) kStep on
    const auto open = [&](const Cursor& p, int& from) {
        const int begin = ((p.s.first >> ts) + p.local) << ts;
        from = max(begin, p.s.first & ~(kStep - 1));
        const int to = min(p.s.len, begin + (p.tiles() << ts));
        return ((to - from + kStep - 1) / kStep - phase + phases - 1) >> (ts - T::kStepLog2);
    };

    // The loads run ahead of the products, over the units' ends: `ahead` is
    // where they are, next_t0 and next_page the step to be loaded next.
    Cursor ahead = c;
    int ahead_from = 0, ahead_j = 0, ahead_steps = 0, next_t0 = 0, next_page = -1;
    bool more = c.left > 0;
    const uint8_t *ahead_k = nullptr, *ahead_v = nullptr;   // of the unit's head
    const auto enter = [&]() {
        const int64_t head = (ahead.unit * side + mine_head) / groups;
        ahead_k = a.cache.k + head * a.cache.k_head;
        ahead_v = a.cache.v + head * a.cache.v_head;
        ahead_steps = open(ahead, ahead_from);
    };
    if (more) enter();
    const auto look = [&]() {
        while (more && ahead_j >= ahead_steps) {
            ahead.next_unit(a, units, ts);
            more = ahead.left > 0;
            ahead_j = 0;
            if (more) enter();
        }
        next_page = -1;
        if (more) {
            next_t0 = ahead_from + (ahead_j++ * phases + phase) * kStep;
            const int t = next_t0 + lane % kStep;
            if (t >= ahead.s.first && t < ahead.s.len) {
                const int pg = a.block_table[int64_t(ahead.b) * a.max_pages + (t >> a.cache.page_shift)];
                next_page = pg < a.cache.num_pages ? pg : -1;
            }
        }
    };
    const auto issue = [&](int stage) -> uint32_t {
        uint32_t mask = __ballot_sync(kFull, next_page >= 0);
        if (kStep == 16) mask &= 0xffffu;
        if (more) load_step<T>(ring_at + stage * T::kStage, a.cache, ahead_k, ahead_v, next_t0, next_page, mask);
        cp_commit();
        look();
        return mask;
    };
    uint32_t masks[kStages];   // of the steps in the ring, the oldest first
    look();
#pragma unroll
    for (int i = 0; i + 1 < kStages; ++i) masks[i] = issue(i);
    int stage = 0;             // of the step that comes next

    // sequences without tokens
    for (int b = blockIdx.x; ranks == 0 && b < a.B; b += gridDim.x)
        if (span_of(a, b, ts).tiles == 0) {
            uint4* o = reinterpret_cast<uint4*>(a.out + int64_t(b) * a.q_heads * D);
            for (int i = threadIdx.x; i < a.q_heads * D / 8; i += kNt) o[i] = make_uint4(0, 0, 0, 0);
            if (a.lse != nullptr)
                for (int i = threadIdx.x; i < a.q_heads; i += kNt) a.lse[int64_t(b) * a.q_heads + i] = -INFINITY;
        }

    Note note = {-1, 0, 0, 0};
    // q, as A: row g (and g + 8) is head h0 + g. For E4M3 the order of the 16 columns of a product is
    // that in which the keys' bytes come out of ldmatrix: 4 quad .. 4 quad + 3.
    uint32_t aq[kD16][4];
    const auto load_q = [&](const Cursor& p) {
        const int at = p.unit * side + mine_head, chunk = at % groups, rows = min(kRows, group - chunk * kRows);
        const int h0 = at / groups * group + chunk * kRows;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = g + 8 * h;
            const uint16_t* q = a.q + int64_t(p.b) * a.q_stride + int64_t(h0 + r) * D;
#pragma unroll
            for (int k = 0; k < kD16; ++k) {
                if constexpr (!E4M3) {
                    aq[k][h] = h < NH && r < rows ? *reinterpret_cast<const uint32_t*>(q + k * 16 + quad * 2) : 0u;
                    aq[k][h + 2] = h < NH && r < rows ? *reinterpret_cast<const uint32_t*>(q + k * 16 + quad * 2 + 8) : 0u;
                } else {
                    const uint2 w = h < NH && r < rows ? *reinterpret_cast<const uint2*>(q + k * 16 + quad * 4) : make_uint2(0u, 0u);
                    aq[k][h] = w.x;
                    aq[k][h + 2] = w.y;
                }
            }
        }
    };
    if (c.left > 0) load_q(c);
    while (c.left > 0) {
        const int at = c.unit * side + mine_head, chunk = at % groups;
        const int rows = min(kRows, group - chunk * kRows), h0 = at / groups * group + chunk * kRows;

        float f_row[NH];   // what a row's scores are multiplied by, with log2 e; and then by score_up
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            f_row[h] = a.score;
            if constexpr (E4M3) {
                float most = 0.0f;
#pragma unroll
                for (int k = 0; k < kD16; ++k)
#pragma unroll
                    for (int z = h; z < 4; z += 2) most = fmaxf(most, fmaxf(finite_size(bf16_lo(aq[k][z])), finite_size(bf16_hi(aq[k][z]))));
                most = fmaxf(most, __shfl_xor_sync(kFull, most, 1));
                most = fmaxf(most, __shfl_xor_sync(kFull, most, 2));
                // f16 holds q times 2^(14 - e), e the exponent of the row's largest finite value (14 for a row without one)
                const int e = most > 0.0f ? max(int(__float_as_uint(most) >> 23) - 127, -112) : 14;
                const float up = __uint_as_float(uint32_t(127 + 14 - e) << 23);
                f_row[h] *= __uint_as_float(uint32_t(127 - 14 + e) << 23);
#pragma unroll
                for (int k = 0; k < kD16; ++k)
#pragma unroll
                    for (int z = h; z < 4; z += 2) aq[k][z] = pack_f16x2(bf16_lo(aq[k][z]) * up, bf16_hi(aq[k][z]) * up);
            }
        }

        // out^T: [16 columns][8 heads][row g: heads 2 quad, 2 quad + 1; row g + 8: the same]
        float o[kD16][NH][4];
        float m[NH], l[NH];
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            m[h] = -INFINITY;
            l[h] = 0.0f;
#pragma unroll
            for (int d = 0; d < kD16; ++d)
#pragma unroll
                for (int z = 0; z < 4; ++z) o[d][h][z] = 0.0f;
        }
        int from = 0;
        const int steps = open(c, from);
        for (int j = 0; j < steps; ++j) {
            cp_wait<kStages - 2>();
            __syncwarp();
            masks[kStages - 1] = issue(stage == 0 ? kStages - 1 : stage - 1);
            const uint32_t ks = ring_at + stage * T::kStage, vs = ks + T::kSide;
            const uint32_t mask = masks[0];
#pragma unroll
            for (int i = 0; i + 1 < kStages; ++i) masks[i] = masks[i + 1];
            stage = stage + 1 == kStages ? 0 : stage + 1;

            float x[kTiles8][4] = {};   // [8 tokens][row g: tokens 2 quad, 2 quad + 1; row g + 8: the same]
#pragma unroll
            for (int t = 0; t < kStep; t += 16) {
                if constexpr (!E4M3) {
                    const int row = t + lane % 8 + (lane & 16) / 2, v = (lane >> 3) & 1;
#pragma unroll
                    for (int k = 0; k < kD16; ++k) {
                        uint32_t r[4];
                        ldsm(r, ks + T::at(row, 2 * k + v));
                        mma<false>(x[t / 8], aq[k], r[0], r[1]);
                        mma<false>(x[t / 8 + 1], aq[k], r[2], r[3]);
                    }
                } else {
                    const int row = t + lane % 16, v = lane >> 4;
#pragma unroll
                    for (int k = 0; k < kD16; k += 2) {
                        uint32_t r[4];
                        ldsm(r, ks + T::at(row, k + v));
#pragma unroll
                        for (int z = 0; z < 4; ++z)
                            mma<true>(x[t / 8 + (z & 1)], aq[k + z / 2], e4m3x2_to_f16x2(r[z]), e4m3x2_to_f16x2(r[z] >> 16));
                    }
                }
            }
            constexpr uint32_t kAll = kStep == 32 ? 0xffffffffu : 0xffffu;
            float top[NH];
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                top[h] = -INFINITY;
#pragma unroll
                for (int n = 0; n < kTiles8; ++n)
#pragma unroll
                    for (int z = 0; z < 2; ++z) x[n][2 * h + z] = x[n][2 * h + z] * f_row[h] * a.score_up;
            }
            if (mask != kAll) {
                const uint32_t seen = mask >> (quad * 2);
#pragma unroll
                for (int n = 0; n < kTiles8; ++n)
#pragma unroll
                    for (int z = 0; z < 2 * NH; ++z)
                        if (!((seen >> (n * 8 + (z & 1))) & 1u)) x[n][z] = -INFINITY;
            }
            bool higher = false;
#pragma unroll
            for (int h = 0; h < NH; ++h) {
#pragma unroll
                for (int n = 0; n < kTiles8; ++n) top[h] = fmaxf(top[h], fmaxf(x[n][2 * h], x[n][2 * h + 1]));
                top[h] = fmaxf(top[h], __shfl_xor_sync(kFull, top[h], 1));
                top[h] = fmaxf(top[h], __shfl_xor_sync(kFull, top[h], 2));
                higher |= top[h] > m[h];
            }
            if (__any_sync(kFull, higher)) {
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    const float now = fmaxf(m[h], top[h]);
                    const float f = now == -INFINITY ? 1.0f : ex2_approx(m[h] - now);
                    m[h] = now;
                    l[h] *= f;
                    const float f0 = __shfl_sync(kFull, f, quad * 8), f1 = __shfl_sync(kFull, f, quad * 8 + 4);
#pragma unroll
                    for (int d = 0; d < kD16; ++d) {
                        o[d][h][0] *= f0;
                        o[d][h][1] *= f1;
                        o[d][h][2] *= f0;
                        o[d][h][3] *= f1;
                    }
                }
            }
            // Weights 2^(x - m), in two terms each: the upper bits of the float and what they leave (the
            // upper alone would cost a bfloat16 result as much as its own rounding, and one of few bits
            // where the values cancel). As f16 (E4M3), 22 bits, they are times 2^15, so that those down to
            // 2^-39 of the largest count. (One f16 term, 11 bits: 175.5 us for 176.2 in 1.08 GB of 8-bit heads
            // of 128 with 8 query heads each, 100.7 for 110.6 in 537 MB with 16.) As bfloat16, 16 bits, the
            // second term is never 0 but at least 2^-20 of the weight, so that an infinite value does not
            // become NaN by it. (A third brought no result nearer to 64 bits: the sums are as coarse.)
            uint32_t p[NH][kTiles8], lo[NH][kTiles8];
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const float base = (m[h] == -INFINITY ? 0.0f : m[h]) - (E4M3 ? 15.0f : 0.0f);
#pragma unroll
                for (int n = 0; n < kTiles8; ++n) {
                    const float p0 = ex2_approx(x[n][2 * h] - base), p1 = ex2_approx(x[n][2 * h + 1] - base);
                    l[h] += p0 + p1;
                    if constexpr (E4M3) {
                        const float u0 = __uint_as_float(__float_as_uint(p0) & 0xffffe000u), u1 = __uint_as_float(__float_as_uint(p1) & 0xffffe000u);
                        p[h][n] = pack_f16x2(u0, u1);
                        lo[h][n] = pack_f16x2(p0 - u0, p1 - u1);
                    } else {
                        p[h][n] = __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632);
                        lo[h][n] = pack_bf16x2(fmaxf(p0 - bf16_lo(p[h][n]), p0 * 0x1p-20f), fmaxf(p1 - bf16_hi(p[h][n]), p1 * 0x1p-20f));
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < kStep; t += 16) {
                if constexpr (!E4M3) {
                    const int row = t + lane % 8 + (lane & 16) / 2, v = (lane >> 3) & 1;
#pragma unroll
                    for (int d = 0; d < kD16; ++d) {
                        uint32_t r[4];
                        ldsm_t(r, vs + T::at(row, 2 * d + v));
#pragma unroll
                        for (int h = 0; h < NH; ++h) {
                            mma<false>(o[d][h], r, p[h][t / 8], p[h][t / 8 + 1]);
                            mma<false>(o[d][h], r, lo[h][t / 8], lo[h][t / 8 + 1]);
                        }
                    }
                } else {
                    // A transposed 16-bit unit is two columns' bytes: row g is column 2 g, row g + 8 column 2 g + 1.
                    const int row = t + lane % 16, v = lane >> 4;
#pragma unroll
                    for (int d = 0; d < kD16; d += 2) {
                        uint32_t r[4];
                        ldsm_t(r, vs + T::at(row, d + v));
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            const uint32_t w0 = r[2 * z], w1 = r[2 * z + 1];
                            const uint32_t f[4] = {e4m3x2_to_f16x2(__byte_perm(w0, 0, 0x4420)), e4m3x2_to_f16x2(__byte_perm(w0, 0, 0x4431)),
                                                   e4m3x2_to_f16x2(__byte_perm(w1, 0, 0x4420)), e4m3x2_to_f16x2(__byte_perm(w1, 0, 0x4431))};
#pragma unroll
                            for (int h = 0; h < NH; ++h) {
                                mma<true>(o[d + z][h], f, p[h][t / 8], p[h][t / 8 + 1]);
                                mma<true>(o[d + z][h], f, lo[h][t / 8], lo[h][t / 8 + 1]);
                            }
                        }
                    }
                }
            }
        }

        // the next unit's q, on its way while this one is finished
        Cursor next = c;
        next.next_unit(a, units, ts);
        if (next.left > 0) load_q(next);

        // this warp's result into the stage that no load is on its way to
        __syncwarp();
        float* const mine = reinterpret_cast<float*>(ring + (stage == 0 ? kStages - 1 : stage - 1) * T::kStage);
        if (lane == 0) s_out[warp] = mine;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            l[h] += __shfl_xor_sync(kFull, l[h], 1);
            l[h] += __shfl_xor_sync(kFull, l[h], 2);
            if (quad == 0 && phases > 1) {
                s_m[warp][g + 8 * h] = m[h];
                s_l[warp][g + 8 * h] = l[h];
            }
        }
        const int seg = c.tiles();
        const bool begins = c.local == 0, ends = c.local + seg == c.s.tiles, whole = begins && ends && ranks == 0;
        const int64_t slot = (2 * int64_t(blockIdx.x) + (begins ? 1 : 0)) * side + mine_head;
        // a row's largest score and sum, where they are the whole unit's: log-sum-exp; else into the workspace
        const auto store_sum = [&](int r, float most, float sum) {
            if (!whole) {
                ws.m[slot * kRows + r] = most;
                ws.l[slot * kRows + r] = sum;
            } else if (a.lse != nullptr) {
                a.lse[int64_t(c.b) * a.q_heads + h0 + r] = (most + log2f(sum) - (E4M3 ? 15.0f : 0.0f)) * kLn2;
            }
        };
        const auto store_row = [&](int r, int d, const float4& y) {
            if (ranks > 0)
                *reinterpret_cast<float4*>(s_co + r * D + d) = y;
            else if (whole)
                *reinterpret_cast<uint2*>(a.out + (int64_t(c.b) * a.q_heads + h0 + r) * D + d) = pack_out(y, a.cache.v_scale);
            else
                *reinterpret_cast<float4*>(ws.o + (slot * unit_rows(group) + r) * D + d) = y;
        };
        constexpr int kHalf = NH / T::kRounds;   // groups of 8 rows of a round
#pragma unroll
        for (int h0r = 0; h0r < NH; h0r += kHalf) {
#pragma unroll
            for (int h = 0; h < kHalf; ++h)
#pragma unroll
                for (int d = 0; d < kD16; ++d)
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const int col = E4M3 ? d * 16 + 2 * g + (z >> 1) : d * 16 + g + 8 * (z >> 1);
                        mine[T::out_at(8 * h + 2 * quad + (z & 1), col)] = o[d][h0r + h][z];
                    }
            const int here = min(rows - 8 * h0r, 8 * kHalf), pieces = here * (D / 4);
            if (phases == 1) {   // a warp has the head to itself
                float f[kHalf];
#pragma unroll
                for (int h = 0; h < kHalf; ++h) {
                    const float sum = l[h0r + h];
                    f[h] = !whole ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
                    if (quad == 0 && g + 8 * (h0r + h) < rows) store_sum(g + 8 * (h0r + h), m[h0r + h], sum);
                }
                __syncwarp();
                for (int i = lane; i - lane < pieces; i += kWarp) {
                    const int r = i / (D / 4), d = i % (D / 4) * 4;
                    float factor = __shfl_sync(kFull, f[0], r % 8 * 4);
                    if (kHalf == 2) {
                        const float other = __shfl_sync(kFull, f[kHalf - 1], r % 8 * 4);
                        factor = r < 8 ? factor : other;
                    }
                    if (i >= pieces) continue;
                    float4 y = *reinterpret_cast<const float4*>(mine + T::out_at(r, d));
                    y.x *= factor;
                    y.y *= factor;
                    y.z *= factor;
                    y.w *= factor;
                    store_row(8 * h0r + r, d, y);
                }
                __syncwarp();   // the next round, or the next loads, take the place of these rows
                continue;
            }
            group_sync(mine_head, phases);
            if (h0r == 0) {
                // what a warp's row counts in the sum of the head's warps, and for a whole unit in the output
                for (int r = phase * kWarp + lane; r < rows; r += phases * kWarp) {
                    float most = -INFINITY, sum = 0.0f;
                    for (int w = mine_head; w < kWarps; w += side) most = fmaxf(most, s_m[w][r]);
                    const float base = most == -INFINITY ? 0.0f : most;
                    for (int w = mine_head; w < kWarps; w += side) sum += ex2_approx(s_m[w][r] - base) * s_l[w][r];
                    const float inv = !whole ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
                    for (int w = mine_head; w < kWarps; w += side) s_f[w][r] = ex2_approx(s_m[w][r] - base) * inv;
                    if (ranks > 0) {
                        s_cm[r] = most;
                        s_cl[r] = sum;
                    } else {
                        store_sum(r, most, sum);
                    }
                }
                group_sync(mine_head, phases);
            }
#pragma unroll 2
            for (int i = phase * kWarp + lane; i < pieces; i += phases * kWarp) {
                const int r = 8 * h0r + i / (D / 4), d = i % (D / 4) * 4;
                float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (int w = mine_head; w < kWarps; w += side) {
                    const float f = s_f[w][r];
                    const float4 z = *reinterpret_cast<const float4*>(s_out[w] + T::out_at(i / (D / 4), d));
                    y.x += f * z.x;
                    y.y += f * z.y;
                    y.z += f * z.z;
                    y.w += f * z.w;
                }
                store_row(r, d, y);
            }
            if (h0r + kHalf < NH) group_sync(mine_head, phases);   // the next round's rows take the place of these
        }
        if (ranks == 0 && begins && !ends) {   // what is left of the unit fills the next runs
            const int rest = c.s.tiles - seg, more_runs = rest <= run ? 1 : (rest + int(run) - 1) / int(run);
            note = {c.b, c.unit, int(blockIdx.x) + more_runs, int(blockIdx.x)};
        }
        if (phases > 1) group_sync(mine_head, phases);   // the stages may be filled again
        c = next;
    }
    if (ranks == 0) {
        if (threadIdx.x == 0) ws.notes[blockIdx.x] = note;
        return;
    }

    // The blocks of a cluster join their shares: each takes some of the rows' columns.
    cluster_sync();
    const int u = blockIdx.x / ranks, unit = u % units, head = unit / groups, chunk = unit % groups;
    const int rows = min(kRows, group - chunk * kRows);
    for (int i = rank * kNt + threadIdx.x; i < rows * (D / 4); i += ranks * kNt) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        float m1[kMaxRanks], l1[kMaxRanks];
        float4 z[kMaxRanks];
#pragma unroll
        for (int k = 0; k < kMaxRanks; ++k) {
            m1[k] = -INFINITY;
            l1[k] = 0.0f;
            if (k < ranks) {
                m1[k] = ld_cluster(s_cm + r, k);
                l1[k] = ld_cluster(s_cl + r, k);
                z[k] = ld_cluster4(s_co + r * D + d, k);
            }
        }
        float most = m1[0], sum = 0.0f;
#pragma unroll
        for (int k = 1; k < kMaxRanks; ++k) most = fmaxf(most, m1[k]);
        const float base = most == -INFINITY ? 0.0f : most;
        float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < kMaxRanks; ++k)
            if (l1[k] != 0.0f) {   // a block without tokens left no output
                const float f = ex2_approx(m1[k] - base);
                sum += f * l1[k];
                y.x += f * z[k].x;
                y.y += f * z[k].y;
                y.z += f * z[k].z;
                y.w += f * z[k].w;
            }
        const int64_t row = int64_t(u / units) * a.q_heads + head * group + chunk * kRows + r;
        const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
        *reinterpret_cast<uint2*>(a.out + row * D + d) = pack_out(make_float4(y.x * f, y.y * f, y.z * f, y.w * f), a.cache.v_scale);
        if (a.lse != nullptr && d == 0) a.lse[row] = (most + log2f(sum) - (E4M3 ? 15.0f : 0.0f)) * kLn2;
    }
    cluster_sync();   // the others may still read this block's share
}

// ---------------------------------------------------------------------------
// Join of the units that several runs share: a warp, or `warps` of them, per
// row (unit, head). Every block gathers the notes for itself.
// ---------------------------------------------------------------------------

constexpr int kJoinWarps = 8;
constexpr int kJoinBatch = 8;        // partial results that a warp asks for at once

template <int D, bool E4M3>
__global__ void __launch_bounds__(kJoinWarps* kWarp) join_kernel(const AttentionArgs a, int groups, int side, int blocks, int warps) {
    constexpr int kLanes = D == 64 ? 16 : 32, kVecs = D / (4 * kLanes), kSub = kWarp / kLanes;   // lanes of a row; rows side by side
    __shared__ Note s_note[kMaxBlocks];
    __shared__ int s_count[kJoinWarps];
    __shared__ float s_m[kJoinWarps], s_l[kJoinWarps];
    __shared__ float4 s_o[kJoinWarps][D / 4];
    pdl_wait_and_release();
    const int heads = a.cache.heads, group = a.q_heads / heads, urows = unit_rows(group), rows_all = side * urows;
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    const Partials ws = partials(a.workspace, blocks * side, urows, D);
    int units = 0;
    for (int r0 = 0; r0 < blocks; r0 += kJoinWarps * kWarp) {
        const int run = r0 + threadIdx.x;
        const Note n = run < blocks ? ws.notes[run] : Note{-1, 0, 0, 0};
        const uint32_t there = __ballot_sync(kFull, n.b >= 0);
        if (lane == 0) s_count[warp] = __popc(there);
        __syncthreads();
        int at = units + __popc(there & ((1u << lane) - 1u));
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
            if (w < warp) at += s_count[w];
            units += s_count[w];
        }
        if (n.b >= 0) s_note[at] = n;
        __syncthreads();
    }
    const int item = (int(blockIdx.x) * kJoinWarps + warp) / warps, sub = warp % warps;
    const int r = item % urows, side_head = item % rows_all / urows;
    const bool in = item < units * rows_all;
    const Note n = in ? s_note[item / rows_all] : Note{};
    const int chunk = (n.unit * side + side_head) % groups, head = (n.unit * side + side_head) / groups;
    const bool valid = in && r < group - chunk * kRows;   // the last group of 16 may be smaller
    const int parts = valid ? n.last - n.run + 1 : 0;
    float m = -INFINITY, l = 0.0f;
    float4 y[kVecs] = {};
    const auto add = [&](float m1, float l1, const float4 (&z)[kVecs]) {
        const float now = fmaxf(m, m1), base = now == -INFINITY ? 0.0f : now;
        const float f = ex2_approx(m - base), f1 = ex2_approx(m1 - base);
        m = now;
        l = l * f + l1 * f1;
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            y[v].x = y[v].x * f + z[v].x * f1;
            y[v].y = y[v].y * f + z[v].y * f1;
            y[v].z = y[v].z * f + z[v].z * f1;
            y[v].w = y[v].w * f + z[v].w * f1;
        }
    };
    const int step = warps * kSub;
    for (int p0 = sub * kSub + lane / kLanes; p0 - lane / kLanes < parts; p0 += step * kJoinBatch) {
        float m1[kJoinBatch], l1[kJoinBatch];
        float4 z[kJoinBatch][kVecs];
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) {
            const int p = p0 + i * step;
            m1[i] = -INFINITY;
            l1[i] = 0.0f;
#pragma unroll
            for (int v = 0; v < kVecs; ++v) z[i][v] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (p < parts) {
                const int64_t slot = (2 * int64_t(n.run + p) + (p == 0 ? 1 : 0)) * side + side_head;
                m1[i] = ws.m[slot * kRows + r];
                l1[i] = ws.l[slot * kRows + r];
#pragma unroll
                for (int v = 0; v < kVecs; ++v)
                    z[i][v] = reinterpret_cast<const float4*>(ws.o + (slot * urows + r) * D)[lane % kLanes + v * kLanes];
            }
        }
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) add(m1[i], l1[i], z[i]);
    }
    if constexpr (kSub == 2) {
        float4 z[kVecs];
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
            z[v] = make_float4(__shfl_xor_sync(kFull, y[v].x, 16), __shfl_xor_sync(kFull, y[v].y, 16),
                               __shfl_xor_sync(kFull, y[v].z, 16), __shfl_xor_sync(kFull, y[v].w, 16));
        add(__shfl_xor_sync(kFull, m, 16), __shfl_xor_sync(kFull, l, 16), z);
    }
    if (warps > 1) {
        if (lane == 0) {
            s_m[warp] = m;
            s_l[warp] = l;
        }
        if (lane < kLanes)
#pragma unroll
            for (int v = 0; v < kVecs; ++v) s_o[warp][lane + v * kLanes] = y[v];
        __syncthreads();
        if (sub == 0)
            for (int w = 1; w < warps; ++w) {
                float4 z[kVecs];
#pragma unroll
                for (int v = 0; v < kVecs; ++v) z[v] = s_o[warp + w][lane % kLanes + v * kLanes];
                add(s_m[warp + w], s_l[warp + w], z);
            }
    }
    if (!valid || sub != 0) return;
    const int64_t row = int64_t(n.b) * a.q_heads + head * group + chunk * kRows + r;
    const float f = l == 0.0f ? 0.0f : 1.0f / l;
    if (lane < kLanes)
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
            *reinterpret_cast<uint2*>(a.out + row * D + (lane + v * kLanes) * 4) =
                pack_out(make_float4(y[v].x * f, y[v].y * f, y[v].z * f, y[v].w * f), a.cache.v_scale);
    if (a.lse != nullptr && lane == 0) a.lse[row] = (m + log2f(l) - (E4M3 ? 15.0f : 0.0f)) * kLn2;
}

template <int D, bool E4M3, int NH>
cudaError_t launch_d(const AttentionArgs& a, int num_sms, cudaStream_t stream) {
    using T = Tile<D, E4M3, NH>;
    static SmemGrant grant;
    auto kernel = attention_kernel<D, E4M3, NH>;
    cudaError_t err = grant.ensure(kernel);
    if (err != cudaSuccess) return err;
    const auto resident = [&](size_t smem) {
        int n = 0;
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kNt, smem) == cudaSuccess && n > 0 ? n : 1;
    };
    constexpr int kShare = NH * 8 * D * 4;   // a block's share of a cluster's unit
    static const int occ = resident(T::kSmem), cluster_occ = resident(T::kSmem + kShare);
    const int group = a.q_heads / a.cache.heads, groups = (group + kRows - 1) / kRows;
    const int64_t table = int64_t(a.max_pages) << a.cache.page_shift, longest = a.window > 0 ? std::min<int64_t>(table, a.window) : table;

    // Units that are few and cannot be long go to clusters of as many blocks as find room at once (heads
    // of 256 in bfloat16: 15 of 8 blocks, not the 19 that SMs / 8 would give), each unit's tokens in equal
    // shares: one kernel and no join. The runs cost 2 to 3 us more, but share all tokens over all blocks,
    // however many units there are and however unlike. What a cluster's block has beyond its share in that
    // (units taken to be 3/4 of the longest on average) may be as many tokens as are read in those 2.5 us;
    // a block is bound by its warps, so that is a number of tokens of a head size and type, not of bytes.
    // GB300, us, clusters / runs: bfloat16 D = 128, 2 units of 2048 tokens 8.8 / 10.3, of 4096 12.6 / 10.5; 8
    // of 2000 9.4 / 10.5, of 4000 13.0 / 12.4; 64 of 4096 28.6 / 31.9, of 1 to 4096 21.9 / 21.9; D = 64, 8 of
    // 4096 10.1 / 10.4, of 8192 14.8 / 11.5; D = 256, 8 of 2048 12.7 / 14.2, 48 windows of 1023 18.5 / 21.5.
    // 8 bits, D = 64, 64 of 1024 9.6 / 11.3, of 1 to 8192 24.0 / 18.3; D = 128, 8 of 2048 9.5 / 11.6, of 8192
    // 18.1 / 14.5, 64 of 1 to 8192 32.9 / 25.2; D = 256, 16 of 2048 14.5 / 15.6, 64 of 1 to 4096 31.0 / 26.5.
    // In 490 such calls of 2 to 256 units the way taken was 13% slower than the other at most.
    static ClusterSlots cluster_slots;
    uint32_t slots[kMaxRanks + 1];
    err = cluster_slots.get(kernel, kNt, T::kSmem + kShare, num_sms * cluster_occ, slots);
    if (err != cudaSuccess) return err;
    const int64_t clusters = int64_t(a.B) * a.cache.heads * groups, everywhere = int64_t(num_sms) * occ;
    constexpr int64_t kAhead = D == 64 ? 520 : D == 256 ? 310 : E4M3 ? 480 : 400;
    int ranks = kMaxRanks;
    while (ranks > 0 && clusters > slots[ranks]) ranks /= 2;
    if (ranks > 0 && longest * (4 * everywhere - 3 * clusters * ranks) <= 4 * kAhead * everywhere * ranks)
        return launch_cluster(kernel, dim3(unsigned(clusters * ranks)), dim3(kNt), ranks, T::kSmem + kShare, stream, a, groups, 1, ranks);
    const int side = heads_at_once(a.cache.heads * groups);
    // no more blocks than the most tiles that these tables can hold need
    const int tile = kWarps / side * T::kStep;
    const int64_t tiles = (longest + tile - 1) / tile + 1 + kUnitCost;
    const int64_t most = (tiles * (a.cache.heads * groups / side) * a.B + kMinTiles - 1) / kMinTiles;
    const int blocks = int(std::max<int64_t>(1, std::min<int64_t>({int64_t(num_sms) * occ, kMaxBlocks, most})));
    err = launch_pdl(kernel, dim3(blocks), dim3(kNt), T::kSmem, stream, a, groups, side, 0);
    if (err != cudaSuccess) return err;
    // Units that may be split: all of them, or the one at each border of two runs. A row of one
    // gets a warp for every 8 of the runs that share it on average.
    const int64_t all = int64_t(a.B) * (a.cache.heads * groups / side);
    const int split = int(std::min<int64_t>(blocks - 1, all));
    if (split == 0) return cudaSuccess;
    int warps = 1;
    while (warps < kJoinWarps && blocks > split * warps * kJoinBatch) warps *= 2;
    const int64_t join_warps = int64_t(split) * side * unit_rows(group) * warps;
    return launch_pdl(join_kernel<D, E4M3>, dim3(unsigned((join_warps + kJoinWarps - 1) / kJoinWarps)), dim3(kJoinWarps * kWarp), 0,
                      stream, a, groups, side, blocks, warps);
}

// Up to 8 heads of a group make one half of a product's rows.
template <int D>
cudaError_t launch_heads(const AttentionArgs& a, int num_sms, cudaStream_t stream) {
    const bool one = a.q_heads / a.cache.heads <= 8;
    if (a.cache.e4m3) return one ? launch_d<D, true, 1>(a, num_sms, stream) : launch_d<D, true, 2>(a, num_sms, stream);
    return one ? launch_d<D, false, 1>(a, num_sms, stream) : launch_d<D, false, 2>(a, num_sms, stream);
}

}  // namespace

size_t paged_attention_workspace(int64_t, int q_heads, int heads, int head_dim) {
    const int group = q_heads / heads;
    const size_t rows = size_t(unit_rows(group));
    const size_t results = size_t(2 * kMaxBlocks * heads_at_once(heads * ((group + kRows - 1) / kRows)));
    return results * (rows * head_dim + 2 * kRows) * sizeof(float) + kMaxBlocks * sizeof(Note);
}

cudaError_t launch_paged_attention(const AttentionArgs& args, int num_sms, cudaStream_t stream) {
    // scale k_scale log2 e may lie far outside float32 where the scores do not, so a power of two of it
    // is a factor of its own. The other stays within 2^-100 .. 2^14 (but for products below 2^-226): with
    // the 2^-126 .. 2^113 of a row of q (E4M3) it is in range, or so small that its scores are 0.
    AttentionArgs a = args;
    int e = 0;
    const double f = frexp(double(a.scale) * double(a.cache.k_scale) * kLog2e, &e);
    const int up = std::max(-126, std::min(127, e > 14 ? e - 14 : e < -100 ? e + 100 : 0));
    a.score = float(ldexp(f, e - up));
    a.score_up = float(ldexp(1.0, up));
    switch (a.cache.head_dim) {
        case 64: return launch_heads<64>(a, num_sms, stream);
        case 128: return launch_heads<128>(a, num_sms, stream);
        case 256: return launch_heads<256>(a, num_sms, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace moe
