// Block tables and slot maps of a decode step, and the return of finished
// requests' pages: whole-number work on a few kilobytes, so latency is what
// counts. One launch each: a cluster of up to 8 blocks, every one of which
// scans all requests for itself (no block waits for another's sums) and then
// takes its share of the tokens. A token finds its request by bisection in the
// prefix sums, held in shared memory.
//
// lengths may be cached itself and free_count_out free_count itself: the
// cluster meets once between the last read of these and the first write.
//
// GB300: 3.4 us for 16 requests with a token each, 6.5 us for 1023 with 32768
// places: two dependent loads, two scans, a bisection per token and its stores.
// Pages given back: 6.1 us for 1024 requests of up to 128 pages. A request's
// are one warp's, a load in front of each store, so long rows take long: 49 us
// for 8192 pages, 753 us for 131072.
#include "few_device.cuh"
#include "moe_launch.h"

namespace moe {
namespace {

constexpr int kNt = 1024;
constexpr int kWarps = kNt / kWarp;

// Sum over the block's threads before this one, and over all of them. Every
// thread calls; s_sum holds kWarps values and may be used again right away.
__device__ __forceinline__ int64_t block_before(int64_t v, int64_t* s_sum, int64_t& total) {
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp, warps = blockDim.x / kWarp;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < kWarp; o <<= 1) {
        const int64_t y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
    }
    if (lane == kWarp - 1) s_sum[warp] = x;
    __syncthreads();
    int64_t w = lane < warps ? s_sum[lane] : 0;
#pragma unroll
    for (int o = 1; o < kWarp; o <<= 1) {
        const int64_t y = __shfl_up_sync(kFull, w, o);
        if (lane >= o) w += y;
    }
    total = __shfl_sync(kFull, w, kWarp - 1);
    const int64_t before = __shfl_sync(kFull, w, warp == 0 ? 0 : warp - 1);
    __syncthreads();
    return (warp == 0 ? 0 : before) + x - v;
}

// 12 bytes of shared memory per request, and the warps' sums (a block may have 227 KB)
static_assert(12 * kMaxRequests + kWarps * sizeof(int64_t) <= 227 * 1024, "all requests fit a block's shared memory");

__device__ __forceinline__ int64_t at_least_zero(int32_t v) { return v > 0 ? v : 0; }

__global__ void __launch_bounds__(kNt) page_table_kernel(const PageTableArgs a) {
    extern __shared__ int32_t smem[];
    __shared__ int64_t s_sum[kWarps];
    int32_t* s_end = smem;             // [B] tokens up to and with request b (at most 2^31 - 1)
    int32_t* s_cached = smem + a.B;    // [B]
    int32_t* s_new = smem + 2 * a.B;   // [B] the step's new pages before request b's; -1: refused
    pdl_wait_and_release();
    const int nt = blockDim.x, P = 1 << a.page_shift;
    const int64_t kMost = 0x7fffffff;
    const int64_t free_count = min(max(int64_t(*a.free_count), int64_t(0)), a.free_capacity);
    const uint32_t rank = blockIdx.x, blocks = gridDim.x;

    // a thread's requests: a run of them, so that its sums follow on each other's
    const int per = (a.B + nt - 1) / nt, b0 = min(a.B, int(threadIdx.x) * per), b1 = min(a.B, b0 + per);
    int64_t sum = 0, tokens = 0;
    for (int b = b0; b < b1; ++b) sum += at_least_zero(a.added[b]);
    int64_t end = block_before(sum, s_sum, tokens), fresh = 0;
    const auto pages = [&](int64_t n) { return (n + P - 1) >> a.page_shift; };
    for (int b = b0; b < b1; ++b) {
        const int64_t c = at_least_zero(a.cached[b]), n = c + at_least_zero(a.added[b]);
        end += n - c;
        const bool fits = pages(n) <= a.max_pages && end <= a.max_tokens;
        s_end[b] = int32_t(min(end, kMost));
        s_cached[b] = int32_t(c);
        s_new[b] = fits ? int32_t(pages(n) - pages(c)) : -1;
        fresh += fits ? pages(n) - pages(c) : 0;
    }
    int64_t wanted = 0, taken = block_before(fresh, s_sum, wanted);
    // the pages handed out end with the last request whose sum the stack covers
    int refused = 0;
    int64_t last = 0;
    for (int b = b0; b < b1; ++b) {
        const int32_t n = s_new[b];
        if (n >= 0) {
            const bool ok = n == 0 || taken + n <= free_count;
            s_new[b] = ok ? int32_t(min(taken, kMost)) : -1;
            taken += n;
            if (taken <= free_count) last = taken;
            refused += !ok;
        } else {
            ++refused;
        }
    }
    // every read of what may be written in place is done
    if (blocks > 1) cluster_sync();
    else __syncthreads();

    const int have_tokens = int(min(tokens, int64_t(a.max_tokens)));
    for (int64_t i64 = int64_t(rank) * nt + threadIdx.x; i64 < a.max_tokens; i64 += int64_t(blocks) * nt) {
        const int i = int(i64);
        int64_t slot = -1;
        int pos = 0;
        if (i < have_tokens) {
            int lo = 0, hi = a.B - 1;   // the first request that ends behind i
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                if (s_end[mid] > i) hi = mid;
                else lo = mid + 1;
            }
            const int32_t base = s_new[lo];
            if (base >= 0) {
                const int c = s_cached[lo];
                pos = c + i - (lo > 0 ? s_end[lo - 1] : 0);
                const int entry = pos >> a.page_shift, have = int(pages(c));
                int32_t* row = a.block_table + int64_t(lo) * a.max_pages;
                int32_t page;
                if (entry < have) {
                    page = row[entry];
                } else {
                    page = a.free_pages[free_count - 1 - (base + entry - have)];
                    if ((pos & (P - 1)) == 0) row[entry] = page;   // a new page's first token is a new one
                }
                if (page >= 0) slot = (int64_t(page) << a.page_shift) + (pos & (P - 1));
            }
        }
        a.positions[i] = pos;
        a.slots[i] = slot;
    }

    if (rank != 0) return;
    for (int b = threadIdx.x; b < a.B; b += nt) {
        const int32_t begin = b > 0 ? s_end[b - 1] : 0;
        a.starts[b] = begin;
        a.lengths[b] = s_cached[b] + (s_new[b] >= 0 ? s_end[b] - begin : 0);
    }
    // sums of the threads' counts, and the largest of their page totals
    int64_t all = 0;
    block_before(refused, s_sum, all);
#pragma unroll
    for (int o = kWarp / 2; o > 0; o >>= 1) last = max(last, __shfl_xor_sync(kFull, last, o));
    if (threadIdx.x % kWarp == 0) s_sum[threadIdx.x / kWarp] = last;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < nt / kWarp; ++w) last = max(last, s_sum[w]);
        a.starts[a.B] = int32_t(min(tokens, kMost));
        *a.free_count_out = int32_t(free_count - last);
        if (a.refused != nullptr) *a.refused = int32_t(all);
    }
}

__global__ void __launch_bounds__(kNt) page_release_kernel(const PageReleaseArgs a) {
    extern __shared__ int32_t smem[];
    __shared__ int64_t s_sum[kWarps];
    int32_t* s_pages = smem;           // [B] pages that request b gives back
    int32_t* s_before = smem + a.B;    // [B] and those of the requests before it (at most 2^31 - 1)
    pdl_wait_and_release();
    const int nt = blockDim.x, P = 1 << a.page_shift;
    const int64_t free_count = min(max(int64_t(*a.free_count), int64_t(0)), a.free_capacity);
    const int per = (a.B + nt - 1) / nt, b0 = min(a.B, int(threadIdx.x) * per), b1 = min(a.B, b0 + per);
    int64_t sum = 0, total = 0;
    for (int b = b0; b < b1; ++b) {
        const int64_t n = a.finished[b] != 0 ? min((at_least_zero(a.lengths[b]) + P - 1) >> a.page_shift, int64_t(a.max_pages)) : 0;
        s_pages[b] = int32_t(n);
        sum += n;
    }
    int64_t before = block_before(sum, s_sum, total);
    for (int b = b0; b < b1; ++b) {
        s_before[b] = int32_t(min(before, int64_t(0x7fffffff)));
        before += s_pages[b];
    }
    const uint32_t rank = blockIdx.x, blocks = gridDim.x;
    if (blocks > 1) cluster_sync();
    else __syncthreads();
    const int warps = nt / kWarp;
    for (int b = int(rank) * warps + threadIdx.x / kWarp; b < a.B; b += int(blocks) * warps) {
        const int32_t* row = a.block_table + int64_t(b) * a.max_pages;
        const int64_t to = free_count + s_before[b];
        for (int i = threadIdx.x % kWarp; i < s_pages[b] && to + i < a.free_capacity; i += kWarp)
            a.free_pages[to + i] = row[i];
        if (threadIdx.x % kWarp == 0 && a.finished[b] != 0) a.lengths[b] = 0;
    }
    if (rank == 0 && threadIdx.x == 0) *a.free_count = int32_t(min(free_count + total, a.free_capacity));
}

// Blocks of the cluster, and threads of a block: one small block where it is
// enough for one item a thread, else up to 8 blocks (the portable limit).
void shape(int64_t items, int& blocks, int& threads) {
    threads = kNt;
    while (threads > 128 && items <= threads / 2) threads /= 2;
    blocks = 1;
    while (blocks < 8 && items > int64_t(blocks) * threads) blocks *= 2;
}

}  // namespace

cudaError_t launch_page_table(const PageTableArgs& a, cudaStream_t stream) {
    static SmemGrant grant;
    const size_t smem = 12 * size_t(a.B);
    if (smem + sizeof(int64_t) * kWarps > 48 * 1024) {
        const cudaError_t err = grant.ensure(page_table_kernel);
        if (err != cudaSuccess) return err;
    }
    int blocks = 1, threads = kNt;
    shape(std::max(a.B, a.max_tokens), blocks, threads);
    return launch_cluster(page_table_kernel, dim3(blocks), dim3(threads), uint32_t(blocks), smem, stream, a);
}

cudaError_t launch_page_release(const PageReleaseArgs& a, cudaStream_t stream) {
    static SmemGrant grant;
    const size_t smem = 8 * size_t(a.B);
    if (smem + sizeof(int64_t) * kWarps > 48 * 1024) {
        const cudaError_t err = grant.ensure(page_release_kernel);
        if (err != cudaSuccess) return err;
    }
    int blocks = 1, threads = kNt;
    shape(int64_t(a.B) * kWarp, blocks, threads);
    return launch_cluster(page_release_kernel, dim3(blocks), dim3(threads), uint32_t(blocks), smem, stream, a);
}

}  // namespace moe
