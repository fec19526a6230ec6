// A whole MoE layer for a few tokens (T <= 32), bfloat16 weights, in two
// kernels: routing and fc1 with SwiGLU, then fc2 with the weighted combine.
//
//   ids, w = top-k of softmax(logits)   (as moe_route)
//   a[t, j, i]  = bf16( w[t, j] * silu(W1g[e] x_t)_i * (W1u[e] x_t)_i ),  e = ids[t, j]
//   out[t, h]   = bf16( sum_j (W2[e_j] a[t, j])_h )
//
// At a few tokens the layer is bound by the bytes of the chosen experts'
// weights, each read once. The routing weight goes into the activation before
// its one rounding (tensor cores take bfloat16 operands), so the combine is a
// plain sum over the concatenated k of all chosen experts, in float32.
//
// Routing is redundant: every block routes the whole batch in shared memory
// (tens of KB of logits at most), so no block waits for another.
//   fc1: an item is 8 R columns of one expert's activation. A tile's 16 A rows
//   are 8 gate rows and the same 8 up rows, so one lane's accumulators hold
//   both halves of a SwiGLU. The block's warps split k; blocks sweep the items
//   grid-stride. The activation is stored compactly, expert-sorted (row
//   off[d] + rank of the token among the expert's), for the tokens routed.
//   fc2: a cluster of C blocks takes 16 R output columns; its warps split the
//   (expert, k) units of all chosen experts. B columns are the tokens
//   themselves, zero where a token is not routed to the expert.
// All sums are taken in a fixed order: results do not depend on timing.
#include "few_device.cuh"
#include "few_route.cuh"
#include "moe_launch.h"
#include "rows_common.cuh"

namespace moe {
namespace {

constexpr int kNw = 8;
constexpr int kNt = kNw * kWarp;
constexpr int kDepth = 2;                         // chunks in flight per warp
// fc1: the block's chunks are numbered item by item; a warp takes chunk
// u = warp, warp + kNw, ... of every item, `per` of them (the last may lie
// outside), so that its ring runs on across items.
template <int R, int NG, int US>
__global__ void __launch_bounds__(kNt, 2) fc1_kernel(LayerArgs a) {
    using Ring = WRing<kWBf16, R, US, kDepth>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ FewRoute s;
    pdl_wait_and_release();
    route_few(a, s, blockIdx.x == 0);
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp, g = lane / 4, q = lane % 4;
    const uint32_t K = uint32_t(a.H), I = uint32_t(a.I);
    const uint32_t rb = row_bytes<kWBf16>(K);
    const uint32_t tiles = (I + 8 * R - 1) / (8 * R);
    const uint32_t per = ((rb + 63) / 64 + US * kNw - 1) / (US * kNw);
    const uint32_t items = uint32_t(s.nd) * tiles;
    const int out_n = a.T * 16 * R;
    float* s_red = reinterpret_cast<float*>(smem + kNw * Ring::kBytes);   // [kNw][T][16 R]
    const uint8_t* w13 = static_cast<const uint8_t*>(a.w13);
    const WStride st = {8ull * rb, uint64_t(I) * rb, 0, 0};

    // the chunk of (item, i-th of this warp's)
    struct Cursor {
        uint32_t item, i;
        WChunk c;
    };
    auto place = [&](Cursor& x) {   // rows of x.item
        x.c.rows = 0;
        if (x.item < items) {
            const uint32_t d = x.item / tiles, j = (x.item - d * tiles) * (8 * R) + g;
            const uint64_t row = uint64_t(s.expert[d]) * 2 * I + j;
            x.c.w = w13 + row * rb + q * 16;
#pragma unroll
            for (int r = 0; r < R; ++r) x.c.rows |= (j + 8 * r < I ? 3u : 0u) << (2 * r);
        }
    };
    auto step = [&](Cursor& x) { x.c.step = (x.i * kNw + warp) * US; };
    auto advance = [&](Cursor& x) {
        if (++x.i == per) {
            x.i = 0;
            x.item += gridDim.x;
            place(x);
        }
        step(x);
    };

    Ring ring;
    ring.init(smem + warp * Ring::kBytes);
    Cursor fw = {blockIdx.x, 0, {w13, nullptr, 0, 0}};   // fetch cursor of the weights, kDepth chunks ahead
    place(fw);
    step(fw);
#pragma unroll
    for (int i = 0; i < kDepth; ++i) {
        ring.fetch(i * Ring::kChunk, fw.c, st, w13, rb);
        Ring::commit();
        advance(fw);
    }
    for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
        const uint32_t d = item / tiles, j0 = (item - d * tiles) * (8 * R);
        const uint32_t tokens = s.tokens[d];
        const int m = __popc(tokens), groups = (m + 7) / 8;
        const uint16_t* xrow[NG];
#pragma unroll
        for (int n = 0; n < NG; ++n)
            xrow[n] = n * 8 + g < m ? a.x + uint64_t(s.row_t[s.off[d] + n * 8 + g]) * K : nullptr;
        float acc[R][NG][4] = {};
        for (uint32_t i = 0; i < per; ++i) {
            const uint32_t s0 = (i * kNw + warp) * US;
            BGran<kWBf16> b0[US];
#pragma unroll
            for (int k = 0; k < US; ++k) load_x<kWBf16>(b0[k], xrow[0], xrow[0] != nullptr, s0 + k, q, K);
            Ring::wait();
            if (s0 * 64u < rb) {
#pragma unroll
                for (int k = 0; k < US; ++k)
                    bf16_step<R, NG>(acc, (1u << groups) - 1u,
                                       [&](AGran& w, int r) { ring.read(w, k, r); },
                                       [&](int n, BGran<kWBf16>& b) {
                                           if (n == 0) b = b0[k];
                                           else load_x<kWBf16>(b, xrow[n], xrow[n] != nullptr, s0 + k, q, K);
                                       });
            }
            __syncwarp();   // the slot is read: refill it
            ring.fetch(ring.slot, fw.c, st, w13, rb);
            Ring::commit();
            ring.next();
            advance(fw);
        }
        store_partial<R, NG>(s_red + warp * out_n, acc, m);
        __syncthreads();
        // thread -> (token of the expert, column); the two halves lie 8 rows apart
        for (int o = threadIdx.x; o < m * 8 * R; o += kNt) {
            const int c = o / (8 * R), i = o % (8 * R);
            const int at = c * (16 * R) + (i / 8) * 16 + i % 8;
            float gate = 0.0f, up = 0.0f;
#pragma unroll
            for (int w = 0; w < kNw; ++w) {
                gate += s_red[w * out_n + at];
                up += s_red[w * out_n + at + 8];
            }
            const uint32_t row = s.off[d] + c;
            if (j0 + i < I) a.act[uint64_t(row) * I + j0 + i] = uint16_t(pack_bf16x2(s.row_w[row] * (silu(gate) * up), 0.0f));
        }
        __syncthreads();
    }
    Ring::drain();
}

// fc2: the chunks of all chosen experts, in order, are dealt to the warps of
// the cluster.
template <int R, int NG, int US>
__global__ void __launch_bounds__(kNt, 2) fc2_kernel(LayerArgs a, uint32_t C) {
    using Ring = WRing<kWBf16, R, US, kDepth>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ FewRoute s;
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp, g = lane / 4, q = lane % 4;
    const uint32_t K = uint32_t(a.I), H = uint32_t(a.H);
    const uint32_t rb = row_bytes<kWBf16>(K);
    const uint32_t rank = blockIdx.x % C, row0 = blockIdx.x / C * (16 * R);
    const uint32_t chunks = ((rb + 63) / 64 + US - 1) / US;   // per expert
    const int out_n = a.T * 16 * R;
    float* s_red = reinterpret_cast<float*>(smem + kNw * Ring::kBytes);   // [kNw][T][16 R]
    float* s_warp = s_red + warp * out_n;
    // Before the wait for fc1: routing from the logits and the first weights.
    // Neither is written by fc1, and fc1 let this kernel start only after its
    // own wait, so whatever wrote them has completed.
    route_few(a, s, false);
    const uint8_t* w2 = static_cast<const uint8_t*>(a.w2);
    const WStride st = {16ull * rb, 8ull * rb, 0, 0};
    uint32_t rows = 0;
#pragma unroll
    for (int i = 0; i < 2 * R; ++i) rows |= uint32_t(row0 + 8 * i + g < H) << i;
    const uint32_t nd = uint32_t(s.nd), stride = C * kNw, sd = stride / chunks, su = stride - sd * chunks;
    struct Cursor {
        uint32_t d, u;
        WChunk c;
    };
    auto place = [&](Cursor& x) {
        x.c.rows = 0;
        if (x.d < nd) {
            const uint64_t row = uint64_t(s.expert[x.d]) * H + row0 + g;
            x.c.w = w2 + row * rb + q * 16;
            x.c.rows = rows;
        }
        x.c.step = x.u * US;
    };
    auto advance = [&](Cursor& x) {
        x.u += su;
        x.d += sd;
        if (x.u >= chunks) {
            x.u -= chunks;
            ++x.d;
        }
        place(x);
    };
    Ring ring;
    ring.init(smem + warp * Ring::kBytes);
    const uint32_t first = rank * kNw + warp;
    Cursor fw = {first / chunks, first % chunks, {w2, nullptr, 0, 0}};
    place(fw);
    Cursor cur = fw;
#pragma unroll
    for (int i = 0; i < kDepth; ++i) {
        ring.fetch(i * Ring::kChunk, fw.c, st, w2, rb);
        Ring::commit();
        advance(fw);
    }
    pdl_wait_and_release();

    float acc[R][NG][4] = {};
    while (cur.d < nd) {
        const uint32_t d = cur.d, s0 = cur.u * US;
        const uint32_t tokens = s.tokens[d], off = s.off[d];
        const int m = __popc(tokens);
        auto load = [&](int n, int k, BGran<kWBf16>& b) {
            const uint32_t c = n * 8 + g;   // column: token c
            const bool mine = (tokens >> c) & 1u;
            const uint32_t row = off + __popc(tokens & ((1u << c) - 1u));
            load_x<kWBf16>(b, a.act + uint64_t(row) * K, mine, s0 + k, q, K);
        };
        uint32_t live = 0;   // groups with a token of this expert: warp-uniform
#pragma unroll
        for (int n = 0; n < NG; ++n)
            live |= uint32_t(((tokens >> (8 * n)) & 0xffu) != 0u) << n;
        BGran<kWBf16> b0[US];
        if (live & 1u) {
#pragma unroll
            for (int k = 0; k < US; ++k) load(0, k, b0[k]);
        }
        Ring::wait();
#pragma unroll
        for (int k = 0; k < US; ++k)
            bf16_step<R, NG>(acc, live, [&](AGran& w, int r) { ring.read(w, k, r); },
                               [&](int n, BGran<kWBf16>& b) {
                                   if (n == 0) b = b0[k];
                                   else load(n, k, b);
                               });
        __syncwarp();   // the slot is read: refill it
        ring.fetch(ring.slot, fw.c, st, w2, rb);
        Ring::commit();
        ring.next();
        advance(fw);
        advance(cur);
    }
    Ring::drain();
    store_partial<R, NG>(s_warp, acc, a.T);
    __syncthreads();
    if (C > 1) {
        for (int o = threadIdx.x; o < out_n; o += kNt) {
            float v = s_red[o];
#pragma unroll
            for (int w = 1; w < kNw; ++w) v += s_red[w * out_n + o];
            s_red[o] = v;   // this thread alone reads and writes column o
        }
        cluster_sync();
    }
    for (int o = threadIdx.x + (C > 1 ? int(rank) * kNt : 0); o < out_n; o += kNt * int(C)) {
        float v;
        if (C > 1) {
            v = ld_cluster(s_red + o, 0);
            for (uint32_t c = 1; c < C; ++c) v += ld_cluster(s_red + o, c);
        } else {
            v = s_red[o];
#pragma unroll
            for (int w = 1; w < kNw; ++w) v += s_red[w * out_n + o];
        }
        const uint32_t t = uint32_t(o) / (16 * R), row = row0 + uint32_t(o) % (16 * R);
        if (row < H) a.out[uint64_t(t) * H + row] = uint16_t(pack_bf16x2(v, 0.0f));
    }
    if (C > 1) cluster_sync();   // the others may still read this block's sums
}

template <int R, int NG, int US>
cudaError_t launch_r(const LayerArgs& a, int num_sms, cudaStream_t stream) {
    auto fc1 = fc1_kernel<R, NG, US>;
    auto fc2 = fc2_kernel<R, NG, US>;
    static SmemGrant grant1, grant2;
    cudaError_t err = grant1.ensure(fc1);
    if (err == cudaSuccess) err = grant2.ensure(fc2);
    if (err != cudaSuccess) return err;
    const size_t smem = kNw * WRing<kWBf16, R, US, kDepth>::kBytes + sizeof(float) * kNw * a.T * 16 * R;
    const uint64_t nd = std::min<uint64_t>(a.E, uint64_t(a.T) * a.k);   // most experts that can be chosen
    const uint64_t items = nd * ((uint64_t(a.I) + 8 * R - 1) / (8 * R));
    const uint32_t grid = uint32_t(std::min<uint64_t>(items, 2ull * num_sms));
    err = launch_pdl(fc1, dim3(grid), dim3(kNt), smem, stream, a);
    if (err != cudaSuccess) return err;
    const uint32_t tiles = (uint32_t(a.H) + 16 * R - 1) / (16 * R);
    const uint32_t C = split_k(tiles, 2u * uint32_t(num_sms), 8);
    return launch_cluster(fc2, dim3(tiles * C), dim3(kNt), C, smem, stream, a, C);
}

}  // namespace

cudaError_t launch_layer_bf16(const LayerArgs& a, int num_sms, cudaStream_t stream) {
    if (a.T <= 8) return launch_r<1, 1, 4>(a, num_sms, stream);
    if (a.T <= 16) return launch_r<1, 2, 4>(a, num_sms, stream);
    return launch_r<1, 4, 4>(a, num_sms, stream);
}

}  // namespace moe
