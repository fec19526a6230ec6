// C-ABI entry points (declared in include/moe_glue.h): argument validation on
// the host, then one launch sequence on the caller's stream. No allocation,
// no synchronisation, no host copies, no fallback path.
#include "moe_glue.h"
#include "moe_launch.h"

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <initializer_list>
#include <utility>

namespace {

using moe::RoutePlan;

constexpr int kMaxDevices = 64;
std::atomic<int> g_sm_count[kMaxDevices];

// SM count of the current device (cached per device; racing first calls all
// store the same value).
cudaError_t current_sm_count(int* out) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev >= 0 && dev < kMaxDevices) {
        const int cached = g_sm_count[dev].load(std::memory_order_relaxed);
        if (cached > 0) { *out = cached; return cudaSuccess; }
    }
    int sms = 0;
    err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess) return err;
    if (dev >= 0 && dev < kMaxDevices) g_sm_count[dev].store(sms, std::memory_order_relaxed);
    *out = sms;
    return cudaSuccess;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

struct Range {
    const void* p;
    uint64_t bytes;
};

bool overlap(Range a, Range b) {
    if (a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

bool any_overlap(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (const Range& i : ins)
            if (overlap(*o, i)) return true;
        for (auto o2 = o + 1; o2 != outs.end(); ++o2)
            if (overlap(*o, *o2)) return true;
    }
    return false;
}

moe_status_t check_route_sizes(int64_t T, int E, int k) {
    if (T < 0 || E < 1 || k < 1 || k > E) return MOE_ERR_INVALID_ARG;
    if (E > MOE_MAX_EXPERTS || k > MOE_MAX_TOPK) return MOE_ERR_UNSUPPORTED;
    if (T * int64_t(k) >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// Rows of bfloat16 vectors: width a multiple of 8 elements (16 bytes).
moe_status_t check_rows(int64_t rows, int width, int64_t slots_mult) {
    if (rows < 0 || width < 1) return MOE_ERR_INVALID_ARG;
    if (width % 8 != 0) return MOE_ERR_MISALIGNED;
    if (rows * slots_mult >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

moe_status_t from_cuda(cudaError_t err) { return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// Local routing arguments: 0 <= e0 < e1 <= E, pad >= 1, padded capacity < 2^31.
moe_status_t check_local(int64_t T, int E, int k, int e0, int e1, int pad, int64_t* rows) {
    moe_status_t st = check_route_sizes(T, E, k);
    if (st != MOE_OK) return st;
    if (e0 < 0 || e1 > E || e0 >= e1 || pad < 1) return MOE_ERR_INVALID_ARG;
    const int64_t r = T * int64_t(k) + int64_t(e1 - e0) * int64_t(pad - 1);
    if (r >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
    if (rows) *rows = r;
    return MOE_OK;
}

}  // namespace

extern "C" {

const char* moe_status_string(moe_status_t status) {
    switch (status) {
        case MOE_OK: return "MOE_OK";
        case MOE_ERR_INVALID_ARG: return "MOE_ERR_INVALID_ARG";
        case MOE_ERR_MISALIGNED: return "MOE_ERR_MISALIGNED";
        case MOE_ERR_UNSUPPORTED: return "MOE_ERR_UNSUPPORTED";
        case MOE_ERR_WORKSPACE: return "MOE_ERR_WORKSPACE";
        case MOE_ERR_CUDA: return "MOE_ERR_CUDA";
    }
    return "MOE_ERR_UNKNOWN";
}

moe_status_t moe_route_workspace_size(int64_t T, int E, int k, size_t* bytes) {
    if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check_route_sizes(T, E, k);
    if (st != MOE_OK) return st;
    *bytes = T == 0 ? 0 : moe::plan_route(T, E, k).ws_bytes;
    return MOE_OK;
}

moe_status_t moe_route(const float* logits, int64_t T, int E, int k, int renorm,
                       int32_t* topk_ids, float* topk_weights, int32_t* expert_counts,
                       int32_t* expert_offsets, int32_t* perm, int32_t* inv_perm,
                       void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    moe_status_t st = check_route_sizes(T, E, k);
    if (st != MOE_OK) return st;
    if (expert_counts == nullptr || expert_offsets == nullptr) return MOE_ERR_INVALID_ARG;
    if (!aligned4(expert_counts) || !aligned4(expert_offsets)) return MOE_ERR_MISALIGNED;
    const uint64_t S = uint64_t(T) * uint64_t(k);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) {
        if (any_overlap({{expert_counts, 4ull * E}, {expert_offsets, 4ull * (E + 1)}}, {}))
            return MOE_ERR_INVALID_ARG;
        cudaError_t err = cudaMemsetAsync(expert_counts, 0, sizeof(int32_t) * E, s);
        if (err == cudaSuccess) err = cudaMemsetAsync(expert_offsets, 0, sizeof(int32_t) * (E + 1), s);
        return from_cuda(err);
    }
    if (logits == nullptr || topk_ids == nullptr || topk_weights == nullptr || perm == nullptr ||
        inv_perm == nullptr)
        return MOE_ERR_INVALID_ARG;
    if (!aligned4(logits) || !aligned4(topk_ids) || !aligned4(topk_weights) || !aligned4(perm) ||
        !aligned4(inv_perm))
        return MOE_ERR_MISALIGNED;
    const RoutePlan plan = moe::plan_route(T, E, k);
    if (plan.ws_bytes > 0) {
        if (workspace == nullptr || workspace_bytes < plan.ws_bytes) return MOE_ERR_WORKSPACE;
        if (!aligned16(workspace)) return MOE_ERR_MISALIGNED;
    }
    const uint64_t ws = plan.ws_bytes;
    if (any_overlap({{topk_ids, 4 * S}, {topk_weights, 4 * S}, {expert_counts, 4ull * E},
                     {expert_offsets, 4ull * (E + 1)}, {perm, 4 * S}, {inv_perm, 4 * S},
                     {workspace, ws}},
                    {{logits, 4ull * uint64_t(T) * E}}))
        return MOE_ERR_INVALID_ARG;
    return from_cuda(moe::launch_route(plan, logits, int(T), E, k, renorm ? 1 : 0, topk_ids,
                                       topk_weights, expert_counts, expert_offsets, perm, inv_perm,
                                       workspace, s));
}

moe_status_t moe_route_expand(const float* logits, int64_t T, int E, int k, int renorm,
                              const moe_bf16_t* x, int H, int32_t* topk_ids, float* topk_weights,
                              int32_t* expert_counts, int32_t* expert_offsets, int32_t* perm,
                              int32_t* inv_perm, moe_bf16_t* expanded_x, void* workspace,
                              size_t workspace_bytes, moe_stream_t stream) {
    moe_status_t st = check_route_sizes(T, E, k);
    if (st != MOE_OK) return st;
    if ((st = check_rows(T, H, k)) != MOE_OK) return st;
    if (T > 0) {
        if (x == nullptr || expanded_x == nullptr) return MOE_ERR_INVALID_ARG;
        if (!aligned16(x) || !aligned16(expanded_x)) return MOE_ERR_MISALIGNED;
        const uint64_t S = uint64_t(T) * uint64_t(k);
        const uint64_t ws = moe::plan_route(T, E, k).ws_bytes;
        // expanded_x against every other buffer of the call
        if (any_overlap({{expanded_x, 2 * S * uint64_t(H)}},
                        {{x, 2 * uint64_t(T) * uint64_t(H)}, {logits, 4ull * uint64_t(T) * E},
                         {topk_ids, 4 * S}, {topk_weights, 4 * S}, {expert_counts, 4ull * E},
                         {expert_offsets, 4ull * (E + 1)}, {perm, 4 * S}, {inv_perm, 4 * S},
                         {workspace, ws}}))
            return MOE_ERR_INVALID_ARG;
        // x is an input of the expansion: no routing output may overlap it
        if (any_overlap({{x, 2 * uint64_t(T) * uint64_t(H)}},
                        {{topk_ids, 4 * S}, {topk_weights, 4 * S}, {expert_counts, 4ull * E},
                         {expert_offsets, 4ull * (E + 1)}, {perm, 4 * S}, {inv_perm, 4 * S},
                         {workspace, ws}}))
            return MOE_ERR_INVALID_ARG;
    }
    const moe::RoutePlan plan = moe::plan_route(T, E, k);
    if (T > 0 && moe::route_expand_fits(plan)) {
        // validate the routing arguments exactly as moe_route does
        if (expert_counts == nullptr || expert_offsets == nullptr || logits == nullptr ||
            topk_ids == nullptr || topk_weights == nullptr || perm == nullptr || inv_perm == nullptr)
            return MOE_ERR_INVALID_ARG;
        if (!aligned4(expert_counts) || !aligned4(expert_offsets) || !aligned4(logits) ||
            !aligned4(topk_ids) || !aligned4(topk_weights) || !aligned4(perm) || !aligned4(inv_perm))
            return MOE_ERR_MISALIGNED;
        const uint64_t S = uint64_t(T) * uint64_t(k);
        if (any_overlap({{topk_ids, 4 * S}, {topk_weights, 4 * S}, {expert_counts, 4ull * E},
                         {expert_offsets, 4ull * (E + 1)}, {perm, 4 * S}, {inv_perm, 4 * S}},
                        {{logits, 4ull * uint64_t(T) * E}}))
            return MOE_ERR_INVALID_ARG;
        int sms = 0;
        if (current_sm_count(&sms) != cudaSuccess) return MOE_ERR_CUDA;
        return from_cuda(moe::launch_route_expand(
            plan, logits, int(T), E, k, renorm ? 1 : 0, topk_ids, topk_weights, expert_counts,
            expert_offsets, perm, inv_perm, x, H, expanded_x, sms, reinterpret_cast<cudaStream_t>(stream)));
    }
    st = moe_route(logits, T, E, k, renorm, topk_ids, topk_weights, expert_counts, expert_offsets,
                   perm, inv_perm, workspace, workspace_bytes, stream);
    if (st != MOE_OK || T == 0) return st;
    return moe_expand(x, T, H, k, inv_perm, expanded_x, stream);
}

moe_status_t moe_route_local_rows(int64_t T, int k, int e0, int e1, int pad, int64_t* rows) {
    if (rows == nullptr || T < 0 || k < 1 || e0 < 0 || e0 >= e1 || pad < 1) return MOE_ERR_INVALID_ARG;
    const int64_t r = T * int64_t(k) + int64_t(e1 - e0) * int64_t(pad - 1);
    if (r >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
    *rows = r;
    return MOE_OK;
}

moe_status_t moe_route_local_workspace_size(int64_t T, int E, int k, int e0, int e1, size_t* bytes) {
    if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check_local(T, E, k, e0, e1, 1, nullptr);
    if (st != MOE_OK) return st;
    *bytes = T == 0 ? 0 : moe::plan_route(T, E, k, e1 - e0).ws_bytes;
    return MOE_OK;
}

moe_status_t moe_route_local(const float* logits, int64_t T, int E, int k, int renorm, int e0,
                             int e1, int pad, int32_t* topk_ids, float* topk_weights,
                             int32_t* expert_counts, int32_t* expert_offsets, int32_t* perm,
                             int32_t* inv_perm, void* workspace, size_t workspace_bytes,
                             moe_stream_t stream) {
    int64_t rows = 0;
    moe_status_t st = check_local(T, E, k, e0, e1, pad, &rows);
    if (st != MOE_OK) return st;
    const int n = e1 - e0;
    if (expert_counts == nullptr || expert_offsets == nullptr) return MOE_ERR_INVALID_ARG;
    if (!aligned4(expert_counts) || !aligned4(expert_offsets)) return MOE_ERR_MISALIGNED;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) {
        if (any_overlap({{expert_counts, 4ull * n}, {expert_offsets, 4ull * (n + 1)}, {perm, 4ull * rows}}, {}))
            return MOE_ERR_INVALID_ARG;
        cudaError_t err = cudaMemsetAsync(expert_counts, 0, sizeof(int32_t) * n, s);
        if (err == cudaSuccess) err = cudaMemsetAsync(expert_offsets, 0, sizeof(int32_t) * (n + 1), s);
        if (err == cudaSuccess && rows > 0) {
            if (perm == nullptr) return MOE_ERR_INVALID_ARG;
            err = cudaMemsetAsync(perm, 0xff, sizeof(int32_t) * rows, s);   // all -1
        }
        return from_cuda(err);
    }
    if (logits == nullptr || topk_ids == nullptr || topk_weights == nullptr || perm == nullptr ||
        inv_perm == nullptr)
        return MOE_ERR_INVALID_ARG;
    if (!aligned4(logits) || !aligned4(topk_ids) || !aligned4(topk_weights) || !aligned4(perm) ||
        !aligned4(inv_perm))
        return MOE_ERR_MISALIGNED;
    const moe::RoutePlan plan = moe::plan_route(T, E, k, n);
    if (plan.ws_bytes > 0) {
        if (workspace == nullptr || workspace_bytes < plan.ws_bytes) return MOE_ERR_WORKSPACE;
        if (!aligned16(workspace)) return MOE_ERR_MISALIGNED;
    }
    const uint64_t S = uint64_t(T) * uint64_t(k);
    if (any_overlap({{topk_ids, 4 * S}, {topk_weights, 4 * S}, {expert_counts, 4ull * n},
                     {expert_offsets, 4ull * (n + 1)}, {perm, 4ull * rows}, {inv_perm, 4 * S},
                     {workspace, plan.ws_bytes}},
                    {{logits, 4ull * uint64_t(T) * E}}))
        return MOE_ERR_INVALID_ARG;
    const moe::LocalRange local{e0, n, pad, int(rows)};
    return from_cuda(moe::launch_route(plan, logits, int(T), E, k, renorm ? 1 : 0, topk_ids,
                                       topk_weights, expert_counts, expert_offsets, perm, inv_perm,
                                       workspace, s, &local));
}

moe_status_t moe_expand_rows(const moe_bf16_t* x, int64_t T, int H, int k, const int32_t* inv_perm,
                             int64_t rows, moe_bf16_t* expanded_x, moe_stream_t stream) {
    if (k < 1) return MOE_ERR_INVALID_ARG;
    if (k > MOE_MAX_TOPK) return MOE_ERR_UNSUPPORTED;
    moe_status_t st = check_rows(T, H, k);
    if (st != MOE_OK) return st;
    if (rows < 0) return MOE_ERR_INVALID_ARG;
    if (rows >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
    if (T == 0 || rows == 0) return MOE_OK;
    if (x == nullptr || inv_perm == nullptr || expanded_x == nullptr) return MOE_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(expanded_x) || !aligned4(inv_perm)) return MOE_ERR_MISALIGNED;
    const uint64_t S = uint64_t(T) * uint64_t(k);
    if (any_overlap({{expanded_x, 2 * uint64_t(rows) * uint64_t(H)}},
                    {{x, 2 * uint64_t(T) * uint64_t(H)}, {inv_perm, 4 * S}}))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if (current_sm_count(&sms) != cudaSuccess) return MOE_ERR_CUDA;
    return from_cuda(moe::launch_expand(x, T, H, k, inv_perm, rows, expanded_x, sms,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_combine_rows(const moe_bf16_t* expert_out, int64_t rows, int64_t T, int H, int k,
                              const float* topk_weights, const int32_t* inv_perm, moe_bf16_t* out,
                              moe_stream_t stream) {
    if (k < 1) return MOE_ERR_INVALID_ARG;
    if (k > MOE_MAX_TOPK) return MOE_ERR_UNSUPPORTED;
    moe_status_t st = check_rows(T, H, k);
    if (st != MOE_OK) return st;
    if (rows < 0) return MOE_ERR_INVALID_ARG;
    if (rows >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    if (topk_weights == nullptr || inv_perm == nullptr || out == nullptr ||
        (rows > 0 && expert_out == nullptr))
        return MOE_ERR_INVALID_ARG;
    if ((rows > 0 && !aligned16(expert_out)) || !aligned16(out) || !aligned4(topk_weights) ||
        !aligned4(inv_perm))
        return MOE_ERR_MISALIGNED;
    const uint64_t S = uint64_t(T) * uint64_t(k);
    if (any_overlap({{out, 2 * uint64_t(T) * uint64_t(H)}},
                    {{expert_out, 2 * uint64_t(rows) * uint64_t(H)}, {topk_weights, 4 * S},
                     {inv_perm, 4 * S}}))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if (current_sm_count(&sms) != cudaSuccess) return MOE_ERR_CUDA;
    return from_cuda(moe::launch_combine(expert_out, rows, T, H, k, topk_weights, inv_perm, out, sms,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_expand(const moe_bf16_t* x, int64_t T, int H, int k, const int32_t* inv_perm,
                        moe_bf16_t* expanded_x, moe_stream_t stream) {
    if (k < 1) return MOE_ERR_INVALID_ARG;
    if (k > MOE_MAX_TOPK) return MOE_ERR_UNSUPPORTED;
    moe_status_t st = check_rows(T, H, k);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    if (x == nullptr || inv_perm == nullptr || expanded_x == nullptr) return MOE_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(expanded_x) || !aligned4(inv_perm)) return MOE_ERR_MISALIGNED;
    const uint64_t S = uint64_t(T) * uint64_t(k);
    if (any_overlap({{expanded_x, 2 * S * uint64_t(H)}},
                    {{x, 2 * uint64_t(T) * uint64_t(H)}, {inv_perm, 4 * S}}))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    cudaError_t err = current_sm_count(&sms);
    if (err != cudaSuccess) return MOE_ERR_CUDA;
    return from_cuda(moe::launch_expand(x, T, H, k, inv_perm, T * k, expanded_x, sms,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_swiglu(const moe_bf16_t* gate_up, int64_t rows, int I, moe_bf16_t* act,
                        moe_stream_t stream) {
    moe_status_t st = check_rows(rows, I, 1);
    if (st != MOE_OK) return st;
    if (rows == 0) return MOE_OK;
    if (gate_up == nullptr || act == nullptr) return MOE_ERR_INVALID_ARG;
    if (!aligned16(gate_up) || !aligned16(act)) return MOE_ERR_MISALIGNED;
    if (any_overlap({{act, 2 * uint64_t(rows) * uint64_t(I)}},
                    {{gate_up, 4 * uint64_t(rows) * uint64_t(I)}}))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    cudaError_t err = current_sm_count(&sms);
    if (err != cudaSuccess) return MOE_ERR_CUDA;
    return from_cuda(moe::launch_swiglu(gate_up, rows, I, act, sms,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_combine(const moe_bf16_t* expert_out, int64_t T, int H, int k,
                         const float* topk_weights, const int32_t* inv_perm, moe_bf16_t* out,
                         moe_stream_t stream) {
    if (k < 1) return MOE_ERR_INVALID_ARG;
    if (k > MOE_MAX_TOPK) return MOE_ERR_UNSUPPORTED;
    moe_status_t st = check_rows(T, H, k);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    if (expert_out == nullptr || topk_weights == nullptr || inv_perm == nullptr || out == nullptr)
        return MOE_ERR_INVALID_ARG;
    if (!aligned16(expert_out) || !aligned16(out) || !aligned4(topk_weights) ||
        !aligned4(inv_perm))
        return MOE_ERR_MISALIGNED;
    const uint64_t S = uint64_t(T) * uint64_t(k);
    if (any_overlap({{out, 2 * uint64_t(T) * uint64_t(H)}},
                    {{expert_out, 2 * S * uint64_t(H)}, {topk_weights, 4 * S}, {inv_perm, 4 * S}}))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    cudaError_t err = current_sm_count(&sms);
    if (err != cudaSuccess) return MOE_ERR_CUDA;
    return from_cuda(moe::launch_combine(expert_out, T * k, T, H, k, topk_weights, inv_perm, out, sms,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_swiglu_mxfp8(const moe_bf16_t* gate_up, int64_t rows, int I, uint8_t* act_codes,
                              uint8_t* act_scales, moe_stream_t stream) {
    moe_status_t st = check_rows(rows, I, 1);
    if (st != MOE_OK) return st;
    if (I % 32 != 0) return MOE_ERR_MISALIGNED;
    if (rows == 0) return MOE_OK;
    if (gate_up == nullptr || act_codes == nullptr || act_scales == nullptr) return MOE_ERR_INVALID_ARG;
    if (!aligned16(gate_up) || !aligned16(act_codes)) return MOE_ERR_MISALIGNED;
    const uint64_t n = uint64_t(rows) * uint64_t(I);
    if (any_overlap({{act_codes, n}, {act_scales, n / 32}}, {{gate_up, 4 * n}}))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if (current_sm_count(&sms) != cudaSuccess) return MOE_ERR_CUDA;
    return from_cuda(moe::launch_swiglu_mxfp8(gate_up, rows, I, act_codes, act_scales, sms,
                                              reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_expand_mxfp8(const moe_bf16_t* x, int64_t T, int H, int k, const int32_t* inv_perm,
                              int64_t rows, uint8_t* codes, uint8_t* scales, moe_stream_t stream) {
    if (k < 1) return MOE_ERR_INVALID_ARG;
    if (k > MOE_MAX_TOPK) return MOE_ERR_UNSUPPORTED;
    moe_status_t st = check_rows(T, H, k);
    if (st != MOE_OK) return st;
    if (H % 32 != 0) return MOE_ERR_MISALIGNED;
    if (rows < 0) return MOE_ERR_INVALID_ARG;
    if (rows >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
    if (T == 0 || rows == 0) return MOE_OK;
    if (x == nullptr || inv_perm == nullptr || codes == nullptr || scales == nullptr)
        return MOE_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(codes) || !aligned4(inv_perm)) return MOE_ERR_MISALIGNED;
    const uint64_t S = uint64_t(T) * uint64_t(k);
    const uint64_t n = uint64_t(rows) * uint64_t(H);
    if (any_overlap({{codes, n}, {scales, n / 32}},
                    {{x, 2 * uint64_t(T) * uint64_t(H)}, {inv_perm, 4 * S}}))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if (current_sm_count(&sms) != cudaSuccess) return MOE_ERR_CUDA;
    return from_cuda(moe::launch_expand_mxfp8(x, T, H, k, inv_perm, rows, codes, scales, sms,
                                              reinterpret_cast<cudaStream_t>(stream)));
}

namespace {

// The FP4 format arguments: a known format, n a multiple of its block, and
// for NVFP4 a finite positive tensor scale.
moe_status_t check_fp4(int format, int n, float global_scale) {
    if (format != MOE_FP4_NVFP4 && format != MOE_FP4_MXFP4) return MOE_ERR_INVALID_ARG;
    if (format == MOE_FP4_NVFP4 && !(global_scale > 0.0f && global_scale <= 3.4028234663852886e38f))
        return MOE_ERR_INVALID_ARG;
    if (n % (format == MOE_FP4_NVFP4 ? 16 : 32) != 0) return MOE_ERR_MISALIGNED;
    return MOE_OK;
}

}  // namespace

moe_status_t moe_swiglu_fp4(const moe_bf16_t* gate_up, int64_t rows, int I, int format,
                            float global_scale, uint8_t* act_codes, uint8_t* act_scales,
                            moe_stream_t stream) {
    moe_status_t st = check_rows(rows, I, 1);
    if (st != MOE_OK) return st;
    if ((st = check_fp4(format, I, global_scale)) != MOE_OK) return st;
    if (rows == 0) return MOE_OK;
    if (gate_up == nullptr || act_codes == nullptr || act_scales == nullptr) return MOE_ERR_INVALID_ARG;
    if (!aligned16(gate_up) || !aligned16(act_codes)) return MOE_ERR_MISALIGNED;
    const uint64_t n = uint64_t(rows) * uint64_t(I);
    const uint64_t block = format == MOE_FP4_NVFP4 ? 16 : 32;
    if (any_overlap({{act_codes, n / 2}, {act_scales, n / block}}, {{gate_up, 4 * n}}))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if (current_sm_count(&sms) != cudaSuccess) return MOE_ERR_CUDA;
    return from_cuda(moe::launch_swiglu_fp4(gate_up, rows, I, format == MOE_FP4_NVFP4, global_scale, act_codes,
                                            act_scales, sms, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_expand_fp4(const moe_bf16_t* x, int64_t T, int H, int k, const int32_t* inv_perm,
                            int64_t rows, int format, float global_scale, uint8_t* codes,
                            uint8_t* scales, moe_stream_t stream) {
    if (k < 1) return MOE_ERR_INVALID_ARG;
    if (k > MOE_MAX_TOPK) return MOE_ERR_UNSUPPORTED;
    moe_status_t st = check_rows(T, H, k);
    if (st != MOE_OK) return st;
    if ((st = check_fp4(format, H, global_scale)) != MOE_OK) return st;
    if (rows < 0) return MOE_ERR_INVALID_ARG;
    if (rows >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
    if (T == 0 || rows == 0) return MOE_OK;
    if (x == nullptr || inv_perm == nullptr || codes == nullptr || scales == nullptr)
        return MOE_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(codes) || !aligned4(inv_perm)) return MOE_ERR_MISALIGNED;
    const uint64_t S = uint64_t(T) * uint64_t(k);
    const uint64_t n = uint64_t(rows) * uint64_t(H);
    const uint64_t block = format == MOE_FP4_NVFP4 ? 16 : 32;
    if (any_overlap({{codes, n / 2}, {scales, n / block}},
                    {{x, 2 * uint64_t(T) * uint64_t(H)}, {inv_perm, 4 * S}}))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if (current_sm_count(&sms) != cudaSuccess) return MOE_ERR_CUDA;
    return from_cuda(moe::launch_expand_fp4(x, T, H, k, inv_perm, rows, format == MOE_FP4_NVFP4, global_scale,
                                            codes, scales, sms, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_qk_rmsnorm(moe_bf16_t* q, moe_bf16_t* k, int64_t T, int num_q_heads,
                            int num_k_heads, int head_dim, const moe_bf16_t* q_weight,
                            const moe_bf16_t* k_weight, float weight_bias, float eps,
                            moe_stream_t stream) {
    if (T < 0 || num_q_heads < 0 || num_k_heads < 0 || num_q_heads + num_k_heads < 1)
        return MOE_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return MOE_ERR_UNSUPPORTED;
    if (T * int64_t(num_q_heads + num_k_heads) >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    if ((num_q_heads > 0 && q == nullptr) || (num_k_heads > 0 && k == nullptr) ||
        q_weight == nullptr || k_weight == nullptr)
        return MOE_ERR_INVALID_ARG;
    if ((num_q_heads > 0 && !aligned16(q)) || (num_k_heads > 0 && !aligned16(k)) ||
        !aligned16(q_weight) || !aligned16(k_weight))
        return MOE_ERR_MISALIGNED;
    const uint64_t qb = 2 * uint64_t(T) * uint64_t(num_q_heads) * uint64_t(head_dim);
    const uint64_t kb = 2 * uint64_t(T) * uint64_t(num_k_heads) * uint64_t(head_dim);
    if (any_overlap({{q, qb}, {k, kb}}, {{q_weight, 2ull * head_dim}, {k_weight, 2ull * head_dim}}))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if (current_sm_count(&sms) != cudaSuccess) return MOE_ERR_CUDA;
    return from_cuda(moe::launch_qk_rmsnorm(q, k, T, num_q_heads, num_k_heads, head_dim, q_weight,
                                            k_weight, weight_bias, eps, sms,
                                            reinterpret_cast<cudaStream_t>(stream)));
}

namespace {

// Common rules of the two norm calls. codes == NULL in the bfloat16 form.
moe_status_t add_rmsnorm(const moe_bf16_t* x, const moe_bf16_t* residual, int64_t T, int H,
                         const moe_bf16_t* weight, float weight_bias, float eps, moe_bf16_t* out,
                         moe_bf16_t* residual_out, uint8_t* codes, uint8_t* scales,
                         moe_stream_t stream) {
    if (residual == nullptr && residual_out != nullptr) return MOE_ERR_INVALID_ARG;
    if ((residual != nullptr && !aligned16(residual)) || (out != nullptr && !aligned16(out)) ||
        (residual_out != nullptr && !aligned16(residual_out)) || !aligned16(x) || !aligned16(weight) ||
        (codes != nullptr && !aligned16(codes)))
        return MOE_ERR_MISALIGNED;
    const uint64_t n = uint64_t(T) * uint64_t(H);
    const Range in_x{x, 2 * n}, in_w{weight, 2ull * H}, in_r{residual, residual != nullptr ? 2 * n : 0};
    const Range o_y{out, out != nullptr ? 2 * n : 0}, o_r{residual_out, residual_out != nullptr ? 2 * n : 0};
    const Range o_c{codes, codes != nullptr ? n : 0}, o_s{scales, codes != nullptr ? n / 32 : 0};
    if (any_overlap({o_y, o_r, o_c, o_s}, {in_x, in_w})) return MOE_ERR_INVALID_ARG;
    if (any_overlap({o_y, o_c, o_s}, {in_r})) return MOE_ERR_INVALID_ARG;
    if (residual_out != residual && overlap(o_r, in_r)) return MOE_ERR_INVALID_ARG;   // in place, or apart
    return from_cuda(moe::launch_add_rmsnorm(x, residual, T, H, weight, weight_bias, eps, out, residual_out,
                                             codes, scales, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

moe_status_t moe_add_rmsnorm(const moe_bf16_t* x, const moe_bf16_t* residual, int64_t T, int H,
                             const moe_bf16_t* weight, float weight_bias, float eps, moe_bf16_t* out,
                             moe_bf16_t* residual_out, moe_stream_t stream) {
    const moe_status_t st = check_rows(T, H, 1);
    if (st != MOE_OK) return st;
    if (!(eps >= 0.0f)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (x == nullptr || weight == nullptr || out == nullptr) return MOE_ERR_INVALID_ARG;
    return add_rmsnorm(x, residual, T, H, weight, weight_bias, eps, out, residual_out, nullptr, nullptr, stream);
}

moe_status_t moe_add_rmsnorm_mxfp8(const moe_bf16_t* x, const moe_bf16_t* residual, int64_t T, int H,
                                   const moe_bf16_t* weight, float weight_bias, float eps,
                                   uint8_t* codes, uint8_t* scales, moe_bf16_t* out,
                                   moe_bf16_t* residual_out, moe_stream_t stream) {
    const moe_status_t st = check_rows(T, H, 1);
    if (st != MOE_OK) return st;
    if (H % 32 != 0) return MOE_ERR_MISALIGNED;
    if (!(eps >= 0.0f)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (x == nullptr || weight == nullptr || codes == nullptr || scales == nullptr) return MOE_ERR_INVALID_ARG;
    return add_rmsnorm(x, residual, T, H, weight, weight_bias, eps, out, residual_out, codes, scales, stream);
}

namespace {

// Sizes of the products for a few tokens: T <= MOE_FEW_MAX_TOKENS, widths up
// to 2^20 (32-bit offsets inside a row).
moe_status_t check_few(int64_t T, int64_t width) {
    if (T < 0 || width < 1) return MOE_ERR_INVALID_ARG;
    if (T > MOE_FEW_MAX_TOKENS || width > (1 << 20)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

uint64_t fp4_scales(uint64_t values, int format) { return values / (format == MOE_FP4_NVFP4 ? 16 : 32); }

}  // namespace

moe_status_t moe_gemv_fp4(const moe_bf16_t* x, int64_t T, int K, const uint8_t* codes,
                          const uint8_t* scales, int N, int format, float global_scale, void* y,
                          int y_float32, moe_stream_t stream) {
    moe_status_t st = check_few(T, K);
    if (st != MOE_OK) return st;
    if (N < 1) return MOE_ERR_INVALID_ARG;
    if ((st = check_fp4(format, K, global_scale)) != MOE_OK) return st;
    if (K % 32 != 0) return MOE_ERR_MISALIGNED;   // a row of codes is whole 16-byte vectors
    if (T == 0) return MOE_OK;
    if (x == nullptr || codes == nullptr || scales == nullptr || y == nullptr) return MOE_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(codes) || !aligned16(scales) || !aligned4(y)) return MOE_ERR_MISALIGNED;
    const uint64_t n = uint64_t(N) * uint64_t(K);
    if (any_overlap({{y, (y_float32 ? 4ull : 2ull) * uint64_t(T) * uint64_t(N)}},
                    {{x, 2 * uint64_t(T) * uint64_t(K)}, {codes, n / 2}, {scales, fp4_scales(n, format)}}))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if (current_sm_count(&sms) != cudaSuccess) return MOE_ERR_CUDA;
    return from_cuda(moe::launch_gemv_fp4(x, int(T), K, codes, scales, N, format == MOE_FP4_NVFP4, global_scale, y,
                                          y_float32 != 0, sms, reinterpret_cast<cudaStream_t>(stream)));
}

namespace {

moe_status_t check_layer_sizes(int64_t T, int E, int k, int H, int I) {
    moe_status_t st = check_route_sizes(T, E, k);
    if (st != MOE_OK) return st;
    if ((st = check_few(T, H)) != MOE_OK) return st;
    if ((st = check_few(T, I)) != MOE_OK) return st;
    if (H % 8 != 0 || I % 8 != 0) return MOE_ERR_MISALIGNED;
    return MOE_OK;
}

// The activation [T k, I] in 16 bits, an exponent for every 8 of it (4-bit
// weights; padded to whole 16 bytes), then the routing that fc1 leaves for fc2.
uint64_t layer_act(int64_t T, int k, int I) { return 2 * uint64_t(T) * uint64_t(k) * uint64_t(I); }
uint64_t layer_exps(int64_t T, int k, int I) { return (layer_act(T, k, I) / 16 + 15) / 16 * 16; }
uint64_t layer_workspace(int64_t T, int k, int I) { return layer_act(T, k, I) + layer_exps(T, k, I) + moe::kFewRouteBytes; }

using LayerLaunch = cudaError_t (*)(const moe::LayerArgs&, int, cudaStream_t);

// Everything of a layer call but its weights; `weights` are their ranges.
moe_status_t run_layer(moe::LayerArgs& a, LayerLaunch launch, const float* logits, int64_t T, int E, int k,
                       int renorm, const moe_bf16_t* x, int H, int I, moe_bf16_t* out, int32_t* topk_ids,
                       float* topk_weights, void* workspace, size_t workspace_bytes, moe_stream_t stream,
                       std::initializer_list<Range> weights) {
    if (logits == nullptr || x == nullptr || out == nullptr) return MOE_ERR_INVALID_ARG;
    if (!aligned4(logits) || !aligned16(x) || !aligned16(out) || (topk_ids != nullptr && !aligned4(topk_ids)) ||
        (topk_weights != nullptr && !aligned4(topk_weights)))
        return MOE_ERR_MISALIGNED;
    const uint64_t S = uint64_t(T) * uint64_t(k), need = layer_workspace(T, k, I);
    if (workspace == nullptr || workspace_bytes < need) return MOE_ERR_WORKSPACE;
    if (!aligned16(workspace)) return MOE_ERR_MISALIGNED;
    const Range o_out{out, 2 * uint64_t(T) * H}, o_id{topk_ids, topk_ids != nullptr ? 4 * S : 0},
        o_w{topk_weights, topk_weights != nullptr ? 4 * S : 0}, o_ws{workspace, need};
    if (any_overlap({o_out, o_id, o_w, o_ws}, {{logits, 4ull * uint64_t(T) * E}, {x, 2 * uint64_t(T) * H}}) ||
        any_overlap({o_out, o_id, o_w, o_ws}, weights))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if (current_sm_count(&sms) != cudaSuccess) return MOE_ERR_CUDA;
    a.logits = logits;
    a.x = x;
    a.out = out;
    a.topk_ids = topk_ids;
    a.topk_weights = topk_weights;
    a.act = static_cast<uint16_t*>(workspace);
    a.act_exps = static_cast<uint8_t*>(workspace) + layer_act(T, k, I);
    a.route = a.act_exps + layer_exps(T, k, I);
    a.T = int(T); a.E = E; a.k = k; a.renorm = renorm ? 1 : 0; a.H = H; a.I = I;
    return from_cuda(launch(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

moe_status_t moe_layer_workspace_size(int64_t T, int E, int k, int H, int I, size_t* bytes) {
    if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check_layer_sizes(T, E, k, H, I);
    if (st != MOE_OK) return st;
    *bytes = T == 0 ? 0 : layer_workspace(T, k, I);
    return MOE_OK;
}

moe_status_t moe_layer(const float* logits, int64_t T, int E, int k, int renorm, const moe_bf16_t* x, int H,
                       int I, const moe_bf16_t* w13, const moe_bf16_t* w2, moe_bf16_t* out,
                       int32_t* topk_ids, float* topk_weights, void* workspace, size_t workspace_bytes,
                       moe_stream_t stream) {
    const moe_status_t st = check_layer_sizes(T, E, k, H, I);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    if (w13 == nullptr || w2 == nullptr) return MOE_ERR_INVALID_ARG;
    if (!aligned16(w13) || !aligned16(w2)) return MOE_ERR_MISALIGNED;
    const uint64_t n = uint64_t(E) * uint64_t(H) * uint64_t(I);
    moe::LayerArgs a = {};
    a.w13 = w13;
    a.w2 = w2;
    return run_layer(a, moe::launch_layer_bf16, logits, T, E, k, renorm, x, H, I, out, topk_ids, topk_weights, workspace,
                     workspace_bytes, stream, {{w13, 4 * n}, {w2, 2 * n}});
}

moe_status_t moe_layer_fp4(const float* logits, int64_t T, int E, int k, int renorm, const moe_bf16_t* x, int H,
                           int I, int format, const uint8_t* w13_codes, const uint8_t* w13_scales,
                           const float* w13_global, const uint8_t* w2_codes, const uint8_t* w2_scales,
                           const float* w2_global, moe_bf16_t* out, int32_t* topk_ids, float* topk_weights,
                           void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    const moe_status_t st = check_layer_sizes(T, E, k, H, I);
    if (st != MOE_OK) return st;
    if (format != MOE_FP4_NVFP4 && format != MOE_FP4_MXFP4) return MOE_ERR_INVALID_ARG;
    if (H % 32 != 0 || I % 32 != 0) return MOE_ERR_MISALIGNED;
    if (T == 0) return MOE_OK;
    if (w13_codes == nullptr || w13_scales == nullptr || w2_codes == nullptr || w2_scales == nullptr)
        return MOE_ERR_INVALID_ARG;
    const bool nv = format == MOE_FP4_NVFP4;
    if (nv && (w13_global == nullptr || w2_global == nullptr)) return MOE_ERR_INVALID_ARG;
    if (!aligned16(w13_codes) || !aligned16(w13_scales) || !aligned16(w2_codes) || !aligned16(w2_scales) ||
        (nv && (!aligned4(w13_global) || !aligned4(w2_global))))
        return MOE_ERR_MISALIGNED;
    const uint64_t n = uint64_t(E) * uint64_t(H) * uint64_t(I), gb = nv ? 4ull * E : 0;
    moe::LayerArgs a = {};
    a.w13 = w13_codes;
    a.w2 = w2_codes;
    a.w13_scales = w13_scales;
    a.w2_scales = w2_scales;
    a.w13_global = w13_global;
    a.w2_global = w2_global;
    return run_layer(a, nv ? moe::launch_layer_nvfp4 : moe::launch_layer_mxfp4, logits, T, E, k, renorm, x, H, I, out, topk_ids,
                     topk_weights, workspace, workspace_bytes, stream,
                     {{w13_codes, n}, {w13_scales, fp4_scales(2 * n, format)}, {w2_codes, n / 2},
                      {w2_scales, fp4_scales(n, format)}, {w13_global, gb}, {w2_global, gb}});
}

namespace {

bool power_of_two(int64_t v) { return v > 0 && (v & (v - 1)) == 0; }

int log2_of(int64_t v) {
    int s = 0;
    while ((int64_t(1) << s) < v) ++s;
    return s;
}

static_assert(moe::kMaxRequests == MOE_MAX_REQUESTS, "the kernels' shared memory is for as many requests as the header allows");

moe_status_t check_pages(int64_t B, int page_size, int max_pages) {
    if (B < 0 || page_size < 1 || max_pages < 1) return MOE_ERR_INVALID_ARG;
    if (!power_of_two(page_size) || page_size > MOE_KV_MAX_PAGE_SIZE) return MOE_ERR_UNSUPPORTED;
    if (int64_t(max_pages) * page_size > (int64_t(1) << 30)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

bool usable_scale(float s) { return s >= 0x1p-126f && s <= 0x1p126f; }   // so is its reciprocal

// The address range of one side of a cache.
moe_status_t cache_range(const void* p, int64_t pages, int64_t page, int64_t tokens, int64_t token, int64_t heads,
                         int64_t head, int64_t row_bytes, int esz, Range* out) {
    if (page < 0 || token < 0 || head < 0) return MOE_ERR_INVALID_ARG;
    const int vec = 16 / esz;
    if (page % vec != 0 || token % vec != 0 || head % vec != 0 || !aligned16(p)) return MOE_ERR_MISALIGNED;
    uint64_t last = 0;
    for (const auto& d : {std::pair<int64_t, int64_t>{pages, page}, {tokens, token}, {heads, head}}) {
        uint64_t step = 0;
        if (__builtin_mul_overflow(uint64_t(d.first - 1), uint64_t(d.second) * esz, &step) || step >> 56 != 0)
            return MOE_ERR_UNSUPPORTED;
        last += step;
    }
    *out = {p, last + uint64_t(row_bytes)};
    return MOE_OK;
}

// The rules of a cache, its view for the kernels and its two address ranges.
moe_status_t check_cache(const moe_kv_cache_t* c, moe::CacheView* view, Range* k, Range* v) {
    if (c == nullptr || c->num_pages < 1 || c->num_heads < 1 || c->page_size < 1) return MOE_ERR_INVALID_ARG;
    if (c->type != MOE_KV_BF16 && c->type != MOE_KV_E4M3) return MOE_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return MOE_ERR_UNSUPPORTED;
    if (!power_of_two(c->page_size) || c->page_size > MOE_KV_MAX_PAGE_SIZE) return MOE_ERR_UNSUPPORTED;
    if (c->num_pages >= (int64_t(1) << 31) || c->num_heads > 1024) return MOE_ERR_UNSUPPORTED;
    if (!usable_scale(c->k_scale) || !usable_scale(c->v_scale)) return MOE_ERR_INVALID_ARG;
    if (c->type == MOE_KV_BF16 && (c->k_scale != 1.0f || c->v_scale != 1.0f)) return MOE_ERR_INVALID_ARG;
    if (c->k == nullptr || c->v == nullptr) return MOE_ERR_INVALID_ARG;
    const int esz = c->type == MOE_KV_E4M3 ? 1 : 2;
    moe_status_t st = cache_range(c->k, c->num_pages, c->k_page_stride, c->page_size, c->k_token_stride, c->num_heads,
                                  c->k_head_stride, int64_t(c->head_dim) * esz, esz, k);
    if (st != MOE_OK) return st;
    st = cache_range(c->v, c->num_pages, c->v_page_stride, c->page_size, c->v_token_stride, c->num_heads,
                     c->v_head_stride, int64_t(c->head_dim) * esz, esz, v);
    if (st != MOE_OK) return st;
    view->k = static_cast<uint8_t*>(c->k);
    view->v = static_cast<uint8_t*>(c->v);
    view->k_page = c->k_page_stride * esz;
    view->k_token = c->k_token_stride * esz;
    view->k_head = c->k_head_stride * esz;
    view->v_page = c->v_page_stride * esz;
    view->v_token = c->v_token_stride * esz;
    view->v_head = c->v_head_stride * esz;
    view->num_pages = c->num_pages;
    view->page_shift = log2_of(c->page_size);
    view->heads = c->num_heads;
    view->head_dim = c->head_dim;
    view->e4m3 = c->type == MOE_KV_E4M3;
    view->k_scale = c->k_scale;
    view->v_scale = c->v_scale;
    return MOE_OK;
}

// Rows of heads * D bfloat16 values, `stride` elements apart.
moe_status_t check_strided(const void* p, int64_t n, int64_t heads, int D, int64_t stride, Range* out) {
    const int64_t row = heads * D;
    if (p == nullptr || stride < row) return MOE_ERR_INVALID_ARG;
    if (stride % 8 != 0 || !aligned16(p)) return MOE_ERR_MISALIGNED;
    if (stride >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
    *out = {p, 2 * (uint64_t(n - 1) * uint64_t(stride) + uint64_t(row))};
    return MOE_OK;
}

}  // namespace

moe_status_t moe_page_table(const int32_t* cached, const int32_t* added, int64_t B, int page_size, int max_pages,
                            int64_t max_tokens, const int32_t* free_pages, int64_t free_capacity,
                            const int32_t* free_count, int32_t* block_table, int32_t* lengths, int32_t* starts,
                            int32_t* positions, int64_t* slots, int32_t* free_count_out, int32_t* refused,
                            moe_stream_t stream) {
    const moe_status_t st = check_pages(B, page_size, max_pages);
    if (st != MOE_OK) return st;
    if (max_tokens < 0 || free_capacity < 0) return MOE_ERR_INVALID_ARG;
    if (B > MOE_MAX_REQUESTS || max_tokens >= (int64_t(1) << 31) || free_capacity >= (int64_t(1) << 31))
        return MOE_ERR_UNSUPPORTED;
    if ((B > 0 && (cached == nullptr || added == nullptr || block_table == nullptr || lengths == nullptr)) ||
        (max_tokens > 0 && (positions == nullptr || slots == nullptr)) || (free_capacity > 0 && free_pages == nullptr) ||
        free_count == nullptr || free_count_out == nullptr || starts == nullptr)
        return MOE_ERR_INVALID_ARG;
    for (const void* p : std::initializer_list<const void*>{cached, added, free_pages, free_count, block_table, lengths,
                                                            starts, positions, free_count_out, refused})
        if (!aligned4(p)) return MOE_ERR_MISALIGNED;
    if ((reinterpret_cast<uintptr_t>(slots) & 7u) != 0) return MOE_ERR_MISALIGNED;
    const uint64_t b4 = 4 * uint64_t(B), n = uint64_t(max_tokens);
    const Range i_c{cached, b4}, i_a{added, b4}, i_p{free_pages, 4 * uint64_t(free_capacity)}, i_f{free_count, 4};
    const Range o_t{block_table, b4 * uint64_t(max_pages)}, o_l{lengths, b4}, o_s{starts, b4 + 4}, o_p{positions, 4 * n},
        o_q{slots, 8 * n}, o_f{free_count_out, 4}, o_r{refused, refused != nullptr ? 4u : 0u};
    if (any_overlap({o_t, o_l, o_s, o_p, o_q, o_f, o_r}, {i_a, i_p}) || any_overlap({o_t, o_s, o_p, o_q, o_r}, {i_c, i_f}) ||
        overlap(o_l, i_f) || overlap(o_f, i_c) || (lengths != cached && overlap(o_l, i_c)))
        return MOE_ERR_INVALID_ARG;
    moe::PageTableArgs a = {};
    a.cached = cached;
    a.added = added;
    a.free_pages = free_pages;
    a.free_count = free_count;
    a.block_table = block_table;
    a.lengths = lengths;
    a.starts = starts;
    a.positions = positions;
    a.slots = slots;
    a.free_count_out = free_count_out;
    a.refused = refused;
    a.free_capacity = free_capacity;
    a.B = int(B);
    a.page_shift = log2_of(page_size);
    a.max_pages = max_pages;
    a.max_tokens = int(max_tokens);
    return from_cuda(moe::launch_page_table(a, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_page_release(const int32_t* finished, int64_t B, int page_size, int max_pages,
                              const int32_t* block_table, int32_t* lengths, int32_t* free_pages,
                              int64_t free_capacity, int32_t* free_count, moe_stream_t stream) {
    const moe_status_t st = check_pages(B, page_size, max_pages);
    if (st != MOE_OK) return st;
    if (free_capacity < 0) return MOE_ERR_INVALID_ARG;
    if (B > MOE_MAX_REQUESTS || free_capacity >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
    if (B == 0) return MOE_OK;
    if (finished == nullptr || block_table == nullptr || lengths == nullptr || free_count == nullptr ||
        (free_capacity > 0 && free_pages == nullptr))
        return MOE_ERR_INVALID_ARG;
    for (const void* p : std::initializer_list<const void*>{finished, block_table, lengths, free_pages, free_count})
        if (!aligned4(p)) return MOE_ERR_MISALIGNED;
    const uint64_t b4 = 4 * uint64_t(B);
    if (any_overlap({{lengths, b4}, {free_pages, 4 * uint64_t(free_capacity)}, {free_count, 4}},
                    {{finished, b4}, {block_table, b4 * uint64_t(max_pages)}}))
        return MOE_ERR_INVALID_ARG;
    moe::PageReleaseArgs a = {};
    a.finished = finished;
    a.block_table = block_table;
    a.lengths = lengths;
    a.free_pages = free_pages;
    a.free_count = free_count;
    a.free_capacity = free_capacity;
    a.B = int(B);
    a.page_shift = log2_of(page_size);
    a.max_pages = max_pages;
    return from_cuda(moe::launch_page_release(a, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_kv_append(const moe_bf16_t* q, int64_t q_stride, const moe_bf16_t* k, int64_t k_stride,
                           const moe_bf16_t* v, int64_t v_stride, int64_t N, int num_q_heads,
                           const int32_t* positions, const int64_t* slots, const float* cos_sin,
                           int64_t max_positions, int rot, int interleaved, const moe_kv_cache_t* cache,
                           moe_bf16_t* q_out, int64_t q_out_stride, moe_bf16_t* k_out, int64_t k_out_stride,
                           moe_stream_t stream) {
    moe::AppendArgs a = {};
    Range ck, cv;
    moe_status_t st = check_cache(cache, &a.cache, &ck, &cv);
    if (st != MOE_OK) return st;
    const int D = cache->head_dim;
    if (N < 0 || num_q_heads < 0 || rot < 0 || rot > D || max_positions < 0 || (rot > 0 && max_positions < 1))
        return MOE_ERR_INVALID_ARG;
    if (rot % 16 != 0) return MOE_ERR_MISALIGNED;
    if (N >= (int64_t(1) << 31) || num_q_heads > 1024 || max_positions > (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
    if (N == 0) return MOE_OK;
    if (slots == nullptr || (rot > 0 && (positions == nullptr || cos_sin == nullptr))) return MOE_ERR_INVALID_ARG;
    Range i_q{nullptr, 0}, i_k, i_v, o_q{nullptr, 0}, o_k{nullptr, 0};
    if (num_q_heads > 0) {
        if ((st = check_strided(q, N, num_q_heads, D, q_stride, &i_q)) != MOE_OK) return st;
        if ((st = check_strided(q_out, N, num_q_heads, D, q_out_stride, &o_q)) != MOE_OK) return st;
    }
    if ((st = check_strided(k, N, cache->num_heads, D, k_stride, &i_k)) != MOE_OK) return st;
    if ((st = check_strided(v, N, cache->num_heads, D, v_stride, &i_v)) != MOE_OK) return st;
    if (k_out != nullptr && (st = check_strided(k_out, N, cache->num_heads, D, k_out_stride, &o_k)) != MOE_OK) return st;
    if ((reinterpret_cast<uintptr_t>(slots) & 7u) != 0 || (rot > 0 && (!aligned4(positions) || !aligned16(cos_sin))))
        return MOE_ERR_MISALIGNED;
    const Range i_s{slots, 8 * uint64_t(N)}, i_p{positions, rot > 0 ? 4 * uint64_t(N) : 0},
        i_c{cos_sin, 4 * uint64_t(max_positions) * uint64_t(rot)};
    // Slices of one array interleave: row by row, an output may lie beside an
    // input, so only arrays with the same stride can be told apart by their rows.
    const auto apart = [](Range x, int64_t xs, int xh, Range y, int64_t ys, int yh, int D) {
        if (!overlap(x, y)) return true;
        if (xs != ys) return false;
        const int64_t d = (reinterpret_cast<intptr_t>(y.p) - reinterpret_cast<intptr_t>(x.p)) / 2;
        const int64_t at = ((d % xs) + xs) % xs;   // y's row begins here inside x's stride
        return at >= int64_t(xh) * D && at + int64_t(yh) * D <= xs;
    };
    const int kh = cache->num_heads;
    const bool q_in_place = q_out == q && q_out_stride == q_stride, k_in_place = k_out == k && k_out_stride == k_stride;
    if (num_q_heads > 0 &&
        ((!q_in_place && !apart(o_q, q_out_stride, num_q_heads, i_q, q_stride, num_q_heads, D)) ||
         !apart(o_q, q_out_stride, num_q_heads, i_k, k_stride, kh, D) ||
         !apart(o_q, q_out_stride, num_q_heads, i_v, v_stride, kh, D)))
        return MOE_ERR_INVALID_ARG;
    if (k_out != nullptr &&
        ((!k_in_place && !apart(o_k, k_out_stride, kh, i_k, k_stride, kh, D)) ||
         (num_q_heads > 0 && (!apart(o_k, k_out_stride, kh, i_q, q_stride, num_q_heads, D) ||
                              !apart(o_k, k_out_stride, kh, o_q, q_out_stride, num_q_heads, D))) ||
         !apart(o_k, k_out_stride, kh, i_v, v_stride, kh, D)))
        return MOE_ERR_INVALID_ARG;
    for (const Range& c : {ck, cv})
        for (const Range& r : {i_q, i_k, i_v, o_q, o_k, i_s, i_p, i_c})
            if (overlap(c, r)) return MOE_ERR_INVALID_ARG;
    for (const Range& o : {o_q, o_k})
        for (const Range& r : {i_s, i_p, i_c})
            if (overlap(o, r)) return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if (current_sm_count(&sms) != cudaSuccess) return MOE_ERR_CUDA;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_out = q_out;
    a.k_out = k_out;
    a.positions = positions;
    a.slots = slots;
    a.cos_sin = cos_sin;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_out_stride = q_out_stride;
    a.k_out_stride = k_out_stride;
    a.max_positions = max_positions;
    a.N = int(N);
    a.q_heads = num_q_heads;
    a.rot = rot;
    a.interleaved = interleaved != 0;
    return from_cuda(moe::launch_kv_append(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

namespace {

moe_status_t check_attention_sizes(int64_t B, int num_q_heads, int num_heads, int head_dim) {
    if (B < 0 || num_q_heads < 1 || num_heads < 1 || num_q_heads % num_heads != 0) return MOE_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return MOE_ERR_UNSUPPORTED;
    if (B >= (int64_t(1) << 24) || num_q_heads > 1024) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

}  // namespace

moe_status_t moe_paged_attention_workspace_size(int64_t B, int num_q_heads, int num_heads, int head_dim,
                                                size_t* bytes) {
    if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check_attention_sizes(B, num_q_heads, num_heads, head_dim);
    if (st != MOE_OK) return st;
    *bytes = B == 0 ? 0 : moe::paged_attention_workspace(B, num_q_heads, num_heads, head_dim);
    return MOE_OK;
}

moe_status_t moe_paged_attention(const moe_bf16_t* q, int64_t q_stride, int64_t B, int num_q_heads,
                                 const moe_kv_cache_t* cache, const int32_t* block_table, int max_pages,
                                 const int32_t* lengths, int window, float scale, moe_bf16_t* out, float* lse,
                                 void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    moe::AttentionArgs a = {};
    Range ck, cv, i_q;
    moe_status_t st = check_cache(cache, &a.cache, &ck, &cv);
    if (st != MOE_OK) return st;
    if ((st = check_attention_sizes(B, num_q_heads, cache->num_heads, cache->head_dim)) != MOE_OK) return st;
    if ((st = check_pages(B, cache->page_size, max_pages)) != MOE_OK) return st;
    if (window < 0 || !(scale >= -3.402823466e38f && scale <= 3.402823466e38f)) return MOE_ERR_INVALID_ARG;
    if (B == 0) return MOE_OK;
    const int D = cache->head_dim;
    if ((st = check_strided(q, B, num_q_heads, D, q_stride, &i_q)) != MOE_OK) return st;
    if (block_table == nullptr || lengths == nullptr || out == nullptr) return MOE_ERR_INVALID_ARG;
    if (!aligned4(block_table) || !aligned4(lengths) || !aligned16(out) || !aligned4(lse)) return MOE_ERR_MISALIGNED;
    const uint64_t need = moe::paged_attention_workspace(B, num_q_heads, cache->num_heads, D);
    if (workspace == nullptr || workspace_bytes < need) return MOE_ERR_WORKSPACE;
    if (!aligned16(workspace)) return MOE_ERR_MISALIGNED;
    const uint64_t heads = uint64_t(B) * uint64_t(num_q_heads);
    if (any_overlap({{out, 2 * heads * D}, {lse, lse != nullptr ? 4 * heads : 0}, {workspace, need}},
                    {i_q, ck, cv, {block_table, 4 * uint64_t(B) * uint64_t(max_pages)}, {lengths, 4 * uint64_t(B)}}))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if (current_sm_count(&sms) != cudaSuccess) return MOE_ERR_CUDA;
    a.q = q;
    a.block_table = block_table;
    a.lengths = lengths;
    a.out = out;
    a.lse = lse;
    a.workspace = workspace;
    a.q_stride = q_stride;
    a.B = int(B);
    a.q_heads = num_q_heads;
    a.max_pages = max_pages;
    a.window = window;
    a.scale = scale;
    return from_cuda(moe::launch_paged_attention(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
