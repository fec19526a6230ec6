// Host-side interface between the C-ABI layer (api.cu) and the kernel
// translation units. Not installed; not part of the public ABI.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace moe {

// Launch geometry of the routing step, a pure function of (T, E, k).
struct RoutePlan {
    int gs = 32;        // lanes that cooperate on one token (8, 16 or 32)
    int epl = 1;        // experts held per lane: E <= gs * epl
    bool fused = false; // one block does everything (small T)
    int nt = 512;       // threads per block
    int G = 1;          // blocks of the two-kernel path
    int tpc = 0;        // tokens per block
    int tpw = 0;        // tokens per warp (contiguous run inside the block)
    int Ep = 0;         // E rounded up to a multiple of 4 (row stride of the count matrix)
    size_t ws_bytes = 0;
    size_t smem_topk = 0;
    size_t smem_scatter = 0;
};

// nloc: number of counted experts (0 = all E); it sets the count-matrix width.
RoutePlan plan_route(int64_t T, int E, int k, int nloc = 0);

// A local routing: experts [e0, e0 + n) are counted, their segments padded
// to a multiple of pad, perm has `rows` entries.
struct LocalRange {
    int e0, n, pad, rows;
};

cudaError_t launch_route(const RoutePlan& plan, const float* logits, int T, int E, int k,
                         int renorm, int32_t* topk_ids, float* topk_weights,
                         int32_t* expert_counts, int32_t* expert_offsets, int32_t* perm,
                         int32_t* inv_perm, void* workspace, cudaStream_t stream,
                         const LocalRange* local = nullptr);

// One-launch route + expand for decode-sized batches (route_expand.cu).
bool route_expand_fits(const RoutePlan& plan);
cudaError_t launch_route_expand(const RoutePlan& plan, const float* logits, int T, int E, int k,
                                int renorm, int32_t* topk_ids, float* topk_weights,
                                int32_t* expert_counts, int32_t* expert_offsets, int32_t* perm,
                                int32_t* inv_perm, const uint16_t* x, int H, uint16_t* expanded_x,
                                int num_sms, cudaStream_t stream);

// rows: rows of expanded_x (T*k, or a padded local capacity); inv_perm
// entries outside [0, rows) are skipped.
cudaError_t launch_expand(const uint16_t* x, int64_t T, int H, int k, const int32_t* inv_perm,
                          int64_t rows, uint16_t* expanded_x, int num_sms, cudaStream_t stream);

cudaError_t launch_swiglu(const uint16_t* gate_up, int64_t rows, int I, uint16_t* act,
                          int num_sms, cudaStream_t stream);

// rows: rows of expert_out; inv_perm entries outside [0, rows) contribute nothing.
cudaError_t launch_combine(const uint16_t* expert_out, int64_t rows, int64_t T, int H, int k,
                           const float* topk_weights, const int32_t* inv_perm, uint16_t* out,
                           int num_sms, cudaStream_t stream);

// SwiGLU / expand with MXFP8 outputs (quant.cu): codes [rows, n] E4M3 bytes,
// scales [rows, n/32] E8M0 bytes; n (I or H) a multiple of 32.
cudaError_t launch_swiglu_mxfp8(const uint16_t* gate_up, int64_t rows, int I, uint8_t* codes,
                                uint8_t* scales, int num_sms, cudaStream_t stream);
cudaError_t launch_expand_mxfp8(const uint16_t* x, int64_t T, int H, int k, const int32_t* inv_perm,
                                int64_t rows, uint8_t* codes, uint8_t* scales, int num_sms,
                                cudaStream_t stream);
// FP4 outputs: NVFP4 (nvfp4, tensor scale g) or MXFP4.
cudaError_t launch_swiglu_fp4(const uint16_t* gate_up, int64_t rows, int I, bool nvfp4, float g,
                              uint8_t* codes, uint8_t* scales, int num_sms, cudaStream_t stream);
cudaError_t launch_expand_fp4(const uint16_t* x, int64_t T, int H, int k, const int32_t* inv_perm,
                              int64_t rows, bool nvfp4, float g, uint8_t* codes, uint8_t* scales,
                              int num_sms, cudaStream_t stream);

// Per-head RMSNorm of q [T, nq, head_dim] and k [T, nk, head_dim] in place
// (qknorm.cu); head_dim 64, 128 or 256.
cudaError_t launch_qk_rmsnorm(uint16_t* q, uint16_t* k, int64_t T, int nq, int nk, int head_dim,
                              const uint16_t* qw, const uint16_t* kw, float bias, float eps,
                              int num_sms, cudaStream_t stream);

// RMS norm of rows with the residual's addition (rmsnorm.cu): residual,
// out and residual_out may be NULL; codes != NULL adds the MXFP8 output.
cudaError_t launch_add_rmsnorm(const uint16_t* x, const uint16_t* residual, int64_t T, int H,
                               const uint16_t* weight, float bias, float eps, uint16_t* out,
                               uint16_t* residual_out, uint8_t* codes, uint8_t* scales,
                               cudaStream_t stream);

// Products of T <= 32 tokens x [T, K] with 4-bit weights [N, K] (gemv_fp4.cu).
cudaError_t launch_gemv_fp4(const uint16_t* x, int T, int K, const uint8_t* codes, const uint8_t* scales,
                            int N, bool nvfp4, float g, void* y, bool y_f32, int num_sms,
                            cudaStream_t stream);

// A whole MoE layer for T <= 32 tokens (layer_bf16.cu, layer_fp4.cuh). Weights:
// bfloat16 (w13, w2), or codes with scales and, for NVFP4, a tensor scale per
// expert. kFewRouteBytes: the routing that fc1 leaves for fc2 (few_route.cuh).
constexpr size_t kFewRouteBytes = 4624;
struct LayerArgs {
    const float* logits;
    const uint16_t* x;
    const void* w13;
    const void* w2;
    const uint8_t* w13_scales;   // 4-bit weights only
    const uint8_t* w2_scales;
    const float* w13_global;     // NVFP4 only, [E]
    const float* w2_global;
    uint16_t* out;
    int32_t* topk_ids;           // may be NULL
    float* topk_weights;         // may be NULL
    uint16_t* act;               // workspace [T*k, I]: bfloat16; f16 for 4-bit weights
    uint8_t* act_exps;           // workspace [T*k, I/8] (4-bit weights): exponents of 8 columns' f16
    void* route;                 // workspace, kFewRouteBytes
    int T, E, k, renorm, H, I;
};
cudaError_t launch_layer_bf16(const LayerArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_layer_nvfp4(const LayerArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_layer_mxfp4(const LayerArgs& a, int num_sms, cudaStream_t stream);

// Block tables and slot maps (page_table.cu). Sums over the requests are 64-bit.
constexpr int kMaxRequests = 16384;   // MOE_MAX_REQUESTS (checked in api.cu and page_table.cu)
struct PageTableArgs {
    const int32_t* cached;       // may be lengths
    const int32_t* added;
    const int32_t* free_pages;
    const int32_t* free_count;   // may be free_count_out
    int32_t* block_table;
    int32_t* lengths;
    int32_t* starts;
    int32_t* positions;
    int64_t* slots;
    int32_t* free_count_out;
    int32_t* refused;            // may be NULL
    int64_t free_capacity;
    int B, page_shift, max_pages, max_tokens;
};
cudaError_t launch_page_table(const PageTableArgs& a, cudaStream_t stream);
struct PageReleaseArgs {
    const int32_t* finished;
    const int32_t* block_table;
    int32_t* lengths;
    int32_t* free_pages;
    int32_t* free_count;
    int64_t free_capacity;
    int B, page_shift, max_pages;
};
cudaError_t launch_page_release(const PageReleaseArgs& a, cudaStream_t stream);

// A paged key-value cache as the kernels see it: strides in bytes.
struct CacheView {
    uint8_t* k;
    uint8_t* v;
    int64_t k_page, k_token, k_head;
    int64_t v_page, v_token, v_head;
    int64_t num_pages;
    int page_shift, heads, head_dim;
    bool e4m3;
    float k_scale, v_scale;
};

// Rotary embedding and the cache's writes (kv_append.cu).
struct AppendArgs {
    CacheView cache;
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    uint16_t* q_out;
    uint16_t* k_out;             // may be NULL
    const int32_t* positions;
    const int64_t* slots;
    const float* cos_sin;
    int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;   // elements
    int64_t max_positions;
    int N, q_heads, rot;
    bool interleaved;
};
cudaError_t launch_kv_append(const AppendArgs& a, int num_sms, cudaStream_t stream);

// Attention of one token per sequence over the cache (paged_attention.cu).
struct AttentionArgs {
    CacheView cache;
    const uint16_t* q;
    const int32_t* block_table;
    const int32_t* lengths;
    uint16_t* out;
    float* lse;                  // may be NULL
    void* workspace;
    int64_t q_stride;            // elements
    int B, q_heads, max_pages, window;
    float scale;
    float score, score_up;       // set by the launch: their product is scale * k_scale * log2 e
};
size_t paged_attention_workspace(int64_t B, int q_heads, int heads, int head_dim);
cudaError_t launch_paged_attention(const AttentionArgs& a, int num_sms, cudaStream_t stream);

}  // namespace moe
