// Parameters and host-side entry points of the serving kernels (internal to libgqa_serve.so).
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

namespace gqa {

// ---------------------------------------------------------------- cache pages
struct CacheState {
    int* table;  // [S, M]
    int* lens;   // [S]
    int* refs;   // [P]
    int S, M, P;
    int page_shift;  // log2(page size)
};

// gqa_cache_resize: key = slots (NULL: 0..n-1), arg = new lengths.
// gqa_cache_fork: key = children, arg = parents.
struct PlanParams {
    CacheState c;
    const int* key;
    const int* arg;
    int n;
    int* status;
};

// The pools [layers, P, page, row_bytes] of both tensors.
struct Pools {
    uint8_t* kv[2];
    long long row_bytes;
    int layers;
};

struct CompactParams {
    CacheState c;
    Pools pools;
    const int* keep;  // [S, T]
    const int* keep_lens;
    const int* tree_lens;  // NULL: T nodes
    int T;
    int* status;
};

cudaError_t launch_resize(const PlanParams& p, cudaStream_t stream);
cudaError_t launch_fork(const PlanParams& p, const Pools& pools, int sms, cudaStream_t stream);
cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream);

// ---------------------------------------------------------------- attention
struct AttnParams {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    long long q_stride, k_stride, v_stride;  // elements between rows
    void* out;
    bool out_bf16;
    float* lse;
    int B, Hq, Hk, d;
    float scale;
    // packed prompts
    const int* cu_q;
    const int* cu_k;
    int total_q, total_k;
    int causal;
    // tree over a cache
    const int* table;  // NULL: dense [B, Sk, Hk, d]
    int M, P, page_shift, Sk;
    const int* seqlens;
    const int* tree_lens;
    const int* mask;
    long long mask_stride;  // words between sequences (0: shared)
    int T, W;
};
cudaError_t launch_attn_varlen(const AttnParams& p, cudaStream_t stream);
cudaError_t launch_attn_tree(const AttnParams& p, cudaStream_t stream);

}  // namespace gqa
