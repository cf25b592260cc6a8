// Parameters and host-side entry points of the serving kernels (internal to libgqa_serve.so).
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

namespace gqa {

// Every kernel here but those of large prompt batches may be brought in while the one before it in the stream still runs
// (programmatic dependent launch): its blocks set themselves up, and wait (wait_before) for all
// that came before to be complete before they touch global memory.  Its own first act is to let
// the next one in (let_next), which costs nothing: that one's blocks come when all of its own are
// placed, and take only room that is free.
#ifdef __CUDACC__
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <class... A>
cudaError_t launch_early(void (*kernel)(A...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                         const A&... args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
#endif

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
cudaError_t launch_compact(const CompactParams& p, int sms, cudaStream_t stream);

// ---------------------------------------------------------------- attention
struct ServeParams;
struct ServePlanParams;

int serve_ctas_per_sm(int nt);
// The attention kernel for head dimension d and nt tiles per unit: packed prompts (seqlens NULL;
// with a list, else by ranges and nt = 1) or a tree over a cache.
cudaError_t launch_serve(const ServeParams& p, int d, int nt, int grid, cudaStream_t stream);
cudaError_t launch_serve_list(const ServePlanParams& p, cudaStream_t stream);
// Device address of this library's status word on the current device (NULL on error).
unsigned int* serve_status_symbol();

}  // namespace gqa
