// C ABI of libgqa_serve.so: argument validation and launches.  See include/gqa_serve.h for
// the contract.
#include "gqa_serve.h"

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "launch_serve.h"

namespace {

struct DeviceInfo {
    int sms = 0;
    bool ok = false;  // sm_100
};

gqa_status device_info(int* dev_out, DeviceInfo* info) {
    static DeviceInfo cache[64];
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();  // leave no error pending for the caller's own checks
        return GQA_ERR_CUDA;
    }
    *dev_out = dev;
    std::lock_guard<std::mutex> lk(mu);
    if (dev >= 0 && dev < 64 && cache[dev].sms > 0) {
        *info = cache[dev];
        return GQA_OK;
    }
    int major = 0, minor = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return GQA_ERR_CUDA;
    }
    info->sms = sms;
    info->ok = major == 10 && minor == 0;
    if (dev >= 0 && dev < 64) cache[dev] = *info;
    return GQA_OK;
}

gqa_status b200(int* dev, DeviceInfo* info) {
    const gqa_status st = device_info(dev, info);
    if (st != GQA_OK) return st;
    return info->ok ? GQA_OK : GQA_ERR_ARCH;
}

gqa_status launched(cudaError_t e) {
    if (e == cudaSuccess) return GQA_OK;
    cudaGetLastError();
    return GQA_ERR_CUDA;
}

bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

bool page_size_ok(int page_size) { return page_size >= 16 && (page_size & (page_size - 1)) == 0; }

int log2_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

// What both attention calls check of heads, head dimension, scale, output and splits.
gqa_status check_heads(int Hq, int Hk, int d, float scale, int out_dtype, int num_splits) {
    if (Hq < 1 || Hk < 1 || num_splits < 0) return GQA_ERR_SHAPE;
    if (out_dtype != GQA_OUT_F32 && out_dtype != GQA_OUT_BF16) return GQA_ERR_SHAPE;
    if (Hq % Hk != 0) return GQA_ERR_HEADS;
    if (d != 64 && d != 128) return GQA_ERR_HEADDIM;
    if (!std::isfinite(scale)) return GQA_ERR_SHAPE;
    return GQA_OK;
}

// A row stride in elements: 0 stands for contiguous rows.
bool stride_ok(long long* stride, long long row) {
    if (*stride == 0) *stride = row;
    return *stride >= row && *stride % 8 == 0 && *stride < (1ll << 38);  // bytes below 2^40: a tensor map's limit
}

gqa_status check_state(const gqa::CacheState& c, int page_size) {
    if (c.S < 1 || c.M < 1 || c.P < 1 || !page_size_ok(page_size)) return GQA_ERR_SHAPE;
    if (((long long)c.M * page_size) >= (1ll << 31) || ((long long)c.P * page_size) >= (1ll << 31)) return GQA_ERR_SHAPE;
    if (!c.table || !c.lens || !c.refs) return GQA_ERR_NULL;
    if (!aligned(c.table, 4) || !aligned(c.lens, 4) || !aligned(c.refs, 4)) return GQA_ERR_ALIGN;
    return GQA_OK;
}

gqa_status check_requests(const int* a, bool need_a, const int* b, int n, const int* status) {
    if (n < 0 || n > GQA_CACHE_MAX_REQUESTS) return GQA_ERR_SHAPE;
    if (n == 0) return GQA_OK;
    if ((need_a && !a) || !b || !status) return GQA_ERR_NULL;
    if (!aligned(a, 4) || !aligned(b, 4) || !aligned(status, 4)) return GQA_ERR_ALIGN;
    return GQA_OK;
}

gqa_status check_pools(const void* k, const void* v, int layers, long long row_bytes) {
    if (layers < 1 || row_bytes < 16 || row_bytes % 16 != 0 || row_bytes > (1ll << 24)) return GQA_ERR_SHAPE;
    if ((long long)layers * row_bytes / 8 >= 65535ll * 128) return GQA_ERR_SHAPE;
    if (!k || !v) return GQA_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16)) return GQA_ERR_ALIGN;
    return GQA_OK;
}

gqa::CacheState state_of(int* table, int* lens, int* refs, int S, int M, int P, int page_size) {
    gqa::CacheState c{};
    c.table = table;
    c.lens = lens;
    c.refs = refs;
    c.S = S;
    c.M = M;
    c.P = P;
    c.page_shift = page_size > 0 ? log2_of(page_size) : 0;
    return c;
}

gqa::Pools pools_of(void* k, void* v, int layers, long long row_bytes) {
    gqa::Pools p{};
    p.kv[0] = static_cast<uint8_t*>(k);
    p.kv[1] = static_cast<uint8_t*>(v);
    p.layers = layers;
    p.row_bytes = row_bytes;
    return p;
}

}  // namespace

extern "C" {

gqa_status gqa_attn_fwd_varlen(const void* q, long long q_row_stride, const void* k,
                               long long k_row_stride, const void* v, long long v_row_stride,
                               const int* cu_seqlens_q, const int* cu_seqlens_k, void* out,
                               int out_dtype, float* lse, int B, int total_q, int total_k, int Hq,
                               int Hk, int d, float scale, int causal, int num_splits,
                               void* stream) {
    if (B < 1 || total_q < 0 || total_k < 0) return GQA_ERR_SHAPE;
    gqa_status st = check_heads(Hq, Hk, d, scale, out_dtype, num_splits);
    if (st != GQA_OK) return st;
    if (!stride_ok(&q_row_stride, (long long)Hq * d) || !stride_ok(&k_row_stride, (long long)Hk * d) ||
        !stride_ok(&v_row_stride, (long long)Hk * d))
        return GQA_ERR_SHAPE;
    // kernel row indices are 32-bit
    if ((long long)total_q * Hq >= (1ll << 31) || (long long)total_k * Hk >= (1ll << 31)) return GQA_ERR_SHAPE;
    if (!cu_seqlens_q || !cu_seqlens_k) return GQA_ERR_NULL;
    if (total_q > 0 && (!q || !out || !lse)) return GQA_ERR_NULL;
    if (total_k > 0 && (!k || !v)) return GQA_ERR_NULL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(lse, 16) ||
        !aligned(cu_seqlens_q, 4) || !aligned(cu_seqlens_k, 4))
        return GQA_ERR_ALIGN;
    int dev = 0;
    DeviceInfo info;
    if ((st = b200(&dev, &info)) != GQA_OK) return st;
    if (total_q == 0) return GQA_OK;
    gqa::AttnParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.q_stride = q_row_stride;
    p.k_stride = k_row_stride;
    p.v_stride = v_row_stride;
    p.cu_q = cu_seqlens_q;
    p.cu_k = cu_seqlens_k;
    p.out = out;
    p.out_bf16 = out_dtype == GQA_OUT_BF16;
    p.lse = lse;
    p.B = B;
    p.total_q = total_q;
    p.total_k = total_k;
    p.Hq = Hq;
    p.Hk = Hk;
    p.d = d;
    p.scale = scale;
    p.causal = causal ? 1 : 0;
    return launched(gqa::launch_attn_varlen(p, static_cast<cudaStream_t>(stream)));
}

gqa_status gqa_attn_fwd_tree(const void* q, const void* k_cache, const void* v_cache,
                             const int* block_table, int max_pages_per_seq, int num_pages,
                             int page_size, const int* cache_seqlens, const int* tree_mask,
                             int mask_shared, const int* tree_lens, void* out, int out_dtype,
                             float* lse, int B, int T, int Sk, int Hq, int Hk, int d, float scale,
                             int num_splits, void* stream) {
    if (B < 1 || T < 1) return GQA_ERR_SHAPE;
    gqa_status st = check_heads(Hq, Hk, d, scale, out_dtype, num_splits);
    if (st != GQA_OK) return st;
    if (!q || !k_cache || !v_cache || !cache_seqlens || !tree_mask || !out || !lse) return GQA_ERR_NULL;
    // kernel row indices and tensor-map coordinates are 32-bit
    if ((long long)B * T * Hq >= (1ll << 31)) return GQA_ERR_SHAPE;
    if (block_table != nullptr) {
        if (max_pages_per_seq < 1 || num_pages < 1 || !page_size_ok(page_size) ||
            (long long)max_pages_per_seq * page_size >= (1ll << 31) ||
            (long long)num_pages * page_size * Hk >= (1ll << 31))
            return GQA_ERR_SHAPE;
    } else if (Sk < 1 || (long long)B * Sk * Hk >= (1ll << 31)) {
        return GQA_ERR_SHAPE;
    }
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
        !aligned(lse, 16) || !aligned(block_table, 4) || !aligned(cache_seqlens, 4) ||
        !aligned(tree_mask, 4) || !aligned(tree_lens, 4))
        return GQA_ERR_ALIGN;
    int dev = 0;
    DeviceInfo info;
    if ((st = b200(&dev, &info)) != GQA_OK) return st;
    gqa::AttnParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k_cache);
    p.v = static_cast<const uint16_t*>(v_cache);
    p.table = block_table;
    p.M = max_pages_per_seq;
    p.P = num_pages;
    p.page_shift = block_table != nullptr ? log2_of(page_size) : 0;
    p.Sk = Sk;
    p.seqlens = cache_seqlens;
    p.tree_lens = tree_lens;
    p.mask = tree_mask;
    p.T = T;
    p.W = (T + 31) / 32;
    p.mask_stride = mask_shared ? 0 : (long long)T * p.W;
    p.out = out;
    p.out_bf16 = out_dtype == GQA_OUT_BF16;
    p.lse = lse;
    p.B = B;
    p.Hq = Hq;
    p.Hk = Hk;
    p.d = d;
    p.scale = scale;
    return launched(gqa::launch_attn_tree(p, static_cast<cudaStream_t>(stream)));
}

gqa_status gqa_cache_resize(int* block_table, int* cache_seqlens, int* page_refs, int S,
                            int max_pages_per_seq, int num_pages, int page_size, const int* slots,
                            const int* new_lens, int n, int* status, void* stream) {
    gqa::PlanParams p{};
    p.c = state_of(block_table, cache_seqlens, page_refs, S, max_pages_per_seq, num_pages, page_size);
    gqa_status st = check_state(p.c, page_size);
    if (st != GQA_OK || (st = check_requests(slots, false, new_lens, n, status)) != GQA_OK) return st;
    int dev = 0;
    DeviceInfo info;
    if ((st = b200(&dev, &info)) != GQA_OK) return st;
    if (n == 0) return GQA_OK;
    p.key = slots;
    p.arg = new_lens;
    p.n = n;
    p.status = status;
    return launched(gqa::launch_resize(p, static_cast<cudaStream_t>(stream)));
}

gqa_status gqa_cache_fork(void* k_pages, void* v_pages, int layers, long long row_bytes,
                          int* block_table, int* cache_seqlens, int* page_refs, int S,
                          int max_pages_per_seq, int num_pages, int page_size, const int* parents,
                          const int* children, int n, int* status, void* stream) {
    gqa::PlanParams p{};
    p.c = state_of(block_table, cache_seqlens, page_refs, S, max_pages_per_seq, num_pages, page_size);
    gqa_status st = check_state(p.c, page_size);
    if (st != GQA_OK || (st = check_pools(k_pages, v_pages, layers, row_bytes)) != GQA_OK ||
        (st = check_requests(parents, true, children, n, status)) != GQA_OK)
        return st;
    int dev = 0;
    DeviceInfo info;
    if ((st = b200(&dev, &info)) != GQA_OK) return st;
    if (n == 0) return GQA_OK;
    p.key = children;
    p.arg = parents;
    p.n = n;
    p.status = status;
    return launched(gqa::launch_fork(p, pools_of(k_pages, v_pages, layers, row_bytes), info.sms,
                                     static_cast<cudaStream_t>(stream)));
}

gqa_status gqa_cache_compact(void* k_pages, void* v_pages, int layers, long long row_bytes,
                             int* block_table, int* cache_seqlens, int* page_refs, int S,
                             int max_pages_per_seq, int num_pages, int page_size, const int* keep,
                             const int* keep_lens, const int* tree_lens, int T, int* status,
                             void* stream) {
    gqa::CompactParams p{};
    p.c = state_of(block_table, cache_seqlens, page_refs, S, max_pages_per_seq, num_pages, page_size);
    gqa_status st = check_state(p.c, page_size);
    if (st != GQA_OK || (st = check_pools(k_pages, v_pages, layers, row_bytes)) != GQA_OK) return st;
    if (T < 1) return GQA_ERR_SHAPE;
    if (!keep || !keep_lens || !status) return GQA_ERR_NULL;
    if (!aligned(keep, 4) || !aligned(keep_lens, 4) || !aligned(tree_lens, 4) || !aligned(status, 4))
        return GQA_ERR_ALIGN;
    int dev = 0;
    DeviceInfo info;
    if ((st = b200(&dev, &info)) != GQA_OK) return st;
    p.pools = pools_of(k_pages, v_pages, layers, row_bytes);
    p.keep = keep;
    p.keep_lens = keep_lens;
    p.tree_lens = tree_lens;
    p.T = T;
    p.status = status;
    return launched(gqa::launch_compact(p, static_cast<cudaStream_t>(stream)));
}

gqa_status gqa_serve_device_status(int reset) {
    (void)reset;
    return GQA_OK;
}

}  // extern "C"
