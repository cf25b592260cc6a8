// C ABI of libgqa_serve.so: argument validation, schedules, TMA tensor maps, scratch and
// launches.  See include/gqa_serve.h for the contract.
#include "gqa_serve.h"

#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <mutex>

#include "launch_serve.h"
#include "serve_params.h"

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

// What both attention calls check of heads, head dimension, scale and output.
gqa_status check_heads(int Hq, int Hk, int d, float scale, int out_dtype) {
    if (Hq < 1 || Hk < 1) return GQA_ERR_SHAPE;
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
    if ((long long)layers * row_bytes >= (1ll << 31)) return GQA_ERR_SHAPE;  // 32-bit columns in the kernels
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

// ---------------------------------------------------------------- tensor maps, scratch, waits

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled get_encode_tiled() {
    static EncodeTiled fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiled>(ptr);
    });
    return fn;
}

// [B, S, H, d] as a 4-D map (d, H, S, B) with 128-byte swizzle, boxes of one row's 128 bytes x
// box_h heads x box_s rows, zero fill out of bounds.  Rows lie row_bytes apart; fp32 tensors are
// outputs, the others bf16.
bool encode(CUtensorMap* m, const void* ptr, long long B, long long S, int H, int d, long long row_bytes,
            int box_h, int box_s, bool f32 = false) {
    EncodeTiled enc = get_encode_tiled();
    if (!enc) return false;
    const cuuint64_t es = f32 ? 4 : 2;
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)S, (cuuint64_t)B};
    // (one batch: its stride is never used, and the packed rows' total may exceed its limit)
    cuuint64_t strides[3] = {(cuuint64_t)d * es, (cuuint64_t)row_bytes, (cuuint64_t)row_bytes * (B > 1 ? S : 1)};
    cuuint32_t box[4] = {(cuuint32_t)(128 / es), (cuuint32_t)box_h, (cuuint32_t)box_s, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
               const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, f32 ? CU_TENSOR_MAP_L2_PROMOTION_NONE : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scratch comes from a stream-ordered pool of this library per device, which keeps what is
// freed.  In a stream capture an allocation becomes the graph's own.
cudaMemPool_t workspace_pool(int dev) {
    static cudaMemPool_t pools[64] = {};
    static std::mutex mu;
    if (dev < 0 || dev >= 64) return nullptr;
    std::lock_guard<std::mutex> lk(mu);
    if (pools[dev] == nullptr) {
        cudaMemPoolProps props{};
        props.allocType = cudaMemAllocationTypePinned;
        props.location.type = cudaMemLocationTypeDevice;
        props.location.id = dev;
        // the first call may be made in a stream capture, which otherwise forbids making a pool
        cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
        cudaThreadExchangeStreamCaptureMode(&mode);
        cudaMemPool_t pool = nullptr;
        const bool made = cudaMemPoolCreate(&pool, &props) == cudaSuccess;
        if (made) {
            uint64_t keep = ~0ull;
            cudaMemPoolSetAttribute(pool, cudaMemPoolAttrReleaseThreshold, &keep);
        } else {
            cudaGetLastError();
        }
        cudaThreadExchangeStreamCaptureMode(&mode);
        if (!made) return nullptr;
        pools[dev] = pool;
    }
    return pools[dev];
}

// One allocation on a stream, freed on it when the object goes (after the launches in between).
class Workspace {
public:
    Workspace(int dev, size_t bytes, cudaStream_t stream) : stream_(stream) {
        cudaMemPool_t pool = workspace_pool(dev);
        if (pool == nullptr || std::getenv("GQA_FAULT_INJECT_ALLOC") != nullptr) return;
        if (cudaMallocFromPoolAsync(&ptr_, bytes, pool, stream) != cudaSuccess) {
            cudaGetLastError();
            ptr_ = nullptr;
        }
    }
    ~Workspace() {
        if (ptr_ != nullptr) cudaFreeAsync(ptr_, stream_);
    }
    Workspace(const Workspace&) = delete;
    Workspace& operator=(const Workspace&) = delete;
    bool ok() const { return ptr_ != nullptr; }
    // the next piece of the allocation, 256-byte aligned
    template <class T>
    T* take(size_t count) {
        T* p = reinterpret_cast<T*>(static_cast<char*>(ptr_) + used_);
        used_ += size_of<T>(count);
        return p;
    }
    template <class T>
    static size_t size_of(size_t count) {
        return (count * sizeof(T) + 255) & ~(size_t)255;
    }

private:
    void* ptr_ = nullptr;
    size_t used_ = 0;
    cudaStream_t stream_;
};

// Limit of each in-kernel wait, as gqa_attn_fwd reads it.
long long timeout_ns() {
    if (const char* e = std::getenv("GQA_WAIT_TIMEOUT_NS")) {
        const long long ns = std::atoll(e);
        return ns < 1 ? 1 : ns;
    }
    const char* e = std::getenv("GQA_WAIT_TIMEOUT_MS");
    const long long ms = e ? std::atoll(e) : 4000;
    return (ms < 1 ? 1 : ms) * 1000000ll;
}

// ---------------------------------------------------------------- attention schedules

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// Heads, rows and waits: what does not depend on where K and V lie.  `queries` is the query rows
// of a sequence (the average one's, for prompts): a tile holds a group's heads side by side
// unless that pads more rows than a tile per head does.
void fill_common(gqa::ServeParams* p, int B, int Hq, int Hk, float scale, long long queries) {
    const int g = Hq / Hk, M = gqa::kServeBlockM;
    p->B = B;
    p->Hq = Hq;
    p->Hk = Hk;
    p->g = g;
    const long long apart = (long long)g * ceil_div(queries, M);
    p->pack = g <= M && ceil_div(queries, M / g) <= apart ? 1 : 0;
    p->pos_per_tile = p->pack ? M / g : M;
    p->rows_valid = p->pack ? g * p->pos_per_tile : M;
    p->n_hg = p->pack ? Hk : Hq;
    p->div_g = gqa::make_fastdiv((uint32_t)g);
    p->div_hg = gqa::make_fastdiv((uint32_t)p->n_hg);
    p->scale_log2 = (float)((double)scale * 1.4426950408889634);
    p->timeout_ns = timeout_ns();
    p->drain_ns = p->timeout_ns > 1000000000ll ? p->timeout_ns : 1000000000ll;
    // host-side fault injection: the kernel stalls on a wait that nothing completes
    p->inject_stall = std::getenv("GQA_FAULT_INJECT_STALL") != nullptr ? 1 : 0;
}

// The ranges schedule: every CTA slot gets an equal share of all key blocks.  Units of at most
// kWholeBlocks blocks are not split: a CTA that walks one alone is done before the partials of
// several would be written and joined, and needs no scratch.  Measured on B200 (a tree of 8 nodes,
// B 1, Hk 8, d 128; whole against split): 256 keys 10.2 and 11.9 us, 512 keys 13.4 and 15.1, 1024
// keys 20.0 and 17.7, 2048 keys 33.3 and 17.4.  A range holds at least two blocks: 8192 keys take
// 28.5 us so, 25.0 with four and 28.8 with eight, 2048 keys 17.4, 22.4 and 26.6.
gqa_status run_ranges(gqa::ServeParams* p, int dev, int sms, int d, int nt, long long most_units, long long most_keys,
                      cudaStream_t stream) {
    constexpr int kWholeBlocks = 4;
    int grid = sms * gqa::serve_ctas_per_sm(nt);
    p->whole = most_keys <= kWholeBlocks * gqa::kServeBlockN ? 1 : 0;
    p->min_blocks = p->whole ? 1 : 2;
    const long long steps = most_units * (p->whole ? 1 : ceil_div(most_keys, gqa::kServeBlockN));
    if (steps < grid) grid = (int)(steps > 1 ? steps : 1);
    const bool prefix = p->B > gqa::kServeOwnPrefix;
    if (p->whole && !prefix) return launched(gqa::launch_serve(*p, d, nt, grid, stream));
    const size_t rows = (size_t)2 * grid * nt * gqa::kServeBlockM;
    using W = Workspace;
    W ws(dev, W::size_of<float>(rows * d) + W::size_of<float>(rows) + W::size_of<gqa::ServeBound>(grid) +
                  (prefix ? W::size_of<long long>((size_t)p->B + 1) : 0), stream);
    if (!ws.ok()) return GQA_ERR_ALLOC;
    p->part_o = ws.take<float>(rows * d);
    p->part_lse = ws.take<float>(rows);
    p->bounds = ws.take<gqa::ServeBound>(grid);
    p->pre = prefix ? ws.take<long long>((size_t)p->B + 1) : nullptr;
    return launched(gqa::launch_serve(*p, d, nt, grid, stream));
}

// The list schedule (two-tile units of prompts).
gqa_status run_list(gqa::ServeParams* p, int dev, int sms, int d, cudaStream_t stream) {
    gqa::ServePlanParams l{};
    l.cu_q = p->cu_q;
    l.cu_k = p->cu_k;
    l.B = p->B;
    l.total_q = p->total_q;
    l.total_k = p->total_k;
    l.causal = p->causal;
    l.pos_per_unit = 2 * p->pos_per_tile;
    // windows of about 12 MB of K and V (the forward's, fitted on B200: the L2 also carries Q and
    // the output), at most kServeWindows of them
    const long long rows = 12000000ll / (4ll * p->Hk * d);
    long long window = rows > 1 ? rows : 1;
    const long long least = ceil_div(p->total_k > 0 ? p->total_k : 1, gqa::kServeWindows);
    if (window < least) window = least;
    l.window_rows = (int)window;
    l.windows = gqa::kServeWindows;
    const long long cap = ceil_div(p->total_q, l.pos_per_unit) + p->B;
    l.list_cap = (int)cap;
    using W = Workspace;
    W ws(dev, W::size_of<int2>((size_t)cap) + W::size_of<int>(1), stream);
    if (!ws.ok()) return GQA_ERR_ALLOC;
    l.list = ws.take<int2>((size_t)cap);
    l.list_len = ws.take<int>(1);
    p->list = l.list;
    p->list_len = l.list_len;
    p->kv_shared = 1;
    if (gqa::launch_serve_list(l, stream) != cudaSuccess) {
        cudaGetLastError();
        return GQA_ERR_CUDA;
    }
    const long long units = cap * p->n_hg;
    return launched(gqa::launch_serve(*p, d, 2, (int)(units < sms ? units : sms), stream));
}

}  // namespace

extern "C" {

gqa_status gqa_attn_fwd_varlen(const void* q, long long q_row_stride, const void* k,
                               long long k_row_stride, const void* v, long long v_row_stride,
                               const int* cu_seqlens_q, const int* cu_seqlens_k, void* out,
                               int out_dtype, float* lse, int B, int total_q, int total_k, int Hq,
                               int Hk, int d, float scale, int causal, void* stream) {
    if (B < 1 || total_q < 0 || total_k < 0) return GQA_ERR_SHAPE;
    gqa_status st = check_heads(Hq, Hk, d, scale, out_dtype);
    if (st != GQA_OK) return st;
    if (!stride_ok(&q_row_stride, (long long)Hq * d) || !stride_ok(&k_row_stride, (long long)Hk * d) ||
        !stride_ok(&v_row_stride, (long long)Hk * d))
        return GQA_ERR_SHAPE;
    // kernel row indices are 32-bit
    if (((long long)total_q + B) * Hq >= (1ll << 31) || (long long)total_k * Hk >= (1ll << 31)) return GQA_ERR_SHAPE;
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
    gqa::ServeParams p{};
    const long long queries = ceil_div(total_q, B);
    fill_common(&p, B, Hq, Hk, scale, queries);
    p.cu_q = cu_seqlens_q;
    p.cu_k = cu_seqlens_k;
    p.total_q = total_q;
    p.total_k = total_k;
    p.causal = causal ? 1 : 0;
    p.out = out_dtype == GQA_OUT_F32 ? static_cast<float*>(out) : nullptr;
    p.out_bf16 = out_dtype == GQA_OUT_BF16 ? static_cast<uint16_t*>(out) : nullptr;
    p.lse = lse;
    const int g = p.g, M = gqa::kServeBlockM;
    const int box_h = p.pack ? g : 1, box_s = p.pos_per_tile;
    if (!encode(&p.tm_q, q, 1, total_q, Hq, d, q_row_stride * 2, box_h, box_s)) return GQA_ERR_CUDA;
    // (without keys nothing is loaded: any mapped address serves)
    const bool keys = total_k > 0;
    if (!encode(&p.tm_k, keys ? k : q, 1, keys ? total_k : 1, keys ? Hk : 1, d, keys ? k_row_stride * 2 : 256, 1, M) ||
        !encode(&p.tm_v, keys ? v : q, 1, keys ? total_k : 1, keys ? Hk : 1, d, keys ? v_row_stride * 2 : 256, 1, M))
        return GQA_ERR_CUDA;
    // Two-tile units from a list when the average sequence fills them and there is one for three in
    // four SMs; else ranges over one-tile units, which also share a long key axis among CTAs.
    // Measured on B200 (Hq 32, Hk 8, d 128, causal; list against ranges): 64 units 22.8 and 16.1 us,
    // 128 units 30.9 and 33.3, 256 units 43 and 52, 1024 units 117 and 173.
    const long long tiles = ceil_div(queries, p.pos_per_tile);
    const long long units = ceil_div(total_q, 2 * p.pos_per_tile) * p.n_hg;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (tiles >= 2 && 4 * units >= 3ll * info.sms) {
        if (!encode(&p.tm_o, out, 1, total_q, Hq, d, (long long)Hq * d * (p.out ? 4 : 2), box_h, box_s, p.out != nullptr))
            return GQA_ERR_CUDA;
        return run_list(&p, dev, info.sms, d, s);
    }
    p.kv_shared = (tiles > 1 || !p.pack) ? 1 : 0;
    return run_ranges(&p, dev, info.sms, d, 1, (ceil_div(total_q, p.pos_per_tile) + B) * p.n_hg, total_k, s);
}

gqa_status gqa_attn_fwd_tree(const void* q, const void* k_cache, const void* v_cache,
                             const int* block_table, int max_pages_per_seq, int num_pages,
                             int page_size, const int* cache_seqlens, const int* tree_mask,
                             int mask_shared, const int* tree_lens, void* out, int out_dtype,
                             float* lse, int B, int T, int Sk, int Hq, int Hk, int d, float scale,
                             void* stream) {
    if (B < 1 || T < 1) return GQA_ERR_SHAPE;
    gqa_status st = check_heads(Hq, Hk, d, scale, out_dtype);
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
    gqa::ServeParams p{};
    fill_common(&p, B, Hq, Hk, scale, T);
    p.seqlens = cache_seqlens;
    p.tree_lens = tree_lens;
    p.mask = tree_mask;
    p.T = T;
    p.W = (T + 31) / 32;
    p.mask_stride = mask_shared ? 0 : (long long)T * p.W;
    p.out = out_dtype == GQA_OUT_F32 ? static_cast<float*>(out) : nullptr;
    p.out_bf16 = out_dtype == GQA_OUT_BF16 ? static_cast<uint16_t*>(out) : nullptr;
    p.lse = lse;
    const long long tiles = ceil_div(T, p.pos_per_tile);
    const int nt = tiles >= 2 ? 2 : 1, M = gqa::kServeBlockM;
    const int box_h = p.pack ? p.g : 1, box_s = p.pos_per_tile;
    if (!encode(&p.tm_q, q, B, T, Hq, d, 2ll * Hq * d, box_h, box_s) ||
        (nt == 2 &&
         !encode(&p.tm_o, out, B, T, Hq, d, (long long)Hq * d * (p.out ? 4 : 2), box_h, box_s, p.out != nullptr)))
        return GQA_ERR_CUDA;
    const long long kv_row = 2ll * Hk * d;
    if (block_table == nullptr) {
        p.cap = Sk;
        if (!encode(&p.tm_k, k_cache, B, Sk, Hk, d, kv_row, 1, M) || !encode(&p.tm_v, v_cache, B, Sk, Hk, d, kv_row, 1, M))
            return GQA_ERR_CUDA;
    } else {
        // the page pools as (d, Hk, page_size, num_pages), boxes of up to 128 rows
        p.cap = max_pages_per_seq * page_size;
        p.block_table = block_table;
        p.table_stride = max_pages_per_seq;
        p.page_shift = log2_of(page_size);
        p.page_rows = page_size < M ? page_size : M;
        p.num_pages = num_pages;
        if (!encode(&p.tm_k, k_cache, num_pages, page_size, Hk, d, kv_row, 1, p.page_rows) ||
            !encode(&p.tm_v, v_cache, num_pages, page_size, Hk, d, kv_row, 1, p.page_rows))
            return GQA_ERR_CUDA;
    }
    p.kv_shared = (tiles > nt || !p.pack) ? 1 : 0;
    return run_ranges(&p, dev, info.sms, d, nt, ceil_div(tiles, nt) * B * p.n_hg, p.cap,
                      static_cast<cudaStream_t>(stream));
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
    return launched(gqa::launch_compact(p, info.sms, static_cast<cudaStream_t>(stream)));
}

gqa_status gqa_serve_device_status(int reset) {
    unsigned int* ptr = gqa::serve_status_symbol();
    if (!ptr) return GQA_ERR_CUDA;
    unsigned int h = 0;
    if (cudaMemcpy(&h, ptr, sizeof(h), cudaMemcpyDeviceToHost) != cudaSuccess) return GQA_ERR_CUDA;
    if (reset) {
        const unsigned int z = 0;
        if (cudaMemcpy(ptr, &z, sizeof(z), cudaMemcpyHostToDevice) != cudaSuccess) return GQA_ERR_CUDA;
    }
    return h ? GQA_ERR_TIMEOUT : GQA_OK;
}

}  // extern "C"
