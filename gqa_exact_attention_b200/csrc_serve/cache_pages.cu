// The pages of a paged KV cache: gqa_cache_resize, gqa_cache_fork, gqa_cache_compact.
//
// Taking pages is a prefix problem: request i, which needs a_i pages, gets those free pages
// (page_refs = 0) whose rank among the free ones, in order of their numbers, lies in
// [a_0 + .. + a_{i-1}, a_0 + .. + a_i).  One cluster of thread blocks does a whole call: it
// validates the requests, gives up and shares pages, counts the free ones per warp, and each
// warp then writes the ranks of its own pages into the table.  The steps are separated by
// cluster barriers (a fraction of a microsecond) instead of launches, and the state stays in
// L2.  Nothing depends on the order in which atomics land: the counts only add up.  What a call
// costs is latency, the dependent reads of its steps (lengths, table entries, counts): measured on
// B200, 4 us for 8 slots of a small cache, 20 us for 256 slots over 131 thousand pages, whose bytes
// alone would take 1 us.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "gqa_serve.h"
#include "launch_serve.h"

namespace gqa {
namespace {

namespace cg = cooperative_groups;

constexpr int kMostCtas = 16;  // of a cluster (8 where 16 cannot be had)
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;  // at most 32: one warp adds them up
constexpr int kEmpty = -1;

__device__ __forceinline__ int pages_of(int len, int shift) { return (len >> shift) + ((len & ((1 << shift) - 1)) != 0); }
__device__ __forceinline__ int clamp_len(int len, const CacheState& c) {
    const long long cap = (long long)c.M << c.page_shift;
    return len < 0 ? 0 : (len > cap ? (int)cap : len);
}
__device__ __forceinline__ bool known(int page, const CacheState& c) { return page >= 0 && page < c.P; }
__device__ __forceinline__ int* row_of(const CacheState& c, int slot) { return c.table + (size_t)slot * c.M; }

// Open-addressing set of slots in shared memory: the lowest request that names each.
struct SlotSet {
    int* keys;
    int* first;
    int mask;  // size - 1, a power of two of at least twice the requests
    __device__ int place(int slot) const { return (int)(((unsigned)slot * 2654435761u) >> 7) & mask; }
    __device__ void insert(int slot, int i) const {
        for (int at = place(slot);; at = (at + 1) & mask) {
            const int was = atomicCAS(&keys[at], kEmpty, slot);
            if (was == kEmpty || was == slot) {
                atomicMin(&first[at], i);
                return;
            }
        }
    }
    // the lowest request that names the slot, or a value past every request
    __device__ int find(int slot) const {
        for (int at = place(slot);; at = (at + 1) & mask) {
            if (keys[at] == slot) return first[at];
            if (keys[at] == kEmpty) return 0x7fffffff;
        }
    }
};

__host__ __device__ constexpr int set_size(int n) {
    int s = 64;
    while (s < 2 * n) s *= 2;
    return s;
}

// Inclusive prefix sum over a block's threads; *total is the block's sum.  64 bits: requests
// may ask for more pages in all than 32 bits count.
__device__ long long block_scan(long long x, long long* warp_sums, long long* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    long long w = lane < kWarps ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    const long long before = __shfl_sync(0xffffffffu, w, warp == 0 ? 0 : warp - 1);
    *total = __shfl_sync(0xffffffffu, w, 31);
    __syncthreads();
    return incl + (warp == 0 ? 0 : before);
}
constexpr int kMost = 0x7fffffff;
__device__ __forceinline__ int saturate(long long x) { return x > kMost ? kMost : (int)x; }

template <bool FORK>
__global__ void __launch_bounds__(kThreads) cache_plan_kernel(const __grid_constant__ PlanParams p) {
    extern __shared__ int smem[];
    __shared__ long long warp_sums[kWarps];
    __shared__ int cta_free;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const CacheState& c = p.c;
    let_next();
    const int n = p.n;
    const int size = set_size(n);
    int* key_ = smem;       // [n] the requests
    int* arg_ = key_ + n;
    int* upto = arg_ + n;   // [n] pages needed by requests 0..i
    int* first = upto + n;  // [n] the first new entry of request i's row
    int* old = first + n;   // [n] entries that request i gives up end here
    int* state = old + n;   // [n] GQA_CACHE_DONE, _INVALID, _SHARED, or one of
    constexpr int kSkip = 8;  // a fork of a slot to itself
    constexpr int kTake = 9;  // as GQA_CACHE_DONE, if its pages can be had
    auto acts = [&](int i) { return state[i] == GQA_CACHE_DONE || state[i] == kTake; };
    const SlotSet keys{state + n, state + n + size, size - 1};
    const SlotSet parents{state + n + 2 * size, state + n + 3 * size, size - 1};  // fork only


    // ---- 1. the requests, by every block alike (nothing of the state changes yet)
    for (int i = tid; i < size; i += kThreads) {
        keys.keys[i] = kEmpty;
        keys.first[i] = 0x7fffffff;
        if constexpr (FORK) {
            parents.keys[i] = kEmpty;
            parents.first[i] = 0x7fffffff;
        }
    }
    wait_before();
    for (int i = tid; i < n; i += kThreads) {
        key_[i] = p.key != nullptr ? p.key[i] : i;
        arg_[i] = p.arg[i];
    }
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
        const int key = key_[i], arg = arg_[i];
        if (key >= 0 && key < c.S) keys.insert(key, i);
        if constexpr (FORK) {
            if (arg >= 0 && arg < c.S) parents.insert(arg, i);
        }
    }
    __syncthreads();
    long long carry = 0;
    const int rounds = (n + kThreads - 1) / kThreads;
    for (int r = 0; r < rounds; ++r) {
        const int i = r * kThreads + tid;
        int need = 0;
        if (i < n) {
            const int key = key_[i], arg = arg_[i];
            int st = GQA_CACHE_INVALID, at = 0, end = 0;
            if (key >= 0 && key < c.S && keys.find(key) == i) {
                const int mine = clamp_len(c.lens[key], c);
                if constexpr (FORK) {
                    if (arg == key) {
                        st = kSkip;
                    } else if (arg >= 0 && arg < c.S && parents.find(key) > n) {
                        const int len = clamp_len(c.lens[arg], c);
                        st = GQA_CACHE_DONE;
                        at = len >> c.page_shift;  // whole pages are shared
                        end = pages_of(mine, c.page_shift);
                        need = pages_of(len, c.page_shift) - at;
                    }
                } else if (arg >= 0 && arg <= ((long long)c.M << c.page_shift)) {
                    st = GQA_CACHE_DONE;
                    const int stay = min(mine, arg);
                    if (arg != mine && (stay & ((1 << c.page_shift) - 1)) != 0) {
                        const int page = row_of(c, key)[stay >> c.page_shift];
                        if (known(page, c) && __ldcg(c.refs + page) > 1) st = GQA_CACHE_SHARED;
                    }
                    if (st == GQA_CACHE_DONE) {
                        const int had = pages_of(mine, c.page_shift), want = pages_of(arg, c.page_shift);
                        need = max(want - had, 0);
                        at = need > 0 ? had : want;  // taken from here, or given up from here
                        end = had;
                    }
                }
            }
            state[i] = need > 0 ? kTake : st;
            first[i] = at;
            old[i] = end;
        }
        long long total;
        const long long incl = carry + block_scan(need, warp_sums, &total);
        if (i < n) upto[i] = saturate(incl);
        carry += total;
    }
    const int needed = saturate(carry);
    auto sync = [&] {
        if (ctas > 1) cluster.sync();
        else __syncthreads();
    };
    sync();  // every block has read the state

    // ---- 2. pages given up, and with FORK the shared ones named; 256 entries per warp and turn
    constexpr int kChunk = 256;
    const int chunks = (c.M + kChunk - 1) / kChunk;
    const long long items = (long long)n * chunks;
    for (long long w = (long long)rank * kWarps + warp; w < items; w += ctas * kWarps) {
        const int i = (int)(w % n), j0 = (int)(w / n) * kChunk;
        if (!acts(i)) continue;
        const int lo = FORK ? 0 : first[i];
        const int hi = FORK ? max(first[i], old[i]) : old[i];
        if (j0 >= hi || j0 + kChunk <= lo) continue;
        int* row = row_of(c, key_[i]);
        const int* from = FORK ? row_of(c, arg_[i]) : nullptr;
        int was[kChunk / 32], now[kChunk / 32];
#pragma unroll
        for (int e = 0; e < kChunk / 32; ++e) {
            const int j = j0 + e * 32 + lane;
            was[e] = (j >= lo && j < old[i]) ? row[j] : -1;
            now[e] = (FORK && j < first[i]) ? from[j] : -1;
        }
#pragma unroll
        for (int e = 0; e < kChunk / 32; ++e) {
            const int j = j0 + e * 32 + lane;
            if (known(was[e], c)) atomicSub(c.refs + was[e], 1);
            if (known(now[e], c)) atomicAdd(c.refs + now[e], 1);
            if (j >= lo && j < hi) row[j] = now[e];
        }
    }

    // ---- 3. the free pages, counted per warp over its own range of page numbers, kFew * 32 at a
    // time so that the loads overlap; bit e of a lane's mask is page 32 e + lane
    constexpr int kFew = 32;
    int free_before = 0, free_all = 0;
    const int per_warp = ((c.P + ctas * kWarps - 1) / (ctas * kWarps) + 31) / 32 * 32;
    const long long p0 = (long long)(rank * kWarps + warp) * per_warp;
    const int p_lo = p0 < c.P ? (int)p0 : c.P;
    const int p_hi = p0 + per_warp < c.P ? (int)(p0 + per_warp) : c.P;
    auto free_mask = [&](int at) {
        int x[kFew];
        unsigned m = 0;
#pragma unroll
        for (int e = 0; e < kFew; ++e) {
            const int page = at + e * 32 + lane;
            x[e] = page < p_hi ? __ldcg(c.refs + page) : 1;
        }
#pragma unroll
        for (int e = 0; e < kFew; ++e) m |= x[e] == 0 ? 1u << e : 0u;
        return m;
    };
    // the first request of lo..hi with upto > r (one has)
    auto first_past = [&](int r, int lo, int hi) {
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (upto[mid] > r) hi = mid;
            else lo = mid + 1;
        }
        return lo;
    };
    if (needed > 0) {
        sync();  // the counts are final
        int mine = 0;
        unsigned first_mask = 0;  // of the warp's first pages: most pools have no more
        for (int at = p_lo; at < p_hi; at += kFew * 32) {
            const unsigned m = free_mask(at);
            if (at == p_lo) first_mask = m;
            mine += __popc(m);
        }
        mine = __reduce_add_sync(0xffffffffu, mine);
        long long total;
        const int incl = (int)block_scan(lane == 31 ? mine : 0, warp_sums, &total);
        // (lane 31 of each warp holds the sum up to and with its warp)
        free_before = __shfl_sync(0xffffffffu, incl, 31) - mine;
        if (tid == 0) cta_free = (int)total;
        sync();
        // (each of the first lanes reads one block's count)
        int x = lane < ctas ? *cluster.map_shared_rank(&cta_free, lane) : 0;
        free_all = __reduce_add_sync(0xffffffffu, x);
        free_before += __reduce_add_sync(0xffffffffu, lane < rank ? x : 0);

        // ---- 4. each warp hands out its own free pages
        for (int at = p_lo; at < p_hi && free_before < needed; at += kFew * 32) {
            unsigned m = at == p_lo ? first_mask : free_mask(at);
            // lane e keeps group e's free lanes, and how many are free in the groups before
            unsigned group = 0;
#pragma unroll
            for (int e = 0; e < kFew; ++e) {
                const unsigned ball = __ballot_sync(0xffffffffu, (m >> e) & 1u);
                if (lane == e) group = ball;
            }
            int upto_group = __popc(group);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, upto_group, o);
                if (lane >= o) upto_group += y;
            }
            const int in_group = upto_group - __popc(group);
            const int here = __shfl_sync(0xffffffffu, upto_group, 31);
            if (here == 0) continue;
            // the requests that these pages go to: few, where requests take many pages
            const int end = min(free_before + here, needed) - 1;
            const int found = first_past(lane == 0 ? free_before : end, 0, n - 1);
            const int req_lo = __shfl_sync(0xffffffffu, found, 0), req_hi = __shfl_sync(0xffffffffu, found, 1);
            while (__any_sync(0xffffffffu, m != 0u)) {  // every lane's next page
                const int e = m != 0u ? __ffs(m) - 1 : 0;
                const unsigned others = __shfl_sync(0xffffffffu, group, e);
                const int r = free_before + __shfl_sync(0xffffffffu, in_group, e) + __popc(others & ((1u << lane) - 1u));
                if (m != 0u && r < needed) {
                    const int lo = first_past(r, req_lo, req_hi);
                    const int entry = first[lo] + (r - (lo > 0 ? upto[lo - 1] : 0));
                    if (upto[lo] <= free_all && entry < c.M) {
                        const int page = at + e * 32 + lane;
                        row_of(c, key_[lo])[entry] = page;
                        c.refs[page] = 1;
                    }
                }
                m &= m - 1u;
            }
            free_before += here;
        }
    }

    // ---- 5. lengths and outcomes
    for (int i = rank * kThreads + tid; i < n; i += ctas * kThreads) {
        int st = state[i];
        if (st == kTake) st = upto[i] <= free_all ? GQA_CACHE_DONE : GQA_CACHE_NO_PAGES;
        if constexpr (FORK) {
            if (acts(i))
                c.lens[key_[i]] = st == GQA_CACHE_DONE ? clamp_len(c.lens[arg_[i]], c) : 0;
        } else {
            if (st == GQA_CACHE_DONE) c.lens[key_[i]] = arg_[i];
        }
        p.status[i] = st == kSkip ? (int)GQA_CACHE_DONE : st;
    }
    if constexpr (FORK) {
        // a child without a page for its last rows gives the shared ones back
        if (needed > free_all) {
            sync();  // no warp looks for free pages any more
            for (int i = rank * kWarps + warp; i < n; i += ctas * kWarps) {
                if (state[i] != kTake || upto[i] <= free_all) continue;
                int* row = row_of(c, key_[i]);
                for (int j = lane; j < first[i]; j += 32) {
                    if (known(row[j], c)) atomicSub(c.refs + row[j], 1);
                    row[j] = -1;
                }
            }
        }
    }
    if (needed > 0) sync();  // a block's count is read by the others until here
}

// The last rows of each fork: [0, len % page) of the parent's last page to the child's, in every
// layer's K and V.  A block belongs to one fork (blockIdx.x) and takes every gridDim.y-th of its
// pieces, 16 KB of one page in one layer; what it has to look up, it looks up once.  A parent's rows
// are read from DRAM once and by its other children from L2.  Measured on B200: 226 MB (240 forks of
// 16 parents, 8 layers) in 40 us, 5.6 TB/s.  Bound by the latency of its reads, which warps wait for
// 57 % of the time: no memory unit is above 71 % (DRAM 49 %).
constexpr int kCopyBytes = 16384;
constexpr int kCopyThreads = 256;

__global__ void __launch_bounds__(kCopyThreads) cache_tail_copy_kernel(const __grid_constant__ PlanParams p,
                                                                       const __grid_constant__ Pools pools) {
    const CacheState& c = p.c;
    const int i = blockIdx.x;
    let_next();
    wait_before();
    const int child = p.key[i], parent = p.arg[i];
    if (p.status[i] != GQA_CACHE_DONE || parent == child) return;
    const int len = clamp_len(__ldcg(c.lens + child), c);
    const int tail = len & ((1 << c.page_shift) - 1);
    if (tail == 0) return;
    const int entry = len >> c.page_shift;
    const int src = __ldcg(row_of(c, parent) + entry), dst = __ldcg(row_of(c, child) + entry);
    if (!known(src, c) || !known(dst, c)) return;
    const long long page_bytes = pools.row_bytes << c.page_shift;
    const long long bytes = tail * pools.row_bytes;
    const int parts = (int)((bytes + kCopyBytes - 1) / kCopyBytes);
    const int pieces = pools.layers * 2 * parts;
    for (int x = blockIdx.y; x < pieces; x += gridDim.y) {
        const int part = x % parts, kv = x / parts & 1, layer = x / parts / 2;
        uint8_t* pool = pools.kv[kv] + (size_t)layer * c.P * page_bytes;
        const uint8_t* from = pool + (size_t)src * page_bytes;
        uint8_t* to = pool + (size_t)dst * page_bytes;
        constexpr int kEach = kCopyBytes / (16 * kCopyThreads);
        uint4 v[kEach];
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const long long at = (long long)part * kCopyBytes + (e * kCopyThreads + threadIdx.x) * 16;
            if (at < bytes) v[e] = *reinterpret_cast<const uint4*>(from + at);
        }
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const long long at = (long long)part * kCopyBytes + (e * kCopyThreads + threadIdx.x) * 16;
            if (at < bytes) *reinterpret_cast<uint4*>(to + at) = v[e];
        }
    }
}

// What gqa_cache_compact does to one slot, decided from the state before the call.
struct CompactSlot {
    int len, base, end;  // old length, context, new length
    int status;
};
__device__ CompactSlot compact_slot(const CompactParams& p, int s) {
    // called by a whole block; the same answer for every thread
    const CacheState& c = p.c;
    CompactSlot r;
    r.len = clamp_len(c.lens[s], c);
    const int nodes = min(max(p.tree_lens != nullptr ? p.tree_lens[s] : p.T, 0), min(p.T, r.len));
    const int m = p.keep_lens[s];
    r.base = r.len - nodes;
    r.end = r.base + m;
    // both checks read before either answers: their look-ups overlap
    const bool range = m >= 0 && m <= nodes;
    bool bad = !range, shared = false;
    const int* keep = p.keep + (size_t)s * p.T;
    if (range) {
        for (int j = threadIdx.x; j < m; j += blockDim.x)
            bad |= keep[j] <= (j > 0 ? keep[j - 1] : -1) || keep[j] >= nodes;
        const int lo = r.base >> c.page_shift, hi = pages_of(r.end, c.page_shift);
        for (int j = lo + threadIdx.x; j < hi; j += blockDim.x) {
            const int page = row_of(c, s)[j];
            shared |= known(page, c) && __ldcg(c.refs + page) > 1;
        }
    }
    bad = __syncthreads_or(bad);
    shared = __syncthreads_or(shared);
    r.status = bad ? GQA_CACHE_INVALID : (shared ? GQA_CACHE_SHARED : GQA_CACHE_DONE);
    return r;
}

// Moves the accepted rows.  A thread owns one 16-byte column of one layer's K or V and walks
// the accepted nodes in order: node keep[j] >= j goes to place j, so a row is overwritten only
// after it was read, and sixteen rows may be read before their sixteen writes.  The rows' places are
// looked up by the block together, kMoveRows at a time.  Bound by the latency of those look-ups and
// two turns of reads: measured on B200, 73 MB (128 slots, trees of 64, 8 layers) in 16 us, 4.5 TB/s.
constexpr int kMoveThreads = 128;
constexpr int kMoveBatch = 16;
constexpr int kMoveRows = 128;
__global__ void __launch_bounds__(kMoveThreads) cache_compact_rows_kernel(const __grid_constant__ CompactParams p) {
    __shared__ int from_[kMoveRows], to_[kMoveRows];  // rows of a layer's pool; -1: not moved
    const CacheState& c = p.c;
    const int s = blockIdx.x;
    let_next();
    wait_before();
    const CompactSlot r = compact_slot(p, s);
    if (blockIdx.y == 0 && threadIdx.x == 0) p.status[s] = r.status;
    if (r.status != GQA_CACHE_DONE) return;
    const int cols = (int)(p.pools.row_bytes / 16);
    const int items = 2 * p.pools.layers * cols;
    const int* row = row_of(c, s);
    const int* keep = p.keep + (size_t)s * p.T;
    const int in_page = (1 << c.page_shift) - 1;
    auto at = [&](int pos) {
        const int page = row[pos >> c.page_shift];
        return known(page, c) ? (page << c.page_shift) + (pos & in_page) : -1;
    };
    const int m = r.end - r.base;
    for (int j0 = 0; j0 < m; j0 += kMoveRows) {
        const int n = min(kMoveRows, m - j0);
        __syncthreads();
        for (int j = threadIdx.x; j < n; j += kMoveThreads) {
            const int node = keep[j0 + j];
            const int to = node > j0 + j ? at(r.base + j0 + j) : -1;
            const int from = to >= 0 ? at(r.base + node) : -1;
            from_[j] = from;
            to_[j] = from >= 0 ? to : -1;
        }
        __syncthreads();
        // (a row that the next kMoveRows read is never written by these: it lies further on)
        for (int item = blockIdx.y * kMoveThreads + threadIdx.x; item < items; item += gridDim.y * kMoveThreads) {
            const int col = item % cols, kv = item / cols & 1, layer = item / cols / 2;
            uint8_t* pool = p.pools.kv[kv] + ((size_t)layer * c.P << c.page_shift) * p.pools.row_bytes + (size_t)col * 16;
            for (int j = 0; j < n; j += kMoveBatch) {
                uint4 x[kMoveBatch];
#pragma unroll
                for (int e = 0; e < kMoveBatch; ++e)
                    if (j + e < n && from_[j + e] >= 0)
                        x[e] = *reinterpret_cast<const uint4*>(pool + (size_t)from_[j + e] * p.pools.row_bytes);
#pragma unroll
                for (int e = 0; e < kMoveBatch; ++e)
                    if (j + e < n && to_[j + e] >= 0)
                        *reinterpret_cast<uint4*>(pool + (size_t)to_[j + e] * p.pools.row_bytes) = x[e];
            }
        }
    }
}

// The lengths and pages after the rows have moved: one warp per slot (a tree spans few pages).
__global__ void __launch_bounds__(128) cache_compact_pages_kernel(const __grid_constant__ CompactParams p) {
    const CacheState& c = p.c;
    const int s = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    let_next();
    wait_before();
    if (s >= c.S || p.status[s] != GQA_CACHE_DONE) return;
    const int len = clamp_len(c.lens[s], c);
    const int nodes = min(max(p.tree_lens != nullptr ? p.tree_lens[s] : p.T, 0), min(p.T, len));
    const int end = len - nodes + p.keep_lens[s];
    __syncwarp();
    int* row = row_of(c, s);
    for (int j = pages_of(end, c.page_shift) + lane; j < pages_of(len, c.page_shift); j += 32) {
        if (known(row[j], c)) atomicSub(c.refs + row[j], 1);
        row[j] = -1;
    }
    if (lane == 0) c.lens[s] = end;
}

// Blocks of the cluster: a block for every 1024 pages of the pool or 8 warp turns of table entries,
// at most 16; one for a small cache, whose steps then need no cluster barrier.  Measured on B200
// with the calls around them: 131 thousand pages and 256 slots of 2048 entries, 20 us a call (25 with
// 8 blocks of twice the threads); 4 thousand pages and 128 slots, a verification step of 34 us
// (39 with a block for every 8192 pages).
int plan_ctas(const PlanParams& p) {
    const long long pages = ((long long)p.c.P + 1023) / 1024, entries = (long long)p.n * ((p.c.M + 255) / 256) / 8;
    int ctas = 1;
    while (ctas < kMostCtas && ctas < (pages > entries ? pages : entries)) ctas *= 2;
    return ctas;
}

template <bool FORK>
cudaError_t launch_plan(const PlanParams& p, cudaStream_t stream) {
    const size_t bytes = sizeof(int) * (6 * (size_t)p.n + (FORK ? 4 : 2) * (size_t)set_size(p.n));
    // per device, set once for the most that a call may need; setting it again is harmless
    static int most_ctas[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {kMostCtas, 1, 1};
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kMostCtas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    int most = dev >= 0 && dev < 64 ? most_ctas[dev] : 0;
    if (most == 0) {
        const size_t largest = sizeof(int) * (6 * (size_t)GQA_CACHE_MAX_REQUESTS +
                                              (FORK ? 4 : 2) * (size_t)set_size(GQA_CACHE_MAX_REQUESTS));
        e = cudaFuncSetAttribute(cache_plan_kernel<FORK>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)largest);
        if (e != cudaSuccess) return e;
        most = 8;  // what every device can place
        int clusters = 0;
        cfg.dynamicSmemBytes = largest;
        if (cudaFuncSetAttribute(cache_plan_kernel<FORK>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
            cudaOccupancyMaxActiveClusters(&clusters, cache_plan_kernel<FORK>, &cfg) == cudaSuccess && clusters > 0)
            most = kMostCtas;
        cudaGetLastError();
        cfg.dynamicSmemBytes = bytes;
        if (dev >= 0 && dev < 64) most_ctas[dev] = most;
    }
    const int ctas = plan_ctas(p) < most ? plan_ctas(p) : most;
    cfg.gridDim = dim3((unsigned)ctas);
    attr[1].val.clusterDim.x = (unsigned)ctas;
    return cudaLaunchKernelEx(&cfg, cache_plan_kernel<FORK>, p);
}

}  // namespace

cudaError_t launch_resize(const PlanParams& p, cudaStream_t stream) { return launch_plan<false>(p, stream); }

cudaError_t launch_fork(const PlanParams& p, const Pools& pools, int sms, cudaStream_t stream) {
    cudaError_t e = launch_plan<true>(p, stream);
    if (e != cudaSuccess) return e;
    // about 48 blocks per SM in all, but none without a piece of a whole page (the case above with
    // its plan: 66 us with 8, 57 with 16, 50 with 48, 52 with 96)
    const long long page_bytes = pools.row_bytes << p.c.page_shift;
    const long long pieces = (page_bytes + kCopyBytes - 1) / kCopyBytes * pools.layers * 2;
    long long each = ((long long)sms * 48 + p.n - 1) / p.n;
    if (each > pieces) each = pieces;
    if (each > 65535) each = 65535;
    return launch_early(cache_tail_copy_kernel, dim3((unsigned)p.n, (unsigned)each), kCopyThreads, 0, stream, p, pools);
}

cudaError_t launch_compact(const CompactParams& p, int sms, cudaStream_t stream) {
    const long long items = 2ll * p.pools.layers * (p.pools.row_bytes / 16);
    // about 7 blocks per SM (what its registers hold) at once, each with some columns
    long long each = ((long long)sms * 7 + p.c.S - 1) / p.c.S;
    const long long most = (items + kMoveThreads - 1) / kMoveThreads;
    if (each > most) each = most;
    cudaError_t e = launch_early(cache_compact_rows_kernel, dim3((unsigned)p.c.S, (unsigned)each), kMoveThreads, 0, stream, p);
    if (e != cudaSuccess) return e;
    return launch_early(cache_compact_pages_kernel, dim3((unsigned)((p.c.S + 3) / 4)), 128, 0, stream, p);
}

}  // namespace gqa
