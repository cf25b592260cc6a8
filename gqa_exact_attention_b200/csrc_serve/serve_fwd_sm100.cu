// Attention over packed prompts and of draft trees over a cache, for sm_100a: persistent,
// warp-specialised, TMA + tcgen05.
//
// The row softmax in one pass: S = Q K^T of a 128-row tile and a 128-key block in tensor
// memory, P = 2^(c s - m) in bf16 over it (c = scale log2 e; the row sums keep the unrounded
// P in fp32), O += P V in tensor memory.  m is a reference maximum that moves only when a
// block's maximum passes it by more than 8 octaves.
//
// Work comes in units: a group of NT tiles of one sequence and head (or head group, whose g
// query heads fold into a tile's rows).  Two schedules over them:
//  - LIST (many tiles: prompts): a sorted list of tile groups, whole units, dealt over the
//    CTAs in alternating direction; bound by the tensor pipe.
//  - ranges (few rows over many keys: trees, short prompts): all units' key blocks in one
//    row, cut into one equal range per CTA.  Without a causal mask every CTA streams the same
//    number of blocks whatever the lengths are.  A causal unit counts all key blocks of its
//    sequence, those past its diagonal too, so CTAs at a prompt's early tiles have less to do
//    than those at its late ones.  A unit that several CTAs share leaves fp32 partials, which a
//    second kernel joins in the order of the keys.  Bound by HBM.
// Roles:
//   warpgroup 0, warp 0   TMA producer: Q tiles once per unit, then a ring of K/V blocks.
//   warpgroup 0, warp 1   MMA issuer (one elected lane).
//   warpgroup 0, warp 3   scheduler: posts the CTA's pieces of units in a short ring.
//   warpgroup 0, warp 2   clears the rows of V behind a sequence's last key in its last block:
//                         they belong to another sequence or to nobody, and 0 * NaN is NaN.
//   warpgroups 1..NT      softmax, one per tile; thread = tile row = TMEM lane.
//   warpgroup NT + 1      (NT = 2 only) epilogue.  With NT = 1 the softmax warpgroup writes.
// NT = 2: one CTA per SM.  NT = 1: two, so that one's unit changes overlap the other's stream.
//
// Measured on B200 (several boxes): 64 causal prompts of 1024 to 2048 tokens (Hq 32, Hk 8, d 128)
// 1.64-1.71 ms, 770-800 TFLOP/s under the power cap (tensor pipe and exponentials each about half
// busy: the chain S, softmax, P V of two tiles is latency; 64-key halves of S, dynamic units and
// programmatic launches were all slower); 64 sequences of up to 16384 keys with 16 drafted tokens
// 0.52-0.62 ms from pages of 16, 4.6-5.5 TB/s, 0.45 ms from pages of 64, 6.2 TB/s; one sequence of
// 8192 keys 28 us; one causal prompt of 2048 in ranges (Hq 8, Hk 2, d 64) 36 us.
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "exp2_poly4.cuh"
#include "launch_serve.h"
#include "ptx_sm100.cuh"
#include "serve_params.h"
#include "serve_ranges.h"

namespace gqa {

__device__ unsigned int g_serve_status = 0;

namespace {

using namespace ptx;

constexpr int kBlockM = kServeBlockM;
constexpr int kBlockN = kServeBlockN;

constexpr int kSegs = 4;  // pieces that the scheduler warp may be ahead

enum Mode { kVarlenRanges, kVarlenList, kTreeDense, kTreePaged };

template <int HD, int NT, bool RANGES>
struct Cfg {
    static constexpr int kRowBytes = 2 * HD;  // one row of Q, K or V
    // a tile is kChunks column chunks of 128 rows x 128 bytes (the swizzle span)
    static constexpr int kChunks = HD / 64;
    static constexpr int kChunkBytes = 128 * 128;
    static constexpr int kTileBytes = kChunks * kChunkBytes;
    static constexpr int kSlots = (NT == 2) ? (HD == 128 ? 4 : 8) : (HD == 128 ? 2 : 5);
    static constexpr int kPvSteps = kBlockN / 16;
    static constexpr uint32_t kPvStepBytes = 16 * 128;  // keys of one step, one chunk
    static constexpr bool kEpilogueWG = (NT == 2);
    static constexpr int kWarpgroups = 1 + NT + (kEpilogueWG ? 1 : 0);
    static constexpr int kThreads = kWarpgroups * 128;
    static constexpr int kCtasPerSm = kEpilogueWG ? 1 : 2;
    // registers at launch (65536 / (threads x CTAs)), then redistributed with setmaxnreg; the
    // sum over the warpgroups stays what the block was launched with
    static constexpr int kLaunchRegs = ((65536 / (kThreads * kCtasPerSm)) / 8) * 8;
    // (the joining epilogue of the ranges schedule takes more than the list's)
    static constexpr int kRegsLoad = NT == 2 && !RANGES ? 104 : 80;
    static constexpr int kRegsSoftmax = NT == 2 ? 168 : 176;
    static constexpr int kRegsEpilogue =
        kEpilogueWG ? kWarpgroups * kLaunchRegs - kRegsLoad - NT * kRegsSoftmax : 0;
    static_assert(kRegsLoad + NT * kRegsSoftmax + kRegsEpilogue == kWarpgroups * kLaunchRegs,
                  "register split must add up to the launch allocation");
    static constexpr int kTmemCols = (NT * 128 + NT * HD) <= 256 ? 256 : 512;
    // d = 64: S and O leave columns for P (two tiles: 384 of 512; one: 192 of 256), so P has its own and
    // the next block's S is computed while this block's softmax runs
    static constexpr bool kSepP = HD == 64;
    static constexpr int kNumBars = 2 * kSlots + 9 * NT + 4 + (kSepP ? 2 * NT : 0) + 2 * kSegs;
    // warps that read the pieces the scheduler posts: producer, MMA, clearing, softmax, epilogue
    static constexpr int kReaders = 3 + 4 * NT + (kEpilogueWG ? 4 : 0);
    static constexpr int kStatsBytes = kEpilogueWG ? 2 * NT * 2 * 128 * 4 : 0;  // (m, l), 2 buffers
    static constexpr int kOStageBytes = kEpilogueWG ? 128 * 128 : 0;
    static constexpr int kPreBytes = (kServeOwnPrefix + 1) * 8;
    static constexpr int kSmemBytes = 1024 /* alignment slack */ + NT * kTileBytes + kSlots * kTileBytes +
                                      kOStageBytes + 8 * kNumBars + kStatsBytes + kPreBytes + 16 + kSegs * 128;
    static_assert(kSmemBytes * kCtasPerSm + 1024 * kCtasPerSm <= 233472, "shared memory per SM");
    // Of each 16 exponential pairs of an unmasked 32-key chunk, this many take the polynomial instead
    // of the special-function unit.  Measured on B200 over 64 causal prompts: d = 64, 0 pairs 2.26 ms,
    // 2 pairs 1.98, 3 pairs 1.92; d = 128, 0 and 2 pairs 1.63 ms, 4 pairs 1.70.
    static constexpr int kPolyPairs = HD == 128 ? 0 : 3;
    static constexpr uint32_t kIdescQK = idesc_bf16_f32(128, 128, false);
    static constexpr uint32_t kIdescPV = idesc_bf16_f32(128, HD, true);
    __device__ static uint64_t sdesc(uint32_t saddr, uint32_t lbo) { return sdesc_sw128(saddr, lbo, 1024); }
    __device__ static void mma_s(uint32_t d, uint64_t a, uint64_t b, uint32_t acc) { mma_ss(d, a, b, kIdescQK, acc); }
    __device__ static void mma_pv(uint32_t d, uint32_t a, uint64_t b, uint32_t acc) { mma_ts(d, a, b, kIdescPV, acc); }
    __host__ __device__ static constexpr int s_col(int t) { return t * 128; }
    __host__ __device__ static constexpr int o_col(int t) { return NT * 128 + t * HD; }
    __host__ __device__ static constexpr int p_col(int t) {
        return kSepP ? NT * 128 + NT * HD + t * 64 : s_col(t);
    }
    static constexpr int kPAfterO = NT * HD;  // separate P lies this many columns past O
};

template <uint32_t R>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <uint32_t R>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// A small input (a bound, a length, a table entry, a mask word).  An ordinary load: the kernel may
// have started before the one that writes it ended, so the read-only path (__ldg) is not for it.
template <class T>
__device__ __forceinline__ T fresh(const T* p) { return *p; }

// ---------------------------------------------------------------- sequences, units, segments

struct Seq {
    int q0, lq;  // first query row (0 for a tree: the batch coordinate selects it) and queries
    int k0, sk;  // first key row (0 for a cache) and keys
    int nodes;   // tree: its nodes, the last keys
};
template <int MODE>
__device__ __forceinline__ Seq seq_of(const ServeParams& p, int b) {
    Seq s;
    if constexpr (MODE == kVarlenRanges || MODE == kVarlenList) {
        s.q0 = min(max(fresh(p.cu_q + b), 0), p.total_q);
        s.lq = min(max(fresh(p.cu_q + b + 1), s.q0), p.total_q) - s.q0;
        s.k0 = min(max(fresh(p.cu_k + b), 0), p.total_k);
        s.sk = min(max(fresh(p.cu_k + b + 1), s.k0), p.total_k) - s.k0;
        s.nodes = 0;
    } else {
        s.q0 = s.k0 = 0;
        s.lq = p.T;
        s.sk = min(max(fresh(p.seqlens + b), 0), p.cap);
        s.nodes = min(max(p.tree_lens != nullptr ? fresh(p.tree_lens + b) : p.T, 0), min(p.T, s.sk));
    }
    return s;
}

// The steps that a unit counts in the ranges schedule: its key blocks (one without keys: its rows
// are written all the same), or one where units are not split.
__device__ __forceinline__ int unit_steps(const ServeParams& p, int sk) {
    return p.whole ? 1 : max((sk + kBlockN - 1) / kBlockN, 1);
}
template <int NT>
__device__ __forceinline__ int tile_groups(const ServeParams& p, int lq) {
    return (lq + NT * p.pos_per_tile - 1) / (NT * p.pos_per_tile);
}

// A CTA's piece of one unit, posted in shared memory by the scheduler warp.
template <int NT>
struct Seg {
    int b, hg, kvh;  // b < 0: no more pieces
    Seq s;
    int pos0[NT];  // first query position of tile t
    int n[NT];     // key blocks of tile t in this piece
    int kb_lo, nblk;
    int parts;  // pieces of the unit (1: this is the whole unit)
    int slot;   // where this piece's partials go
    // rows of V behind the last key in the last block: they are cleared before P V
    __device__ __forceinline__ bool dirty() const { return nblk > 0 && (kb_lo + nblk) * kBlockN > s.sk; }
};

struct Walk {
    long long x, x0, x_end;  // ranges: position in the row of blocks; list: unit
    long long all;           // blocks or units in all
    int ctas;                // CTAs that take part
    int b;
    ServeBound bound;  // ranges: the unit of the first piece
};
// the last sequence that starts at or before step x
__device__ __forceinline__ int seq_at(const ServeParams& p, const long long* pre, long long x) {
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The unit that step x of sequence b belongs to, and how CTAs share it.
struct UnitAt {
    Seq s;
    int hg, mt;
    int blk, steps;  // x is its step blk of `steps`
    UnitShares by;
};
template <int NT, int MODE>
__device__ __forceinline__ UnitAt unit_at(const ServeParams& p, const long long* pre, const Walk& w, int b, long long x) {
    UnitAt u;
    u.s = seq_of<MODE>(p, b);
    u.steps = unit_steps(p, u.s.sk);
    const long long y = x - pre[b];
    const int unit = (int)mul_div(y, 1, u.steps);
    u.blk = (int)(y - (long long)unit * u.steps);
    const int groups = tile_groups<NT>(p, u.s.lq);
    u.hg = unit / groups;
    u.mt = unit - u.hg * groups;
    if (p.whole) u.by = {0, 1, 0};
    else u.by = unit_shares(w.all, w.ctas, x - u.blk, u.steps);
    return u;
}

template <int NT, int MODE>
__device__ __forceinline__ Walk walk_begin(const ServeParams& p, const long long* pre) {
    Walk w{};
    if constexpr (MODE == kVarlenList) {
        w.ctas = (int)gridDim.x;
        w.all = (long long)fresh(p.list_len) * p.n_hg;
        w.x = blockIdx.x;
        w.x_end = w.all;
    } else {
        w.all = pre[p.B];
        w.ctas = range_ctas(w.all, p.min_blocks, (int)gridDim.x);
        if ((int)blockIdx.x < w.ctas && w.all > 0) {
            w.x = w.x0 = range_start(w.all, w.ctas, (int)blockIdx.x);
            w.x_end = range_start(w.all, w.ctas, (int)blockIdx.x + 1);
            w.b = seq_at(p, pre, w.x);
        }
    }
    return w;
}

template <int NT, int MODE>
__device__ __forceinline__ bool next_seg(Walk& w, Seg<NT>& g, const ServeParams& p, const long long* pre) {
    if (w.x >= w.x_end) return false;
    int mt, hi;
    if constexpr (MODE == kVarlenList) {
        // dealt in alternating direction: round r gives its k-th unit to CTA k or ctas - 1 - k
        const int u = (int)w.x, r = u / w.ctas, k = u - r * w.ctas;
        const int at = (r & 1) && (long long)(r + 1) * w.ctas <= w.all ? r * w.ctas + w.ctas - 1 - k : u;
        uint32_t pair, hg;
        fastdivmod((uint32_t)at, p.div_hg, pair, hg);
        const int2 e = fresh(p.list + pair);
        g.b = e.x;
        g.hg = (int)hg;
        mt = e.y;
        g.s = seq_of<MODE>(p, g.b);
        g.kb_lo = 0;
        hi = 0x7fffffff;
        g.parts = 1;
        g.slot = 0;
        w.x += w.ctas;
    } else {
        while (w.x >= pre[w.b + 1]) ++w.b;
        g.b = w.b;
        const UnitAt u = unit_at<NT, MODE>(p, pre, w, g.b, w.x);
        const int len = (int)min((long long)(u.steps - u.blk), w.x_end - w.x);
        g.s = u.s;
        g.hg = u.hg;
        mt = u.mt;
        g.kb_lo = p.whole ? 0 : u.blk;
        hi = p.whole ? 0x7fffffff : u.blk + len;
        g.parts = u.by.parts;
        g.slot = piece_slot((int)blockIdx.x, w.x == w.x0);
        if (w.x == w.x0)
            w.bound = {g.b, u.hg, u.mt, u.s.q0, u.s.lq, u.by.cta0, u.blk > 0 ? u.by.parts : 0, u.by.first_slot};
        w.x += len;
    }
    g.kvh = p.pack ? g.hg : (int)fastdiv((uint32_t)g.hg, p.div_g);
    g.nblk = 0;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        g.pos0[t] = (mt * NT + t) * p.pos_per_tile;
        int end = 0;
        if (g.pos0[t] < g.s.lq) {
            int keys = g.s.sk;
            if constexpr (MODE == kVarlenRanges || MODE == kVarlenList) {
                // causal: bottom-right aligned to the sequence's own lengths
                const int last = min(g.pos0[t] + p.pos_per_tile, g.s.lq) - 1;
                if (p.causal) keys = max(0, min(keys, last + 1 + (g.s.sk - g.s.lq)));
            } else {
                if (g.pos0[t] >= g.s.nodes) keys = 0;  // padding rows only
            }
            end = (keys + kBlockN - 1) / kBlockN;
        }
        g.n[t] = max(0, min(hi, end) - g.kb_lo);
        g.nblk = max(g.nblk, g.n[t]);
    }
    return true;
}

// a[t] for a run-time t without dynamic indexing (keeps the arrays in registers)
template <int NT>
__device__ __forceinline__ int pick(const int (&a)[NT], int t) {
    int v = a[0];
#pragma unroll
    for (int i = 1; i < NT; ++i) v = (t == i) ? a[i] : v;
    return v;
}

// Row r of a tile -> (query position, q-head); ok when it is an output row.
struct RowMap {
    int pos, head;
    bool ok;
};
__device__ __forceinline__ RowMap row_map(const ServeParams& p, int lq, int pos0, int hg, int row) {
    RowMap m;
    if (p.pack) {
        uint32_t pr, hh;
        fastdivmod((uint32_t)row, p.div_g, pr, hh);
        m.pos = pos0 + (int)pr;
        m.head = hg * p.g + (int)hh;
        m.ok = row < p.rows_valid && m.pos < lq;
    } else {
        m.pos = pos0 + row;
        m.head = hg;
        m.ok = m.pos < lq;
    }
    return m;
}

// Where row (pos, head) of a sequence lies in out (element index) and lse.
template <int MODE>
__device__ __forceinline__ size_t out_row(const ServeParams& p, int b, const Seq& s, const RowMap& m) {
    if constexpr (MODE == kTreeDense || MODE == kTreePaged)
        return ((size_t)b * p.T + m.pos) * p.Hq + m.head;
    else
        return (size_t)(s.q0 + m.pos) * p.Hq + m.head;
}
template <int MODE>
__device__ __forceinline__ size_t lse_row(const ServeParams& p, int b, const Seq& s, const RowMap& m) {
    if constexpr (MODE == kTreeDense || MODE == kTreePaged)
        return ((size_t)b * p.Hq + m.head) * p.T + m.pos;
    else
        return (size_t)m.head * p.total_q + s.q0 + m.pos;
}

constexpr float kLn2 = 0.69314718055994530942f;

// 8 N columns of a row, scaled, to fp32 or bf16 output
template <int N>
__device__ __forceinline__ void store_cols(const ServeParams& p, size_t at, const float (&f)[8 * N], float inv) {
    if (p.out_bf16 != nullptr) {
        uint4* dst = reinterpret_cast<uint4*>(p.out_bf16 + at);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float* x = f + 8 * i;
            dst[i] = make_uint4(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv),
                                pack_bf16x2(x[4] * inv, x[5] * inv), pack_bf16x2(x[6] * inv, x[7] * inv));
        }
    } else {
        float4* dst = reinterpret_cast<float4*>(p.out + at);
#pragma unroll
        for (int i = 0; i < 2 * N; ++i)
            dst[i] = make_float4(f[4 * i] * inv, f[4 * i + 1] * inv, f[4 * i + 2] * inv, f[4 * i + 3] * inv);
    }
}

// Four columns of a row of a partial tile.  The tile's 128 rows lie side by side, so that a warp,
// whose lanes are rows, writes and reads whole lines.
template <int HD>
__device__ __forceinline__ float4* part_at(const ServeParams& p, int tile, int col4, int row) {
    return reinterpret_cast<float4*>(p.part_o) + ((size_t)tile * (HD / 4) + col4) * 128 + row;
}

// Writes one tile row from TMEM: O / l and LSE = (m + log2 l) ln 2 to out and lse, or (PART) the
// same in fp32 and log2 units to the piece's slot.  `has`: the tile had keys in this piece;
// `valid`: the row's result counts (a tree's padding rows give 0 and -inf).  Arrives on o_empty
// once O is in registers, so the next unit's PV may overwrite it.
template <int HD, int NT, int MODE, bool PART>
__device__ __forceinline__ void write_row(const ServeParams& p, uint32_t o_addr, const RowMap& rm, const Seg<NT>& g,
                                          int t, int row, bool has, bool idle, bool valid, float m, float l,
                                          uint32_t o_empty_bar) {
    // (no key: 0, whatever V holds; a NaN sum is not 0)
    const bool zero = !has || !valid || l == 0.f;
    const float inv_l = zero ? 0.f : 1.f / l;
    const float lse2 = zero ? -INFINITY : m + __log2f(l);
    const size_t at = PART ? 0 : out_row<MODE>(p, g.b, g.s, rm) * HD;
#pragma unroll
    for (int ch = 0; ch < HD / 32; ++ch) {
        uint32_t r[32];
        if (has && !idle) {
            tmem_ld32(o_addr + ch * 32, r);
            tmem_wait_ld();
        }
        if (has && ch == HD / 32 - 1) {
            tc_fence_before();
            mbar_arrive(o_empty_bar);
        }
        if (!rm.ok || idle) continue;
        if constexpr (PART) {
            if (zero) continue;  // (the join skips a part whose LSE is -inf)
            const float* f = reinterpret_cast<const float*>(r);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                __stcg(part_at<HD>(p, g.slot * NT + t, ch * 8 + i, row),
                       make_float4(f[4 * i] * inv_l, f[4 * i + 1] * inv_l, f[4 * i + 2] * inv_l, f[4 * i + 3] * inv_l));
        } else {
            if (zero) {
#pragma unroll
                for (int i = 0; i < 32; ++i) r[i] = 0u;
            }
            store_cols<4>(p, at + ch * 32, reinterpret_cast<const float(&)[32]>(r), inv_l);
        }
    }
    if (rm.ok) {
        if constexpr (PART) __stcg(p.part_lse + ((size_t)g.slot * NT + t) * 128 + row, lse2);
        else p.lse[lse_row<MODE>(p, g.b, g.s, rm)] = lse2 * kLn2;
    }
}
// Either of the two, by the unit's pieces.
template <int HD, int NT, int MODE>
__device__ __forceinline__ void write_piece(const ServeParams& p, uint32_t o_addr, const RowMap& rm, const Seg<NT>& g,
                                            int t, int row, bool has, bool idle, bool valid, float m, float l,
                                            uint32_t o_empty_bar) {
    if (g.parts == 1) write_row<HD, NT, MODE, false>(p, o_addr, rm, g, t, row, has, idle, valid, m, l, o_empty_bar);
    else write_row<HD, NT, MODE, true>(p, o_addr, rm, g, t, row, has, idle, valid, m, l, o_empty_bar);
}

// Paged KV: the block-table entries of one sequence, cached in the producer warp's
// registers 32 at a time (lane i holds entry base + i), with the next 32 already loaded
// (lane i of w1 holds base + 32 + i) so that moving on does not wait for memory.
// Warp-collective: every lane calls it with the same arguments.
struct PageCache {
    int b = -1;
    int base = 0;
    int w0 = -1, w1 = -1;
};
__device__ __forceinline__ int table_entry(const ServeParams& p, int b, int i) {
    return (i < p.table_stride) ? fresh(p.block_table + (size_t)b * p.table_stride + i) : -1;
}
__device__ __forceinline__ int page_of(PageCache& pc, const ServeParams& p, int b, int page_i,
                                       int lane) {
    if (b != pc.b || page_i < pc.base || page_i >= pc.base + 64) {
        pc.b = b;
        pc.base = page_i & ~31;
        pc.w0 = table_entry(p, b, pc.base + lane);
        pc.w1 = table_entry(p, b, pc.base + 32 + lane);
    } else if (page_i >= pc.base + 32) {
        pc.base += 32;
        pc.w0 = pc.w1;
        pc.w1 = table_entry(p, b, pc.base + 32 + lane);
    }
    return __shfl_sync(0xffffffffu, pc.w0, page_i - pc.base);
}

// Bounded wait on an mbarrier phase.  Returns false when the CTA is aborting or when this wait
// ran past the time limit (then it records the timeout and starts the abort).
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag,
                                             const ServeParams& p) {
    if (mbar_try_wait(bar, parity)) return true;
    uint64_t t0 = globaltimer();
    uint32_t spins = 0;
    while (!mbar_try_wait(bar, parity)) {
        if ((++spins & 255u) == 0) {
            if (*abort_flag) return false;
            if ((long long)(globaltimer() - t0) > p.timeout_ns) {
                *abort_flag = 1u;
                atomicOr(&g_serve_status, 1u);
                return false;
            }
        }
    }
    return true;
}

// Wait used during teardown: ignores the abort flag, gives up silently at its own limit
// (p.drain_ns, at least 1 s: copies and MMAs already issued must land before the CTA's shared
// and tensor memory are released).
__device__ __forceinline__ void wait_drain(uint32_t bar, uint32_t parity, const ServeParams& p) {
    uint64_t t0 = globaltimer();
    while (!mbar_try_wait(bar, parity)) {
        if ((long long)(globaltimer() - t0) > p.drain_ns) return;
    }
}

// Word i of a row's mask over the tree's nodes (32 of them): before the tree every key is seen,
// behind its last node none is.  No mask: a row whose result is not kept.
__device__ __forceinline__ uint32_t tree_word(const int* row, int i, int nodes) {
    if (i < 0) return 0xffffffffu;
    const int left = nodes - i * 32;
    if (left <= 0) return 0u;
    const uint32_t w = row != nullptr ? (uint32_t)fresh(row + i) : 0xffffffffu;
    return left >= 32 ? w : w & ((1u << left) - 1u);
}

// pre[b] = key blocks of all units of the sequences before b, by all threads of a block; the
// caller synchronises afterwards.
template <int NT, int MODE, int THREADS>
__device__ void block_prefix(const ServeParams& p, long long* pre) {
    __shared__ long long sums[THREADS / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long carry = 0;
    for (int b0 = 0; b0 < p.B; b0 += THREADS) {
        const int b = b0 + (int)threadIdx.x;
        long long x = 0;
        if (b < p.B) {
            const Seq s = seq_of<MODE>(p, b);
            x = (long long)p.n_hg * tile_groups<NT>(p, s.lq) * unit_steps(p, s.sk);
        }
        long long incl = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) sums[warp] = incl;
        __syncthreads();
        long long before = 0, total = 0;
#pragma unroll
        for (int i = 0; i < THREADS / 32; ++i) {
            if (i < warp) before += sums[i];
            total += sums[i];
        }
        if (b < p.B) pre[b + 1] = carry + before + incl;
        carry += total;
        __syncthreads();
    }
    if (threadIdx.x == 0) pre[0] = 0;
}

template <int HD, int NT, int MODE>
__global__ void __launch_bounds__(Cfg<HD, NT, MODE != kVarlenList>::kThreads, Cfg<HD, NT, MODE != kVarlenList>::kCtasPerSm)
    serve_fwd_kernel(const __grid_constant__ ServeParams p) {
    using C = Cfg<HD, NT, MODE != kVarlenList>;
    constexpr bool kPaged = MODE == kTreePaged;
    constexpr bool kTree = MODE == kTreePaged || MODE == kTreeDense;
    constexpr bool kRanges = MODE != kVarlenList;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);

    const uint32_t sQ = base;
    const uint32_t sKV = base + NT * C::kTileBytes;
    const uint32_t sO = sKV + C::kSlots * C::kTileBytes;  // 1024-aligned staging (NT == 2)
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + NT * C::kTileBytes + C::kSlots * C::kTileBytes +
                                                 C::kOStageBytes);
    float* stats = reinterpret_cast<float*>(bars + C::kNumBars);  // [2][NT][2][128]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(stats) + C::kStatsBytes);
    const uint32_t bar0 = smem_u32(bars);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    // blocks before each sequence (the ranges schedule)
    long long* own_pre = reinterpret_cast<long long*>(tmem_slot + 4);
    Seg<NT>* segs = reinterpret_cast<Seg<NT>*>(own_pre + kServeOwnPrefix + 1);
    static_assert(sizeof(Seg<NT>) <= 128, "room for a piece");
    auto seg_full = [&](uint32_t i) { return bar0 + 8u * (C::kNumBars - 2 * kSegs + i % kSegs); };
    auto seg_empty = [&](uint32_t i) { return bar0 + 8u * (C::kNumBars - kSegs + i % kSegs); };

    auto kv_full = [&](int s) { return bar0 + 8u * s; };
    auto kv_empty = [&](int s) { return bar0 + 8u * (C::kSlots + s); };
    auto q_full = [&](int t) { return bar0 + 8u * (2 * C::kSlots + t); };
    auto q_empty = [&](int t) { return bar0 + 8u * (2 * C::kSlots + NT + t); };
    auto s_full = [&](int t) { return bar0 + 8u * (2 * C::kSlots + 2 * NT + t); };
    auto p_full = [&](int t) { return bar0 + 8u * (2 * C::kSlots + 3 * NT + t); };
    auto o_full = [&](int t) { return bar0 + 8u * (2 * C::kSlots + 4 * NT + t); };
    auto o_empty = [&](int t) { return bar0 + 8u * (2 * C::kSlots + 5 * NT + t); };
    // One barrier per statistics buffer: the softmax may post a unit's statistics before
    // the epilogue has waited for the previous unit's (a one-block unit's S needs nothing
    // from the epilogue), and a parity wait must never fall two phases behind.  Per buffer,
    // the next post needs the epilogue to have released O_t of the unit before.
    auto st_full = [&](int t, uint32_t buf) { return bar0 + 8u * (2 * C::kSlots + 6 * NT + 2 * t + buf); };
    const uint32_t mma_done = bar0 + 8u * (2 * C::kSlots + 8 * NT);
    // never arrived on: the injected stall waits on it (failure-detection tests)
    const uint32_t stall_bar = bar0 + 8u * (2 * C::kSlots + 8 * NT + 1);
    // a V block with rows behind a sequence's last key has landed (MMA -> warp 2), and they are
    // cleared (warp 2 -> MMA).  Warp 2 does not follow the ring by itself: it would miss phases.
    const uint32_t v_dirty = bar0 + 8u * (2 * C::kSlots + 8 * NT + 3);
    const uint32_t v_clean = bar0 + 8u * (2 * C::kSlots + 8 * NT + 2);
    // the first half of P_t (64 keys) is there: its P V runs while the softmax does the second
    // (not with separate P: there S runs meanwhile, and the hand-off cost 2 % at d = 64; at
    // d = 128 it gains 1-4 %)
    [[maybe_unused]] auto p_half = [&](int t) { return bar0 + 8u * (2 * C::kSlots + 8 * NT + 4 + t); };
    // separate P (kSepP): S_t read into registers (softmax -> MMA), P_t.V done (MMA -> softmax)
    [[maybe_unused]] auto s_free = [&](int t) { return bar0 + 8u * (2 * C::kSlots + 9 * NT + 4 + t); };
    [[maybe_unused]] auto p_free = [&](int t) { return bar0 + 8u * (2 * C::kSlots + 9 * NT + 4 + NT + t); };

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int wg = warp >> 2;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kSlots; ++s) {
            mbar_init(kv_full(s), 1);
            mbar_init(kv_empty(s), 1);
        }
        for (int t = 0; t < NT; ++t) {
            mbar_init(q_full(t), 1);
            mbar_init(q_empty(t), 1);
            mbar_init(s_full(t), 1);
            mbar_init(p_half(t), 128);
            mbar_init(p_full(t), 128);
            mbar_init(o_full(t), 1);
            mbar_init(o_empty(t), 128);
            mbar_init(st_full(t, 0), 128);
            mbar_init(st_full(t, 1), 128);
        }
        mbar_init(mma_done, 1);
        mbar_init(stall_bar, 1);
        mbar_init(v_dirty, 1);
        mbar_init(v_clean, 1);
        for (uint32_t i = 0; i < kSegs; ++i) {
            mbar_init(seg_full(i), 1);
            mbar_init(seg_empty(i), C::kReaders);
        }
        if constexpr (C::kSepP) {
            for (int t = 0; t < NT; ++t) {
                mbar_init(s_free(t), 128);
                mbar_init(p_free(t), 1);
            }
        }
        *abort_flag = 0u;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&p.tm_q);
        prefetch_tmap(&p.tm_k);
        prefetch_tmap(&p.tm_v);
    }
    if (warp == 1) {
        tmem_alloc<C::kTmemCols>(smem_u32(tmem_slot));
        tmem_relinquish();
        tc_fence_before();
    }
    if constexpr (kRanges) wait_before();
    const long long* pre = p.pre;
    if constexpr (kRanges) {
        // the blocks of each sequence's units, summed up by every CTA for itself
        if (pre == nullptr) {
            block_prefix<NT, MODE, C::kThreads>(p, own_pre);
            pre = own_pre;
        }
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // (the next kernel's CTAs come when every CTA here has its tensor memory: they never hold what
    // one of these still waits for)
    if constexpr (kRanges) let_next();

    // The next piece for this warp (its si-th), or NULL: none, or the CTA is aborting (ok false).
    auto next_piece = [&](uint32_t si, bool& ok) -> const Seg<NT>* {
        ok = __all_sync(0xffffffffu, wait_bounded(seg_full(si), (si / kSegs) & 1u, abort_flag, p));
        const Seg<NT>* g = segs + si % kSegs;
        return ok && g->b >= 0 ? g : nullptr;
    };
    // This warp has read its si-th piece.
    auto done_piece = [&](uint32_t si) {
        __syncwarp();
        if (lane == 0) mbar_arrive(seg_empty(si));
    };

    if (wg == 0) {
        regs_dec<C::kRegsLoad>();
        if (warp == 0) {
            // -------------------------------------------------------- TMA producer
            // The whole warp runs the loop (so its values stay warp-uniform); one elected
            // lane issues the copies.
            uint32_t ld = 0;       // K/V ring loads issued (K and V each count one)
            uint32_t qn[NT] = {};  // Q loads issued per tile
            bool ok = true;
            PageCache pcache;      // paged KV only
            // Q_t of a unit, once the previous unit's last S_t has read the buffer
            auto load_q = [&](const Seg<NT>& g, int t) {
                if (g.n[t] == 0 || !ok) return;
                if (qn[t] > 0)
                    ok = __all_sync(0xffffffffu, wait_bounded(q_empty(t), (qn[t] - 1) & 1u, abort_flag, p));
                if (!ok) return;
                if (elect_one()) {
                    const int rows = p.pack ? p.rows_valid : kBlockM;
                    mbar_arrive_expect_tx(q_full(t), (uint32_t)(rows * C::kRowBytes));
                    const int hcoord = p.pack ? g.hg * p.g : g.hg;
#pragma unroll
                    for (int c = 0; c < C::kChunks; ++c)
                        tma_load_4d_hint(sQ + t * C::kTileBytes + c * C::kChunkBytes, &p.tm_q,
                                         q_full(t), c * 64, hcoord, g.s.q0 + g.pos0[t], kTree ? g.b : 0,
                                         l2_policy_evict_first());
                }
                __syncwarp();
                ++qn[t];
            };
            // Injected stall (failure-detection tests): a wait that nothing completes runs
            // out at the wait limit and aborts the CTA, as a copy that never lands would.
            if (p.inject_stall) ok = __all_sync(0xffffffffu, wait_bounded(stall_bar, 0u, abort_flag, p));
            // Load order per unit: Q_0, K_0, Q_1.., V_0, K_1, V_1, ...  The MMA warp may
            // issue a unit's first S_0 while the unit before still runs on tile 1, so K_0
            // must not queue behind Q_1 (which waits for that unit's last S_1).
            for (uint32_t si = 0; ok; ++si) {
                const Seg<NT>* const piece = next_piece(si, ok);
                if (piece == nullptr) break;
                const Seg<NT> g = *piece;
                done_piece(si);
                load_q(g, 0);
                for (int it = 0; it < g.nblk && ok; ++it) {
                    const int kpos = (g.kb_lo + it) * kBlockN;
                    // paged KV: the block's 128 keys come from 128 / page_rows pages (one
                    // page row range each); sub-ranges at or past this sequence's key count
                    // take a page coordinate past the pool, which TMA fills with zeros
                    // (masked anyway), so no table entry past the sequence is used
                    [[maybe_unused]] int pg[8], prow[8];
                    [[maybe_unused]] const int nsub = kPaged ? kBlockN / p.page_rows : 1;
                    if constexpr (kPaged) {
#pragma unroll
                        for (int sub = 0; sub < 8; ++sub) {
                            if (sub >= nsub) break;
                            const int key0 = kpos + sub * p.page_rows;
                            const int page = page_of(pcache, p, g.b, key0 >> p.page_shift, lane);
                            pg[sub] = key0 < g.s.sk ? page : p.num_pages;
                            prow[sub] = key0 & ((1 << p.page_shift) - 1);
                        }
                    }
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const int slot = ld % C::kSlots;
                        if (ld >= (uint32_t)C::kSlots)
                            ok = __all_sync(0xffffffffu, wait_bounded(kv_empty(slot), ((ld / C::kSlots) - 1) & 1u, abort_flag, p));
                        if (!ok) break;
                        if (elect_one()) {
                            mbar_arrive_expect_tx(kv_full(slot), (uint32_t)C::kTileBytes);
                            const void* tm = w == 0 ? (const void*)&p.tm_k : (const void*)&p.tm_v;
                            const uint64_t pol = p.kv_shared ? l2_policy_evict_last() : l2_policy_evict_first();
                            if constexpr (!kPaged) {
#pragma unroll
                                for (int c = 0; c < C::kChunks; ++c)
                                    tma_load_4d_hint(sKV + slot * C::kTileBytes + c * C::kChunkBytes, tm,
                                                     kv_full(slot), c * 64, g.kvh, g.s.k0 + kpos, kTree ? g.b : 0, pol);
                            } else {
#pragma unroll
                                for (int sub = 0; sub < 8; ++sub) {
                                    if (sub >= nsub) break;
#pragma unroll
                                    for (int c = 0; c < C::kChunks; ++c)
                                        tma_load_4d_hint(sKV + slot * C::kTileBytes + c * C::kChunkBytes +
                                                             sub * p.page_rows * 128,
                                                         tm, kv_full(slot), c * 64, g.kvh, prow[sub],
                                                         pg[sub], pol);
                                }
                            }
                        }
                        __syncwarp();
                        ++ld;
                        if (it == 0 && w == 0) {
#pragma unroll
                            for (int t = 1; t < NT; ++t) load_q(g, t);
                        }
                    }
                }
            }
            if (!ok) {
                // let the copies already issued land before the CTA's memory is released
                const uint32_t first = ld > (uint32_t)C::kSlots ? ld - C::kSlots : 0u;
                for (uint32_t l = first; l < ld; ++l)
                    wait_drain(kv_full(l % C::kSlots), (l / C::kSlots) & 1u, p);
                for (int t = 0; t < NT; ++t)
                    if (qn[t] > 0) wait_drain(q_full(t), (qn[t] - 1) & 1u, p);
            }
            __syncwarp();
        } else if (warp == 1) {
            // -------------------------------------------------------- MMA issuer
            // The whole warp runs the loop: barrier waits and descriptors are warp-uniform,
            // and one elected lane issues each group of MMAs and its commit.
            uint32_t ld = 0;
            uint32_t qn[NT] = {}, pn[NT] = {}, on[NT] = {};
            uint32_t vc = 0;  // cleared V blocks waited for
            bool ok = true;
            // descriptors built once; each MMA advances them by a constant offset
            const uint64_t q_desc0 = C::sdesc(sQ, 16);
            const uint64_t k_desc0 = C::sdesc(sKV, 16);
            const uint64_t v_desc0 = C::sdesc(sKV, C::kChunkBytes);  // MN-major: chunks along d
            // Issue a group of MMAs; before its last MMA, probe (without blocking) the
            // barrier the next group will wait on, so the probe's latency overlaps that
            // MMA instead of leaving the tensor pipe idle.  Returns the probe's result.
            auto issue_s = [&](int t, int slot, uint32_t probe_bar, uint32_t probe_par) {
                const uint64_t a0 = sdesc_add(q_desc0, t * C::kTileBytes);
                const uint64_t b0 = sdesc_add(k_desc0, slot * C::kTileBytes);
                const uint32_t d = tmem + C::s_col(t);
                bool ready = false;
                if (elect_one()) {
                    // 32 bytes of the row per MMA: 16 elements of d
                    constexpr int kSteps = C::kRowBytes / 32;
#pragma unroll
                    for (int kk = 0; kk < kSteps; ++kk) {
                        const uint32_t off = (kk >> 2) * C::kChunkBytes + (kk & 3) * 32;
                        if (kk == kSteps - 1 && probe_bar != 0u) ready = mbar_test_wait(probe_bar, probe_par);
                        C::mma_s(d, sdesc_add(a0, off), sdesc_add(b0, off), kk > 0 ? 1u : 0u);
                    }
                }
                return __ballot_sync(0xffffffffu, ready) != 0u;  // only the issuing lane probed
            };
            // O_t += P_t V over half h of the block's keys; before the last MMA, probe as above
            auto issue_pv = [&](int t, int slot, int h, bool accumulate, uint32_t probe_bar, uint32_t probe_par) {
                constexpr int kSteps = C::kPvSteps / 2;
                const uint64_t b0 = sdesc_add(v_desc0, slot * C::kTileBytes + h * kSteps * C::kPvStepBytes);
                const uint32_t d = tmem + C::o_col(t);
                const uint32_t a = tmem + C::p_col(t) + h * kSteps * 8;
                bool ready = false;
                if (elect_one()) {
                    // 8 TMEM columns of P (16 keys) per MMA
#pragma unroll
                    for (int kk = 0; kk < kSteps; ++kk) {
                        if (kk == kSteps - 1 && probe_bar != 0u) ready = mbar_test_wait(probe_bar, probe_par);
                        C::mma_pv(d, a + kk * 8, sdesc_add(b0, kk * C::kPvStepBytes), (accumulate || kk > 0) ? 1u : 0u);
                    }
                }
                return __ballot_sync(0xffffffffu, ready) != 0u;  // only the issuing lane probed
            };
            auto commit = [&](uint32_t bar) {
                if (elect_one()) mma_commit(bar);
                __syncwarp();
            };
            auto wait = [&](uint32_t bar, uint32_t parity) {
                return __all_sync(0xffffffffu, wait_bounded(bar, parity, abort_flag, p));
            };

            if constexpr (C::kSepP) {
            // Separate P: per key block, first S of the next block for every tile (once its
            // softmax has taken this block's S into registers), then P.V of this block.
            uint32_t sf[NT] = {};
            for (uint32_t si = 0; ok; ++si) {
                const Seg<NT>* const piece = next_piece(si, ok);
                if (piece == nullptr) break;
                const Seg<NT> g = *piece;
                done_piece(si);
                if (g.nblk == 0) continue;
                int slot_k = ld % C::kSlots;
                ok = wait(kv_full(slot_k), (ld / C::kSlots) & 1u);
                if (!ok) break;
                ++ld;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    if (g.n[t] == 0 || !ok) continue;
                    ok = wait(q_full(t), qn[t] & 1u);
                    if (!ok) break;
                    ++qn[t];
                    tc_fence_after();
                    issue_s(t, slot_k, 0u, 0u);
                    commit(s_full(t));
                    if (g.n[t] == 1) commit(q_empty(t));
                }
                if (!ok) break;
                commit(kv_empty(slot_k));
                for (int it = 0; it < g.nblk && ok; ++it) {
                    const int slot_v = ld % C::kSlots;
                    ok = wait(kv_full(slot_v), (ld / C::kSlots) & 1u);
                    if (!ok) break;
                    ++ld;
                    if (it + 1 == g.nblk && g.dirty()) {
                        if (lane == 0) mbar_arrive(v_dirty);
                        ok = wait(v_clean, vc++ & 1u);
                        if (!ok) break;
                    }
                    if (it + 1 < g.nblk) {
                        const int slot_n = ld % C::kSlots;
                        ok = wait(kv_full(slot_n), (ld / C::kSlots) & 1u);
                        if (!ok) break;
                        ++ld;
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            if (it + 1 >= g.n[t] || !ok) continue;
                            ok = wait(s_free(t), sf[t] & 1u);
                            if (!ok) break;
                            ++sf[t];
                            tc_fence_after();
                            issue_s(t, slot_n, 0u, 0u);
                            commit(s_full(t));
                            if (it + 2 == g.n[t]) commit(q_empty(t));
                        }
                        if (!ok) break;
                        commit(kv_empty(slot_n));
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        if (it >= g.n[t] || !ok) continue;
                        ok = wait(p_full(t), pn[t] & 1u);
                        if (!ok) break;
                        ++pn[t];
                        if (it == 0 && on[t] > 0) {
                            // the previous unit's epilogue must have read O_t out
                            ok = wait(o_empty(t), (on[t] - 1) & 1u);
                            if (!ok) break;
                        }
                        tc_fence_after();
                        issue_pv(t, slot_v, 0, it > 0, 0u, 0u);
                        issue_pv(t, slot_v, 1, true, 0u, 0u);
                        commit(p_free(t));
                        if (it + 1 == g.n[t]) {
                            commit(o_full(t));
                            ++on[t];
                        }
                    }
                    if (!ok) break;
                    commit(kv_empty(slot_v));
                }
            }
            } else {
            // A tile that finishes its unit starts the next unit at once: its first S_t is
            // issued right after its last PV_t (the tensor pipe runs MMAs in issue order,
            // so S_t may overwrite the P_t that PV_t reads), instead of after every tile's
            // last PV.  early[t]: the current unit's first S_t was issued that way.
            bool early[NT] = {};
            Seg<NT> g{}, gn{};
            bool have_next = false;
            {
                const Seg<NT>* const piece = next_piece(0, ok);
                if (piece != nullptr) {
                    gn = *piece;
                    have_next = true;
                    done_piece(0);
                }
            }
            for (uint32_t si = 1; have_next && ok; ++si) {
                // the piece after this one, already: key blocks per tile (0 when there is none)
                g = gn;
                int n_next[NT] = {};
                const Seg<NT>* const piece = next_piece(si, ok);
                have_next = piece != nullptr;
                if (!ok) break;
                if (have_next) {
                    gn = *piece;
                    done_piece(si);
#pragma unroll
                    for (int t = 0; t < NT; ++t) n_next[t] = gn.n[t];
                }
                bool early_next[NT] = {};
                if (g.nblk == 0) continue;
                // first key block: S_t for every tile that has keys (and was not started)
                const uint32_t ld_unit = ld;  // ring index of this unit's first K block
                int slot_k = ld % C::kSlots;
                ok = wait(kv_full(slot_k), (ld / C::kSlots) & 1u);
                if (!ok) break;
                ++ld;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    if (g.n[t] == 0 || early[t] || !ok) continue;
                    ok = wait(q_full(t), qn[t] & 1u);
                    if (!ok) break;
                    ++qn[t];
                    tc_fence_after();
                    issue_s(t, slot_k, 0u, 0u);
                    commit(s_full(t));
                    if (g.n[t] == 1) commit(q_empty(t));
                }
                if (!ok) break;
                commit(kv_empty(slot_k));

                bool v_ready = false;  // the next V block's barrier was already seen complete
                for (int it = 0; it < g.nblk && ok; ++it) {
                    const int slot_v = ld % C::kSlots;
                    if (!v_ready) ok = wait(kv_full(slot_v), (ld / C::kSlots) & 1u);
                    if (!ok) break;
                    ++ld;
                    if (it + 1 == g.nblk && g.dirty()) {
                        if (lane == 0) mbar_arrive(v_dirty);
                        ok = wait(v_clean, vc++ & 1u);
                        if (!ok) break;
                    }
                    // K of the next block: waited for only when its first S is issued
                    const bool next = it + 1 < g.nblk;
                    const uint32_t ld_n = ld;
                    const int slot_n = ld_n % C::kSlots;
                    const uint32_t kbar = kv_full(slot_n), kpar = (ld_n / C::kSlots) & 1u;
                    bool k_ready = false;
                    if (next) ++ld;
                    // the V block after next: probed at the end of this iteration
                    const uint32_t vbar = next ? kv_full(ld % C::kSlots) : 0u;
                    const uint32_t vpar = (ld / C::kSlots) & 1u;
                    v_ready = false;
                    tc_fence_after();
                    bool p_ready = false;  // this tile's P was already seen complete
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        if (it >= g.n[t] || !ok) continue;
                        if (!p_ready) ok = wait(p_half(t), pn[t] & 1u);
                        if (!ok) break;
                        if (it == 0 && on[t] > 0) {
                            // the previous unit's epilogue must have read O_t out
                            ok = wait(o_empty(t), (on[t] - 1) & 1u);
                            if (!ok) break;
                        }
                        tc_fence_after();
                        if (!issue_pv(t, slot_v, 0, it > 0, p_full(t), pn[t] & 1u)) ok = wait(p_full(t), pn[t] & 1u);
                        if (!ok) break;
                        ++pn[t];
                        tc_fence_after();
                        const bool more = it + 1 < g.n[t];
                        // probe what comes next: this tile's next K, else the next tile's P
                        const bool has_next_tile = (t + 1 < NT) && (it < g.n[t + 1 < NT ? t + 1 : t]);
                        const uint32_t pbar_next = has_next_tile ? p_half(t + 1 < NT ? t + 1 : t) : 0u;
                        const uint32_t ppar_next = has_next_tile ? (pn[t + 1 < NT ? t + 1 : t] & 1u) : 0u;
                        bool probed = issue_pv(t, slot_v, 1, true,
                                               more && !k_ready ? kbar : pbar_next,
                                               more && !k_ready ? kpar : ppar_next);
                        if (more) {
                            if (!k_ready) {
                                if (!probed) ok = wait(kbar, kpar);
                                if (!ok) break;
                                k_ready = true;
                                tc_fence_after();
                            }
                            p_ready = issue_s(t, slot_n, has_next_tile ? pbar_next : vbar,
                                              has_next_tile ? ppar_next : vpar);
                            if (!has_next_tile) {
                                v_ready = p_ready;
                                p_ready = false;
                            }
                            commit(s_full(t));
                            if (it + 2 == g.n[t]) commit(q_empty(t));
                        } else {
                            p_ready = has_next_tile && probed;
                            commit(o_full(t));
                            ++on[t];
                            // The next unit's K_0 sits at ring index ld_unit + 2 nblk.  Taking
                            // it now is safe when the ring entry it replaces was consumed and
                            // released by an earlier iteration (or the prologue): then its
                            // barrier phase is current and the producer is not blocked on
                            // anything issued later.
                            if (n_next[t] > 0 && 2 * (g.nblk - it) <= C::kSlots) {
                                const uint32_t kq = ld_unit + 2u * (uint32_t)g.nblk;
                                ok = wait(kv_full(kq % C::kSlots), (kq / C::kSlots) & 1u);
                                if (ok) ok = wait(q_full(t), qn[t] & 1u);
                                if (!ok) break;
                                ++qn[t];
                                tc_fence_after();
                                issue_s(t, kq % C::kSlots, 0u, 0u);
                                commit(s_full(t));
                                if (n_next[t] == 1) commit(q_empty(t));
                                early_next[t] = true;
                            }
                        }
                    }
                    if (!ok) break;
                    commit(kv_empty(slot_v));
                    if (next) commit(kv_empty(slot_n));
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) early[t] = early_next[t];
            }
            }
            // every MMA issued so far must be complete before TMEM is released
            commit(mma_done);
            wait_drain(mma_done, 0u, p);
            __syncwarp();
        } else if (warp == 2) {
            // -------------------------------------------------------- rows behind the last key
            // The copies of a sequence's last block bring rows of its neighbour (or whatever the
            // cache holds there); P is 0 for them, and so must V be.  Rows lie 128 bytes apart in
            // each chunk, and the swizzle moves 16-byte pieces within a row only.
            uint32_t ld = 0, vd = 0;
            bool ok = true;
            for (uint32_t si = 0; ok; ++si) {
                const Seg<NT>* const piece = next_piece(si, ok);
                if (piece == nullptr) break;
                const Seg<NT>& g = *piece;
                if (g.dirty()) {
                    ok = __all_sync(0xffffffffu, wait_bounded(v_dirty, vd++ & 1u, abort_flag, p));
                    if (!ok) break;
                    // (the copy's own barrier too: its phase cannot move on before V is used)
                    const uint32_t at = ld + 2u * (uint32_t)g.nblk - 1u;
                    const int slot = at % C::kSlots;
                    ok = __all_sync(0xffffffffu, wait_bounded(kv_full(slot), (at / C::kSlots) & 1u, abort_flag, p));
                    if (!ok) break;
                    const int first = g.s.sk - (g.kb_lo + g.nblk - 1) * kBlockN;
                    const uint32_t v0 = sKV + slot * C::kTileBytes;
#pragma unroll
                    for (int c = 0; c < C::kChunks; ++c)
                        for (int i = first * 8 + lane; i < kBlockN * 8; i += 32)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(v0 + c * C::kChunkBytes + i * 16),
                                         "r"(0)
                                         : "memory");
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(v_clean);
                }
                ld += 2u * (uint32_t)g.nblk;
                done_piece(si);
            }
            __syncwarp();
        } else {
            // -------------------------------------------------------- scheduler
            bool ok = true, more = true;
            Walk w = walk_begin<NT, MODE>(p, pre);
            for (uint32_t si = 0; more && ok; ++si) {
                if (si >= kSegs)
                    ok = __all_sync(0xffffffffu, wait_bounded(seg_empty(si), (si / kSegs - 1) & 1u, abort_flag, p));
                if (!ok) break;
                Seg<NT> g;
                g.b = -1;
                more = next_seg<NT, MODE>(w, g, p, pre);
                if (lane == 0) {
                    segs[si % kSegs] = g;
                    mbar_arrive(seg_full(si));
                    if constexpr (kRanges) {
                        // the unit that this CTA's range begins in, for the joining kernel
                        if (si == 0 && !p.whole) p.bounds[blockIdx.x] = w.bound;
                    }
                }
                __syncwarp();
            }
        }
    } else if (wg <= NT) {
        // ------------------------------------------------------------ softmax, tile t
        regs_inc<C::kRegsSoftmax>();
        const int t = wg - 1;
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t s_addr = tmem + ((uint32_t)(quarter * 32) << 16) + C::s_col(t);
        const uint32_t o_addr = tmem + ((uint32_t)(quarter * 32) << 16) + C::o_col(t);
        static_assert(!C::kSepP || (C::p_col(0) - C::o_col(0) == C::kPAfterO &&
                                    C::p_col(NT - 1) - C::o_col(NT - 1) == C::kPAfterO),
                      "separate P lies a fixed distance past O");
        // P's columns: S's own, or (separate P) a fixed distance past O's
        const uint32_t p_addr = C::kSepP ? o_addr + C::kPAfterO : s_addr;
        const float c = p.scale_log2;
        const float kNegInf = -INFINITY;
        const float fill = (c >= 0.f) ? -INFINITY : INFINITY;  // masked keys drop out of the extremum
        uint32_t sn = 0, stn = 0, sn_o = 0;
        bool ok = true;

        for (uint32_t si = 0; ok; ++si) {
            const Seg<NT>* const piece = next_piece(si, ok);
            if (piece == nullptr) break;
            const Seg<NT>& g = *piece;
            const int n_t = pick<NT>(g.n, t);
            const RowMap rm = row_map(p, g.s.lq, pick<NT>(g.pos0, t), g.hg, row);
            const bool valid = !kTree || rm.pos < g.s.nodes;
            if (n_t == 0) {
                if constexpr (!C::kEpilogueWG) {
                    write_piece<HD, NT, MODE>(p, o_addr, rm, g, t, row, false, false, valid, -INFINITY, 0.f, 0u);
                }
                done_piece(si);
                continue;
            }
            // exclusive key bound of this row (causal: j <= pos + keys - queries)
            const int kmax = !kTree && p.causal ? min(g.s.sk, rm.pos + 1 + (g.s.sk - g.s.lq)) : g.s.sk;
            // keys that every row of a tree sees, and this row's mask of the others
            [[maybe_unused]] const int ctx = g.s.sk - g.s.nodes;
            [[maybe_unused]] const int* mask_row = nullptr;
            if constexpr (kTree) {
                if (rm.ok && valid) mask_row = p.mask + g.b * p.mask_stride + (long long)rm.pos * p.W;
            }
            // A warp whose 32 rows are all padding (short query axis, e.g. decode) only
            // keeps the handshake: its P and O rows feed nothing that is stored.
            const bool idle = __all_sync(0xffffffffu, !rm.ok);
            if (idle) {
                for (int it = 0; it < n_t && ok; ++it) {
                    ok = __all_sync(0xffffffffu, wait_bounded(s_full(t), sn & 1u, abort_flag, p));
                    if (!ok) break;
                    ++sn;
                    tc_fence_after();
                    tc_fence_before();
                    if constexpr (C::kSepP) {
                        if (it + 1 < n_t) mbar_arrive(s_free(t));
                        // The next S may already be issued, so this warp could reach the
                        // next block before the others finish this block's P: its early
                        // arrivals would then complete this block's p_full.  Waiting for
                        // the previous P.V keeps one arrival per thread per phase.
                        // sn - 1 blocks of this tile came before this one
                        if (sn > 1) {
                            ok = __all_sync(0xffffffffu, wait_bounded(p_free(t), sn & 1u, abort_flag, p));
                            if (!ok) break;
                        }
                    }
                    if constexpr (!C::kSepP) mbar_arrive(p_half(t));
                    mbar_arrive(p_full(t));
                }
                if (!ok) break;
                if constexpr (C::kEpilogueWG) {
                    mbar_arrive(st_full(t, stn & 1u));
                    ++stn;
                } else {
                    ok = __all_sync(0xffffffffu, wait_bounded(o_full(t), sn_o & 1u, abort_flag, p));
                    if (!ok) break;
                    ++sn_o;
                    tc_fence_after();
                    write_piece<HD, NT, MODE>(p, o_addr, rm, g, t, row, true, true, valid, kNegInf, 0.f, o_empty(t));
                }
                done_piece(si);
                continue;
            }

            const int kb_lo = g.kb_lo, nodes = g.s.nodes;
            float m = kNegInf;  // reference max of c*s (log2 units), see below
            float l = 0.f;
            for (int it = 0; it < n_t; ++it) {
                ok = __all_sync(0xffffffffu, wait_bounded(s_full(t), sn & 1u, abort_flag, p));
                if (!ok) break;
                ++sn;
                tc_fence_after();
                float s[128];
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) {
                    uint32_t r[32];
                    tmem_ld32(s_addr + ch * 32, r);
#pragma unroll
                    for (int i = 0; i < 32; ++i) s[ch * 32 + i] = __uint_as_float(r[i]);
                }
                tmem_wait_ld();
                if constexpr (C::kSepP) {
                    // S is in registers: the next block's S may be written over it
                    if (it + 1 < n_t) {
                        tc_fence_before();
                        mbar_arrive(s_free(t));
                    }
                }
                const int key0 = (kb_lo + it) * kBlockN;
                // The mask, per 32-key chunk: every key allowed for all 32 rows of the warp
                // (full), none for any of them (empty), or in between.  The branches on it are
                // warp-uniform, as the warp-collective tcgen05.st in the exponential loop
                // requires.  Unmasked blocks skip all of it.
                [[maybe_unused]] int lim = 0, lim_lo = 0, lim_hi = 0;  // prompts: keys [0, lim)
                [[maybe_unused]] uint32_t bits[4] = {};                // trees: bit i of chunk ch
                [[maybe_unused]] uint32_t all_of = 0, none_of = 0;     // chunks full, empty
                bool masked, nothing;
                if constexpr (!kTree) {
                    lim = kmax - key0;
                    lim_lo = __reduce_min_sync(0xffffffffu, lim);
                    lim_hi = __reduce_max_sync(0xffffffffu, lim);
                    masked = lim_lo < kBlockN;
                    nothing = lim <= 0;
                } else {
                    masked = key0 + kBlockN > ctx;
                    nothing = false;
                    if (masked) {
                        const int node0 = key0 - ctx;
                        uint32_t word[5];
#pragma unroll
                        for (int i = 0; i < 5; ++i) word[i] = tree_word(mask_row, (node0 >> 5) + i, nodes);
#pragma unroll
                        for (int ch = 0; ch < 4; ++ch) {
                            bits[ch] = __funnelshift_r(word[ch], word[ch + 1], node0 & 31);
                            if (__all_sync(0xffffffffu, bits[ch] == 0xffffffffu)) all_of |= 1u << ch;
                            if (__all_sync(0xffffffffu, bits[ch] == 0u)) none_of |= 1u << ch;
                        }
                        nothing = (bits[0] | bits[1] | bits[2] | bits[3]) == 0u;
                    }
                }
                auto chunk_empty = [&](int ch) { return kTree ? ((none_of >> ch) & 1u) != 0u : ch * 32 >= lim_hi; };
                auto chunk_full = [&](int ch) { return kTree ? ((all_of >> ch) & 1u) != 0u : ch * 32 + 32 <= lim_lo; };
                // key i of chunk ch, by this row's mask
                auto sees = [&](int ch, int i) {
                    return kTree ? ((bits[ch] >> i) & 1u) != 0u : ch * 32 + i < lim;
                };
                // extremum of the raw scores over the allowed keys (max for c >= 0, min for
                // c < 0); disallowed keys of a partial chunk take the fill value first
                auto extremum = [&](auto op3, auto op2) -> float {
                    if (!masked) {
                        float e[8];  // eight chains of three-input max/min
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            e[k] = op3(s[k], s[k + 8], s[k + 16]);
#pragma unroll
                            for (int i = 3; i < 15; i += 2) e[k] = op3(e[k], s[k + 8 * i], s[k + 8 * i + 8]);
                            e[k] = op2(e[k], s[k + 120]);
                        }
                        return op2(op3(e[0], e[1], e[2]), op3(e[3], e[4], op3(e[5], e[6], e[7])));
                    }
                    float acc = fill;
#pragma unroll
                    for (int ch = 0; ch < 4; ++ch) {
                        if (chunk_empty(ch)) continue;
                        const int b0 = ch * 32;
                        if (!chunk_full(ch)) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) s[b0 + i] = sees(ch, i) ? s[b0 + i] : fill;
                        }
                        float e[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            e[k] = op3(s[b0 + k], s[b0 + k + 4], s[b0 + k + 8]);
                            e[k] = op3(e[k], s[b0 + k + 12], s[b0 + k + 16]);
                            e[k] = op3(e[k], s[b0 + k + 20], s[b0 + k + 24]);
                            e[k] = op2(e[k], s[b0 + k + 28]);
                        }
                        acc = op3(acc, op3(e[0], e[1], e[2]), e[3]);
                    }
                    return acc;
                };
                float e[1];
                if (c >= 0.f)
                    e[0] = extremum([](float x, float y, float z) { return max_nan(x, y, z); },
                                    [](float x, float y) { return max_nan(x, y); });
                else
                    e[0] = extremum([](float x, float y, float z) { return min_nan(x, y, z); },
                                    [](float x, float y) { return min_nan(x, y); });
                const float mx = nothing ? kNegInf : e[0] * c;
                // Reference max m (log2 units): the max of the row's first block with a key, exactly
                // (so that the largest weight is 1 and a row with one key gives its value back), then
                // moved only when a block's max passes m + 8, which keeps every p <= 256 and spares
                // most rows the rescaling of O.
                const bool grow = mx > m + 8.0f || (l == 0.f && mx > m);
                float alpha = 1.f;
                if (grow) {
                    alpha = (l == 0.f) ? 0.f : ex2_approx(m - mx);  // nothing summed: O is 0
                    l *= alpha;
                    m = mx;
                }
                // P = 2^(c*s - m) as bf16, written over S in TMEM (S is in registers).  A
                // disallowed key gets the exponent -inf, i.e. p = 0, for any sign of c.
                // Scores that are not finite: one that is NaN or +inf makes the row's sum NaN, and
                // by it the row's output and LSE (the exponentials alone would not: the polynomial's
                // exponent bits turn a NaN into a number).  -inf is a weight of 0 (2^-126 in the
                // polynomial), and while a row has seen nothing else m stays -inf: 0 in its place.
                const float neg_m = m == kNegInf ? 0.f : -m;
                float ls0 = mx < INFINITY ? 0.f : NAN, ls1 = 0.f;
                // One 32-key chunk: P = 2^(c s - m) as 16 columns of bf16 pairs; with kSelect, keys
                // that the row does not see get the exponent -inf (p = 0 for either sign of c).
                // bf16 is the matrix unit's input: the sum keeps the unrounded p.
                // the pairs of a chunk that take the polynomial, spread over the chunk
                auto use_poly = [](int ch, int i) { return ((i * 5 + ch * 3) & 15) < C::kPolyPairs; };
                auto exp_chunk = [&](auto select_c, int ch) {
                    constexpr bool kSelect = decltype(select_c)::value;
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int j = ch * 32 + 2 * i;
                        float x0, x1;
                        fma2(s[j], s[j + 1], c, c, neg_m, neg_m, x0, x1);
                        if constexpr (kSelect) {
                            x0 = sees(ch, 2 * i) ? x0 : kNegInf;
                            x1 = sees(ch, 2 * i + 1) ? x1 : kNegInf;
                        }
                        float p0, p1;
                        if (!kSelect && use_poly(ch, i)) {
                            exp2_poly4(x0, x1, p0, p1);
                        } else {
                            p0 = ex2_approx(x0);
                            p1 = ex2_approx(x1);
                        }
                        add2(ls0, ls1, p0, p1, ls0, ls1);
                        pk[i] = pack_bf16x2(p0, p1);
                    }
                    tmem_st16(p_addr + ch * 16, pk);
                };
                auto exp_range = [&](auto masked_c, int ch0, int ch1) {
                    constexpr bool kMasked = decltype(masked_c)::value;
#pragma unroll
                    for (int ch = ch0; ch < ch1; ++ch) {
                        if (!kMasked || chunk_full(ch)) {
                            exp_chunk(std::false_type{}, ch);
                        } else if (chunk_empty(ch)) {
                            uint32_t pk[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) pk[i] = 0u;
                            tmem_st16(p_addr + ch * 16, pk);
                        } else {
                            exp_chunk(std::true_type{}, ch);
                        }
                    }
                };
                if constexpr (C::kSepP) {
                    // the previous block's P.V must be done before P and O are written again
                    // P.V of block sn - 2 (this tile's previous one, if any)
                    if (sn > 1) {
                        ok = __all_sync(0xffffffffu, wait_bounded(p_free(t), sn & 1u, abort_flag, p));
                        if (!ok) break;
                        tc_fence_after();
                    }
                }
                if (masked) exp_range(std::true_type{}, 0, 2);
                else exp_range(std::false_type{}, 0, 2);
                // O rescale: PV of the previous block is complete, because this block's S
                // was issued after it.
                if (it > 0 && __any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int ch = 0; ch < HD / 32; ++ch) {
                        uint32_t r[32];
                        tmem_ld32(o_addr + ch * 32, r);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
                        tmem_st32(o_addr + ch * 32, r);
                    }
                }
                if constexpr (!C::kSepP) {
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(p_half(t));
                }
                // second half: keys 64..127
                if (masked) exp_range(std::true_type{}, 2, 4);
                else exp_range(std::false_type{}, 2, 4);
                l += ls0 + ls1;
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(p_full(t));
            }
            if (!ok) break;
            if (m == kNegInf) l *= 0.f;  // scores of -inf only: no key (and NaN stays)
            if constexpr (C::kEpilogueWG) {
                // row statistics for the epilogue warpgroup (double-buffered by unit)
                float* st = stats + ((stn & 1u) * NT + t) * 256;
                st[row] = m;
                st[128 + row] = l;
                mbar_arrive(st_full(t, stn & 1u));
                ++stn;
            } else {
                ok = __all_sync(0xffffffffu, wait_bounded(o_full(t), sn_o & 1u, abort_flag, p));
                if (!ok) break;
                ++sn_o;
                tc_fence_after();
                write_piece<HD, NT, MODE>(p, o_addr, rm, g, t, row, true, false, valid, m, l, o_empty(t));
            }
            done_piece(si);
        }
    } else if constexpr (C::kEpilogueWG) {
        // ------------------------------------------------------------ epilogue
        // O / l goes out through a swizzled shared-memory stage and TMA tensor stores, a
        // 32-column chunk at a time, so every global write is a full line; LSE is stored
        // directly.
        if constexpr (C::kRegsEpilogue < C::kLaunchRegs) regs_dec<C::kRegsEpilogue>();
        if constexpr (C::kRegsEpilogue > C::kLaunchRegs) regs_inc<C::kRegsEpilogue>();
        constexpr uint32_t kEpiBar = 1;  // named barrier of the four epilogue warps
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const bool issuer = (threadIdx.x == (1 + NT) * 128);
        uint32_t on[NT] = {}, stn[NT] = {};
        bool ok = true;
        for (uint32_t si = 0; ok; ++si) {
            const Seg<NT>* const piece = next_piece(si, ok);
            // one decision for the whole warpgroup before its named barriers
            ok = named_bar_and(kEpiBar, 128, ok);
            if (!ok || piece == nullptr) break;
            const Seg<NT>& g = *piece;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (!ok) break;
                if (g.pos0[t] >= g.s.lq) continue;  // a tile wholly past the queries (uniform)
                const RowMap rm = row_map(p, g.s.lq, g.pos0[t], g.hg, row);
                const bool valid = !kTree || rm.pos < g.s.nodes;
                const bool has = g.n[t] > 0;
                const bool idle = __all_sync(0xffffffffu, !rm.ok);
                float m = -INFINITY, l = 0.f;
                if (has) {
                    ok = __all_sync(0xffffffffu, wait_bounded(st_full(t, stn[t] & 1u), (stn[t] >> 1) & 1u,
                                                              abort_flag, p));
                    if (ok) {
                        const float* st = stats + ((stn[t] & 1u) * NT + t) * 256;
                        m = st[row];
                        l = st[128 + row];
                        ++stn[t];
                        ok = __all_sync(0xffffffffu, wait_bounded(o_full(t), on[t] & 1u, abort_flag, p));
                        ++on[t];
                    }
                }
                // one decision for the whole warpgroup before its named barriers
                ok = named_bar_and(kEpiBar, 128, ok);
                if (!ok) break;
                tc_fence_after();
                const uint32_t o_addr = tmem + ((uint32_t)(quarter * 32) << 16) + C::o_col(t);
                if (kRanges && g.parts > 1) {
                    write_row<HD, NT, MODE, true>(p, o_addr, rm, g, t, row, has, idle, valid, m, l, o_empty(t));
                    continue;
                }
                // (no key: 0, whatever V holds; a NaN sum is not 0)
                const bool zero = !has || idle || !valid || l == 0.f;
                const float inv_l = zero ? 0.f : 1.f / l;
                const float lse_v = zero ? -INFINITY : (m + __log2f(l)) * kLn2;
                // A stage row is 128 bytes: 32 fp32 or 64 bf16 columns.  A full tile leaves by a TMA
                // store; in a tile that the sequence's end cuts, the rows behind it belong to the
                // next sequence, and its own are stored one by one.  (A tree's tiles end where the
                // output's T does, and the tensor map cuts them.)
                const bool cut = !kTree && g.pos0[t] + p.pos_per_tile > g.s.lq;
                const int hcoord = p.pack ? g.hg * p.g : g.hg;
                const bool bf16_out = p.out_bf16 != nullptr;
                auto flush = [&](int col0) {
                    fence_proxy_async_smem();
                    named_bar_sync(kEpiBar, 128);
                    if (!cut) {
                        if (issuer) {
                            tma_store_4d_hint(&p.tm_o, sO, col0, hcoord, g.s.q0 + g.pos0[t], kTree ? g.b : 0,
                                              l2_policy_evict_first());
                            bulk_commit_group();
                        }
                    } else {
                        const int piece = threadIdx.x & 7;
#pragma unroll 1
                        for (int r = (threadIdx.x & 127) >> 3; r < 128; r += 16) {
                            const RowMap rr = row_map(p, g.s.lq, g.pos0[t], g.hg, r);
                            if (!rr.ok) continue;
                            uint4 x;
                            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                         : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                                         : "r"(sO + r * 128 + ((uint32_t)(piece ^ (r & 7)) << 4)));
                            const size_t at = out_row<MODE>(p, g.b, g.s, rr) * HD + col0;
                            if (bf16_out) *reinterpret_cast<uint4*>(p.out_bf16 + at + piece * 8) = x;
                            else *reinterpret_cast<uint4*>(p.out + at + piece * 4) = x;
                        }
                    }
                };
#pragma unroll
                for (int ch = 0; ch < HD / 32; ++ch) {
                    uint32_t r[32];
                    if (has && !idle) {
                        tmem_ld32(o_addr + ch * 32, r);
                        tmem_wait_ld();
                    }
                    if (zero) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) r[i] = 0u;
                    }
                    if (has && ch == HD / 32 - 1) {
                        // O_t is in registers: the next unit's PV may overwrite it
                        tc_fence_before();
                        mbar_arrive(o_empty(t));
                    }
                    const int half = bf16_out ? (ch & 1) : 0;
                    if (half == 0) {
                        // the stage is free once the previous store has read it
                        if (issuer) bulk_wait_read_all();
                        named_bar_sync(kEpiBar, 128);
                    }
                    const float* f = reinterpret_cast<const float*>(r);
                    const uint32_t dst = sO + row * 128;
                    if (bf16_out) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t a = dst + ((uint32_t)((half * 4 + j) ^ (row & 7)) << 4);
                            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a),
                                         "r"(pack_bf16x2(f[8 * j] * inv_l, f[8 * j + 1] * inv_l)),
                                         "r"(pack_bf16x2(f[8 * j + 2] * inv_l, f[8 * j + 3] * inv_l)),
                                         "r"(pack_bf16x2(f[8 * j + 4] * inv_l, f[8 * j + 5] * inv_l)),
                                         "r"(pack_bf16x2(f[8 * j + 6] * inv_l, f[8 * j + 7] * inv_l))
                                         : "memory");
                        }
                        if (half == 1) flush((ch >> 1) * 64);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint32_t a = dst + ((uint32_t)(i ^ (row & 7)) << 4);
                            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(f[4 * i] * inv_l),
                                         "f"(f[4 * i + 1] * inv_l), "f"(f[4 * i + 2] * inv_l), "f"(f[4 * i + 3] * inv_l)
                                         : "memory");
                        }
                        flush(ch * 32);
                    }
                }
                if (rm.ok) p.lse[lse_row<MODE>(p, g.b, g.s, rm)] = lse_v;
            }
            done_piece(si);
        }
        if (issuer) bulk_wait_all();
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<C::kTmemCols>(tmem);
    }
}

// ---------------------------------------------------------------- joining the parts
// A unit is shared where a CTA's range begins inside it: boundary c is the begin of CTA c's range.
// The blocks of boundary c (blockIdx.x = c - 1) join a share of its unit's rows, 1 of parts - 1,
// so that units in many parts are spread over as many blocks.  With L_i = log2 of part i's sum,
// M = max L_i and w_i = 2^(L_i - M), O = sum w_i O_i / sum w_i and LSE = (M + log2 sum w_i) ln 2,
// in the order of the keys.  The partials come from L2, and the latency of those reads is what
// it costs: a warp joins 32 columns of 32 rows (lane = row) part by part, eight reads in flight,
// or of a unit in more than four parts 8 columns, four parts at a time.
constexpr int kJoinThreads = 128;
constexpr int kJoinBlocks = 4;  // per boundary
template <int HD, int NT, int MODE>
__global__ void __launch_bounds__(kJoinThreads) serve_join_kernel(const __grid_constant__ ServeParams p) {
    const int lane = threadIdx.x & 31;
    const int c = (int)blockIdx.x + 1;
    let_next();
    wait_before();
    const ServeBound u = p.bounds[c];
    if (u.parts == 0) return;
    Seq s{};
    s.q0 = u.q0;
    s.lq = u.lq;
    auto tile_of = [&](int i, int t) { return part_slot(u.cta0, u.first_slot, i) * NT + t; };
    auto lse_of = [&](int i, int t, int row) { return __ldcg(p.part_lse + (size_t)tile_of(i, t) * 128 + row); };
    auto join = [&](auto wide_c, auto ahead_c) {
        constexpr int kWide = decltype(wide_c)::value, kAhead = decltype(ahead_c)::value;
        constexpr int kCols = HD / (8 * kWide), kItems = NT * 4 * kCols;
        // of the unit's items, 32 rows x (8 kWide) columns, this boundary's share
        const JoinShare mine = join_share(kItems, c, u.cta0, u.parts, (int)blockIdx.y, kJoinBlocks);
        for (int item = mine.lo + (threadIdx.x >> 5); item < mine.hi; item += kJoinThreads / 32) {
            const int col = item % kCols, t = item / kCols / 4, row = item / kCols % 4 * 32 + lane;
            const RowMap rm = row_map(p, s.lq, (u.mt * NT + t) * p.pos_per_tile, u.hg, row);
            if (!rm.ok) continue;
            float M = -INFINITY;
#pragma unroll 4
            for (int i = 0; i < u.parts; ++i) M = fmaxf(M, lse_of(i, t, row));
            float sum = 0.f, acc[8 * kWide] = {};
            for (int i0 = 0; i0 < u.parts; i0 += kAhead) {
                float w[kAhead];
                float4 v[kAhead][2 * kWide];
#pragma unroll
                for (int a = 0; a < kAhead; ++a) {
                    const float li = i0 + a < u.parts ? lse_of(i0 + a, t, row) : -INFINITY;
                    // 0: no keys, and nothing was written.  A NaN sum passes through as NaN.
                    w[a] = li == -INFINITY ? 0.f : ex2_approx(li - M);
                }
#pragma unroll
                for (int a = 0; a < kAhead; ++a)
#pragma unroll
                    for (int e = 0; e < 2 * kWide; ++e)
                        v[a][e] = w[a] != 0.f ? __ldcg(part_at<HD>(p, tile_of(i0 + a, t), col * 2 * kWide + e, row))
                                              : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int a = 0; a < kAhead; ++a) {
                    sum += w[a];
#pragma unroll
                    for (int e = 0; e < 2 * kWide; ++e) {
                        acc[4 * e] += w[a] * v[a][e].x, acc[4 * e + 1] += w[a] * v[a][e].y;
                        acc[4 * e + 2] += w[a] * v[a][e].z, acc[4 * e + 3] += w[a] * v[a][e].w;
                    }
                }
            }
            store_cols<kWide>(p, out_row<MODE>(p, u.b, s, rm) * HD + col * 8 * kWide, acc, sum == 0.f ? 0.f : 1.f / sum);
            if (col == 0) p.lse[lse_row<MODE>(p, u.b, s, rm)] = sum == 0.f ? -INFINITY : (M + __log2f(sum)) * kLn2;
        }
    };
    using W = std::integral_constant<int, 4>;
    using N = std::integral_constant<int, 1>;
    if (u.parts <= 4) join(W{}, N{});
    else join(N{}, W{});
}

// ---------------------------------------------------------------- schedules in front

// The sums of block_prefix for batches above kServeOwnPrefix.
template <int NT, int MODE>
__global__ void __launch_bounds__(1024) serve_prefix_kernel(const __grid_constant__ ServeParams p, long long* pre) {
    let_next();
    wait_before();
    block_prefix<NT, MODE, 1024>(p, pre);
}

// The list of the tile groups of packed prompts, one CTA.  Sequences are taken in windows of
// about p.window_rows keys, so that a window's K and V stay in L2 between their readers; within a
// window the groups with the most key blocks come first (a counting sort over kServeBuckets
// ranges of block counts), so that the CTAs finish a window, and the call, with light ones.
// The order within a bucket is the atomics' and changes nothing but which CTA takes what.
__global__ void __launch_bounds__(1024) serve_list_kernel(const __grid_constant__ ServePlanParams p) {
    constexpr int kKeys = kServeWindows * kServeBuckets;
    __shared__ int count[kKeys];
    __shared__ int warp_sums[32];
    __shared__ int most;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < kKeys; i += 1024) count[i] = 0;
    if (tid == 0) most = 1;
    __syncthreads();
    auto bounds = [](const int* cu, int b, int total, int* lo, int* n) {
        *lo = min(max(fresh(cu + b), 0), total);
        *n = min(max(fresh(cu + b + 1), *lo), total) - *lo;
    };
    auto start = [&](int b) { return min(max(fresh(p.cu_q + b), 0), p.total_q); };
    bool back = false;
    for (int b = tid; b < p.B; b += 1024) {
        int k0, sk;
        bounds(p.cu_k, b, p.total_k, &k0, &sk);
        atomicMax(&most, (sk + kServeBlockN - 1) / kServeBlockN);
        back |= start(b + 1) < start(b);
    }
    // Where bounds decrease, a sequence that starts before the end of an earlier one is left out:
    // its rows are unspecified, and the groups of the others fit the list and leave no row out.
    const bool tangled = __syncthreads_or(back) != 0;
    const int per_bucket = (most + kServeBuckets - 1) / kServeBuckets;
    // a warp per sequence, a lane per tile group
    auto each = [&](auto f) {
        int reach = 0;  // (tangled) the largest bound so far
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const int b = b0 + warp;
            if (tangled) {
                int x = b0 + lane < p.B ? start(b0 + lane) : 0;
                const int mine = __shfl_sync(0xffffffffu, x, warp);
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o) x = max(x, y);
                }
                const bool in_order = mine >= max(reach, __shfl_sync(0xffffffffu, x, warp));
                reach = max(reach, __shfl_sync(0xffffffffu, x, 31));
                if (!in_order) continue;
            }
            if (b >= p.B) break;
            int q0, lq, k0, sk;
            bounds(p.cu_q, b, p.total_q, &q0, &lq);
            bounds(p.cu_k, b, p.total_k, &k0, &sk);
            const int window = min(k0 / p.window_rows, p.windows - 1);
            for (int mt = lane; mt * p.pos_per_unit < lq; mt += 32) {
                const int last = min((mt + 1) * p.pos_per_unit, lq) - 1;
                const int keys = p.causal ? max(0, min(sk, last + 1 + sk - lq)) : sk;
                const int blocks = (keys + kServeBlockN - 1) / kServeBlockN;
                const int bucket = kServeBuckets - 1 - min(max(blocks - 1, 0) / per_bucket, kServeBuckets - 1);
                f(window * kServeBuckets + bucket, b, mt);
            }
        }
    };
    each([&](int key, int, int) { atomicAdd(&count[key], 1); });
    __syncthreads();
    // exclusive prefix sums of the counts, four per thread
    static_assert(kKeys == 4 * 1024, "four counts per thread");
    int own[4], tot = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        own[j] = count[tid * 4 + j];
        tot += own[j];
    }
    int incl = tot;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int ws = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, ws, o);
        if (lane >= o) ws += y;
    }
    const int before = __shfl_sync(0xffffffffu, ws, warp == 0 ? 0 : warp - 1);
    int base = incl - tot + (warp == 0 ? 0 : before);
    if (tid == 1023) *p.list_len = min(base + tot, p.list_cap);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        count[tid * 4 + j] = base;
        base += own[j];
    }
    __syncthreads();
    // (the list has room for them all: the sequences are apart)
    each([&](int key, int b, int mt) {
        const int at = atomicAdd(&count[key], 1);
        if (at < p.list_cap) p.list[at] = make_int2(b, mt);
    });
}

template <int HD, int NT, int MODE>
cudaError_t launch_t(const ServeParams& p, int grid, cudaStream_t stream) {
    using C = Cfg<HD, NT, MODE != kVarlenList>;
    // the attribute is per device; setting it again is idempotent, so the race is benign
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !configured[dev]) {
        e = cudaFuncSetAttribute(serve_fwd_kernel<HD, NT, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 C::kSmemBytes);
        if (e != cudaSuccess) return e;
        // setmaxnreg redistributes the registers that the CTA was launched with: refuse a build
        // whose register count differs from the split's assumption
        cudaFuncAttributes attr{};
        e = cudaFuncGetAttributes(&attr, serve_fwd_kernel<HD, NT, MODE>);
        if (e != cudaSuccess) return e;
        if (attr.numRegs != C::kLaunchRegs) return cudaErrorInvalidConfiguration;
        if (dev >= 0 && dev < 64) configured[dev] = true;
    }
    if constexpr (MODE != kVarlenList) {
        if (p.pre != nullptr) {
            e = launch_early(serve_prefix_kernel<NT, MODE>, dim3(1), 1024, 0, stream, p, const_cast<long long*>(p.pre));
            if (e != cudaSuccess) return e;
        }
    }
    if constexpr (MODE == kVarlenList) {
        // Not let in early, lets nothing in, and neither does its list: measured on B200 the large
        // prompt batches lose 1-11 % with it (the short calls and trees gain 5-20 %).
        serve_fwd_kernel<HD, NT, MODE><<<grid, C::kThreads, C::kSmemBytes, stream>>>(p);
        e = cudaGetLastError();
    } else {
        e = launch_early(serve_fwd_kernel<HD, NT, MODE>, dim3((unsigned)grid), C::kThreads, C::kSmemBytes, stream, p);
        if (e == cudaSuccess && !p.whole && grid > 1)
            e = launch_early(serve_join_kernel<HD, NT, MODE>, dim3((unsigned)grid - 1, kJoinBlocks), kJoinThreads, 0, stream, p);
    }
    return e;
}

}  // namespace

int serve_ctas_per_sm(int nt) { return nt == 2 ? 1 : 2; }

cudaError_t launch_serve_list(const ServePlanParams& p, cudaStream_t stream) {
    serve_list_kernel<<<1, 1024, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_serve(const ServeParams& p, int d, int nt, int grid, cudaStream_t stream) {
    if (p.seqlens == nullptr) {
        if (p.list != nullptr)
            return d == 128 ? launch_t<128, 2, kVarlenList>(p, grid, stream) : launch_t<64, 2, kVarlenList>(p, grid, stream);
        return d == 128 ? launch_t<128, 1, kVarlenRanges>(p, grid, stream)
                        : launch_t<64, 1, kVarlenRanges>(p, grid, stream);
    }
    if (p.block_table != nullptr) {
        if (nt == 2)
            return d == 128 ? launch_t<128, 2, kTreePaged>(p, grid, stream) : launch_t<64, 2, kTreePaged>(p, grid, stream);
        return d == 128 ? launch_t<128, 1, kTreePaged>(p, grid, stream) : launch_t<64, 1, kTreePaged>(p, grid, stream);
    }
    if (nt == 2)
        return d == 128 ? launch_t<128, 2, kTreeDense>(p, grid, stream) : launch_t<64, 2, kTreeDense>(p, grid, stream);
    return d == 128 ? launch_t<128, 1, kTreeDense>(p, grid, stream) : launch_t<64, 1, kTreeDense>(p, grid, stream);
}

unsigned int* serve_status_symbol() {
    void* ptr = nullptr;
    if (cudaGetSymbolAddress(&ptr, g_serve_status) != cudaSuccess) {
        cudaGetLastError();
        return nullptr;
    }
    return static_cast<unsigned int*>(ptr);
}

}  // namespace gqa
