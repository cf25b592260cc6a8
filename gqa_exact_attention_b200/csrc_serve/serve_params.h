// Parameters shared by the host plan (serve_api.cpp) and the serving attention kernel.
#pragma once

#include <cuda.h>
#include <cstdint>

#include "fast_divmod.h"

namespace gqa {

constexpr int kServeBlockM = 128;  // rows of one tile (the tcgen05 M)
constexpr int kServeBlockN = 128;  // keys of one K/V block
// sequences whose schedule each CTA sums up for itself (in shared memory); above, a kernel
// in front of the attention writes the sums to global memory
constexpr int kServeOwnPrefix = 1024;

// The unit that a CTA's range begins in, when it begins inside it (else parts is 0).
struct ServeBound {
    int b, hg, mt;
    int q0, lq;      // its sequence's first query row and queries
    int cta0;        // the CTA that begins it
    int parts;       // CTAs that share it
    int first_slot;  // where the first one's partials are
};

struct ServeParams {
    CUtensorMap tm_q;  // varlen: q as (d, Hq, total_q, 1); tree: (d, Hq, T, B)
    CUtensorMap tm_k;  // varlen: (d, Hk, total_k, 1); tree: (d, Hk, Sk, B) or the page pool
    CUtensorMap tm_v;
    CUtensorMap tm_o;  // out like q, for full tiles' TMA stores (two-tile kernels)

    float* out;          // fp32 output, or
    uint16_t* out_bf16;  // bf16 output (the other is NULL)
    float* lse;
    int B, Hq, Hk;
    int g;             // Hq / Hk
    int pack;          // 1: a tile holds g heads x pos_per_tile positions
    int pos_per_tile;  // positions of one tile (packed: floor(128 / g); else 128)
    int rows_valid;    // rows of a tile that map to (position, head)
    int n_hg;          // heads or groups: Hq (unpacked) or Hk (packed)
    FastDiv div_g, div_hg;
    float scale_log2;  // scale * log2(e)

    // packed prompts
    const int* cu_q;
    const int* cu_k;
    int total_q, total_k;
    int causal;

    // a tree over a cache of `cap` keys per sequence
    const int* seqlens;
    const int* tree_lens;  // NULL: T nodes
    const int* mask;       // rows of W words
    long long mask_stride;  // words between sequences (0: one mask for all)
    int T, W, cap;
    const int* block_table;  // paged cache (see gqa_attn_fwd_paged)
    int table_stride, page_shift, page_rows, num_pages;

    // schedule: list (a sorted list of tile groups) or pre (block counts before each sequence)
    const int2* list;         // (sequence, tile group), heaviest first within a window
    const int* list_len;      // its entries
    const long long* pre;     // [B + 1], NULL: summed up in the kernel
    int whole;                // units are not split (no partials)
    int min_blocks;           // a CTA's range holds at least this many blocks (if there are)
    float* part_o;            // [2 * grid][NT][128][d]
    float* part_lse;          // [2 * grid][NT][128], log2 units
    ServeBound* bounds;       // [grid]

    int kv_shared;  // K/V blocks are read by several units: ask L2 to keep them
    long long timeout_ns, drain_ns;
    int inject_stall;
};

struct ServePlanParams {
    const int* cu_q;
    const int* cu_k;
    int B, total_q, total_k, causal;
    int pos_per_unit;  // query positions of one tile group
    int window_rows;   // key rows of one window
    int windows;       // at most kServeWindows
    int2* list;
    int list_cap;
    int* list_len;
};
constexpr int kServeWindows = 64;
constexpr int kServeBuckets = 64;

}  // namespace gqa
