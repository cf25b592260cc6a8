// Attention over packed prompts and of draft trees over a cache: one warp per output row.
//
// O_i = sum_j w_j v_j / sum_j w_j with w_j = exp(scale q_i.k_j - m) over the row's allowed
// keys, in one pass: the running maximum m and sum rescale what came before when the maximum
// moves.  A lane holds d / 32 elements of the query and of O; the sums are fp32.  Bound by
// the instructions of the dot product's shuffles (about 25 per key), far above the bytes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cmath>

#include "launch_serve.h"

namespace gqa {
namespace {

__device__ const uint16_t zeros[128] = {};  // a key of a page outside the pool

__device__ __forceinline__ float bf16(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

template <int HD>
struct Row {
    static constexpr int kPer = HD / 32;
    float q[kPer], o[kPer];
    float m = -INFINITY, l = 0.f;
    __device__ void load(const uint16_t* src, int lane, float scale) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            q[e] = bf16(src + lane * kPer + e) * scale;
            o[e] = 0.f;
        }
    }
    __device__ void key(const uint16_t* k, const uint16_t* v, int lane) {
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < kPer; ++e) x += q[e] * bf16(k + lane * kPer + e);
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
        const float top = fmaxf(m, x);
        const float keep = (m == top) ? 1.f : expf(m - top);
        const float w = expf(x - top);
        m = top;
        l = l * keep + w;
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[e] = o[e] * keep + w * bf16(v + lane * kPer + e);
    }
    __device__ void store(const AttnParams& p, long long at, long long lse_at, int lane) const {
        const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const long long i = at + lane * kPer + e;
            if (p.out_bf16) static_cast<__nv_bfloat16*>(p.out)[i] = __float2bfloat16_rn(o[e] * inv);
            else static_cast<float*>(p.out)[i] = o[e] * inv;
        }
        if (lane == 0) p.lse[lse_at] = l > 0.f ? m + logf(l) : -INFINITY;
    }
};

// Warps stride over the rows of q; each finds its sequence by bisection in cu_seqlens_q.
template <int HD>
__global__ void __launch_bounds__(256) attn_varlen_kernel(const __grid_constant__ AttnParams p) {
    const int lane = threadIdx.x & 31;
    const long long rows = (long long)p.total_q * p.Hq;
    const int g = p.Hq / p.Hk;
    for (long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); r < rows; r += (long long)gridDim.x * 8) {
        const int t = (int)(r / p.Hq), h = (int)(r % p.Hq);
        int lo = 0, hi = p.B;  // the last sequence that starts at or before t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.cu_q[mid] <= t) lo = mid;
            else hi = mid - 1;
        }
        if (lo >= p.B || p.cu_q[lo] > t) continue;
        const int q0 = max(p.cu_q[lo], 0), q1 = min(p.cu_q[lo + 1], p.total_q);
        if (t >= q1) continue;
        const int k0 = min(max(p.cu_k[lo], 0), p.total_k), k1 = min(max(p.cu_k[lo + 1], k0), p.total_k);
        const int end = p.causal ? min(k1 - k0, t - q0 + 1 + (k1 - k0) - (q1 - q0)) : k1 - k0;
        Row<HD> row;
        row.load(p.q + t * p.q_stride + (long long)h * HD, lane, p.scale);
        for (int j = 0; j < end; ++j) {
            const long long at = k0 + j;
            row.key(p.k + at * p.k_stride + (h / g) * HD, p.v + at * p.v_stride + (h / g) * HD, lane);
        }
        row.store(p, ((long long)t * p.Hq + h) * HD, (long long)h * p.total_q + t, lane);
    }
}

template <int HD>
__global__ void __launch_bounds__(256) attn_tree_kernel(const __grid_constant__ AttnParams p) {
    const int lane = threadIdx.x & 31;
    const long long rows = (long long)p.B * p.T * p.Hq;
    const int g = p.Hq / p.Hk;
    for (long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); r < rows; r += (long long)gridDim.x * 8) {
        const int h = (int)(r % p.Hq), i = (int)(r / p.Hq % p.T), b = (int)(r / p.Hq / p.T);
        const long long cap = p.table != nullptr ? (long long)p.M << p.page_shift : p.Sk;
        const int L = (int)min((long long)max(p.seqlens[b], 0), cap);
        const int n = min(max(p.tree_lens != nullptr ? p.tree_lens[b] : p.T, 0), min(p.T, L));
        const int* mask = p.mask + b * p.mask_stride + (long long)i * p.W;
        Row<HD> row;
        row.load(p.q + r * HD, lane, p.scale);
        if (i < n) {
            for (int j = 0; j < L; ++j) {
                const int node = j - (L - n);
                if (node >= 0 && ((mask[node >> 5] >> (node & 31)) & 1) == 0) continue;
                long long at;
                if (p.table != nullptr) {
                    const int page = p.table[(long long)b * p.M + (j >> p.page_shift)];
                    if (page < 0 || page >= p.P) {
                        row.key(zeros, zeros, lane);
                        continue;
                    }
                    at = ((long long)page << p.page_shift) + (j & ((1 << p.page_shift) - 1));
                } else {
                    at = (long long)b * p.Sk + j;
                }
                row.key(p.k + (at * p.Hk + h / g) * HD, p.v + (at * p.Hk + h / g) * HD, lane);
            }
        }
        row.store(p, r * HD, ((long long)b * p.Hq + h) * p.T + i, lane);
    }
}

int blocks_for(long long rows) {
    const long long b = (rows + 7) / 8;
    return (int)(b < 148 * 64 ? b : 148 * 64);
}

}  // namespace

cudaError_t launch_attn_varlen(const AttnParams& p, cudaStream_t stream) {
    const int blocks = blocks_for((long long)p.total_q * p.Hq);
    if (p.d == 128) attn_varlen_kernel<128><<<blocks, 256, 0, stream>>>(p);
    else attn_varlen_kernel<64><<<blocks, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_attn_tree(const AttnParams& p, cudaStream_t stream) {
    const int blocks = blocks_for((long long)p.B * p.T * p.Hq);
    if (p.d == 128) attn_tree_kernel<128><<<blocks, 256, 0, stream>>>(p);
    else attn_tree_kernel<64><<<blocks, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace gqa
