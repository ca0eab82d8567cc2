// What the cross-attention kernels share: the arguments of a call, the rows and keys of a sequence, and
// the way to the key rows, packed or through a block table.
//
//   out[i][h] = sum_j softmax_j(scale q[i][h] . k[j][h / G]) v[j][h / G],   j < keys of the sequence
//
// G = H / Hkv query heads share a key head.  Row R of a sequence's (key head) problem is query R / G,
// head R % G of the group: the queries of all hypotheses and of all heads of a group are rows of one
// tile against the same keys.  A sequence without keys gets zeros, and so does a row whose every score is -inf.
#pragma once

#include "host_common.h"
#include "ptx.cuh"

namespace oasr {

// A row's maximum before its first key: lowest of the finite values, so that scores of -inf have the weight zero.
constexpr float kLowest = -3.402823466e38f;

struct CrossArgs {
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride;   // elements from row to row (pools: from slot to slot)
    const int32_t* cu_q;                      // [N + 1]
    const int32_t* cu_k;                      // packed: [N + 1]
    const int32_t* lens;                      // paged: [N]
    const int32_t* table;                     // paged: [N][mbps]; null: packed
    int mbps, bs, num_blocks;
    int N, H, Hkv, G, total_q, total_k;
    void* out;                                // [total_q][H][64]
    float c;                                  // scale * log2(e)
    int splits, tiles;                        // CTAs that share the keys of a row tile; row tiles at a time
    unsigned* status;
};

// Queries [q0, q0 + nq) and the first of nk keys (packed: a row of k; paged: 0) of sequence s; offsets
// outside their tensors are clamped and flagged.
struct CrossSeq {
    int q0, nq, k0, nk;
    CrossSeq() = default;
    __device__ __forceinline__ CrossSeq(const CrossArgs& a, int s, unsigned& err)
    {
        int q1 = __ldg(a.cu_q + s + 1);
        q0 = __ldg(a.cu_q + s);
        clamp(q0, q1, a.total_q, err);
        nq = q1 - q0;
        if (a.table) {
            const int n = __ldg(a.lens + s);
            k0 = 0;
            nk = min(max(n, 0), a.mbps * a.bs);
            if (nk != n) err |= kErrBounds;
        } else {
            int k1 = __ldg(a.cu_k + s + 1);
            k0 = __ldg(a.cu_k + s);
            clamp(k0, k1, a.total_k, err);
            nk = k1 - k0;
        }
    }
    static __device__ __forceinline__ void clamp(int& x0, int& x1, int total, unsigned& err)
    {
        if (x0 < 0 || x1 < x0 || x1 > total) {
            err |= kErrBounds;
            x0 = min(max(x0, 0), total);
            x1 = min(max(x1, x0), total);
        }
    }
};

// Row of k and v that key j < nk of sequence s is in; -1 (zeros, flagged) where its page names no block.
template <bool PAGED>
__device__ __forceinline__ int cross_row(const CrossArgs& a, const CrossSeq& t, int s, int j, unsigned& err)
{
    if (!PAGED) return t.k0 + j;
    const int page = static_cast<unsigned>(j) / static_cast<unsigned>(a.bs);
    const int id = __ldg(a.table + static_cast<long long>(s) * a.mbps + page);
    if (id < 0 || id >= a.num_blocks) {
        err |= kErrBounds;
        return -1;
    }
    return id * a.bs + (j - page * a.bs);
}

// The tensor-core form (cross_tc.cu), and whether it takes the call's heads and pages.
bool cross_tc_takes(const CrossArgs& a);
oasr_status cross_tc(const CrossArgs& a, int max_q, cudaStream_t stream);

}  // namespace oasr
