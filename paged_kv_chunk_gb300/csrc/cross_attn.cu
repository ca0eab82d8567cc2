// oasr_cross_attn_packed and oasr_cross_attn_paged: a decoder's tokens over the encoder's states of their
// utterance (cross.cuh has the formula).  Here: the entry points, the kernel for few rows a sequence
// (single tokens, beams) or few tiles in bf16, and the fp32 kernel.  Many rows in many tiles go to the kernel of cross_tc.cu.
//
// Few rows: every key row is read once for at most 16 rows, so the bytes of k and v are the cost and what counts is
// how many of them are on the way.  A warp takes 16 keys at a time from a ring of its own in shared memory, three
// chunks (12 KB) ahead, by asynchronous copies of whole 128-byte lines; no other warp waits for it until the shares are
// joined.  Scores are computed with the keys as the matrix instruction's rows (S^T = K . Q^T, O^T = V^T . P^T), so that eight
// query rows fill its columns.  The contraction of q . k may run over the 64 dimensions in any order, and the rows of O^T
// stand for any dimensions, so the order is taken in which a lane's part of a row is 16 bytes: lane 4 g + c has dimensions
// 8 c .. 8 c + 7 and 32 + 8 c .. 32 + 8 c + 7 of keys g and 8 + g (K) and 8 g .. 8 g + 7 of keys 2 c, 2 c + 1, 8 + 2 c and
// 9 + 2 c (V, whose pairs of keys are interleaved by byte permutes).  The weights are rounded to bf16, as the instruction takes
// them and v in one type; their sum is of the unrounded ones.  Against 64 bits a result is off by 0.0022 of its size in rms,
// of which its own rounding alone makes 0.0017.  The keys of a sequence are shared by the warps of a
// CTA and, where that leaves SMs idle, by a cluster of CTAs.
//
// A beam of 8 over 256 utterances of 50 to 1500 keys, 8 heads, in pages (410 MB): 73 us, 0.83 of the copy rate; 456 heads of
// 3480 keys, one wave: 0.99 of it.  With keys in registers, a lane loading what it uses, 86.5: half a row of K at a time, its
// lines came twice from L2, and so did copies by lane (88).
#include <type_traits>

#include "cluster.cuh"
#include "cross.cuh"

namespace oasr {
namespace {

constexpr int kHd = 64;
constexpr int kXWarps = 4, kXThreads = 32 * kXWarps, kXRows = 16, kXKeys = 16;
constexpr int kXRing = 4, kXChunk = 4096, kXCtas = 3;   // chunks of a warp's ring, bytes of one; CTAs an SM
constexpr int kXSplits = 8;   // CTAs of a cluster at most (the portable size)

__device__ __forceinline__ void store_out(__nv_bfloat16* o, float v) { *o = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_out(float* o, float v) { *o = v; }

// Shares of a tile's rows: each with its maximum (in log2 units), its sum of exponentials and its unnormalised
// output.  A share without keys, or with scores of -inf alone, has the sum zero and is left out.
template <int SHARES, int ROWS, int THREADS>
struct Shares {
    static constexpr int kThreads = THREADS, kDims = ROWS * kHd / THREADS;   // a thread joins kDims dimensions of a row
    float o[SHARES][ROWS][kHd + 4];
    float m[SHARES][ROWS], l[SHARES][ROWS];
};

// Join the warps' shares (into share 0, and those of a cluster's CTAs then) and write the rows.  n: rows of the tile; row r
// is written to dst(r).
template <typename Elem, bool CLUSTER, typename AllShares, typename Dst>
__device__ __forceinline__ void join_shares(AllShares& s, int shares, int splits, int n, Dst dst)
{
    constexpr int W = AllShares::kDims;
    const int tid = threadIdx.x, r = tid / (kHd / W), d0 = tid % (kHd / W) * W;
    __syncthreads();
    float m = -INFINITY;
    for (int w = 0; w < shares; ++w)
        if (s.l[w][r] != 0.f) m = fmaxf(m, s.m[w][r]);
    float l = 0.f, o[W] = {};
    for (int w = 0; w < shares; ++w) {
        if (s.l[w][r] == 0.f) continue;   // no keys
        const float f = exp2f(s.m[w][r] - m);
        l += s.l[w][r] * f;
#pragma unroll
        for (int i = 0; i < W; ++i) o[i] += s.o[w][r][d0 + i] * f;
    }
    if constexpr (CLUSTER) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < W; ++i) s.o[0][r][d0 + i] = o[i];
        if (d0 == 0) s.m[0][r] = m, s.l[0][r] = l;
        cluster_sync();
        uint32_t rank;
        asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
        // four dimensions of a row at a time, a run of them to each CTA; every remote load of a step on the way at once
        const int run = (n * (kHd / 4) + splits - 1) / splits, end = min(n * (kHd / 4), static_cast<int>(rank + 1) * run);
        for (int i = rank * run + tid; i < end; i += AllShares::kThreads) {
            const int row = i / (kHd / 4), d = i % (kHd / 4) * 4;
            float lp[kXSplits], mp[kXSplits], top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int p = 0; p < kXSplits; ++p) {
                lp[p] = p < splits ? ld_shared_cluster(smem_addr(&s.l[0][row]), p) : 0.f;
                mp[p] = p < splits ? ld_shared_cluster(smem_addr(&s.m[0][row]), p) : 0.f;
            }
            float4 op[kXSplits], v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int p = 0; p < kXSplits; ++p)
                if (p < splits) op[p] = ld_shared_cluster4(smem_addr(&s.o[0][row][d]), p);
#pragma unroll
            for (int p = 0; p < kXSplits; ++p)
                if (lp[p] != 0.f) top = fmaxf(top, mp[p]);
#pragma unroll
            for (int p = 0; p < kXSplits; ++p) {
                if (lp[p] == 0.f) continue;   // no keys
                const float f = exp2f(mp[p] - top);
                sum += lp[p] * f;
                v.x += op[p].x * f, v.y += op[p].y * f, v.z += op[p].z * f, v.w += op[p].w * f;
            }
            const float f = sum == 0.f ? 0.f : 1.f / sum;
            Elem* to = static_cast<Elem*>(dst(row)) + d;
            store_out(to, v.x * f), store_out(to + 1, v.y * f), store_out(to + 2, v.z * f), store_out(to + 3, v.w * f);
        }
        cluster_sync();   // no CTA leaves or starts its next tile while another one reads its shares
    } else {
        if (r < n) {
            const float f = l == 0.f ? 0.f : 1.f / l;
            Elem* to = static_cast<Elem*>(dst(r)) + d0;
            if constexpr (sizeof(Elem) == 2) {
                static_assert(W == 8);
                uint4 w;
                w.x = pack_bf16(o[0] * f, o[1] * f), w.y = pack_bf16(o[2] * f, o[3] * f);
                w.z = pack_bf16(o[4] * f, o[5] * f), w.w = pack_bf16(o[6] * f, o[7] * f);
                *reinterpret_cast<uint4*>(to) = w;
            } else {
#pragma unroll
                for (int i = 0; i < W; ++i) to[i] = o[i] * f;
            }
        }
        __syncthreads();
    }
}

// An 8 x 8 matrix of 16-bit elements, a row's two neighbours in each lane, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// The work of a CTA: one sequence, key head, share of the keys and every tiles-th row tile from `tile`.
struct CrossItem {
    int s, h, tile, split;
    __device__ __forceinline__ CrossItem(const CrossArgs& a, unsigned x)
    {
        split = x % a.splits;
        x /= a.splits;
        h = x % a.Hkv;
        x /= a.Hkv;
        tile = x % a.tiles;
        s = x / a.tiles;
    }
};

// 16 bytes of a key, copied without passing registers; zeros where there is none.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_sent() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until all but the last LEFT groups of the thread's copies have arrived.
template <int LEFT>
__device__ __forceinline__ void copies_there()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// NT: eights of rows; P^T comes from S^T by two 8 x 8 transpositions.
template <bool PAGED, int NT, bool CLUSTER>
__global__ void __launch_bounds__(kXThreads, kXCtas) cross_few_kernel(const CrossArgs a)
{
    using Elem = __nv_bfloat16;
    constexpr int RT = 8 * NT;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    using WarpShares = Shares<kXWarps, kXRows, kXThreads>;
    WarpShares& s_sh = *reinterpret_cast<WarpShares*>(smem_raw);   // once the rings are done with
    grid_dep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const CrossItem it(a, blockIdx.x);
    unsigned err = 0;
    const CrossSeq t(a, it.s, err);
    const int rows = t.nq * a.G;
    // chunks of 16 keys of this CTA; its warps take them in turn
    const int chunks = (t.nk + kXKeys - 1) / kXKeys, share = (chunks + a.splits - 1) / a.splits;
    const int first = it.split * share, last = min(first + share, chunks);
    const Elem* kb = static_cast<const Elem*>(a.k) + it.h * kHd;
    const Elem* vb = static_cast<const Elem*>(a.v) + it.h * kHd;
    // K of keys g, 8 + g (two words of 16 bytes each), V of keys 2c, 2c + 1, 8 + 2c, 9 + 2c
    using Chunk = uint4[8];
    const uint8_t* ring = smem_raw + warp * (kXRing * kXChunk);
    auto row_of = [&](int chunk) {   // lanes 0 .. 15: the row of the chunk's key
        const int j = chunk * kXKeys + (lane & 15);
        return chunk < last && j < t.nk ? cross_row<PAGED>(a, t, it.s, j, err) : -1;
    };
    // A chunk in the warp's ring: 16 rows of K, then of V, of 128 bytes each.  The 16 bytes of a row change places so that
    // the lanes' reads below meet no bank twice.  Eight lanes copy a row: whole lines (with a lane copying what it will
    // read, half a row of K at a time, the lines of K came twice from L2).
    auto k_at = [](int r, int piece) { return 128 * r + 16 * (piece ^ (r & 1) << 2); };
    auto v_at = [](int r, int piece) { return 2048 + 128 * r + 16 * (piece ^ (r & 7)); };
    auto request = [&](int row, int slot) {
        const uint32_t to = smem_addr(ring + slot * kXChunk);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int r = 4 * u + (lane >> 3), piece = lane & 7, at = __shfl_sync(0xffffffffu, row, r);
            const long long from = max(at, 0);
            copy16(to + k_at(r, piece), kb + from * a.k_stride + 8 * piece, at >= 0);
            copy16(to + v_at(r, piece), vb + from * a.v_stride + 8 * piece, at >= 0);
        }
        copies_sent();
    };
    for (int tile = it.tile; tile * RT < rows; tile += a.tiles) {
        const int r0 = tile * RT, n = min(rows - r0, RT);
        // a lane's part of query row g of each eight: the dimensions that it has of a key
        uint32_t q[NT][8];
#pragma unroll
        for (int e = 0; e < NT; ++e) {
            uint4 x = make_uint4(0, 0, 0, 0), y = x;
            if (8 * e + g < n) {
                const int R = r0 + 8 * e + g, i = R / a.G, hd = it.h * a.G + R - i * a.G;
                const uint4* p = reinterpret_cast<const uint4*>(static_cast<const Elem*>(a.q) + (t.q0 + i) * a.q_stride +
                                                                hd * kHd + 8 * c);
                x = __ldg(p);
                y = __ldg(p + 4);
            }
            q[e][0] = x.x, q[e][1] = x.y, q[e][2] = x.z, q[e][3] = x.w, q[e][4] = y.x, q[e][5] = y.y, q[e][6] = y.z, q[e][7] = y.w;
        }
        // a lane has rows 2 c and 2 c + 1 of each eight: their maxima, its keys' sums, and dimensions 8 g + 2 d (+ 1) of O
        float o[NT][4][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int e = 0; e < NT; ++e) {
            m[e][0] = m[e][1] = kLowest, l[e][0] = l[e][1] = 0.f;
#pragma unroll
            for (int d = 0; d < 4; ++d) o[e][d][0] = o[e][d][1] = o[e][d][2] = o[e][d][3] = 0.f;
        }
        auto work = [&](int chunk, const Chunk& kv) {
            uint32_t p[NT][2];
#pragma unroll
            for (int e = 0; e < NT; ++e) {
                float s[4] = {0.f, 0.f, 0.f, 0.f};   // keys g (0, 1) and 8 + g (2, 3) of rows 2c, 2c + 1
                const uint32_t kg[8] = {kv[0].x, kv[0].y, kv[0].z, kv[0].w, kv[1].x, kv[1].y, kv[1].z, kv[1].w};
                const uint32_t k8[8] = {kv[2].x, kv[2].y, kv[2].z, kv[2].w, kv[3].x, kv[3].y, kv[3].z, kv[3].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t kf[4] = {kg[2 * k], k8[2 * k], kg[2 * k + 1], k8[2 * k + 1]};
                    mma_bf16_16816(s, kf, q[e][2 * k], q[e][2 * k + 1]);
                }
                // keys past the sequence's end do not count
                const int left = t.nk - chunk * kXKeys;
                if (left < kXKeys) {
                    if (g >= left) s[0] = s[1] = -INFINITY;
                    if (8 + g >= left) s[2] = s[3] = -INFINITY;
                }
                float top[2] = {fmaxf(s[0], s[2]), fmaxf(s[1], s[3])};
#pragma unroll
                for (int x = 4; x < 32; x <<= 1)
#pragma unroll
                    for (int r = 0; r < 2; ++r) top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], x));
                top[0] *= a.c, top[1] *= a.c;
                // the reference moves only when a row's maximum has grown by more than 2^8: weights stay below 2^8
                const bool grown0 = top[0] > m[e][0] + 8.f, grown1 = top[1] > m[e][1] + 8.f;
                if (__any_sync(0xffffffffu, grown0 || grown1)) {
                    const float f0 = grown0 ? ex2_approx(m[e][0] - top[0]) : 1.f, f1 = grown1 ? ex2_approx(m[e][1] - top[1]) : 1.f;
                    if (grown0) m[e][0] = top[0];
                    if (grown1) m[e][1] = top[1];
                    l[e][0] *= f0, l[e][1] *= f1;
#pragma unroll
                    for (int d = 0; d < 4; ++d) o[e][d][0] *= f0, o[e][d][1] *= f1, o[e][d][2] *= f0, o[e][d][3] *= f1;
                }
                float w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = ex2_approx(fmaf(s[i], a.c, -m[e][i & 1]));
                l[e][0] += w[0] + w[2], l[e][1] += w[1] + w[3];
                p[e][0] = transposed(pack_bf16(w[0], w[1]));
                p[e][1] = transposed(pack_bf16(w[2], w[3]));
            }
            const uint32_t v[4][4] = {{kv[4].x, kv[4].y, kv[4].z, kv[4].w}, {kv[5].x, kv[5].y, kv[5].z, kv[5].w},
                                      {kv[6].x, kv[6].y, kv[6].z, kv[6].w}, {kv[7].x, kv[7].y, kv[7].z, kv[7].w}};
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const uint32_t vf[4] = {__byte_perm(v[0][d], v[1][d], 0x5410), __byte_perm(v[0][d], v[1][d], 0x7632),
                                        __byte_perm(v[2][d], v[3][d], 0x5410), __byte_perm(v[2][d], v[3][d], 0x7632)};
#pragma unroll
                for (int e = 0; e < NT; ++e) mma_bf16_16816(o[e][d], vf, p[e][0], p[e][1]);
            }
        };
        // kXRing - 1 chunks on the way, and the row of the next one looked up
        int row[kXRing];
#pragma unroll
        for (int i = 0; i < kXRing; ++i) row[i] = row_of(first + warp + i * kXWarps);
#pragma unroll
        for (int i = 0; i < kXRing - 1; ++i) request(row[i], i);
        int next = row[kXRing - 1], slot = 0;
        for (int chunk = first + warp; chunk < last; chunk += kXWarps) {
            copies_there<kXRing - 2>();
            __syncwarp();   // every lane's copies
            const uint8_t* from = ring + slot * kXChunk;
            auto get = [&](int at) { return *reinterpret_cast<const uint4*>(from + at); };
            const Chunk kv = {get(k_at(g, c)),         get(k_at(g, 4 + c)),         get(k_at(8 + g, c)),     get(k_at(8 + g, 4 + c)),
                              get(v_at(2 * c, g)),     get(v_at(2 * c + 1, g)),     get(v_at(8 + 2 * c, g)), get(v_at(9 + 2 * c, g))};
            request(next, slot == 0 ? kXRing - 1 : slot - 1);   // where the last chunk was
            next = row_of(chunk + kXRing * kXWarps);
            work(chunk, kv);
            if (++slot == kXRing) slot = 0;
        }
        copies_there<0>();
        __syncthreads();   // the rings become the shares' place
#pragma unroll
        for (int e = 0; e < NT; ++e)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[e][r] += __shfl_xor_sync(0xffffffffu, l[e][r], x);
                const int R = 8 * e + 2 * c + r;
                if (g == 0) s_sh.m[warp][R] = m[e][r], s_sh.l[warp][R] = l[e][r];
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    *reinterpret_cast<float2*>(&s_sh.o[warp][R][8 * g + 2 * d]) = make_float2(o[e][d][r], o[e][d][2 + r]);
            }
        join_shares<Elem, CLUSTER>(s_sh, kXWarps, a.splits, n, [&](int r) {
            const int R = r0 + r, i = R / a.G;
            return static_cast<Elem*>(a.out) + (static_cast<long long>(t.q0 + i) * a.H + it.h * a.G + R - i * a.G) * kHd;
        });
    }
    grid_dep_trigger();
    if (err) atomicOr(a.status, err);
}

// fp32: a tile's rows and some keys in shared memory, fp32 products (no TF32).  RG warps have eight rows each, and the 4 / RG
// groups of them each their own 32 KL of the keys, joined at the end.  A lane has KL keys of the eight rows of q . k, then two
// dimensions of the eight rows of P . V: of 16 bytes that all lanes load alike (q, P) a warp takes 16 from shared memory, of
// others 512, and with two keys to a lane these are as long as the products.  The next keys are on the way while the weights
// are worked on, the next values during the scores.  64 utterances of 200 rows over 775 states, 8 heads: 746 us (27
// TFLOP/s), 1093 with two rows of four keys to a lane; 8 heads of 8 rows over 8000 keys 28 and 58.
template <int RG, int KL>
struct CrossF32 {
    static constexpr int kRows = 8 * RG, kGroups = kXWarps / RG, kWarpKeys = 32 * KL, kKeys = kGroups * kWarpKeys;
    static constexpr int kLoad = kKeys / kXWarps;   // keys that a warp loads: its own, where RG is 1
    static_assert(kLoad <= 32);
    struct Smem {
        float q[kRows][kHd];
        float k[kKeys][kHd + 4], v[kKeys][kHd];   // the padding puts eight keys' 16 bytes side by side into different banks
        float p[kXWarps][8][kWarpKeys];
        Shares<kGroups, kRows, kXThreads> sh;
    };
};

template <bool PAGED, int RG, int KL>
__global__ void __launch_bounds__(kXThreads, 3) cross_f32_kernel(const CrossArgs a)
{
    using F = CrossF32<RG, KL>;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    typename F::Smem& sm = *reinterpret_cast<typename F::Smem*>(smem_raw);
    grid_dep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rg = warp % RG, kg = warp / RG;
    const CrossItem it(a, blockIdx.x);
    unsigned err = 0;
    const CrossSeq t(a, it.s, err);
    const int rows = t.nq * a.G;
    const int chunks = (t.nk + F::kKeys - 1) / F::kKeys, share = (chunks + a.splits - 1) / a.splits;
    const int first = it.split * share, last = min(first + share, chunks);
    const float* kb = static_cast<const float*>(a.k) + it.h * kHd;
    const float* vb = static_cast<const float*>(a.v) + it.h * kHd;
    const int key0 = kg * F::kWarpKeys;   // of a chunk
    auto sync = [&] { RG == 1 ? __syncwarp() : __syncthreads(); };   // the warps that share keys

    for (int tile = it.tile; tile * F::kRows < rows; tile += a.tiles) {
        const int r0 = tile * F::kRows, n = min(rows - r0, F::kRows);
        const bool has_rows = 8 * rg < n;
        auto row_of = [&](int chunk) {   // of key `lane` of those that the warp loads; -1: none
            const int j = chunk * F::kKeys + warp * F::kLoad + (lane & (F::kLoad - 1));
            return chunk < last && j < t.nk ? cross_row<PAGED>(a, t, it.s, j, err) : -1;
        };
        auto request = [&](auto& to, const float* from, long long stride, int row, bool any) {
            if (any)
#pragma unroll
                for (int u = 0; u < F::kLoad / 2; ++u) {
                    const int i = 2 * u + (lane >> 4), part = 4 * (lane & 15), r = __shfl_sync(0xffffffffu, row, i);
                    copy16(smem_addr(&to[warp * F::kLoad + i][part]), from + max(r, 0) * stride + part, r >= 0);
                }
            copies_sent();
        };
        int row = row_of(first);
        request(sm.k, kb, a.k_stride, row, first < last);
        request(sm.v, vb, a.v_stride, row, first < last);
        row = row_of(first + 1);
        for (int i = tid; i < F::kRows * kHd / 4; i += kXThreads) {
            const int r = i >> 4, R = r0 + r, qi = R / a.G;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < n)
                x = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + (t.q0 + qi) * a.q_stride +
                                                          (it.h * a.G + R - qi * a.G) * kHd) + (i & 15));
            *reinterpret_cast<float4*>(&sm.q[r][4 * (i & 15)]) = x;
        }
        __syncthreads();
        float2 o[8][2] = {};   // dimensions 2 lane and 2 lane + 1, sums over even and odd keys
        float m[8], l[8];      // the maximum, the same in every lane; the lane's part of the sum
#pragma unroll
        for (int r = 0; r < 8; ++r) m[r] = kLowest, l[r] = 0.f;
        for (int chunk = first; chunk < last; ++chunk) {
            const int left = t.nk - chunk * F::kKeys - key0;   // keys from the warp's first on
            const bool works = has_rows && left > 0;
            copies_there<1>();
            sync();   // the keys are there
            float s[8][KL];
            if (works) {
                float2 s2[8][KL] = {};   // sums of even and odd terms: two products an instruction
#pragma unroll 2
                for (int d = 0; d < kHd; d += 4) {
                    float4 k[KL];
#pragma unroll
                    for (int i = 0; i < KL; ++i) k[i] = *reinterpret_cast<const float4*>(&sm.k[key0 + lane + 32 * i][d]);
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const float4 q = *reinterpret_cast<const float4*>(&sm.q[8 * rg + r][d]);
#pragma unroll
                        for (int i = 0; i < KL; ++i) {
                            s2[r][i] = __ffma2_rn(make_float2(q.x, q.y), make_float2(k[i].x, k[i].y), s2[r][i]);
                            s2[r][i] = __ffma2_rn(make_float2(q.z, q.w), make_float2(k[i].z, k[i].w), s2[r][i]);
                        }
                    }
                }
#pragma unroll
                for (int r = 0; r < 8; ++r)
#pragma unroll
                    for (int i = 0; i < KL; ++i) s[r][i] = lane + 32 * i < left ? (s2[r][i].x + s2[r][i].y) * a.c : -INFINITY;
            }
            sync();   // the keys are done with
            request(sm.k, kb, a.k_stride, row, chunk + 1 < last);
            if (works) {
                float x[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    x[r] = s[r][0];
#pragma unroll
                    for (int i = 1; i < KL; ++i) x[r] = fmaxf(x[r], s[r][i]);
                }
#pragma unroll
                for (int e = 16; e; e >>= 1)
#pragma unroll
                    for (int r = 0; r < 8; ++r) x[r] = fmaxf(x[r], __shfl_xor_sync(0xffffffffu, x[r], e));
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    x[r] = fmaxf(x[r], m[r]);
                    const float f = exp2f(m[r] - x[r]);
                    m[r] = x[r];
                    l[r] *= f;
#pragma unroll
                    for (int i = 0; i < KL; ++i) {
                        const float p = exp2f(s[r][i] - x[r]);
                        l[r] += p;
                        sm.p[warp][r][lane + 32 * i] = p;
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) o[r][e].x *= f, o[r][e].y *= f;
                }
            }
            copies_there<1>();
            sync();   // the weights and the values are there
            if (works) {
#pragma unroll 2
                for (int j = 0; j < min(F::kWarpKeys, left); j += 4) {
                    float2 v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const float2*>(&sm.v[key0 + j + i][2 * lane]);
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const float4 p = *reinterpret_cast<const float4*>(&sm.p[warp][r][j]);
                        o[r][0] = __ffma2_rn(make_float2(p.x, p.y), make_float2(v[0].x, v[1].x), o[r][0]);
                        o[r][1] = __ffma2_rn(make_float2(p.x, p.y), make_float2(v[0].y, v[1].y), o[r][1]);
                        o[r][0] = __ffma2_rn(make_float2(p.z, p.w), make_float2(v[2].x, v[3].x), o[r][0]);
                        o[r][1] = __ffma2_rn(make_float2(p.z, p.w), make_float2(v[2].y, v[3].y), o[r][1]);
                    }
                }
            }
            sync();   // the values are done with
            request(sm.v, vb, a.v_stride, row, chunk + 1 < last);
            row = row_of(chunk + 2);
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            *reinterpret_cast<float2*>(&sm.sh.o[kg][8 * rg + r][2 * lane]) =
                make_float2(o[r][0].x + o[r][0].y, o[r][1].x + o[r][1].y);
#pragma unroll
            for (int e = 16; e; e >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], e);
            if (lane == 0) sm.sh.m[kg][8 * rg + r] = m[r], sm.sh.l[kg][8 * rg + r] = l[r];
        }
        join_shares<float, true>(sm.sh, F::kGroups, a.splits, n, [&](int r) {
            const int R = r0 + r, i = R / a.G;
            return static_cast<float*>(a.out) + (static_cast<long long>(t.q0 + i) * a.H + it.h * a.G + R - i * a.G) * kHd;
        });
    }
    copies_there<0>();
    grid_dep_trigger();
    if (err) atomicOr(a.status, err);
}

// --------------------------------------------------------------------------- host

int g_smem_done_x32[6][64], g_smem_done_few[8][64];

constexpr int kXMaxSeqs = 65536, kXMaxHeads = 1024;

oasr_status cross_dispatch(CrossArgs a, int max_q, int max_k, oasr_dtype dt, cudaStream_t stream)
{
    const int sms = sm_count();
    if (!sms || !a.status) return OASR_ERR_CUDA;
    const bool f32 = dt == OASR_F32, paged = a.table != nullptr;
    const long long max_rows = static_cast<long long>(max_q) * a.G, items = static_cast<long long>(a.N) * a.Hkv;
    // Tiles of 128 rows where the tiles of 16 are more than two an SM: few tiles leave SMs idle, and up to one an SM the keys
    // are shared by a cluster (8 heads over 1500 keys: 32 rows 7.4 us, 15.0 in tiles of 128; 128 rows 9.3 and 16.5).  With 153
    // to 304 tiles of 16 rows they take 0.8 of the other's time over 100 or 300 keys, 0.9 over 700, 1.01 over 1500 and 1.04
    // over 3000; with 320, a second round of CTAs, 0.93, 1.1, 1.25 and 1.33.
    if (!f32 && max_rows > kXRows && items * ((max_rows + kXRows - 1) / kXRows) > 2LL * sms && cross_tc_takes(a))
        return cross_tc(a, max_q, stream);
    // row tiles side by side, as many as the longest sequence has (a longer one is walked through)
    // fp32: 32 rows to a tile where those fill the SMs (64 utterances, 200 rows over 775 states: 764 us, 922 with 16), 16 where
    // they do not (5 utterances, 20 rows of 4 heads over 170 states: 8.5 us, 12.9 with 32)
    const int tile_rows = max_rows <= 8 ? 8 : f32 && max_rows > kXRows && items * ((max_rows + 31) / 32) >= sms ? 32 : kXRows;
    long long tiles = (max_rows + tile_rows - 1) / tile_rows;
    while (tiles > 1 && items * tiles > (1 << 24)) tiles = (tiles + 1) / 2;
    if (items * tiles > 0x7fffffffLL / 8) return OASR_ERR_UNSUPPORTED;
    a.tiles = static_cast<int>(tiles);
    // as many shares of the keys as two CTAs an SM leave room for, while each has keys for its four warps (64 rows of a key head
    // over 1500 keys: 8.8 us with four shares, 13.4 with seven, which a wave of clusters does not take)
    // (fp32, as many as there are tiles of keys: 192 keys 6.9 us, 9.3 where a share had two)
    const int least = !f32 ? 2 * kXWarps * kXKeys : tile_rows == 32 ? CrossF32<4, 2>::kKeys : CrossF32<2, 2>::kKeys;
    static_assert(CrossF32<1, 1>::kKeys == CrossF32<2, 2>::kKeys);
    const long long room = 2LL * sms / (items * tiles), wanted = (static_cast<long long>(max_k) + (f32 ? least - 1 : 0)) / least;
    a.splits = static_cast<int>(room < 1 || wanted < 1 ? 1 : room < wanted ? room : wanted);
    if (a.splits > kXSplits) a.splits = kXSplits;
    const dim3 grid(static_cast<unsigned>(items * tiles * a.splits)), block(kXThreads);
    if (f32) {
        auto by_rows = [&](auto rg, auto kl) {
            constexpr int smem = sizeof(typename CrossF32<rg.value, kl.value>::Smem);
            auto kern = paged ? cross_f32_kernel<true, rg.value, kl.value> : cross_f32_kernel<false, rg.value, kl.value>;
            if (!ensure_smem(kern, smem, g_smem_done_x32[2 * (rg.value / 2) + paged])) return OASR_ERR_CUDA;
            return launch_pdl_cluster(kern, grid, block, smem, a.splits, stream, static_cast<const CrossArgs>(a));
        };
        constexpr std::integral_constant<int, 1> one;
        constexpr std::integral_constant<int, 2> two;
        constexpr std::integral_constant<int, 4> four;
        return tile_rows == 8 ? by_rows(one, one) : tile_rows == kXRows ? by_rows(two, two) : by_rows(four, two);
    }
    auto by_pages = [&](auto nt, auto cluster) {
        constexpr int ring = kXWarps * kXRing * kXChunk;
        auto kern = paged ? cross_few_kernel<true, nt.value, cluster.value> : cross_few_kernel<false, nt.value, cluster.value>;
        if (!ensure_smem(kern, ring, g_smem_done_few[4 * (nt.value - 1) + 2 * cluster.value + paged])) return OASR_ERR_CUDA;
        return launch_pdl_cluster(kern, grid, block, ring, a.splits, stream, static_cast<const CrossArgs>(a));
    };
    using std::false_type, std::true_type;
    if (tile_rows == 8) {
        constexpr std::integral_constant<int, 1> nt;
        return a.splits > 1 ? by_pages(nt, true_type()) : by_pages(nt, false_type());
    }
    constexpr std::integral_constant<int, 2> nt;
    return a.splits > 1 ? by_pages(nt, true_type()) : by_pages(nt, false_type());
}

// Arguments that both entry points have.
oasr_status cross_check(const CrossArgs& a, int max_q, int max_k, int D, float scale, oasr_dtype dt)
{
    if (!a.q || !a.k || !a.v || !a.cu_q || !a.out) return OASR_ERR_INVALID_ARG;
    if (a.N <= 0 || a.H <= 0 || a.Hkv <= 0 || a.H % a.Hkv || max_q <= 0 || max_k <= 0 || a.total_q <= 0 || D <= 0)
        return OASR_ERR_INVALID_ARG;
    if (!(scale > 0.f) || scale > 2e38f) return OASR_ERR_INVALID_ARG;
    if ((dt != OASR_F32 && dt != OASR_BF16) || D != kHd || a.N > kXMaxSeqs || a.H > kXMaxHeads) return OASR_ERR_UNSUPPORTED;
    const long long es = dt == OASR_F32 ? 4 : 2;
    if (a.q_stride < a.H * kHd || a.k_stride < a.Hkv * kHd || a.v_stride < a.Hkv * kHd || (a.q_stride * es) % 16 ||
        (a.k_stride * es) % 16 || (a.v_stride * es) % 16)
        return OASR_ERR_INVALID_ARG;
    if (!aligned16(a.q) || !aligned16(a.k) || !aligned16(a.v) || !aligned16(a.out)) return OASR_ERR_INVALID_ARG;
    // rows of a sequence (queries times the heads of a group) are counted in 32 bits
    if (static_cast<long long>(a.total_q) * a.G > 0x7fffffffLL - 256 || static_cast<long long>(max_q) * a.G > 0x7fffffffLL - 256)
        return OASR_ERR_UNSUPPORTED;
    return OASR_OK;
}

}  // namespace
}  // namespace oasr

extern "C" oasr_status oasr_cross_attn_packed(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                              int64_t v_stride, const int32_t* cu_q, const int32_t* cu_k, int num_seqs,
                                              int max_q, int max_k, int total_q, int total_k, void* out, int H, int Hkv, int D,
                                              float scale, oasr_dtype dt, cudaStream_t stream)
{
    using namespace oasr;
    CrossArgs a = {};
    a.q = q, a.k = k, a.v = v, a.out = out;
    a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
    a.cu_q = cu_q, a.cu_k = cu_k;
    a.N = num_seqs, a.H = H, a.Hkv = Hkv, a.G = Hkv > 0 ? H / Hkv : 1;
    a.total_q = total_q, a.total_k = total_k;
    const oasr_status bad = cross_check(a, max_q, max_k, D, scale, dt);
    if (bad != OASR_OK) return bad;
    if (!cu_k || total_k <= 0) return OASR_ERR_INVALID_ARG;
    if (total_k > 0x7fffffff - 256) return OASR_ERR_UNSUPPORTED;   // keys are counted in 32 bits, a tile at a time
    a.c = scale * 1.4426950408889634f;
    a.status = status_word();
    return cross_dispatch(a, max_q, max_k, dt, stream);
}

extern "C" oasr_status oasr_cross_attn_paged(const void* q, int64_t q_stride, const void* k_pool, const void* v_pool,
                                             int num_blocks, int block_size, const int32_t* block_table,
                                             int max_blocks_per_seq, const int32_t* cache_seqlens, const int32_t* cu_q,
                                             int num_seqs, int max_q, int max_k, int total_q, void* out, int H, int Hkv, int D,
                                             float scale, oasr_dtype dt, cudaStream_t stream)
{
    using namespace oasr;
    CrossArgs a = {};
    a.q = q, a.k = k_pool, a.v = v_pool, a.out = out;
    a.q_stride = q_stride, a.k_stride = a.v_stride = static_cast<long long>(Hkv) * kHd;
    a.cu_q = cu_q, a.lens = cache_seqlens, a.table = block_table;
    a.mbps = max_blocks_per_seq, a.bs = block_size, a.num_blocks = num_blocks;
    a.N = num_seqs, a.H = H, a.Hkv = Hkv, a.G = Hkv > 0 ? H / Hkv : 1;
    a.total_q = total_q;
    const oasr_status bad = cross_check(a, max_q, max_k, D, scale, dt);
    if (bad != OASR_OK) return bad;
    if (!block_table || !cache_seqlens || num_blocks <= 0 || block_size <= 0 || max_blocks_per_seq <= 0)
        return OASR_ERR_INVALID_ARG;
    if (static_cast<long long>(num_blocks) * block_size > 0x7fffffffLL ||
        static_cast<long long>(max_blocks_per_seq) * block_size > 0x7fffffffLL - 256)
        return OASR_ERR_UNSUPPORTED;
    a.c = scale * 1.4426950408889634f;
    a.status = status_word();
    return cross_dispatch(a, max_q, max_k, dt, stream);
}
