// oasr_cross_attn_packed and oasr_cross_attn_paged: a decoder's tokens over the encoder's states of their
// utterance (cross.cuh has the formula).  Here: the entry points, the kernel for few rows a sequence
// (single tokens, beams) in bf16, and the fp32 kernel.  Many rows go to the tensor-core kernel of cross_tc.cu.
//
// Few rows: every key row is read once for at most 16 rows, so the bytes of k and v are the cost and what counts is
// how many of them are on the way.  A warp takes 16 keys at a time straight into the registers that the
// matrix instructions read, without shared memory, and requests the next 16 before it works on these.
// The contraction of q . k may run over the 64 dimensions in any order, and the columns of P . V stand for
// any dimensions, so the order is taken in which a lane's share of a row is contiguous: lane 4 g + c
// holds dimensions 16 c .. 16 c + 15 of keys g and 8 + g (K) and 8 g .. 8 g + 7 of keys 2 c, 2 c + 1, 8 + 2 c and
// 9 + 2 c (V, whose pairs of keys are interleaved by byte permutes).  The keys of a sequence are shared by the
// warps of a CTA and, where that leaves SMs idle, by a cluster of CTAs.
#include "cluster.cuh"
#include "cross.cuh"
#include "e4m3.cuh"

namespace oasr {
namespace {

constexpr int kHd = 64;
constexpr int kXWarps = 4, kXThreads = 32 * kXWarps, kXRows = 16, kXKeys = 16;

__device__ __forceinline__ float ld_shared_cluster(uint32_t addr, uint32_t rank)
{
    float v;
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ void store_out(__nv_bfloat16* o, float v) { *o = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_out(float* o, float v) { *o = v; }

// Shares of 16 rows: each with its maximum (in log2 units), its sum of exponentials and its unnormalised
// output.  A share without keys has the maximum -inf and is left out.
struct Shares {
    float o[kXWarps][kXRows][kHd + 4];
    float m[kXWarps][kXRows], l[kXWarps][kXRows];
};

// Join the warps' shares into share 0, then the cluster's, and write the rows.  n: rows of the tile; row r
// is written to dst(r).
template <typename Elem, typename Dst>
__device__ __forceinline__ void join_shares(Shares& s, int shares, int splits, int n, Dst dst)
{
    const int tid = threadIdx.x, r = tid >> 3, d0 = (tid & 7) * 8;   // a thread: a row, eight dimensions
    __syncthreads();
    float m = -INFINITY;
    for (int w = 0; w < shares; ++w)
        if (s.l[w][r] != 0.f) m = fmaxf(m, s.m[w][r]);
    float l = 0.f, o[8] = {};
    for (int w = 0; w < shares; ++w) {
        if (s.l[w][r] == 0.f) continue;   // no keys
        const float f = exp2f(s.m[w][r] - m);
        l += s.l[w][r] * f;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] += s.o[w][r][d0 + i] * f;
    }
    if (splits > 1) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) s.o[0][r][d0 + i] = o[i];
        if ((tid & 7) == 0) s.m[0][r] = m, s.l[0][r] = l;
        cluster_sync();
        uint32_t rank;
        asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
        // CTA `rank` finishes rows rank, rank + splits, ...
        for (int i = tid; i < kXRows * kHd; i += kXThreads) {
            const int row = i / kHd, d = i % kHd;
            if (row >= n || row % splits != static_cast<int>(rank)) continue;
            float top = -INFINITY;
            for (int p = 0; p < splits; ++p)
                if (ld_shared_cluster(smem_addr(&s.l[0][row]), p) != 0.f)
                    top = fmaxf(top, ld_shared_cluster(smem_addr(&s.m[0][row]), p));
            float sum = 0.f, v = 0.f;
            for (int p = 0; p < splits; ++p) {
                const float lp = ld_shared_cluster(smem_addr(&s.l[0][row]), p);
                if (lp == 0.f) continue;
                const float f = exp2f(ld_shared_cluster(smem_addr(&s.m[0][row]), p) - top);
                sum += lp * f;
                v += ld_shared_cluster(smem_addr(&s.o[0][row][d]), p) * f;
            }
            store_out(static_cast<Elem*>(dst(row)) + d, sum == 0.f ? 0.f : v / sum);
        }
        cluster_sync();   // no CTA leaves or starts its next tile while another one reads its shares
    } else {
        if (r < n) {
            const float f = l == 0.f ? 0.f : 1.f / l;
            Elem* to = static_cast<Elem*>(dst(r)) + d0;
            if constexpr (sizeof(Elem) == 2) {
                uint4 w;
                w.x = pack_bf16(o[0] * f, o[1] * f), w.y = pack_bf16(o[2] * f, o[3] * f);
                w.z = pack_bf16(o[4] * f, o[5] * f), w.w = pack_bf16(o[6] * f, o[7] * f);
                *reinterpret_cast<uint4*>(to) = w;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) to[i] = o[i] * f;
            }
        }
        __syncthreads();
    }
}

// The work of a CTA: one sequence, key head, share of the keys and every tiles-th row tile from `tile`.
struct CrossItem {
    int s, h, tile, split;
    __device__ __forceinline__ explicit CrossItem(const CrossArgs& a)
    {
        unsigned x = blockIdx.x;
        split = x % a.splits;
        x /= a.splits;
        h = x % a.Hkv;
        x /= a.Hkv;
        tile = x % a.tiles;
        s = x / a.tiles;
    }
};

template <bool PAGED>
__global__ void __launch_bounds__(kXThreads, 4) cross_few_kernel(const CrossArgs a)
{
    using Elem = __nv_bfloat16;
    __shared__ Shares s_sh;
    grid_dep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const CrossItem it(a);
    unsigned err = 0;
    const CrossSeq t(a, it.s, err);
    const int rows = t.nq * a.G;
    // chunks of 16 keys of this CTA; its warps take them in turn
    const int chunks = (t.nk + kXKeys - 1) / kXKeys, share = (chunks + a.splits - 1) / a.splits;
    const int first = it.split * share, last = min(first + share, chunks);
    const Elem* kb = static_cast<const Elem*>(a.k) + it.h * kHd;
    const Elem* vb = static_cast<const Elem*>(a.v) + it.h * kHd;

    for (int tile = it.tile; tile * kXRows < rows; tile += a.tiles) {
        const int r0 = tile * kXRows, n = min(rows - r0, kXRows);
        // a lane's part of query rows g and g + 8: dimensions 16 c .. 16 c + 15
        uint32_t qa[8], qb[8];
        auto load_q = [&](int r, uint32_t (&w)[8]) {
            uint4 x = make_uint4(0, 0, 0, 0), y = x;
            if (r < n) {
                const int R = r0 + r, i = R / a.G, hd = it.h * a.G + R - i * a.G;
                const uint4* p = reinterpret_cast<const uint4*>(static_cast<const Elem*>(a.q) + (t.q0 + i) * a.q_stride +
                                                                hd * kHd + 16 * c);
                x = __ldg(p);
                y = __ldg(p + 1);
            }
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w, w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
        };
        load_q(g, qa);
        load_q(g + 8, qb);

        float o[8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

        uint4 kv[8];   // K of keys g, 8 + g (two words of 16 bytes each), V of keys 2c, 2c + 1, 8 + 2c, 9 + 2c
        auto row_of = [&](int chunk) {   // lanes 0 .. 15: the row of the chunk's key
            const int j = chunk * kXKeys + (lane & 15);
            return chunk < last && j < t.nk ? cross_row<PAGED>(a, t, it.s, j, err) : -1;
        };
        auto request = [&](int row) {
            auto get = [&](const Elem* base, long long stride, int j, int at) {
                const int r = __shfl_sync(0xffffffffu, row, j);
                return r < 0 ? static_cast<const uint4*>(nullptr) : reinterpret_cast<const uint4*>(base + r * stride + at);
            };
            const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint4* p = get(kb, a.k_stride, 8 * u + g, 16 * c);
                kv[2 * u] = p ? __ldg(p) : zero;
                kv[2 * u + 1] = p ? __ldg(p + 1) : zero;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint4* p = get(vb, a.v_stride, 8 * (u >> 1) + 2 * c + (u & 1), 8 * g);
                kv[4 + u] = p ? __ldg(p) : zero;
            }
        };
        request(row_of(first + warp));
        int next_row = row_of(first + warp + kXWarps);
        for (int chunk = first + warp; chunk < last; chunk += kXWarps) {
            uint4 now[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) now[i] = kv[i];
            request(next_row);
            next_row = row_of(chunk + 2 * kXWarps);
            float s[2][4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                s[u][0] = s[u][1] = s[u][2] = s[u][3] = 0.f;
                const uint32_t w[8] = {now[2 * u].x,     now[2 * u].y,     now[2 * u].z,     now[2 * u].w,
                                       now[2 * u + 1].x, now[2 * u + 1].y, now[2 * u + 1].z, now[2 * u + 1].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t qf[4] = {qa[2 * k], qb[2 * k], qa[2 * k + 1], qb[2 * k + 1]};
                    mma_bf16_16816(s[u], qf, w[2 * k], w[2 * k + 1]);
                }
            }
            // keys past the sequence's end do not count
            const int left = t.nk - chunk * kXKeys - 2 * c;
            if (left < 16) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (8 * u + (i & 1) >= left) s[u][i] = -INFINITY;
            }
            uint32_t p[4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {   // rows g, g + 8
                float x = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2)) * a.c;
                if (x > m[r]) {
                    const float f = ex2_approx(m[r] - x);
                    m[r] = x;
                    l[r] *= f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i][2 * r] *= f, o[i][2 * r + 1] *= f;
                }
                float e[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) e[i] = ex2_approx(fmaf(s[i >> 1][2 * r + (i & 1)], a.c, -m[r]));
                l[r] += (e[0] + e[1]) + (e[2] + e[3]);
                p[r] = pack_bf16(e[0], e[1]);
                p[2 + r] = pack_bf16(e[2], e[3]);
            }
            const uint32_t v[4][4] = {{now[4].x, now[4].y, now[4].z, now[4].w}, {now[5].x, now[5].y, now[5].z, now[5].w},
                                      {now[6].x, now[6].y, now[6].z, now[6].w}, {now[7].x, now[7].y, now[7].z, now[7].w}};
#pragma unroll
            for (int d = 0; d < 8; ++d) {   // dimension 8 g + d
                const uint32_t sel = d & 1 ? 0x7632 : 0x5410;
                mma_bf16_16816(o[d], p, __byte_perm(v[0][d >> 1], v[1][d >> 1], sel),
                               __byte_perm(v[2][d >> 1], v[3][d >> 1], sel));
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            if (c == 0) s_sh.m[warp][g + 8 * r] = m[r], s_sh.l[warp][g + 8 * r] = l[r];
            float* to = &s_sh.o[warp][g + 8 * r][16 * c];   // column 2c + e of product d: dimension 16 c + 8 e + d
#pragma unroll
            for (int d = 0; d < 8; ++d) to[d] = o[d][2 * r], to[8 + d] = o[d][2 * r + 1];
        }
        join_shares<Elem>(s_sh, kXWarps, a.splits, n, [&](int r) {
            const int R = r0 + r, i = R / a.G;
            return static_cast<Elem*>(a.out) + (static_cast<long long>(t.q0 + i) * a.H + it.h * a.G + R - i * a.G) * kHd;
        });
    }
    grid_dep_trigger();
    if (err) atomicOr(a.status, err);
}

// fp32: tiles of 16 rows and 64 keys in shared memory, fp32 products (no TF32).  A thread has one key of eight rows
// of q . k, then one dimension of eight rows of P . V.
constexpr int kFKeys = 64;

struct CrossF32Smem {
    float q[kXRows][kHd];
    float k[kFKeys][kHd + 4], v[kFKeys][kHd + 4];
    float p[kXRows][kFKeys];
    float f[kXRows];
    Shares sh;
};

template <bool PAGED>
__global__ void __launch_bounds__(kXThreads) cross_f32_kernel(const CrossArgs a)
{
    extern __shared__ __align__(16) uint8_t smem_raw[];
    CrossF32Smem& sm = *reinterpret_cast<CrossF32Smem*>(smem_raw);
    grid_dep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const CrossItem it(a);
    unsigned err = 0;
    const CrossSeq t(a, it.s, err);
    const int rows = t.nq * a.G;
    const int chunks = (t.nk + kFKeys - 1) / kFKeys, share = (chunks + a.splits - 1) / a.splits;
    const int first = it.split * share, last = min(first + share, chunks);
    const float* kb = static_cast<const float*>(a.k) + it.h * kHd;
    const float* vb = static_cast<const float*>(a.v) + it.h * kHd;
    const int col = tid & 63, half = tid >> 6;   // key, then dimension; rows 8 half .. 8 half + 7

    for (int tile = it.tile; tile * kXRows < rows; tile += a.tiles) {
        const int r0 = tile * kXRows, n = min(rows - r0, kXRows);
        for (int i = tid; i < kXRows * kHd / 4; i += kXThreads) {
            const int r = i >> 4, R = r0 + r, qi = R / a.G;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < n)
                x = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + (t.q0 + qi) * a.q_stride +
                                                          (it.h * a.G + R - qi * a.G) * kHd) + (i & 15));
            *reinterpret_cast<float4*>(&sm.q[r][4 * (i & 15)]) = x;
        }
        float m[4], l[4], o[8] = {};   // of rows 4 warp .. 4 warp + 3, the same in every lane
#pragma unroll
        for (int r = 0; r < 4; ++r) m[r] = -INFINITY, l[r] = 0.f;
        for (int chunk = first; chunk < last; ++chunk) {
            const int j0 = chunk * kFKeys;
            __syncthreads();
            for (int i = tid; i < kFKeys * 16; i += kXThreads) {   // 16 threads to a row, so each row is looked up by 16
                const int j = i >> 4, row = j0 + j < t.nk ? cross_row<PAGED>(a, t, it.s, j0 + j, err) : -1;
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
                if (row >= 0) {
                    x = __ldg(reinterpret_cast<const float4*>(kb + row * a.k_stride) + (i & 15));
                    y = __ldg(reinterpret_cast<const float4*>(vb + row * a.v_stride) + (i & 15));
                }
                *reinterpret_cast<float4*>(&sm.k[j][4 * (i & 15)]) = x;
                *reinterpret_cast<float4*>(&sm.v[j][4 * (i & 15)]) = y;
            }
            __syncthreads();
            float s[8] = {};
#pragma unroll 4
            for (int d = 0; d < kHd; d += 4) {
                const float4 k = *reinterpret_cast<const float4*>(&sm.k[col][d]);
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const float4 q = *reinterpret_cast<const float4*>(&sm.q[8 * half + r][d]);
                    s[r] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, s[r]))));
                }
            }
#pragma unroll
            for (int r = 0; r < 8; ++r) sm.p[8 * half + r][col] = j0 + col < t.nk ? s[r] * a.c : -INFINITY;
            __syncthreads();
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float* p = sm.p[4 * warp + r];
                const float x0 = p[lane], x1 = p[lane + 32];
                float x = fmaxf(x0, x1);
#pragma unroll
                for (int e = 16; e; e >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, e));
                x = fmaxf(x, m[r]);
                const float f = exp2f(m[r] - x), e0 = exp2f(x0 - x), e1 = exp2f(x1 - x);
                float sum = e0 + e1;
#pragma unroll
                for (int e = 16; e; e >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, e);
                m[r] = x;
                l[r] = l[r] * f + sum;
                p[lane] = e0;
                p[lane + 32] = e1;
                if (lane == 0) sm.f[4 * warp + r] = f;
            }
            __syncthreads();
#pragma unroll
            for (int r = 0; r < 8; ++r) o[r] *= sm.f[8 * half + r];
#pragma unroll 4
            for (int j = 0; j < kFKeys; j += 4) {
                const float v0 = sm.v[j][col], v1 = sm.v[j + 1][col], v2 = sm.v[j + 2][col], v3 = sm.v[j + 3][col];
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const float4 p = *reinterpret_cast<const float4*>(&sm.p[8 * half + r][j]);
                    o[r] = fmaf(p.x, v0, fmaf(p.y, v1, fmaf(p.z, v2, fmaf(p.w, v3, o[r]))));
                }
            }
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) sm.sh.o[0][8 * half + r][col] = o[r];
        if (lane == 0)
#pragma unroll
            for (int r = 0; r < 4; ++r) sm.sh.m[0][4 * warp + r] = m[r], sm.sh.l[0][4 * warp + r] = l[r];
        join_shares<float>(sm.sh, 1, a.splits, n, [&](int r) {
            const int R = r0 + r, i = R / a.G;
            return static_cast<float*>(a.out) + (static_cast<long long>(t.q0 + i) * a.H + it.h * a.G + R - i * a.G) * kHd;
        });
    }
    grid_dep_trigger();
    if (err) atomicOr(a.status, err);
}

// --------------------------------------------------------------------------- host

int g_smem_done_x32[2][64];

constexpr int kXMaxSeqs = 65536, kXMaxHeads = 1024;

oasr_status cross_dispatch(CrossArgs a, int max_q, int max_k, oasr_dtype dt, cudaStream_t stream)
{
    const int sms = sm_count();
    if (!sms || !a.status) return OASR_ERR_CUDA;
    const bool f32 = dt == OASR_F32, paged = a.table != nullptr;
    if (!f32 && static_cast<long long>(max_q) * a.G > kXRows && cross_tc_takes(a)) return cross_tc(a, max_q, stream);
    // row tiles side by side, as many as the longest sequence has (a longer one is walked through)
    const long long want = (static_cast<long long>(max_q) * a.G + kXRows - 1) / kXRows, items = static_cast<long long>(a.N) * a.Hkv;
    long long tiles = want;
    while (tiles > 1 && items * tiles > (1 << 24)) tiles = (tiles + 1) / 2;
    if (items * tiles > 0x7fffffffLL / 8) return OASR_ERR_UNSUPPORTED;
    a.tiles = static_cast<int>(tiles);
    // shares of the keys while SMs would stay idle and every share has keys for its four warps
    const int least = f32 ? kFKeys : 2 * kXWarps * kXKeys;
    a.splits = 1;
    while (a.splits < 8 && items * tiles * a.splits < 2LL * sms && max_k >= 2 * a.splits * least) a.splits *= 2;
    const dim3 grid(static_cast<unsigned>(items * tiles * a.splits)), block(kXThreads);
    const int smem = f32 ? static_cast<int>(sizeof(CrossF32Smem)) : 0;
    if (f32) {
        auto kern = paged ? cross_f32_kernel<true> : cross_f32_kernel<false>;
        if (!ensure_smem(kern, smem, g_smem_done_x32[paged])) return OASR_ERR_CUDA;
        return launch_pdl_cluster(kern, grid, block, smem, a.splits, stream, static_cast<const CrossArgs>(a));
    }
    return launch_pdl_cluster(paged ? cross_few_kernel<true> : cross_few_kernel<false>, grid, block, smem, a.splits, stream,
                              static_cast<const CrossArgs>(a));
}

// Arguments that both entry points have.
oasr_status cross_check(const CrossArgs& a, int max_q, int max_k, int D, float scale, oasr_dtype dt)
{
    if (!a.q || !a.k || !a.v || !a.cu_q || !a.out) return OASR_ERR_INVALID_ARG;
    if (a.N <= 0 || a.H <= 0 || a.Hkv <= 0 || a.H % a.Hkv || max_q <= 0 || max_k <= 0 || a.total_q <= 0 || D <= 0)
        return OASR_ERR_INVALID_ARG;
    if (!(scale > 0.f) || scale > 3e38f) return OASR_ERR_INVALID_ARG;
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
