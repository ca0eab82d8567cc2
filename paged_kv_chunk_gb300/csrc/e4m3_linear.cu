// 8-bit floating-point products with a scale for each block of 128:
//
//   oasr_quantize_blocks  e = max(-100, least e with max|x_block| <= 448 2^e), x8 = e4m3(x 2^-e), byte e + 127
//   oasr_linear_e4m3      out[i][n] = sum_b 2^(ex[i][b] + ew[n][b]) sum_{k in b} x8[i][k] w8[n][k] + bias[n]
//
// A block is 128 neighbouring values of a row, of activations and weights alike; the last of a row may be
// shorter.  The format is the 8-bit cache's (e4m3.cuh) with 128 values to a scale.
//
// A scale is a power of two, its byte the one that tcgen05's block-scaled products take (kind::mxf8f6f4, one for each 32 of
// K): a block's byte serves four steps, and the sums come out of the tensor core scaled, without a pass over the
// accumulators per block.  Products of two e4m3 values are exact in fp32.
//
// What bounds a large product is what it copies into shared memory: 40 KB a step of 128 of K and 128 x 192 outputs, 12 TB/s
// over the GPU at 65537 x 1024 x 512 (43 us, 1.6 PFLOP/s, 168 MB of HBM traffic); 8191 x 4096 x 1024 takes 36 us (1.89 PFLOP/s;
// the int8 product 51).  Pairs of CTAs on 256 x 192 (cta_group::2), half of w each, were right and slower: 69 us.
#include <type_traits>

#include "cluster.cuh"
#include "e4m3.cuh"
#include "host_common.h"
#include "linear.cuh"

namespace oasr {
namespace {

constexpr int kBlk = 128;   // values that share a scale

// ------------------------------------------------------------------ rows to 8 bits

// Eight values as they come, the fp32 bits of the largest magnitude among them and the block's other lanes' (the bits order
// as the values do, NaN above infinity), and the values in fp32.
struct Raw8Bf16 {
    uint4 w;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void clear() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ uint32_t largest(unsigned mask) const
    {
        constexpr uint32_t A = 0x7fff7fffu;
        uint32_t m = __vmaxu2(__vimax3_u16x2(w.x & A, w.y & A, w.z & A), w.w & A);
#pragma unroll
        for (int o = 8; o; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(mask, m, o));
        return max(m << 16, m & 0xffff0000u);
    }
    __device__ __forceinline__ void values(float (&x)[8]) const { unpack8(w, x); }
};
struct Raw8F32 {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p)
    {
        a = __ldcs(reinterpret_cast<const float4*>(p));
        b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ uint32_t largest(unsigned mask) const
    {
        float x[8];
        values(x);
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[e]) & 0x7fffffffu);
#pragma unroll
        for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(mask, m, o));
        return m;
    }
    __device__ __forceinline__ void values(float (&x)[8]) const
    {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
};

// Sixteen lanes to a block, eight values each; four blocks at a time, every load ahead of the first use.  Bound by HBM: 2
// or 4 bytes in, one out per value.  EVEN: rows are whole blocks, and block i begins at value 128 i (the division of a
// block's number by the blocks of a row took half of the time).
constexpr int kQBlocks = 4;

template <bool EVEN, typename Elem>
__global__ void __launch_bounds__(256) quantize_blocks_kernel(const Elem* __restrict__ x, uint8_t* __restrict__ x8,
                                                              uint8_t* __restrict__ scale, int M, int K, int kb, unsigned recip)
{
    grid_dep_wait();
    const int l = threadIdx.x & 15;
    const unsigned mask = 0xffffu << (threadIdx.x & 16);
    const long long blocks = static_cast<long long>(M) * kb;
    const long long i0 = static_cast<long long>(blockIdx.x) * (16 * kQBlocks) + (threadIdx.x >> 4);
    std::conditional_t<sizeof(Elem) == 2, Raw8Bf16, Raw8F32> raw[kQBlocks];
    long long at[kQBlocks];   // the lane's first value; -1: none
#pragma unroll
    for (int u = 0; u < kQBlocks; ++u) {
        const long long i = i0 + 16 * u;
        at[u] = -1;
        if (i < blocks) {
            if (EVEN) {
                at[u] = i * kBlk + 8 * l;
            } else {
                // i / kb by the reciprocal 2^32 / kb, rounded up: at most one too many below 2^31; 64-bit divisions beyond
                long long row = kb == 1 ? i : blocks >> 31 ? i / kb : __umulhi(static_cast<unsigned>(i), recip);
                if (row * kb > i) --row;
                const int k = static_cast<int>(i - row * kb) * kBlk + 8 * l;
                if (k < K) at[u] = row * K + k;
            }
        }
        raw[u].clear();
        if (at[u] >= 0) raw[u].load(x + at[u]);
    }
#pragma unroll
    for (int u = 0; u < kQBlocks; ++u) {
        const uint32_t most = raw[u].largest(mask);
        float v[8];
        raw[u].values(v);
        uint32_t byte = kE4NanScale;
        uint2 q = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
        if (most < 0x7f800000u) {
            byte = e4m3_scale_byte(__uint_as_float(most));
            const float f = e4m3_scale_inverse(byte);
            q.x = e4m3_pack2(v[0] * f, v[1] * f) | (e4m3_pack2(v[2] * f, v[3] * f) << 16);
            q.y = e4m3_pack2(v[4] * f, v[5] * f) | (e4m3_pack2(v[6] * f, v[7] * f) << 16);
        }
        if (at[u] >= 0) *reinterpret_cast<uint2*>(x8 + at[u]) = q;
        if (l == 0 && i0 + 16 * u < blocks) scale[i0 + 16 * u] = static_cast<uint8_t>(byte);
    }
    grid_dep_trigger();
}

// --------------------------------------------------------------------- products

struct E4Problem {
    const uint8_t *x, *w;     // [M][K], [N][K]
    const uint8_t *xs, *ws;   // [M][kb], [N][kb]
    const void* bias;         // null: none
    int M, N, K, kb;
};

__device__ __forceinline__ void unpack16(const uint4& w, float (&v)[16])
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = e4m3_unpack2(u[i] & 0xffffu), b = e4m3_unpack2(u[i] >> 16);
        v[4 * i] = a.x, v[4 * i + 1] = a.y, v[4 * i + 2] = b.x, v[4 * i + 3] = b.y;
    }
}

// A few rows (one to six tokens, which of them goes by K: dispatch_e4): every weight byte is used once per row.  One warp
// per output channel, 16 values per lane and step (within one block), products in fp32 (exact) and their sums too.
constexpr int kE4FewRows = 6;   // the most that dispatch_e4's estimate ever prefers: 7 rows of 512 cost 3820 ns against 3800

template <int MR, typename Elem>
__global__ void __launch_bounds__(256) linear_e4m3_few_kernel(const E4Problem p, Elem* __restrict__ out)
{
    grid_dep_wait();
    const int n = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int m0 = blockIdx.y * MR, rows = min(MR, p.M - m0);
    if (n < p.N) {
        float acc[MR] = {};
        const uint8_t* w = p.w + static_cast<long long>(n) * p.K;
        for (int k = 16 * lane; k < p.K; k += 512) {
            const int b = k / kBlk;
            float wv[16];
            unpack16(__ldg(reinterpret_cast<const uint4*>(w + k)), wv);
            const float ws = e4m3_scale(__ldg(p.ws + static_cast<long long>(n) * p.kb + b));
#pragma unroll
            for (int m = 0; m < MR; ++m) {
                if (m < rows) {
                    const long long row = m0 + m;
                    float xv[16], s = 0.f;
                    unpack16(__ldg(reinterpret_cast<const uint4*>(p.x + row * p.K + k)), xv);
#pragma unroll
                    for (int i = 0; i < 16; ++i) s = fmaf(xv[i], wv[i], s);
                    // the scales' product first: a power of two and exact, where s times one of them may leave fp32's range
                    acc[m] += s * (e4m3_scale(__ldg(p.xs + row * p.kb + b)) * ws);
                }
            }
        }
#pragma unroll
        for (int m = 0; m < MR; ++m)
#pragma unroll
            for (int o = 16; o; o >>= 1) acc[m] += __shfl_xor_sync(0xffffffffu, acc[m], o);
        const float bias = p.bias ? bias_at(static_cast<const Elem*>(p.bias), n) : 0.f;
#pragma unroll
        for (int m = 0; m < MR; ++m)
            if (lane == m && m < rows) put(out + static_cast<long long>(m0 + m) * p.N + n, acc[m] + bias);
    }
    grid_dep_trigger();
}

// Warps of the tensor-core kernel: eight for the epilogue, four for the scales, the issuer, the TMA producer.  The
// producer brings 128 bytes of K of the tile's rows into a ring; the scale warps write the scales of four
// blocks (a word a row) into tensor memory, where every quadrant of lanes has them once; the issuer's products take
// them from there, a block's scale for each of its four steps of 32.  Two accumulators let a tile's
// epilogue overlap the next tile's products.
constexpr int kE4EpiWarps = 8, kE4ScaleWarps = 4, kE4Issuer = kE4EpiWarps + kE4ScaleWarps;
constexpr int kE4Threads = 32 * (kE4Issuer + 2);
constexpr int kE4Splits = 8;   // CTAs of a cluster at most (the portable size)

template <int BN>
struct E4Smem {
    static constexpr int tile_a = 128 * 128, tile = (128 + BN) * 128;   // x rows, then w rows
    static constexpr int stages = BN > 128 ? 4 : BN > 64 ? 5 : 6;
    static constexpr int off_out = stages * tile;                       // [8 warps][2][32 rows][64 bytes] or [8 warps][32 rows][128 bytes]
    static constexpr int off_bias = off_out + kE4EpiWarps * 2 * 32 * 64;    // [8 warps][BN / 2] floats
    static constexpr int off_bar = off_bias + kE4EpiWarps * BN / 2 * 4;   // full, empty, scales full[2], free[2], acc full[2], free[2], drain
    static constexpr int off_misc = off_bar + (2 * stages + 9) * 8;
    static constexpr int bytes = off_misc + 16 + 1024;
    static constexpr int part_row = BN + 4;                             // floats of a row of a split tile's sums, in the ring
    static_assert(128 * part_row * 4 <= stages * tile);
    static constexpr int sb_cols = (BN + 127) / 128 * 4;                // columns of w's scales
    static constexpr int sf_cols = 4 + sb_cols, off_sf = 2 * BN;        // x's, then w's; two buffers
    static constexpr int used = off_sf + 2 * sf_cols;
    static constexpr int cols = used <= 128 ? 128 : used <= 256 ? 256 : 512;
};

struct E4Args {
    E4Problem p;
    void* out;
    int nt, tiles;
    int by_tma;   // the output's rows suit TMA: stored by it
    int splits, share;   // CTAs that share a tile's blocks of K, blocks of each
    unsigned* status;
};

// D [+]= (A . B) with the scales at sa (A's rows) and sb (B's), one for each 32 of K.
__device__ __forceinline__ void umma_e4m3_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t sa, uint32_t sb,
                                                 int acc)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(id), "r"(sa), "r"(sb), "r"(acc));
}

template <int N>
__device__ __forceinline__ void tmem_st(uint32_t at, const uint32_t* w)
{
    static_assert(N == 2 || N == 4 || N == 8, "columns of a store");
    if constexpr (N == 2)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(at), "r"(w[0]), "r"(w[1]) : "memory");
    else if constexpr (N == 4)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3])
                     : "memory");
    else
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(at), "r"(w[0]),
                     "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
}

// The scale bytes of blocks b .. b + 3 of rows first + 32 j + the lane, j < N; 2^0 for rows past the matrix and blocks past
// the row, whose values come as zeros.  Every load goes out before the first is used (a branch for each row had the
// loads of one wait for the other's: 3 us a tile at K = 240).
template <int N>
__device__ __forceinline__ void scale_words(const uint8_t* s, int first, int rows, int kb, int b, uint32_t* w)
{
    const int lane = threadIdx.x & 31;
    const uint8_t* p[N];
#pragma unroll
    for (int j = 0; j < N; ++j) p[j] = s + static_cast<long long>(min(first + 32 * j + lane, rows - 1)) * kb;
    if (!((kb | b | static_cast<int>(reinterpret_cast<uintptr_t>(s))) & 3)) {
#pragma unroll
        for (int j = 0; j < N; ++j) w[j] = __ldg(reinterpret_cast<const uint32_t*>(p[j] + b));
    } else {
        uint32_t byte[N][4];
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) byte[j][i] = __ldg(p[j] + min(b + i, kb - 1));
#pragma unroll
        for (int j = 0; j < N; ++j) {
            w[j] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[j] |= (b + i < kb ? byte[j][i] : 0x7fu) << (8 * i);
        }
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (first + 32 * j + lane >= rows) w[j] = 0x7f7f7f7fu;
}

// SPLIT: the blocks of K of a CTA's one tile are shared by a cluster, whose sums meet in shared memory: each CTA adds up
// its part of the tile from all of them, in their order.
template <int BN, typename Elem, bool SPLIT>
__global__ void __launch_bounds__(kE4Threads, 1) linear_e4m3_kernel(const __grid_constant__ CUtensorMap tm_x,
                                                                    const __grid_constant__ CUtensorMap tm_w,
                                                                    const __grid_constant__ CUtensorMap tm_out, const E4Args a)
{
    using SP = E4Smem<BN>;
    constexpr int S = SP::stages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_addr(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(sm + SP::off_misc);
    volatile int* s_abort = reinterpret_cast<volatile int*>(sm + SP::off_misc + 4);
    const uint32_t bar_full = sb + SP::off_bar, bar_empty = bar_full + 8 * S;
    const uint32_t bar_sf = bar_empty + 8 * S, bar_sf_free = bar_sf + 16;
    const uint32_t bar_acc_full = bar_sf_free + 16, bar_acc_free = bar_acc_full + 16, bar_drain = bar_acc_free + 16;
    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(bar_full + 8 * i, 1);
            mbar_init(bar_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_sf + 8 * i, kE4ScaleWarps);
            mbar_init(bar_sf_free + 8 * i, 1);
            mbar_init(bar_acc_full + 8 * i, 1);
            mbar_init(bar_acc_free + 8 * i, kE4EpiWarps);
        }
        mbar_init(bar_drain, 1);
        fence_mbar_init();
        *s_abort = 0;
    }
    if (warp == kE4Issuer + 1 && lane == 0) {
        prefetch_tensormap(&tm_x);
        prefetch_tensormap(&tm_w);
        if (a.by_tma) prefetch_tensormap(&tm_out);
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(s_tmem)), "r"(SP::cols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    grid_dep_wait();

    // tiles blockIdx.x, + gridDim.x, ... are the CTA's, a row of tiles after the other
    const int rank = SPLIT ? blockIdx.x % a.splits : 0;
    const int first = SPLIT ? blockIdx.x / a.splits : blockIdx.x, stride = SPLIT ? a.tiles : gridDim.x;
    const int my_tiles = first < a.tiles ? (a.tiles - 1 - first) / stride + 1 : 0;
    const int k0 = rank * a.share, ksteps = SPLIT ? min(a.share, a.p.kb - k0) : a.p.kb;   // blocks
    const int groups = (ksteps + 3) / 4;   // of four blocks

    if (warp == kE4Issuer + 1) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            int i = 0;
            bool ok = true;
            for (int lt = 0; lt < my_tiles && ok; ++lt) {
                const int t = first + lt * stride, mt = t / a.nt, nt = t - mt * a.nt;
                for (int kb = 0; kb < ksteps; ++kb, ++i) {
                    const int slot = i % S;
                    if (i >= S && !sleep_or_abort(bar_empty + 8 * slot, ((i / S) - 1) & 1, s_abort)) {
                        ok = false;
                        break;
                    }
                    // rows past M or N and bytes past K come as zeros
                    const uint32_t dst = sb + slot * SP::tile, bar = bar_full + 8 * slot;
                    mbar_arrive_expect_tx(bar, SP::tile);
                    tma_load_2d(dst, &tm_x, bar, 128 * (k0 + kb), mt * 128);
                    tma_load_2d(dst + SP::tile_a, &tm_w, bar, 128 * (k0 + kb), nt * BN);
                }
            }
            // no copy may still be landing when the CTA exits
            for (int u = i - S; u < i; ++u)
                if (u >= 0 && !mbar_wait(bar_full + 8 * (u % S), (u / S) & 1)) *s_abort = 1;
        }
    } else if (warp == kE4Issuer) {
        // ------------------------------------------------------------- MMA issuer
        if (lane == 0) {
            // e4m3 A and B, fp32 D, UE8M0 scales, M = 128
            constexpr uint32_t id = (static_cast<uint32_t>(BN >> 3) << 17) | (1u << 23) | (1u << 27);
            int i = 0, gi = 0, nacc = 0, nfree = 0;
            bool ok = true;
            for (int lt = 0; lt < my_tiles && ok; ++lt) {
                const int buf = lt & 1;
                if (lt >= 2 && !sleep_or_abort(bar_acc_free + 8 * buf, ((lt >> 1) - 1) & 1, s_abort)) break;
                for (int kb = 0; kb < ksteps; ++kb, ++i) {
                    const int slot = i % S, sf = gi & 1;
                    if ((!(kb & 3) && !sleep_or_abort(bar_sf + 8 * sf, (gi >> 1) & 1, s_abort)) ||
                        !sleep_or_abort(bar_full + 8 * slot, (i / S) & 1, s_abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t base = sb + slot * SP::tile, sa = tmem + SP::off_sf + sf * SP::sf_cols;
                    const uint32_t idk = id | (static_cast<uint32_t>(kb & 3) << 4) | (static_cast<uint32_t>(kb & 3) << 29);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_e4m3_scaled(tmem + buf * BN, sdesc(base + 32 * k), sdesc(base + SP::tile_a + 32 * k), idk, sa, sa + 4,
                                         kb > 0 || k > 0);
                    umma_commit(bar_empty + 8 * slot);
                    ++nfree;
                    if ((kb & 3) == 3 || kb == ksteps - 1) {
                        umma_commit(bar_sf_free + 8 * sf);
                        ++gi;
                    }
                }
                if (!ok) break;
                umma_commit(bar_acc_full + 8 * buf);
                ++nacc;
            }
            // drain: every MMA issued has finished and every arrival it owes has landed
            umma_commit(bar_drain);
            bool drained = mbar_wait(bar_drain, 0);
            for (int u = nacc - 2; u < nacc; ++u)
                if (u >= 0) drained = mbar_wait(bar_acc_full + 8 * (u & 1), (u >> 1) & 1) && drained;
            for (int u = gi - 2; u < gi; ++u)
                if (u >= 0) drained = mbar_wait(bar_sf_free + 8 * (u & 1), (u >> 1) & 1) && drained;
            for (int u = nfree - S; u < nfree; ++u)
                if (u >= 0) drained = mbar_wait(bar_empty + 8 * (u % S), (u / S) & 1) && drained;
            if (!drained) *s_abort = 1;
        }
    } else if (warp >= kE4EpiWarps) {
        // --------------------------------------------------------------- scales
        // lane l of each quadrant: the words of rows l, l + 32, ... in neighbouring columns
        constexpr int NB = BN / 32, NBS = NB <= 2 ? 2 : NB <= 4 ? 4 : 8;
        const uint32_t quad = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + SP::off_sf;
        int gi = 0;
        bool ok = true;
        for (int lt = 0; lt < my_tiles && ok; ++lt) {
            const int t = first + lt * stride, mt = t / a.nt, nt = t - mt * a.nt;
            for (int g = 0; g < groups; ++g, ++gi) {
                uint32_t wa[4], wb[NBS];
                scale_words<4>(a.p.xs, mt * 128, a.p.M, a.p.kb, k0 + 4 * g, wa);
                scale_words<NB>(a.p.ws, nt * BN, a.p.N, a.p.kb, k0 + 4 * g, wb);
#pragma unroll
                for (int j = NB; j < NBS; ++j) wb[j] = 0u;
                const int sf = gi & 1;
                if (gi >= 2 && !__all_sync(0xffffffffu, sleep_or_abort(bar_sf_free + 8 * sf, ((gi >> 1) - 1) & 1, s_abort))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                tmem_st<4>(quad + sf * SP::sf_cols, wa);
                tmem_st<NBS>(quad + sf * SP::sf_cols + 4, wb);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_release(bar_sf + 8 * sf);
            }
        }
    } else {
        // --------------------------------------------------------------- epilogue
        // warp: 32 rows (its TMEM lanes, warp % 4) of one half of the tile's columns (warp / 4)
        constexpr int HN = BN / 2;
        const int rq = warp & 3, half = warp >> 2, M = a.p.M, N = a.p.N;
        const uint32_t tl = tmem + (static_cast<uint32_t>(32 * rq) << 16) + half * HN;
        float* s_bias = reinterpret_cast<float*>(sm + SP::off_bias) + warp * HN;
        uint8_t* s_out = sm + SP::off_out + warp * 2 * 32 * 64;
        const Elem* bias = static_cast<const Elem*>(a.p.bias);
        int staged = 0;   // tiles handed to TMA
        for (int lt = 0; lt < my_tiles; ++lt) {
            const int t = first + lt * stride, mt = t / a.nt, nt = t - mt * a.nt, buf = lt & 1;
            const int row0 = mt * 128 + 32 * rq, col0 = nt * BN + half * HN;
            __syncwarp();
            for (int j = lane; j < HN; j += 32) s_bias[j] = bias && col0 + j < N ? bias_at(bias, col0 + j) : 0.f;
            __syncwarp();
            if (!__all_sync(0xffffffffu, sleep_or_abort(bar_acc_full + 8 * buf, (lt >> 1) & 1, s_abort))) break;
            tc_fence_after();
            // the lane's row of the half tile into registers, so that the accumulator is free for the tile after next
            uint32_t acc[HN];
#pragma unroll
            for (int c = 0; c < HN; c += 32) {
                uint32_t* r = acc + c;
                OASR_TMEM_LD32(tl + buf * BN + c, r);
            }
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_release(bar_acc_free + 8 * buf);
            if constexpr (SPLIT) {   // every product has read the ring: the sums' place
                float* to = reinterpret_cast<float*>(sm) + (32 * rq + lane) * SP::part_row + half * HN;
#pragma unroll
                for (int c = 0; c < HN; c += 4)
                    *reinterpret_cast<uint4*>(to + c) = make_uint4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
                continue;
            }
            // no rows of this warp's: nothing staged, as a staging tile is free again only by a store made after its last use
            if (row0 >= M) continue;
            auto sum = [&](int j) { return __uint_as_float(acc[j]) + s_bias[j]; };
            if (a.by_tma) {
                // 64 bytes of every row at a time, staged in turn in two tiles and stored by TMA
                constexpr int CB = 64 / sizeof(Elem);
#pragma unroll
                for (int c = 0; c < HN; c += CB) {
                    if (col0 + c < N) {
                        uint8_t* to = s_out + (staged++ & 1) * 32 * 64;
                        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");   // the tile's last use
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 4; ++j) {   // 16 bytes
                            uint4 o;
                            if constexpr (sizeof(Elem) == 2)
                                o = make_uint4(pack_bf16(sum(c + 8 * j), sum(c + 8 * j + 1)), pack_bf16(sum(c + 8 * j + 2), sum(c + 8 * j + 3)),
                                               pack_bf16(sum(c + 8 * j + 4), sum(c + 8 * j + 5)),
                                               pack_bf16(sum(c + 8 * j + 6), sum(c + 8 * j + 7)));
                            else
                                o = make_uint4(__float_as_uint(sum(c + 4 * j)), __float_as_uint(sum(c + 4 * j + 1)),
                                               __float_as_uint(sum(c + 4 * j + 2)), __float_as_uint(sum(c + 4 * j + 3)));
                            *reinterpret_cast<uint4*>(to + 64 * lane + 16 * (j ^ ((lane >> 1) & 3))) = o;
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) tma_store_2d(&tm_out, smem_addr(to), (col0 + c) * static_cast<int>(sizeof(Elem)), row0);
                    }
                }
            } else {
                // rows of any alignment: 32 columns at a time, staged as the lanes' rows and written row by row, a lane
                // a column
                constexpr int RB = 32 * sizeof(Elem), PV = 16 / sizeof(Elem);   // bytes of a staged row, values of 16 bytes
                auto place = [](int r, int v) { return RB * r + 16 * (v ^ (RB == 64 ? r >> 1 & 3 : r & 7)); };
#pragma unroll
                for (int c = 0; c < HN; c += 32) {
                    if (col0 + c < N) {
                        __syncwarp();
#pragma unroll
                        for (int v = 0; v < RB / 16; ++v) {
                            uint4 o;
                            const int j = c + PV * v;
                            if constexpr (sizeof(Elem) == 2)
                                o = make_uint4(pack_bf16(sum(j), sum(j + 1)), pack_bf16(sum(j + 2), sum(j + 3)),
                                               pack_bf16(sum(j + 4), sum(j + 5)), pack_bf16(sum(j + 6), sum(j + 7)));
                            else
                                o = make_uint4(__float_as_uint(sum(j)), __float_as_uint(sum(j + 1)), __float_as_uint(sum(j + 2)),
                                               __float_as_uint(sum(j + 3)));
                            *reinterpret_cast<uint4*>(s_out + place(lane, v)) = o;
                        }
                        __syncwarp();
                        if (col0 + c + lane < N) {
                            Elem* to = static_cast<Elem*>(a.out) + static_cast<long long>(row0) * N + col0 + c + lane;
                            auto at = [&](int r) {
                                return reinterpret_cast<const Elem*>(s_out + place(r, lane / PV))[lane % PV];
                            };
                            if (row0 + 32 <= M) {
#pragma unroll 16
                                for (int r = 0; r < 32; ++r) to[static_cast<long long>(r) * N] = at(r);
                            } else {
                                for (int r = 0; r < M - row0; ++r) to[static_cast<long long>(r) * N] = at(r);
                            }
                        }
                    }
                }
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");   // every store has been made
    }
    if constexpr (SPLIT) {
        __syncwarp();
        cluster_sync();
        const int mt = first / a.nt, nt = first - mt * a.nt;
        const Elem* bias = static_cast<const Elem*>(a.p.bias);
        // four columns of a row at a time, a run of them to each CTA
        const int all = min(128, a.p.M - mt * 128) * (BN / 4), run = (all + a.splits - 1) / a.splits;
        for (int i = rank * run + tid; i < min(all, (rank + 1) * run); i += kE4Threads) {
            const int r = i / (BN / 4), c = i % (BN / 4) * 4, row = mt * 128 + r, col = nt * BN + c;
            if (col >= a.p.N) continue;
            const uint32_t at = sb + (r * SP::part_row + c) * 4;
            float4 part[kE4Splits];
#pragma unroll
            for (int p = 0; p < kE4Splits; ++p)
                if (p < a.splits) part[p] = ld_shared_cluster4(at, p);
            float v[4] = {part[0].x, part[0].y, part[0].z, part[0].w};
#pragma unroll
            for (int p = 1; p < kE4Splits; ++p)
                if (p < a.splits) v[0] += part[p].x, v[1] += part[p].y, v[2] += part[p].z, v[3] += part[p].w;
            Elem* to = static_cast<Elem*>(a.out) + static_cast<long long>(row) * a.p.N + col;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < a.p.N) put(to + e, v[e] + (bias ? bias_at(bias, col + e) : 0.f));
        }
        cluster_sync();   // no CTA leaves while another one reads its sums
    }
    grid_dep_trigger();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(SP::cols));
    }
    if (tid == 0 && *s_abort) atomicOr(a.status, kErrTimeout);
}

// --------------------------------------------------------------------------- host

constexpr int kE4MaxRows = 0x7fffff00, kE4MaxK = 65536;

int g_smem_done_e4l[8][64];

// splits > 1 (SPLIT): CTAs that share a tile's K, at most one tile a CTA
template <int BN, typename Elem, bool SPLIT = false>
oasr_status launch_e4(const E4Problem& p, void* out, int slot, int sms, cudaStream_t stream, int splits = 1, int share = 0)
{
    using SP = E4Smem<BN>;
    const long long mt = (p.M + 127LL) / 128, nt = (p.N + BN - 1LL) / BN, row = p.N * static_cast<long long>(sizeof(Elem));
    if (mt * nt > 0x7fffffffLL - sms) return OASR_ERR_UNSUPPORTED;
    auto kern = linear_e4m3_kernel<BN, Elem, SPLIT>;
    if (!ensure_smem(kern, SP::bytes, g_smem_done_e4l[slot])) return OASR_ERR_CUDA;
    CUtensorMap tm_x, tm_w, tm_out = {};
    const bool by_tma = !SPLIT && row % 16 == 0 && row <= 0x7fffffffLL;
    if (!encode_bytes128(&tm_x, p.x, p.M, p.K, 128) || !encode_bytes128(&tm_w, p.w, p.N, p.K, BN) ||
        (by_tma && !encode_bytes(&tm_out, out, p.M, static_cast<int>(row), 32, true)))
        return OASR_ERR_INVALID_ARG;
    const E4Args a = {p, out, static_cast<int>(nt), static_cast<int>(mt * nt), by_tma, splits, share, status_word()};
    if (!a.status) return OASR_ERR_CUDA;
    if (SPLIT)
        return launch_pdl_cluster(kern, dim3(a.tiles * splits), dim3(kE4Threads), SP::bytes, splits, stream, tm_x, tm_w,
                                  tm_out, a);
    return launch_pdl(kern, dim3(a.tiles < sms ? a.tiles : sms), dim3(kE4Threads), SP::bytes, stream, tm_x, tm_w, tm_out, a);
}

template <typename Elem>
oasr_status dispatch_e4(const E4Problem& p, void* out, cudaStream_t stream)
{
    // A few rows without tiles, where that is the shorter of the two: about 1300 ns and 90 for each row and 128 of K (512 at a
    // time, and up to 2048 columns), against 2600 and 300 for each 128 of K.  2 x 512 x 2048: 3.8 and 5.0 us, 4 x 2048 x
    // 512 2.5 and 3.7, 6 x 512 x 512 2.9 and 3.6, 6 x 4096 x 1024 11.1 and 6.2, 6 x 512 x 2048 7.4 and 5.5.  That K may be shared
    // by a cluster below is not weighed here: 4 x 512 x 2560 takes 8.0 us and would 5.9, 3 x 512 x 4096 14.4 and 6.8.
    const long long steps = (p.K + 511LL) / 512 * 4, few = 1300 + 90LL * p.M * steps * (p.N > 2048 ? p.N : 2048) / 2048;
    if (p.M == 1 || (p.M <= kE4FewRows && few < 2600 + 300LL * p.kb)) {
        const dim3 grid((p.N + 7) / 8);
        auto go = [&](auto kern) { return launch_pdl(kern, grid, dim3(256), 0, stream, p, static_cast<Elem*>(out)); };
        if (p.M == 1) return go(linear_e4m3_few_kernel<1, Elem>);
        if (p.M == 2) return go(linear_e4m3_few_kernel<2, Elem>);
        if (p.M <= 4) return go(linear_e4m3_few_kernel<4, Elem>);
        return go(linear_e4m3_few_kernel<kE4FewRows, Elem>);
    }
    const int sms = sm_count();
    if (!sms) return OASR_ERR_CUDA;
    constexpr int s = sizeof(Elem) == 4 ? 3 : 0;
    // Tile: the one of the least estimated time.  A step of 128 of K costs 470 ns in 128 x 192, 430 in 128 x 128 and 380 in
    // 128 x 64 (the copies into shared memory are the cost), a tile's hand-over 250, 100 and 50, the last epilogue 1000, 700
    // and 400.  Bf16 results, in this order: 8191 x 4096 x 1024 36.4, 43.4 and 74.9 us; 4096 x 512 x 2048 9.2, 8.8 and 13.4;
    // 1024 x 768 x 256 4.3, 3.9 and 3.8.
    constexpr struct { int n, step, tile, end; } kinds[] = {{192, 470, 250, 1000}, {128, 430, 100, 700}, {64, 380, 50, 400}};
    int best = 0;
    long long least = 0x7fffffffffffffffLL;
    for (int k = 0; k < 3; ++k) {
        const long long tiles = ((p.M + 127LL) / 128) * ((p.N + kinds[k].n - 1LL) / kinds[k].n);
        const long long ns = (tiles + sms - 1) / sms * (static_cast<long long>(p.kb) * kinds[k].step + kinds[k].tile) + kinds[k].end;
        if (ns < least) least = ns, best = k;
    }
    // Few tiles of 128 x 64: K shared by a cluster, 2700 ns for its start and the sums' way (64 x 512 x 2048 5.9 us, 7.3
    // without; 64 x 512 x 4096 6.5 and 12.0; 64 x 1024 x 8192 10.5 and 22.0; 16 x 512 x 1024 5.2 and 5.0, so not shared).  On more
    // than half of the SMs the clusters wait for one another (300 x 512 x 2048 on 144 SMs 11.6 us, 7.5 without).
    const long long tiles = ((p.M + 127LL) / 128) * ((p.N + 63LL) / 64);
    int share = p.kb;
    for (int n = 2; n <= kE4Splits && 2 * tiles * n <= sms; ++n) {
        const int each = (p.kb + n - 1) / n;
        const long long ns = each * 380LL + 50 + 400 + 2700;
        if (ns < least) least = ns, share = each, best = 3;
    }
    if (best == 3)
        return launch_e4<64, Elem, true>(p, out, s ? 7 : 6, sms, stream, (p.kb + share - 1) / share, share);
    if (best == 0) return launch_e4<192, Elem>(p, out, s, sms, stream);
    if (best == 1) return launch_e4<128, Elem>(p, out, s + 1, sms, stream);
    return launch_e4<64, Elem>(p, out, s + 2, sms, stream);
}

}  // namespace
}  // namespace oasr

extern "C" oasr_status oasr_quantize_blocks(const void* x, void* x8, void* scale, int M, int K, oasr_dtype dt,
                                            cudaStream_t stream)
{
    using namespace oasr;
    if (!x || !x8 || !scale || M <= 0 || K <= 0) return OASR_ERR_INVALID_ARG;
    if ((dt != OASR_F32 && dt != OASR_BF16) || K % 16) return OASR_ERR_UNSUPPORTED;
    if (!aligned16(x) || !aligned16(x8)) return OASR_ERR_INVALID_ARG;
    const int kb = (K - 1) / kBlk + 1;
    const long long ctas = (static_cast<long long>(M) * kb + 16 * kQBlocks - 1) / (16 * kQBlocks);
    if (ctas > 0x7fffffffLL) return OASR_ERR_UNSUPPORTED;
    auto go = [&](auto* src) {
        using E = std::remove_const_t<std::remove_pointer_t<decltype(src)>>;
        return launch_pdl(K % kBlk ? quantize_blocks_kernel<false, E> : quantize_blocks_kernel<true, E>,
                          dim3(static_cast<unsigned>(ctas)), dim3(256), 0, stream, src, static_cast<uint8_t*>(x8),
                          static_cast<uint8_t*>(scale), M, K, kb,
                          kb > 1 ? static_cast<unsigned>(0xffffffffu / kb + 1) : 0u);
    };
    return dt == OASR_F32 ? go(static_cast<const float*>(x)) : go(static_cast<const __nv_bfloat16*>(x));
}

extern "C" oasr_status oasr_linear_e4m3(const void* x8, const void* x_scale, const void* w8, const void* w_scale,
                                        const void* bias, void* out, int M, int N, int K, oasr_dtype dt, cudaStream_t stream)
{
    using namespace oasr;
    if (!x8 || !x_scale || !w8 || !w_scale || !out || M <= 0 || N <= 0 || K <= 0) return OASR_ERR_INVALID_ARG;
    if ((dt != OASR_F32 && dt != OASR_BF16) || K % 16 || K > kE4MaxK || M > kE4MaxRows || N > kE4MaxRows)
        return OASR_ERR_UNSUPPORTED;
    const void* ptrs[] = {x8, w8, bias ? bias : x8, out};
    for (const void* p : ptrs)
        if (!aligned16(p)) return OASR_ERR_INVALID_ARG;
    const E4Problem p = {static_cast<const uint8_t*>(x8),      static_cast<const uint8_t*>(w8),
                         static_cast<const uint8_t*>(x_scale), static_cast<const uint8_t*>(w_scale),
                         bias, M, N, K, (K + kBlk - 1) / kBlk};
    return dt == OASR_F32 ? dispatch_e4<float>(p, out, stream) : dispatch_e4<__nv_bfloat16>(p, out, stream);
}
