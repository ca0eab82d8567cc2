// 8-bit integer products with a scale per token and per output channel:
//
//   oasr_quantize_rows         m = max(max|x_row|, 2^-100), x8 = rint(x (127 (1 / m))), scale = m / 127
//   oasr_linear_w8a8           out[i][n] = (sum_k x8[i][k] w8[n][k]) x_scale[i] w_scale[n] + bias[n]
//   oasr_project_qkv_pos_w8a8  the same for a step's q, k, v and its position table, in one launch
//
// This GPU's tensor cores have next to no 8-bit integer rate, but an 8-bit integer is exact in fp16
// and a product of two exact in fp32, so the sums run on tcgen05's fp16 rate: converter warps
// read the 8-bit rows and write them as fp16 into the swizzled tiles the matrix instructions
// read.  A sum stays within 2^24 for K <= 1024, where fp32 holds every integer: the accumulated
// sum is the integer sum.  For longer K it is that of an fp32 accumulation.  Few rows (dispatch_i8) go through
// integer dot products, whose sum is the integer whatever K is, rounded once to fp32.
//
// What bounds a large product is shared memory: of a K step of 64, a tile's rows come in as bytes,
// are read, written as fp16 and read by the matrix unit.  A pair of CTAs on one 256 x 256 tile
// (cta_group::2) holds and converts each w row once for both, 96 KB of traffic per CTA and step
// where a CTA alone on 128 x 256 has 144.  8191 x 4096 x 1024: 57 us in fp32, 51 in bf16
// (1.2 and 1.35 PFLOP/s); with 128 x 128 tiles 87 and 79.
#include <type_traits>

#include "attn_core.cuh"
#include "cluster.cuh"
#include "e4m3.cuh"
#include "host_common.h"
#include "linear.cuh"

namespace oasr {
namespace {

// ------------------------------------------------------------------ rows to 8 bits

constexpr float kLeastMax = 7.8886090522101181e-31f;   // 2^-100

// TPR threads per row, each with NC chunks of eight values in registers (NC 0: a longer row, read a second
// time for its quantisation).  Bound by HBM: 2 or 4 bytes in, one out per value.
template <typename Elem, int TPR, int NC>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const Elem* __restrict__ x, int8_t* __restrict__ x8,
                                                            float* __restrict__ scale, int M, int K)
{
    grid_dep_wait();
    const int row = blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
    const int l = threadIdx.x % TPR, chunks = K / 8;
    const bool on = row < M;
    const Elem* src = x + static_cast<long long>(on ? row : 0) * K;
    constexpr int N = NC ? NC : 1;
    float v[N][8];
    float m = 0.f;
    auto largest = [&](const float (&w)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fabsf(w[e]) < INFINITY ? fmaxf(m, fabsf(w[e])) : INFINITY;
    };
    if constexpr (NC > 0) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
            if (l + TPR * i < chunks) load8(src + 8 * (l + TPR * i), v[i]);
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) largest(v[i]);
    } else {
#pragma unroll 4
        for (int c = l; c < chunks; c += TPR) {
            load8(src + 8 * c, v[0]);
            largest(v[0]);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if constexpr (TPR > 32) {
        __shared__ float s_m[8];
        if ((threadIdx.x & 31) == 0) s_m[threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < TPR / 32; ++w) m = fmaxf(m, s_m[w]);
    }
    const bool bad = m == INFINITY;
    m = fmaxf(m, kLeastMax);
    const float f = __fmul_rn(__frcp_rn(m), 127.f);
    if (on) {
        if (l == 0) scale[row] = bad ? NAN : __fdiv_rn(m, 127.f);
        int8_t* dst = x8 + static_cast<long long>(row) * K;
        auto put8 = [&](int c, const float (&w)[8]) {
            uint32_t q[2] = {0u, 0u};
#pragma unroll
            for (int e = 0; e < 8; ++e)
                q[e >> 2] |= (static_cast<uint32_t>(__float2int_rn(__fmul_rn(w[e], f))) & 255u) << (8 * (e & 3));
            *reinterpret_cast<uint2*>(dst + 8 * c) = bad ? make_uint2(0u, 0u) : make_uint2(q[0], q[1]);
        };
        if constexpr (NC > 0) {
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (l + TPR * i < chunks) put8(l + TPR * i, v[i]);
        } else {
#pragma unroll 2
            for (int c = l; c < chunks; c += TPR) {
                load8(src + 8 * c, v[0]);
                put8(c, v[0]);
            }
        }
    }
    grid_dep_trigger();
}

// --------------------------------------------------------------------- products

struct I8Problem {
    const int8_t* x;        // [M][K]
    const int8_t* w;        // [N][K]
    const float* xs;
    const float* ws;
    const void* bias;       // null: none
    int M, N;
};

struct I8Args {
    I8Problem p[2];
    void* out[4];           // problem 0: column block n / width into out[n / width]; problem 1: out[3]
    int width;
    int K, nt0, nt1, tiles0, tiles;   // column tiles of each problem; tiles of problem 0, of both
    int by_tma;             // the outputs' rows suit TMA: stored by it
    unsigned* status;
};

// Four sums times their row's scale x and columns' scales w, plus the bias b; each operation rounded.
__device__ __forceinline__ float4 scaled(const uint32_t* s, float x, float4 w, float4 b)
{
    auto one = [&](uint32_t v, float wj, float bj) { return __fadd_rn(__fmul_rn(__fmul_rn(__uint_as_float(v), x), wj), bj); };
    return make_float4(one(s[0], w.x, b.x), one(s[1], w.y, b.y), one(s[2], w.z, b.z), one(s[3], w.w, b.w));
}

// Eight 8-bit integers (natural order) to fp16: with its sign bit flipped a byte b is b + 128 as
// an unsigned number, which under the exponent of 1024 reads 1152 + b.
__device__ __forceinline__ uint32_t i8_sub(uint32_t x)
{
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0x64806480u));
    return r;
}
__device__ __forceinline__ uint4 i8_to_f16(uint32_t w0, uint32_t w1)
{
    w0 ^= 0x80808080u;
    w1 ^= 0x80808080u;
    return make_uint4(i8_sub(__byte_perm(w0, 0x64646464u, 0x4140)), i8_sub(__byte_perm(w0, 0x64646464u, 0x4342)),
                      i8_sub(__byte_perm(w1, 0x64646464u, 0x4140)), i8_sub(__byte_perm(w1, 0x64646464u, 0x4342)));
}

// Warps: eight for the epilogue, four groups of four converters, the issuer, the TMA producer.  The producer
// brings 8-bit tiles of 64 K into a ring; the converter groups take its slots in turn (one group's proxy
// fence and waits pass while the others convert: 59.8 us where two groups of eight warps take 63.1) and write
// the fp16 ring that the products read; two accumulators let a tile's epilogue overlap the next tile's products.
// In a pair both CTAs do so with their own rows, and the even one issues the products of both: the odd one's
// issuer passes on that a slot is written.
constexpr int kI8EpiWarps = 8, kI8Group = 128, kI8Groups = 4;
constexpr int kI8Conv0 = 32 * kI8EpiWarps;                        // first converter thread
constexpr int kI8Issuer = kI8EpiWarps + kI8Groups * kI8Group / 32;   // its warp; the producer's is the next
constexpr int kI8Threads = 32 * (kI8Issuer + 2);

template <int BN, bool PAIR>
struct I8Smem {
    static constexpr int b_rows = PAIR ? BN / 2 : BN;                  // of a tile's w rows, the CTA's
    static constexpr int rows = 128 + b_rows;                          // x rows, then w rows
    static constexpr int tile_a = 128 * 128, tile = rows * 128;        // fp16, 64 of K
    static constexpr int raw = rows * 64;                              // 8-bit, 64 of K
    static constexpr int stages = 4, raws = 4;
    static constexpr int off_raw = stages * tile;
    static constexpr bool tma_out = BN >= 128;
    static constexpr int off_out = off_raw + raws * raw;               // [8 warps][32 rows][64 bytes]
    static constexpr int off_ws = off_out + kI8EpiWarps * 32 * 64;   // [8 warps][2][BN / 2] floats
    static constexpr int off_bar = off_ws + kI8EpiWarps * BN * 4;      // full, empty, raw full, raw empty, acc full[2], acc free[2], drain
    static constexpr int off_misc = off_bar + (2 * stages + 2 * raws + 5) * 8;
    static constexpr int bytes = off_misc + 16 + 1024;
    static constexpr int cols = 2 * BN < 32 ? 32 : 2 * BN;
    // a group's last wait on a slot's barrier was for the phase before (it comes by every slot in turn)
    static_assert(stages % kI8Groups == 0 && raws % kI8Groups == 0, "a wait is one phase behind at most");
};

struct I8Outs {
    CUtensorMap m[4];   // of I8Args::out
};

template <int BN, bool PAIR, typename Elem>
__global__ void __launch_bounds__(kI8Threads, 1) linear_i8_kernel(
    const __grid_constant__ CUtensorMap tm_x0, const __grid_constant__ CUtensorMap tm_w0,
    const __grid_constant__ CUtensorMap tm_x1, const __grid_constant__ CUtensorMap tm_w1,
    const __grid_constant__ I8Outs outs, const I8Args a)
{
    using SP = I8Smem<BN, PAIR>;
    constexpr int CTAS = PAIR ? 2 : 1;
    constexpr int S = SP::stages, R = SP::raws;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_addr(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(sm + SP::off_misc);
    volatile int* s_abort = reinterpret_cast<volatile int*>(sm + SP::off_misc + 4);
    const uint32_t bar_full = sb + SP::off_bar, bar_empty = bar_full + 8 * S;
    const uint32_t bar_raw = bar_empty + 8 * S, bar_raw_free = bar_raw + 8 * R;
    const uint32_t bar_acc_full = bar_raw_free + 8 * R, bar_acc_free = bar_acc_full + 16;
    const uint32_t bar_drain = bar_acc_free + 16;
    const int ksteps = (a.K + 63) / 64;
    const int rank = PAIR ? blockIdx.x & 1 : 0;   // in the pair; 0 issues the products of both
    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(bar_full + 8 * i, kI8Group + (PAIR && rank == 0));
            mbar_init(bar_empty + 8 * i, 1);
        }
        for (int i = 0; i < R; ++i) {
            mbar_init(bar_raw + 8 * i, 1);
            mbar_init(bar_raw_free + 8 * i, kI8Group);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_acc_full + 8 * i, 1);
            mbar_init(bar_acc_free + 8 * i, CTAS * kI8EpiWarps);
        }
        mbar_init(bar_drain, 1);
        fence_mbar_init();
        *s_abort = 0;
    }
    if (warp == kI8Issuer + 1 && lane == 0) {
        prefetch_tensormap(&tm_x0);
        prefetch_tensormap(&tm_w0);
        prefetch_tensormap(&tm_x1);
        prefetch_tensormap(&tm_w1);
    }
    if (warp == 0) {
        if constexpr (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(s_tmem)),
                         "r"(SP::cols));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(s_tmem)),
                         "r"(SP::cols));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        }
    }
    tc_fence_before();
    if constexpr (PAIR)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    grid_dep_wait();

    auto decode = [&](int t, int& g, int& mt, int& nt) {
        g = t >= a.tiles0;
        if (g) t -= a.tiles0;
        const int n = g ? a.nt1 : a.nt0;
        mt = t / n;
        nt = t - mt * n;
    };
    // tiles first, first + stride, ... are the CTA's (the pair's)
    const int first = blockIdx.x / CTAS, stride = gridDim.x / CTAS;
    const int my_tiles = first < a.tiles ? (a.tiles - 1 - first) / stride + 1 : 0;
    const int iters = my_tiles * ksteps;

    if (warp == kI8Issuer + 1) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            int i = 0;
            bool ok = true;
            for (int lt = 0; lt < my_tiles && ok; ++lt) {
                int g, mt, nt;
                decode(first + lt * stride, g, mt, nt);
                for (int kb = 0; kb < ksteps; ++kb, ++i) {
                    const int slot = i % R;
                    if (i >= R && !sleep_or_abort(bar_raw_free + 8 * slot, ((i / R) - 1) & 1, s_abort)) {
                        ok = false;
                        break;
                    }
                    // rows past M or N and bytes past K come as zeros
                    const uint32_t dst = sb + SP::off_raw + slot * SP::raw, bar = bar_raw + 8 * slot;
                    mbar_arrive_expect_tx(bar, SP::raw);
                    tma_load_2d(dst, g ? &tm_x1 : &tm_x0, bar, 64 * kb, (mt * CTAS + rank) * 128);
                    tma_load_2d(dst + 128 * 64, g ? &tm_w1 : &tm_w0, bar, 64 * kb, nt * BN + rank * SP::b_rows);
                }
            }
            // no copy may still be landing when the CTA exits
            for (int u = i - R; u < i; ++u)
                if (u >= 0 && !mbar_wait(bar_raw + 8 * (u % R), (u / R) & 1)) *s_abort = 1;
        }
    } else if (warp == kI8Issuer) {
        // ------------------------------------------------------------- MMA issuer
        if (lane == 0 && rank) {
            // passes on to the other CTA that this one's rows of a slot are written
            for (int i = 0; i < iters; ++i) {
                if (!sleep_or_abort(bar_full + 8 * (i % S), (i / S) & 1, s_abort)) break;
                fence_release_smem_cluster();
                mbar_arrive_cluster_relaxed(bar_full + 8 * (i % S), 0);
            }
            // the other's commits have landed before this CTA ends
            for (int u = iters - S; u < iters; ++u)
                if (u >= 0 && !sleep_or_abort(bar_empty + 8 * (u % S), (u / S) & 1, s_abort)) break;
            if (!mbar_wait(bar_drain, 0)) *s_abort = 1;
        } else if (lane == 0) {
            // fp16 A and B, fp32 D
            constexpr uint32_t id = (1u << 4) | (static_cast<uint32_t>(BN >> 3) << 17) | ((CTAS * 128u >> 4) << 24);
            auto commit = [](uint32_t bar) {
                if constexpr (PAIR)
                    umma_commit_pair(bar);
                else
                    umma_commit(bar);
            };
            int i = 0, nacc = 0, nfree = 0;
            bool ok = true;
            for (int lt = 0; lt < my_tiles && ok; ++lt) {
                const int buf = lt & 1;
                if (lt >= 2 && !sleep_or_abort<PAIR>(bar_acc_free + 8 * buf, ((lt >> 1) - 1) & 1, s_abort)) break;
                for (int kb = 0; kb < ksteps; ++kb, ++i) {
                    const int slot = i % S;
                    if (!sleep_or_abort<PAIR>(bar_full + 8 * slot, (i / S) & 1, s_abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t base = sb + slot * SP::tile;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint64_t da = sdesc(base + 32 * k), db = sdesc(base + SP::tile_a + 32 * k);
                        if constexpr (PAIR)
                            umma_ss_pair(tmem + buf * BN, da, db, id, kb > 0 || k > 0);
                        else
                            umma_ss(tmem + buf * BN, da, db, id, kb > 0 || k > 0);
                    }
                    commit(bar_empty + 8 * slot);
                    ++nfree;
                }
                if (!ok) break;
                commit(bar_acc_full + 8 * buf);
                ++nacc;
            }
            // drain: every MMA issued has finished and every arrival it owes has landed
            commit(bar_drain);
            bool drained = mbar_wait(bar_drain, 0);
            for (int u = nacc - 2; u < nacc; ++u)
                if (u >= 0) drained = mbar_wait(bar_acc_full + 8 * (u & 1), (u >> 1) & 1) && drained;
            for (int u = nfree - S; u < nfree; ++u)
                if (u >= 0) drained = mbar_wait(bar_empty + 8 * (u % S), (u / S) & 1) && drained;
            if (!drained) *s_abort = 1;
        }
    } else if (warp >= kI8EpiWarps) {
        // ------------------------------------------------------------ converters
        // thread: 16 bytes (chunk c) of rows r0, r0 + CR, ...
        constexpr int CR = kI8Group / 4, NU = (SP::rows + CR - 1) / CR;   // rows of a pass, passes
        const int grp = (tid - kI8Conv0) / kI8Group, ct = (tid - kI8Conv0) % kI8Group, c = ct & 3, r0 = ct >> 2;
        for (int i = grp; i < iters; i += kI8Groups) {
            const int rs = i % R, slot = i % S;
            if (!__all_sync(0xffffffffu, sleep_or_abort(bar_raw + 8 * rs, (i / R) & 1, s_abort))) break;
            const uint8_t* src = sm + SP::off_raw + rs * SP::raw + 16 * ct;
            uint4 buf[NU];
#pragma unroll
            for (int u = 0; u < NU; ++u)
                if (r0 + CR * u < SP::rows) buf[u] = *reinterpret_cast<const uint4*>(src + 64 * CR * u);
            if (i >= S && !__all_sync(0xffffffffu, sleep_or_abort(bar_empty + 8 * slot, ((i / S) - 1) & 1, s_abort))) break;
            uint8_t* lo = sm + slot * SP::tile + swz128(r0, 2 * c);
            uint8_t* hi = sm + slot * SP::tile + swz128(r0, 2 * c + 1);
#pragma unroll
            for (int u = 0; u < NU; ++u)   // a multiple of 8 rows on, the same swizzle
                if (r0 + CR * u < SP::rows) {
                    *reinterpret_cast<uint4*>(lo + 128 * CR * u) = i8_to_f16(buf[u].x, buf[u].y);
                    *reinterpret_cast<uint4*>(hi + 128 * CR * u) = i8_to_f16(buf[u].z, buf[u].w);
                }
            fence_proxy_async_smem();
            mbar_arrive_release(bar_full + 8 * slot);
            // the raw slot is released only here, its words converted: an arrival right behind the loads can
            // overtake them (they wait in another unit's queue), and a copy then lands under them
            mbar_arrive_release(bar_raw_free + 8 * rs);
        }
    } else {
        // --------------------------------------------------------------- epilogue
        // warp: 32 rows (its TMEM lanes, warp % 4) of one half of the tile's columns (warp / 4)
        constexpr int HN = BN / 2, NC = HN / 16;
        const int rq = warp & 3, half = warp >> 2;
        const uint32_t tl = tmem + (static_cast<uint32_t>(32 * rq) << 16) + half * HN;
        float* s_ws = reinterpret_cast<float*>(sm + SP::off_ws) + warp * BN;   // w scales, then biases
        uint8_t* s_out = sm + SP::off_out + warp * 32 * 64;
        for (int lt = 0; lt < my_tiles; ++lt) {
            int g, mt, nt;
            decode(first + lt * stride, g, mt, nt);
            const I8Problem& p = a.p[g];
            const int M = p.M, N = p.N, buf = lt & 1;
            const Elem* bias = static_cast<const Elem*>(p.bias);
            const int row0 = (mt * CTAS + rank) * 128 + 32 * rq, col0 = nt * BN + half * HN;
            __syncwarp();
#pragma unroll
            for (int j = lane; j < HN; j += 32) {
                const int n = col0 + j;
                s_ws[j] = n < N ? __ldg(p.ws + n) : 0.f;
                s_ws[HN + j] = bias && n < N ? bias_at(bias, n) : 0.f;
            }
            const float x = row0 + lane < M ? __ldg(p.xs + row0 + lane) : 0.f;
            __syncwarp();
            if (!__all_sync(0xffffffffu, sleep_or_abort(bar_acc_full + 8 * buf, (lt >> 1) & 1, s_abort))) break;
            tc_fence_after();
            // the output of the block's columns (a block of 16 lies within one: widths are multiples of 64, or
            // there is one) and the block's first column there
            const int width = g ? N : a.width;
            int which = g ? 3 : col0 / width, at = g ? col0 : col0 - which * width;
            if (SP::tma_out && a.by_tma) {
                // 64 bytes of every row at a time, staged and stored by TMA
                constexpr int CB = 64 / sizeof(Elem);
#pragma unroll 1
                for (int c = 0; c < HN / CB; ++c) {
                    const int col = col0 + CB * c;
                    if (col >= N) break;
                    uint32_t r[CB];
                    OASR_TMEM_LD16(tl + buf * BN + CB * c, r);
                    if constexpr (CB == 32) {
                        uint32_t* r1 = r + 16;
                        OASR_TMEM_LD16(tl + buf * BN + CB * c + 16, r1);
                    }
                    tmem_wait_ld();
                    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");   // the tile's last use
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 4; ++j) {   // 16 bytes
                        uint32_t o[4];
#pragma unroll
                        for (int q = 0; q < CB / 16; ++q) {
                            const int e = (CB / 4) * j + 4 * q;
                            const float4 w = *reinterpret_cast<const float4*>(s_ws + CB * c + e);
                            const float4 b = *reinterpret_cast<const float4*>(s_ws + HN + CB * c + e);
                            const float4 v = scaled(r + e, x, w, b);
                            if constexpr (sizeof(Elem) == 2) {
                                o[2 * q] = pack_bf16(v.x, v.y);
                                o[2 * q + 1] = pack_bf16(v.z, v.w);
                            } else {
                                o[0] = __float_as_uint(v.x), o[1] = __float_as_uint(v.y);
                                o[2] = __float_as_uint(v.z), o[3] = __float_as_uint(v.w);
                            }
                        }
                        *reinterpret_cast<uint4*>(s_out + 64 * lane + 16 * (j ^ ((lane >> 1) & 3))) =
                            make_uint4(o[0], o[1], o[2], o[3]);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && row0 < M)
                        tma_store_2d(&outs.m[which], smem_addr(s_out), at * static_cast<int>(sizeof(Elem)), row0);
                    if ((at += CB) == width && !g) {
                        at = 0;
                        ++which;
                    }
                }
            } else {
                // a lane's row straight from its registers, in whole 32-byte sectors where they are aligned
                const long long row = row0 + lane;
#pragma unroll 1
                for (int c = 0; c < NC; ++c) {
                    const int col = col0 + 16 * c;
                    if (col >= N) break;
                    uint32_t r[16];
                    OASR_TMEM_LD16(tl + buf * BN + 16 * c, r);
                    tmem_wait_ld();
                    constexpr int W = sizeof(Elem) * 16 / 4;   // words of the row
                    uint32_t o[W];
                    float v[16];
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const float4 w = *reinterpret_cast<const float4*>(s_ws + 16 * c + j);
                        const float4 b = *reinterpret_cast<const float4*>(s_ws + HN + 16 * c + j);
                        const float4 t = scaled(r + j, x, w, b);
                        v[j] = t.x, v[j + 1] = t.y, v[j + 2] = t.z, v[j + 3] = t.w;
                    }
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        if constexpr (sizeof(Elem) == 2)
                            o[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
                        else
                            o[j] = __float_as_uint(v[j]);
                    void* ob = which == 0 ? a.out[0] : which == 1 ? a.out[1] : which == 2 ? a.out[2] : a.out[3];
                    Elem* to = static_cast<Elem*>(ob) + row * width + at;
                    const int row_bytes = width * static_cast<int>(sizeof(Elem));
                    if (col + 16 <= N && !(row_bytes & 15)) {
                        if (row >= M) {
                        } else if (!((row_bytes | reinterpret_cast<uintptr_t>(ob)) & 31)) {
#pragma unroll
                            for (int j = 0; j < W; j += 8) st_32bytes(reinterpret_cast<uint32_t*>(to) + j, o + j);
                        } else {
#pragma unroll
                            for (int j = 0; j < W; j += 4)
                                *reinterpret_cast<uint4*>(reinterpret_cast<uint32_t*>(to) + j) = make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                        }
                    } else {
                        // rows of any alignment, or the last columns: 16 lanes to a row
                        float* s_f = reinterpret_cast<float*>(s_out);
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            *reinterpret_cast<float4*>(s_f + 16 * lane + 4 * (j ^ ((lane >> 1) & 3))) =
                                make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                        __syncwarp();
                        const int j = lane & 15;
                        Elem* base = to + (static_cast<long long>(lane >> 4) - lane) * width + j;
#pragma unroll 4
                        for (int i = 0; i < 16; ++i) {
                            const int rr = 2 * i + (lane >> 4);
                            if (row0 + rr < M && col + j < N)
                                put(base + 2LL * i * width, s_f[16 * rr + 4 * ((j >> 2) ^ (i & 3)) + (j & 3)]);
                        }
                    }
                    if ((at += 16) == width && !g) {
                        at = 0;
                        ++which;
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR)
                    mbar_arrive_cluster_relaxed(bar_acc_free + 8 * buf, 0);   // nothing but the accumulators passes on
                else
                    mbar_arrive(bar_acc_free + 8 * buf);
            }
        }
        if (SP::tma_out && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");   // every store has been made
    }
    grid_dep_trigger();
    tc_fence_before();
    if constexpr (PAIR)
        cluster_sync();
    else
        __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        if constexpr (PAIR)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(SP::cols));
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(SP::cols));
    }
    if (tid == 0 && *s_abort) atomicOr(a.status, kErrTimeout);
}

// A few rows (one to eight tokens): every weight byte is used once per row, so the weights' bytes
// are the cost.  One warp per output channel, 16 bytes per lane and step, integer dot products.
constexpr int kI8FewRows = 8;

template <int MR, typename Elem>
__global__ void __launch_bounds__(256) linear_i8_few_kernel(const I8Problem p, Elem* __restrict__ out, int K)
{
    grid_dep_wait();
    const int n = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (n < p.N) {
        int acc[MR];
#pragma unroll
        for (int m = 0; m < MR; ++m) acc[m] = 0;
        const int8_t* w = p.w + static_cast<long long>(n) * K;
        for (int k = 16 * lane; k < K; k += 512) {
            const int4 b = __ldg(reinterpret_cast<const int4*>(w + k));
#pragma unroll
            for (int m = 0; m < MR; ++m) {
                if (m < p.M) {
                    const int4 x = __ldg(reinterpret_cast<const int4*>(p.x + static_cast<long long>(m) * K + k));
                    acc[m] = __dp4a(b.x, x.x, __dp4a(b.y, x.y, __dp4a(b.z, x.z, __dp4a(b.w, x.w, acc[m]))));
                }
            }
        }
#pragma unroll
        for (int m = 0; m < MR; ++m)
#pragma unroll
            for (int o = 16; o; o >>= 1) acc[m] += __shfl_xor_sync(0xffffffffu, acc[m], o);
        const float ws = __ldg(p.ws + n);
        const float bias = p.bias ? bias_at(static_cast<const Elem*>(p.bias), n) : 0.f;
#pragma unroll
        for (int m = 0; m < MR; ++m)
            if (lane == m && m < p.M)
                put(out + static_cast<long long>(m) * p.N + n,
                    __fadd_rn(__fmul_rn(__fmul_rn(static_cast<float>(acc[m]), __ldg(p.xs + m)), ws), bias));
    }
    grid_dep_trigger();
}

// Some rows (nine to some dozens): a warp takes 16 rows and four output channels, its lanes every 32nd 16 bytes
// of K, integer dot products; KS warps share the K of the same outputs.  A K step of the tensor-core kernel costs
// 0.28 us whatever its tile holds, which is what these shapes would wait for: 16 x 512 x 4096 takes 8.1 us here and
// 20.9 there, 9 x 512 x 2048 3.6 and 11.9, 64 x 512 x 2048 5.7 and 12.0 (K over 512 with KS = 1: 26.8, 9.2, 14.4).
constexpr int kI8SomeRows = 16, kI8SomeCols = 4;

template <int KS, typename Elem>
__global__ void __launch_bounds__(128) linear_i8_some_kernel(const I8Problem p, Elem* __restrict__ out, int K)
{
    grid_dep_wait();
    constexpr int MR = kI8SomeRows, NC = kI8SomeCols, G = 4 / KS;   // groups of KS warps in the block
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n0 = (blockIdx.x * G + warp / KS) * NC, m0 = blockIdx.y * MR;
    int acc[MR * NC];
#pragma unroll
    for (int i = 0; i < MR * NC; ++i) acc[i] = 0;
    const int8_t* w[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) w[c] = p.w + static_cast<long long>(min(n0 + c, p.N - 1)) * K;   // surplus: not stored
    for (int k = 16 * (lane + 32 * (warp % KS)); k < K; k += 512 * KS) {
        int4 b[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) b[c] = __ldg(reinterpret_cast<const int4*>(w[c] + k));
        const int8_t* x = p.x + static_cast<long long>(m0) * K + k;
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            if (m0 + m < p.M) {
                const int4 a = __ldg(reinterpret_cast<const int4*>(x + static_cast<long long>(m) * K));
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    acc[m * NC + c] = __dp4a(b[c].x, a.x, __dp4a(b[c].y, a.y, __dp4a(b[c].z, a.z, __dp4a(b[c].w, a.w, acc[m * NC + c]))));
            }
        }
    }
    // sums over the lanes, half of the values handed on at each step: lane L ends with values 2 L and 2 L + 1
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < 2 * o; ++i) {
            const int give = up ? acc[i] : acc[i + 2 * o], keep = up ? acc[i + 2 * o] : acc[i];
            acc[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
    if constexpr (KS > 1) {
        __shared__ int s_sum[4][MR * NC];
        s_sum[warp][2 * lane] = acc[0];
        s_sum[warp][2 * lane + 1] = acc[1];
        __syncthreads();
        if (warp % KS == 0)
#pragma unroll
            for (int j = 1; j < KS; ++j) {
                acc[0] += s_sum[warp + j][2 * lane];
                acc[1] += s_sum[warp + j][2 * lane + 1];
            }
    }
    if (warp % KS == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int m = m0 + (2 * lane + e) / NC, n = n0 + (2 * lane + e) % NC;
            if (m < p.M && n < p.N) {
                const float bias = p.bias ? bias_at(static_cast<const Elem*>(p.bias), n) : 0.f;
                put(out + static_cast<long long>(m) * p.N + n,
                    __fadd_rn(__fmul_rn(__fmul_rn(static_cast<float>(acc[e]), __ldg(p.xs + m)), __ldg(p.ws + n)), bias));
            }
        }
    }
    grid_dep_trigger();
}

// --------------------------------------------------------------------------- host

int g_smem_done_i8[8][64];

template <int BN, bool PAIR, typename Elem>
oasr_status launch_i8(I8Args a, int slot, int sms, cudaStream_t stream)
{
    using SP = I8Smem<BN, PAIR>;
    constexpr int MT = PAIR ? 256 : 128;
    auto tiles_of = [](const I8Problem& p) { return static_cast<long long>((p.M + MT - 1LL) / MT) * ((p.N + BN - 1) / BN); };
    const long long t0 = tiles_of(a.p[0]), t1 = a.p[1].M ? tiles_of(a.p[1]) : 0;
    if (t0 + t1 > 0x7fffffffLL - sms) return OASR_ERR_UNSUPPORTED;
    a.nt0 = (a.p[0].N + BN - 1) / BN;
    a.nt1 = a.p[1].M ? (a.p[1].N + BN - 1) / BN : 1;
    a.tiles0 = static_cast<int>(t0);
    a.tiles = static_cast<int>(t0 + t1);
    auto kern = linear_i8_kernel<BN, PAIR, Elem>;
    if (!ensure_smem(kern, SP::bytes, g_smem_done_i8[slot])) return OASR_ERR_CUDA;
    CUtensorMap tm[4];
    for (int g = 0; g < 2; ++g) {
        const I8Problem& p = a.p[a.p[1].M ? g : 0];   // one problem: its maps stand in for the other's
        if (!encode_bytes(&tm[2 * g], p.x, p.M, a.K, 128) || !encode_bytes(&tm[2 * g + 1], p.w, p.N, a.K, SP::b_rows))
            return OASR_ERR_INVALID_ARG;
    }
    I8Outs outs = {};
    for (int o = 0; SP::tma_out && o < 4; ++o) {
        if (!a.out[o]) continue;
        const I8Problem& p = a.p[o == 3];
        const long long bytes = (o == 3 ? p.N : a.width) * static_cast<long long>(sizeof(Elem));
        a.by_tma = bytes % 16 == 0 && bytes <= 0x7fffffffLL;
        if (!a.by_tma) break;
        if (!encode_bytes(&outs.m[o], a.out[o], p.M, static_cast<int>(bytes), 32, true)) return OASR_ERR_INVALID_ARG;
    }
    if constexpr (PAIR)
        return launch_pdl_cluster(kern, dim3(2 * (a.tiles < sms / 2 ? a.tiles : sms / 2)), dim3(kI8Threads), SP::bytes, 2, stream,
                                  tm[0], tm[1], tm[2], tm[3], outs, static_cast<const I8Args>(a));
    else
        return launch_pdl(kern, dim3(a.tiles < sms ? a.tiles : sms), dim3(kI8Threads), SP::bytes, stream, tm[0], tm[1], tm[2],
                          tm[3], outs, static_cast<const I8Args>(a));
}

template <typename Elem>
oasr_status some_rows(const I8Problem& p, void* out, int K, cudaStream_t stream)
{
    const unsigned groups = (p.N + kI8SomeCols - 1) / kI8SomeCols, rows = (p.M + kI8SomeRows - 1) / kI8SomeRows;
    if (K > 512)
        return launch_pdl(linear_i8_some_kernel<4, Elem>, dim3(groups, rows), dim3(128), 0, stream, p, static_cast<Elem*>(out), K);
    return launch_pdl(linear_i8_some_kernel<1, Elem>, dim3((groups + 3) / 4, rows), dim3(128), 0, stream, p,
                      static_cast<Elem*>(out), K);
}

// Tile: the one of the least estimated time.  Measured per K step of 64 (ns, by the slope over K): 375 for a
// pair's 256 x 256, 315 for 128 x 128, 285 and 275 for 128 x 64 and 128 x 32, where the steps' latency is the cost;
// a tile's epilogue takes 2400, 1300, 600 and 400, half of which the next tile's products hide.  8191 x 4096 x 1024
// in fp32: 57 us in pairs, 87 in 128 x 128; 1024 x 768 x 256 in bf16: 7.0 in pairs, 5.2, 4.5 in 128 x 64 and 5.5 in
// 128 x 32.  256 x 128 in pairs and 128 x 256 without were nowhere the fastest.
template <typename Elem>
oasr_status dispatch_i8(const I8Args& a, cudaStream_t stream)
{
    const int sms = sm_count();
    if (!sms || !a.status) return OASR_ERR_CUDA;
    constexpr struct { int m, n, ctas, step, epilogue; } kinds[] = {
        {256, 256, 2, 375, 2400}, {128, 128, 1, 315, 1300}, {128, 64, 1, 285, 600}, {128, 32, 1, 275, 400}};
    int best = 0;
    long long least = 0x7fffffffffffffffLL;
    for (int k = 0; k < 4; ++k) {
        const auto& t = kinds[k];
        long long tiles = 0;
        for (const I8Problem& p : a.p)
            if (p.M) tiles += ((p.M + t.m - 1LL) / t.m) * ((p.N + t.n - 1) / t.n);
        const long long waves = (tiles * t.ctas + sms - 1) / sms, steps = static_cast<long long>((a.K + 63) / 64) * t.step;
        const long long wave = steps > t.epilogue / 2 ? steps + t.epilogue / 2 : t.epilogue;
        if (waves * wave + t.epilogue < least) {
            least = waves * wave + t.epilogue;
            best = k;
        }
    }
    // the integer kernel: blocks of 16 x 4 outputs (16 x 16 up to K = 512), four of them on an SM at a time, each
    // 0.5 us and 2.0 for every round of its K.  Over 128 rows its reads of x pass the caches: 256 x 512 x 2048 takes
    // 17.9 us there, 12.0 here
    if (!a.p[1].M && a.p[0].M <= 128) {
        const long long split = a.K > 512 ? 4 : 1, blocks = ((a.p[0].M + 15) / 16) * ((a.p[0].N + 16 / split - 1) / (16 / split));
        const long long round = 500 + 2000 * ((a.K + 512 * split - 1) / (512 * split)), full = 4LL * sms;
        if ((blocks > full ? round * blocks / full : round) < least) return some_rows<Elem>(a.p[0], a.out[0], a.K, stream);
    }
    constexpr int s = sizeof(Elem) == 4 ? 4 : 0;
    if (best == 0) return launch_i8<256, true, Elem>(a, s, sms, stream);
    if (best == 1) return launch_i8<128, false, Elem>(a, s + 1, sms, stream);
    if (best == 2) return launch_i8<64, false, Elem>(a, s + 2, sms, stream);
    return launch_i8<32, false, Elem>(a, s + 3, sms, stream);
}

template <typename Elem>
oasr_status few_rows(const I8Problem& p, void* out, int K, cudaStream_t stream)
{
    const dim3 grid((p.N + 7) / 8);
    auto go = [&](auto kern) { return launch_pdl(kern, grid, dim3(256), 0, stream, p, static_cast<Elem*>(out), K); };
    if (p.M == 1) return go(linear_i8_few_kernel<1, Elem>);
    if (p.M <= 4) return go(linear_i8_few_kernel<4, Elem>);
    return go(linear_i8_few_kernel<kI8FewRows, Elem>);
}

constexpr int kI8MaxK = 65536;   // integer sums of K products of at most 2^14 stay below 2^31
constexpr int kI8MaxRows = 0x7fffff00;   // the rows and columns of whole tiles are 32-bit numbers

}  // namespace
}  // namespace oasr

extern "C" oasr_status oasr_quantize_rows(const void* x, void* x8, float* scale, int M, int K, oasr_dtype dt,
                                          cudaStream_t stream)
{
    using namespace oasr;
    if (!x || !x8 || !scale || M <= 0 || K <= 0) return OASR_ERR_INVALID_ARG;
    if ((dt != OASR_F32 && dt != OASR_BF16) || K % 16) return OASR_ERR_UNSUPPORTED;
    if (!aligned16(x) || !aligned16(x8) || !aligned16(scale)) return OASR_ERR_INVALID_ARG;
    // a warp per row while its values fit the warp's registers, a block per longer row
    auto go = [&](auto* src, auto kern, int rows_per_block) {
        return launch_pdl(kern, dim3((static_cast<unsigned>(M) + rows_per_block - 1) / rows_per_block), dim3(256), 0, stream,
                          src, static_cast<int8_t*>(x8), scale, M, K);
    };
    auto by_length = [&](auto* src) {
        using E = std::remove_const_t<std::remove_pointer_t<decltype(src)>>;
        if (K <= 256) return go(src, quantize_rows_kernel<E, 32, 1>, 8);
        if (K <= 512) return go(src, quantize_rows_kernel<E, 32, 2>, 8);
        if (K <= 1024) return go(src, quantize_rows_kernel<E, 32, 4>, 8);
        if (K <= 8192) return go(src, quantize_rows_kernel<E, 256, 4>, 1);
        return go(src, quantize_rows_kernel<E, 256, 0>, 1);
    };
    return dt == OASR_F32 ? by_length(static_cast<const float*>(x)) : by_length(static_cast<const __nv_bfloat16*>(x));
}

extern "C" oasr_status oasr_linear_w8a8(const void* x8, const float* x_scale, const void* w8, const float* w_scale,
                                        const void* bias, void* out, int M, int N, int K, oasr_dtype dt,
                                        cudaStream_t stream)
{
    using namespace oasr;
    if (!x8 || !x_scale || !w8 || !w_scale || !out || M <= 0 || N <= 0 || K <= 0) return OASR_ERR_INVALID_ARG;
    if ((dt != OASR_F32 && dt != OASR_BF16) || K % 16 || K > kI8MaxK || M > kI8MaxRows || N > kI8MaxRows)
        return OASR_ERR_UNSUPPORTED;
    const void* ptrs[] = {x8, x_scale, w8, w_scale, bias ? bias : x8, out};
    for (const void* p : ptrs)
        if (!aligned16(p)) return OASR_ERR_INVALID_ARG;
    I8Args a = {};
    a.p[0] = {static_cast<const int8_t*>(x8), static_cast<const int8_t*>(w8), x_scale, w_scale, bias, M, N};
    a.out[0] = out;
    a.width = N;
    a.K = K;
    a.status = status_word();
    if (M <= kI8FewRows)
        return dt == OASR_F32 ? few_rows<float>(a.p[0], out, K, stream) : few_rows<__nv_bfloat16>(a.p[0], out, K, stream);
    return dt == OASR_F32 ? dispatch_i8<float>(a, stream) : dispatch_i8<__nv_bfloat16>(a, stream);
}

extern "C" oasr_status oasr_project_qkv_pos_w8a8(const void* x8, const float* x_scale, const void* w_qkv8,
                                                 const float* w_qkv_scale, const void* b_qkv, const void* pos8,
                                                 const float* pos_scale, const void* w_pos8,
                                                 const float* w_pos_scale, void* q, void* k, void* v, void* rel,
                                                 int M, int R, int d_model, int H, oasr_dtype dt,
                                                 cudaStream_t stream)
{
    using namespace oasr;
    const void* ptrs[] = {x8, x_scale, w_qkv8, w_qkv_scale, b_qkv, pos8, pos_scale, w_pos8, w_pos_scale, q, k, v, rel};
    for (const void* p : ptrs)
        if (!p || !aligned16(p)) return OASR_ERR_INVALID_ARG;
    if (M <= 0 || R <= 0 || d_model <= 0 || H <= 0) return OASR_ERR_INVALID_ARG;
    if ((dt != OASR_F32 && dt != OASR_BF16) || d_model % kHeadDim || d_model / kHeadDim != H || d_model > kI8MaxK / 4 ||
        M > kI8MaxRows || R > kI8MaxRows)
        return OASR_ERR_UNSUPPORTED;
    I8Args a = {};
    a.p[0] = {static_cast<const int8_t*>(x8), static_cast<const int8_t*>(w_qkv8), x_scale, w_qkv_scale, b_qkv, M,
              3 * d_model};
    a.p[1] = {static_cast<const int8_t*>(pos8), static_cast<const int8_t*>(w_pos8), pos_scale, w_pos_scale, nullptr, R,
              d_model};
    a.out[0] = q;
    a.out[1] = k;
    a.out[2] = v;
    a.out[3] = rel;
    a.width = d_model;
    a.K = d_model;
    a.status = status_word();
    return dt == OASR_F32 ? dispatch_i8<float>(a, stream) : dispatch_i8<__nv_bfloat16>(a, stream);
}
