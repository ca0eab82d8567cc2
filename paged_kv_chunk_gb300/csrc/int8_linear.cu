// 8-bit integer products with a scale per token and per output channel:
//
//   oasr_quantize_rows         m = max(max|x_row|, 2^-100), x8 = rint(x (127 (1 / m))), scale = m / 127
//   oasr_linear_w8a8           out[i][n] = (sum_k x8[i][k] w8[n][k]) x_scale[i] w_scale[n] + bias[n]
//   oasr_project_qkv_pos_w8a8  the same for a step's q, k, v and its position table, in one launch
//
// This GPU's tensor cores have next to no 8-bit integer rate, but an 8-bit integer is exact in fp16
// and a product of two exact in fp32, so the sums run on tcgen05's fp16 rate: converter warps
// read the 8-bit rows and write them as fp16 into the swizzled tiles the matrix instructions
// read.  A sum stays below 2^24 for K <= 1024, where fp32 holds every integer: the accumulated
// sum is the integer sum.  For longer K it is that of an fp32 accumulation.
#include "attn_core.cuh"
#include "e4m3.cuh"
#include "host_common.h"
#include "tcgen05.cuh"

namespace oasr {
namespace {

// ------------------------------------------------------------------ rows to 8 bits

constexpr float kLeastMax = 7.8886090522101181e-31f;   // 2^-100
constexpr int kKeep = 4;   // chunks of eight values a thread keeps between its two passes

// TPR threads per row; each takes every TPR-th chunk of eight values.
template <typename Elem, int TPR>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const Elem* __restrict__ x, int8_t* __restrict__ x8,
                                                            float* __restrict__ scale, int M, int K)
{
    grid_dep_wait();
    const int row = blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
    const int l = threadIdx.x % TPR, chunks = K / 8;
    const bool on = row < M;
    const Elem* src = x + static_cast<long long>(on ? row : 0) * K;
    float keep[kKeep][8];
    float m = 0.f;
    for (int i = 0, c = l; c < chunks; ++i, c += TPR) {
        float v[8];
        load8(src + 8 * c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fabsf(v[e]) < INFINITY ? fmaxf(m, fabsf(v[e])) : INFINITY;
#pragma unroll
        for (int k = 0; k < kKeep; ++k)
            if (k == i)
#pragma unroll
                for (int e = 0; e < 8; ++e) keep[k][e] = v[e];
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
    const float f = bad ? 0.f : __fmul_rn(__frcp_rn(m), 127.f);
    if (on) {
        if (l == 0) scale[row] = bad ? NAN : __fdiv_rn(m, 127.f);
        int8_t* dst = x8 + static_cast<long long>(row) * K;
        for (int i = 0, c = l; c < chunks; ++i, c += TPR) {
            float v[8];
            bool kept = false;
#pragma unroll
            for (int k = 0; k < kKeep; ++k)
                if (k == i) {
                    kept = true;
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = keep[k][e];
                }
            if (!kept) load8(src + 8 * c, v);
            uint32_t w[2] = {0u, 0u};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int q = bad ? 0 : __float2int_rn(__fmul_rn(v[e], f));
                w[e >> 2] |= (static_cast<uint32_t>(q) & 255u) << (8 * (e & 3));
            }
            *reinterpret_cast<uint2*>(dst + 8 * c) = make_uint2(w[0], w[1]);
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
    unsigned* status;
};

__device__ __forceinline__ float bias_at(const float* b, int n) { return __ldg(b + n); }
__device__ __forceinline__ float bias_at(const __nv_bfloat16* b, int n) { return __bfloat162float(b[n]); }
__device__ __forceinline__ void put(float* o, float v) { *o = v; }
__device__ __forceinline__ void put(__nv_bfloat16* o, float v) { *o = __float2bfloat16_rn(v); }

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

constexpr int kI8Threads = 13 * 32;   // four epilogue warps, the issuer, eight converter warps
constexpr int kI8Conv = 256;

template <int BN>
struct I8Smem {
    static constexpr int tile_a = 128 * 128, tile = tile_a + BN * 128;   // fp16, 64 of K
    static constexpr int stages = BN == 128 ? 6 : 8;
    static constexpr int off_ws = stages * tile;             // [4 warps][2 * BN] floats
    static constexpr int off_bar = off_ws + 4 * 2 * BN * 4;  // full, empty, acc full[2], acc free[2], drain
    static constexpr int off_misc = off_bar + (2 * stages + 5) * 8;
    static constexpr int bytes = off_misc + 16 + 1024;
    static constexpr int cols = 2 * BN < 32 ? 32 : 2 * BN;
};

template <int BN, typename Elem>
__global__ void __launch_bounds__(kI8Threads, 1) linear_i8_kernel(const I8Args a)
{
    using SP = I8Smem<BN>;
    constexpr int S = SP::stages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_addr(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(sm + SP::off_misc);
    volatile int* s_abort = reinterpret_cast<volatile int*>(sm + SP::off_misc + 4);
    const uint32_t bar_full = sb + SP::off_bar, bar_empty = bar_full + 8 * S;
    const uint32_t bar_acc_full = bar_empty + 8 * S, bar_acc_free = bar_acc_full + 16;
    const uint32_t bar_drain = bar_acc_free + 16;
    const int ksteps = (a.K + 63) / 64;
    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(bar_full + 8 * i, kI8Conv);
            mbar_init(bar_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_acc_full + 8 * i, 1);
            mbar_init(bar_acc_free + 8 * i, 4);
        }
        mbar_init(bar_drain, 1);
        fence_mbar_init();
        *s_abort = 0;
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(s_tmem)),
                     "r"(SP::cols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
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
    const int my_tiles = static_cast<int>(blockIdx.x) < a.tiles ? (a.tiles - 1 - blockIdx.x) / gridDim.x + 1 : 0;

    if (warp >= 5) {
        // ------------------------------------------------------------ converters
        // thread: 16 bytes (chunk c) of rows r0, r0 + 64, ... of the tile's x rows, then its w rows
        constexpr int NU = (128 + BN + 63) / 64;
        const int ct = tid - 160, c = ct & 3, r0 = ct >> 2;
        const int iters = my_tiles * ksteps;
        int lt = -1, lk = ksteps;           // the next step to load: tile, K step
        const int8_t* src[NU];
        auto load = [&](uint4 (&buf)[NU]) {
            if (++lk >= ksteps) {
                lk = 0;
                ++lt;
                int g, mt, nt;
                decode(blockIdx.x + lt * gridDim.x, g, mt, nt);
                const I8Problem& p = a.p[g];
#pragma unroll
                for (int u = 0; u < NU; ++u) {
                    const int r = r0 + 64 * u;
                    src[u] = nullptr;
                    if (r < 128) {
                        if (mt * 128 + r < p.M) src[u] = p.x + static_cast<long long>(mt * 128 + r) * a.K + 16 * c;
                    } else if (r < 128 + BN) {
                        const int n = nt * BN + r - 128;
                        if (n < p.N) src[u] = p.w + static_cast<long long>(n) * a.K + 16 * c;
                    }
                }
            }
            const bool in = 64 * lk + 16 * c < a.K;
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                buf[u] = make_uint4(0u, 0u, 0u, 0u);
                if (in && src[u]) buf[u] = __ldg(reinterpret_cast<const uint4*>(src[u] + 64 * lk));
            }
        };
        auto convert = [&](int i, const uint4 (&buf)[NU]) {
            const int slot = i % S;
            if (i >= S && !wait_or_abort(bar_empty + 8 * slot, ((i / S) - 1) & 1, s_abort)) return false;
            uint8_t* base = sm + slot * SP::tile;
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                const int r = r0 + 64 * u;      // w rows follow the x rows: 128 bytes each
                if (r < 128 + BN) {
                    *reinterpret_cast<uint4*>(base + swz128(r, 2 * c)) = i8_to_f16(buf[u].x, buf[u].y);
                    *reinterpret_cast<uint4*>(base + swz128(r, 2 * c + 1)) = i8_to_f16(buf[u].z, buf[u].w);
                }
            }
            fence_proxy_async_smem();
            mbar_arrive_release(bar_full + 8 * slot);
            return true;
        };
        uint4 b0[NU], b1[NU];
        if (iters > 0) load(b0);
        if (iters > 1) load(b1);
        for (int i = 0; i < iters; i += 2) {
            if (!convert(i, b0)) break;
            if (i + 2 < iters) load(b0);
            if (i + 1 < iters) {
                if (!convert(i + 1, b1)) break;
                if (i + 3 < iters) load(b1);
            }
        }
    } else if (warp == 4) {
        // ------------------------------------------------------------- MMA issuer
        if (lane == 0) {
            // fp16 A and B, fp32 D
            constexpr uint32_t id = (1u << 4) | (static_cast<uint32_t>(BN >> 3) << 17) | ((128u >> 4) << 24);
            int i = 0, nacc = 0, nfree = 0;
            bool ok = true;
            for (int lt = 0; lt < my_tiles && ok; ++lt) {
                const int buf = lt & 1;
                if (lt >= 2 && !wait_or_abort(bar_acc_free + 8 * buf, ((lt >> 1) - 1) & 1, s_abort)) break;
                for (int kb = 0; kb < ksteps; ++kb, ++i) {
                    const int slot = i % S;
                    if (!wait_or_abort(bar_full + 8 * slot, (i / S) & 1, s_abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t base = sb + slot * SP::tile;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_ss(tmem + buf * BN, sdesc(base + 32 * k), sdesc(base + SP::tile_a + 32 * k), id,
                                (kb > 0 || k > 0) ? 1 : 0);
                    umma_commit(bar_empty + 8 * slot);
                    ++nfree;
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
            for (int u = nfree - S; u < nfree; ++u)
                if (u >= 0) drained = mbar_wait(bar_empty + 8 * (u % S), (u / S) & 1) && drained;
            if (!drained) *s_abort = 1;
        }
    } else {
        // --------------------------------------------------------------- epilogue
        const uint32_t tl = tmem + (static_cast<uint32_t>(32 * warp) << 16);
        float* s_ws = reinterpret_cast<float*>(sm + SP::off_ws) + warp * 2 * BN;   // w scales, then biases
        for (int lt = 0; lt < my_tiles; ++lt) {
            int g, mt, nt;
            decode(blockIdx.x + lt * gridDim.x, g, mt, nt);
            const I8Problem& p = a.p[g];
            const int buf = lt & 1;
            const Elem* bias = static_cast<const Elem*>(p.bias);
            __syncwarp();
            for (int j = lane; j < BN; j += 32) {
                const int n = nt * BN + j;
                s_ws[j] = n < p.N ? __ldg(p.ws + n) : 0.f;
                s_ws[BN + j] = bias && n < p.N ? bias_at(bias, n) : 0.f;
            }
            const int row = mt * 128 + 32 * warp + lane;
            const float xs = row < p.M ? __ldg(p.xs + row) : 0.f;
            __syncwarp();
            if (!__all_sync(0xffffffffu, wait_or_abort(bar_acc_full + 8 * buf, (lt >> 1) & 1, s_abort))) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < BN / 32; ++c) {
                uint32_t r[32];
                OASR_TMEM_LD32(tl + buf * BN + 32 * c, r);
                tmem_wait_ld();
                const int col = nt * BN + 32 * c;
                if (row < p.M && col < p.N) {
                    // a block of 32 columns lies within one output (widths are multiples of 64,
                    // or there is one output)
                    const int which = g ? 3 : col / a.width;
                    const int width = g ? p.N : a.width;
                    void* ob = which == 0 ? a.out[0] : which == 1 ? a.out[1] : which == 2 ? a.out[2] : a.out[3];
                    Elem* dst = static_cast<Elem*>(ob) + static_cast<long long>(row) * width + (col - (g ? 0 : which * a.width));
                    float v[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        v[j] = __fadd_rn(__fmul_rn(__fmul_rn(__uint_as_float(r[j]), xs), s_ws[32 * c + j]), s_ws[BN + 32 * c + j]);
                    if (col + 32 <= p.N && (width & 7) == 0) {
                        if constexpr (sizeof(Elem) == 2) {
#pragma unroll
                            for (int j = 0; j < 32; j += 8)
                                *reinterpret_cast<uint4*>(dst + j) =
                                    make_uint4(pack_bf16(v[j], v[j + 1]), pack_bf16(v[j + 2], v[j + 3]),
                                               pack_bf16(v[j + 4], v[j + 5]), pack_bf16(v[j + 6], v[j + 7]));
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; j += 4)
                                *reinterpret_cast<float4*>(dst + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (col + j < p.N) put(dst + j, v[j]);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_acc_free + 8 * buf);
        }
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

// --------------------------------------------------------------------------- host

int g_smem_done_i8[6][64];

template <int BN, typename Elem>
oasr_status launch_i8(I8Args a, int slot, int sms, cudaStream_t stream)
{
    auto tiles_of = [](const I8Problem& p) { return static_cast<long long>((p.M + 127LL) / 128) * ((p.N + BN - 1) / BN); };
    const long long t0 = tiles_of(a.p[0]), t1 = a.p[1].M ? tiles_of(a.p[1]) : 0;
    if (t0 + t1 > 0x7fffffffLL - sms) return OASR_ERR_UNSUPPORTED;
    a.nt0 = (a.p[0].N + BN - 1) / BN;
    a.nt1 = a.p[1].M ? (a.p[1].N + BN - 1) / BN : 1;
    a.tiles0 = static_cast<int>(t0);
    a.tiles = static_cast<int>(t0 + t1);
    auto kern = linear_i8_kernel<BN, Elem>;
    if (!ensure_smem(kern, I8Smem<BN>::bytes, g_smem_done_i8[slot])) return OASR_ERR_CUDA;
    return launch_pdl(kern, dim3(a.tiles < sms ? a.tiles : sms), dim3(kI8Threads), I8Smem<BN>::bytes, stream,
                      static_cast<const I8Args>(a));
}

// The widest of 128, 64 and 32 columns whose tiles cover the SMs.
template <typename Elem>
oasr_status dispatch_i8(const I8Args& a, cudaStream_t stream)
{
    const int sms = sm_count();
    if (!sms || !a.status) return OASR_ERR_CUDA;
    auto tiles = [&](int bn) {
        long long n = 0;
        for (const I8Problem& p : a.p)
            if (p.M) n += ((p.M + 127LL) / 128) * ((p.N + bn - 1) / bn);
        return n;
    };
    constexpr int s = sizeof(Elem) == 4 ? 3 : 0;
    if (tiles(128) >= sms) return launch_i8<128, Elem>(a, s, sms, stream);
    if (tiles(64) >= sms) return launch_i8<64, Elem>(a, s + 1, sms, stream);
    return launch_i8<32, Elem>(a, s + 2, sms, stream);
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

}  // namespace
}  // namespace oasr

extern "C" oasr_status oasr_quantize_rows(const void* x, void* x8, float* scale, int M, int K, oasr_dtype dt,
                                          cudaStream_t stream)
{
    using namespace oasr;
    if (!x || !x8 || !scale || M <= 0 || K <= 0) return OASR_ERR_INVALID_ARG;
    if ((dt != OASR_F32 && dt != OASR_BF16) || K % 16) return OASR_ERR_UNSUPPORTED;
    if (!aligned16(x) || !aligned16(x8) || !aligned16(scale)) return OASR_ERR_INVALID_ARG;
    auto go = [&](auto* src, auto warp_kern, auto block_kern) {
        // a warp per row keeps up to 1024 values in registers; longer rows take a block each
        const bool warp = K <= 32 * 8 * kKeep;
        const unsigned grid = warp ? (static_cast<unsigned>(M) + 7) / 8 : static_cast<unsigned>(M);
        return launch_pdl(warp ? warp_kern : block_kern, dim3(grid), dim3(256), 0, stream, src,
                          static_cast<int8_t*>(x8), scale, M, K);
    };
    if (dt == OASR_F32)
        return go(static_cast<const float*>(x), quantize_rows_kernel<float, 32>, quantize_rows_kernel<float, 256>);
    return go(static_cast<const __nv_bfloat16*>(x), quantize_rows_kernel<__nv_bfloat16, 32>,
              quantize_rows_kernel<__nv_bfloat16, 256>);
}

extern "C" oasr_status oasr_linear_w8a8(const void* x8, const float* x_scale, const void* w8, const float* w_scale,
                                        const void* bias, void* out, int M, int N, int K, oasr_dtype dt,
                                        cudaStream_t stream)
{
    using namespace oasr;
    if (!x8 || !x_scale || !w8 || !w_scale || !out || M <= 0 || N <= 0 || K <= 0) return OASR_ERR_INVALID_ARG;
    if ((dt != OASR_F32 && dt != OASR_BF16) || K % 16 || K > kI8MaxK) return OASR_ERR_UNSUPPORTED;
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
    if ((dt != OASR_F32 && dt != OASR_BF16) || d_model % kHeadDim || d_model / kHeadDim != H || d_model > kI8MaxK / 4)
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
