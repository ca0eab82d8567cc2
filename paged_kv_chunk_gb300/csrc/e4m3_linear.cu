// 8-bit floating-point products with a scale for each block of 128:
//
//   oasr_quantize_blocks  e = max(-100, least e with max|x_block| <= 448 2^e), x8 = e4m3(x 2^-e), byte e + 127
//   oasr_linear_e4m3      out[i][n] = sum_b 2^(ex[i][b] + ew[n][b]) sum_{k in b} x8[i][k] w8[n][k] + bias[n]
//
// A block is 128 neighbouring values of a row, of activations and weights alike; the last of a row may be
// shorter.  The format is the 8-bit cache's (e4m3.cuh) with 128 values to a scale.
#include <type_traits>

#include "e4m3.cuh"
#include "host_common.h"

namespace oasr {
namespace {

constexpr int kBlk = 128;   // values that share a scale

// ------------------------------------------------------------------ rows to 8 bits

// Sixteen lanes to a block, eight values each.
template <typename Elem>
__global__ void __launch_bounds__(256) quantize_blocks_kernel(const Elem* __restrict__ x, uint8_t* __restrict__ x8,
                                                              uint8_t* __restrict__ scale, int M, int K, int kb)
{
    grid_dep_wait();
    const int l = threadIdx.x & 15;
    const long long blocks = static_cast<long long>(M) * kb, stride = static_cast<long long>(gridDim.x) * 16;
    for (long long i = static_cast<long long>(blockIdx.x) * 16 + (threadIdx.x >> 4); i < blocks; i += stride) {
        const long long row = i / kb;
        const int b = static_cast<int>(i - row * kb), k = b * kBlk + 8 * l;
        float v[8] = {};
        if (k < K) load8(x + row * K + k, v);
        uint32_t most = 0;   // the bits of magnitudes order as the values do, NaN above infinity
#pragma unroll
        for (int e = 0; e < 8; ++e) most = max(most, __float_as_uint(v[e]) & 0x7fffffffu);
        const unsigned mask = 0xffffu << (threadIdx.x & 16);
#pragma unroll
        for (int o = 8; o; o >>= 1) most = max(most, __shfl_xor_sync(mask, most, o));
        uint32_t byte = kE4NanScale;
        uint2 q = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
        if (most < 0x7f800000u) {
            byte = e4m3_scale_byte(__uint_as_float(most));
            const float f = e4m3_scale_inverse(byte);
            q.x = e4m3_pack2(v[0] * f, v[1] * f) | (e4m3_pack2(v[2] * f, v[3] * f) << 16);
            q.y = e4m3_pack2(v[4] * f, v[5] * f) | (e4m3_pack2(v[6] * f, v[7] * f) << 16);
        }
        if (k < K) *reinterpret_cast<uint2*>(x8 + row * K + k) = q;
        if (l == 0) scale[i] = static_cast<uint8_t>(byte);
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

__device__ __forceinline__ float bias_at(const float* b, int n) { return __ldg(b + n); }
__device__ __forceinline__ float bias_at(const __nv_bfloat16* b, int n) { return __bfloat162float(b[n]); }
__device__ __forceinline__ void put(float* o, float v) { *o = v; }
__device__ __forceinline__ void put(__nv_bfloat16* o, float v) { *o = __float2bfloat16_rn(v); }

__device__ __forceinline__ void unpack16(const uint4& w, float (&v)[16])
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = e4m3_unpack2(u[i] & 0xffffu), b = e4m3_unpack2(u[i] >> 16);
        v[4 * i] = a.x, v[4 * i + 1] = a.y, v[4 * i + 2] = b.x, v[4 * i + 3] = b.y;
    }
}

// A few rows (one to eight tokens): every weight byte is used once per row.  One warp per output channel, 16
// values per lane and step (within one block), products in fp32 (exact) and their sums too.
constexpr int kE4FewRows = 8;

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
                    acc[m] += s * e4m3_scale(__ldg(p.xs + row * p.kb + b)) * ws;
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

// --------------------------------------------------------------------------- host

constexpr int kE4MaxRows = 0x7fffff00, kE4MaxK = 65536;

template <typename Elem>
oasr_status dispatch_e4(const E4Problem& p, void* out, cudaStream_t stream)
{
    const long long groups = (p.M + kE4FewRows - 1LL) / kE4FewRows;
    if (groups > 65535) return OASR_ERR_UNSUPPORTED;
    const dim3 grid((p.N + 7) / 8, static_cast<unsigned>(groups));
    if (p.M == 1) return launch_pdl(linear_e4m3_few_kernel<1, Elem>, grid, dim3(256), 0, stream, p, static_cast<Elem*>(out));
    return launch_pdl(linear_e4m3_few_kernel<kE4FewRows, Elem>, grid, dim3(256), 0, stream, p, static_cast<Elem*>(out));
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
    const int sms = sm_count(), kb = (K + kBlk - 1) / kBlk;
    if (!sms) return OASR_ERR_CUDA;
    const long long ctas = (static_cast<long long>(M) * kb + 15) / 16, most = 8LL * sms;
    const dim3 grid(static_cast<unsigned>(ctas < most ? ctas : most));
    auto go = [&](auto* src) {
        using E = std::remove_const_t<std::remove_pointer_t<decltype(src)>>;
        return launch_pdl(quantize_blocks_kernel<E>, grid, dim3(256), 0, stream, src, static_cast<uint8_t*>(x8),
                          static_cast<uint8_t*>(scale), M, K, kb);
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
