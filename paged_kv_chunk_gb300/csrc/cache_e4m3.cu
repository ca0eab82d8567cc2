// oasr_paged_append_e4m3 and oasr_paged_read_e4m3: the chunk's K/V rows quantised into the
// 8-bit pools, and cached rows read back dense (format: e4m3.cuh).
//
// The 8-bit pools are [num_blocks][H][block_size][64] and the scales [num_blocks][H][K, V][block_size]:
// one head's rows of a page are one contiguous run (1 KB for 16 frames), and so are its scales
// (32 bytes), because an attention program reads one head of a stream.
//
// Both calls move a row's 64 + 1 bytes on the 8-bit side and 128 (bf16) or 256 (fp32) on the other: 64 streams'
// 1024 positions of 8 heads are read to bf16 in 34.7 us (0.86 of the measured copy rate), chunks of 64 frames of
// 256 streams and 8 heads written in 11.1 (0.67, launch and tail included).
#include <type_traits>

#include "e4m3.cuh"
#include "host_common.h"

namespace oasr {
namespace {

// Page of position p (below 2^31) and its place there: a shift where block_size is a power of two (shift
// >= 0), else a 32-bit division (64-bit ones took half of the append's time).
__device__ __forceinline__ int page_of(int p, int block_size, int shift, int& slot)
{
    const int lb = shift >= 0 ? p >> shift : static_cast<int>(static_cast<unsigned>(p) / static_cast<unsigned>(block_size));
    slot = p - lb * block_size;
    return lb;
}

// Sixteen values of a row as they come, and the largest magnitude's fp32 bits among them: the bits order as the
// values do, with NaN above infinity.
struct Raw16Bf16 {
    uint4 w[2];
    __device__ __forceinline__ void load(const __nv_bfloat16* p)
    {
        w[0] = __ldg(reinterpret_cast<const uint4*>(p));
        w[1] = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    }
    __device__ __forceinline__ uint32_t largest(unsigned mask) const   // of the row: in all of its four lanes
    {
        constexpr uint32_t A = 0x7fff7fffu;
        uint32_t m = __vimax3_u16x2(w[0].x & A, w[0].y & A, w[0].z & A);
        m = __vimax3_u16x2(m, w[0].w & A, w[1].x & A);
        m = __vimax3_u16x2(m, w[1].y & A, w[1].z & A);
        m = __vmaxu2(m, w[1].w & A);
        m = __vmaxu2(m, __shfl_xor_sync(mask, m, 1));
        m = __vmaxu2(m, __shfl_xor_sync(mask, m, 2));
        return max(m << 16, m & 0xffff0000u);
    }
    __device__ __forceinline__ float2 pair(int i) const
    {
        const uint4& v = w[i >> 2];
        const uint32_t b = (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
        return make_float2(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u));
    }
};

struct Raw16F32 {
    uint4 w[4];
    __device__ __forceinline__ void load(const float* p)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ uint32_t largest(unsigned mask) const
    {
        constexpr uint32_t A = 0x7fffffffu;
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m = __vimax3_u32(m, w[i].x & A, w[i].y & A);
            m = __vimax3_u32(m, w[i].z & A, w[i].w & A);
        }
        m = max(m, __shfl_xor_sync(mask, m, 1));
        return max(m, __shfl_xor_sync(mask, m, 2));
    }
    __device__ __forceinline__ float2 pair(int i) const
    {
        const uint4& v = w[i >> 1];
        return i & 1 ? make_float2(__uint_as_float(v.z), __uint_as_float(v.w)) : make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
    }
};

template <typename Elem>
using Raw16 = std::conditional_t<sizeof(Elem) == 2, Raw16Bf16, Raw16F32>;

// As e4m3_quantise8, the row in four neighbouring lanes with sixteen values each.
template <typename Raw>
__device__ __forceinline__ uint32_t e4m3_quantise16(const Raw& x, unsigned mask, uint4& q)
{
    const uint32_t amax = x.largest(mask);
    if (amax >= 0x7f800000u) {
        q = make_uint4(0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);
        return kE4NanScale;
    }
    const uint32_t byte = e4m3_scale_byte(__uint_as_float(amax));
    const float s = e4m3_scale_inverse(byte);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = __fmul2_rn(x.pair(2 * i), make_float2(s, s)), b = __fmul2_rn(x.pair(2 * i + 1), make_float2(s, s));
        o[i] = __byte_perm(e4m3_pack2(a.x, a.y), e4m3_pack2(b.x, b.y), 0x5410);
    }
    q = make_uint4(o[0], o[1], o[2], o[3]);
    return byte;
}

// Four lanes per row; rows of one stream in the order (K or V, head, frame), so neighbouring groups write
// neighbouring rows and scale bytes of a page.  Eight lanes a row took twice the instructions a row, which bounded
// it: 13.3 us for 262144 bf16 rows, 11.1 with four; two and four rows a thread 11.5 and 12.0.
// grid: blocks_per_stream blocks of 64 rows for each stream; over_T: floor(2^32 / T), or 2^32 - 1 for T = 1.
template <typename Elem>
__global__ void __launch_bounds__(256) append_e4m3_kernel(
    const Elem* __restrict__ k_new, const Elem* __restrict__ v_new, uint8_t* __restrict__ k_pool,
    uint8_t* __restrict__ v_pool, uint8_t* __restrict__ kv_scale, int num_blocks, int block_size, int shift,
    const int32_t* __restrict__ block_table, int mbps, const int32_t* __restrict__ cache_seqlens,
    int T, int H, uint32_t over_T, int blocks_per_stream, unsigned* status)
{
    grid_dep_wait();     // the previous grid on the stream has finished (programmatic launch)
    const int b = blockIdx.x / blocks_per_stream;
    const int r0 = (blockIdx.x - b * blocks_per_stream) * 64 + (threadIdx.x >> 2);
    const int l4 = threadIdx.x & 3, rows = 2 * H * T;
    const uint32_t r = min(r0, rows - 1);    // surplus groups redo the last row and store nothing
    uint32_t rh = __umulhi(r, over_T), rt = r - rh * T;   // r / T, or one less
    if (rt >= static_cast<uint32_t>(T)) {
        ++rh;
        rt -= T;
    }
    const int t = rt, kv = static_cast<int>(rh) >= H, h = rh - (kv ? H : 0);
    Raw16<Elem> x;
    x.load((kv ? v_new : k_new) + (static_cast<long long>(b) * T * H + (t * H + h)) * kE4Row + 16 * l4);   // T H < 2^29
    const int C = __ldg(cache_seqlens + b);
    unsigned err = 0;
    uint4 q;
    const uint32_t byte = e4m3_quantise16(x, 0xffffffffu, q);
    if (r0 < rows) {
        const int p = static_cast<int>(static_cast<unsigned>(C) + t);   // negative when it passes 2^31 too
        int slot, blk = -1;
        const int lb = page_of(p, block_size, shift, slot);
        if (p >= 0 && lb < mbps) blk = __ldg(block_table + static_cast<long long>(b) * mbps + lb);
        if (blk < 0 || blk >= num_blocks) {
            err = kErrBounds;
        } else {
            const long long page = static_cast<long long>(blk) * H + h;
            *reinterpret_cast<uint4*>((kv ? v_pool : k_pool) + (page * block_size + slot) * kE4Row + 16 * l4) = q;
            if (l4 == 0) kv_scale[(2 * page + kv) * block_size + slot] = static_cast<uint8_t>(byte);
        }
    }
    grid_dep_trigger();
    if (err && l4 == 0) atomicOr(status, err);
}

__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&x)[16])
{
    uint4* d = reinterpret_cast<uint4*>(p);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        d[i] = make_uint4(pack_bf16(x[8 * i], x[8 * i + 1]), pack_bf16(x[8 * i + 2], x[8 * i + 3]),
                          pack_bf16(x[8 * i + 4], x[8 * i + 5]), pack_bf16(x[8 * i + 6], x[8 * i + 7]));
}

__device__ __forceinline__ void store16(float* p, const float (&x)[16])
{
    float4* d = reinterpret_cast<float4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}

// Four lanes per row (16 bytes of e4m3 each), K and V of the row together; rows of a stream in
// the order (head, position), so a warp reads 512 contiguous bytes of a page.  Positions the
// stream does not hold give zeros.
template <typename Elem>
__global__ void __launch_bounds__(256) read_e4m3_kernel(
    const uint8_t* __restrict__ k_pool, const uint8_t* __restrict__ v_pool,
    const uint8_t* __restrict__ kv_scale, int num_blocks, int block_size, int shift,
    const int32_t* __restrict__ block_table, int mbps, const int32_t* __restrict__ cache_seqlens,
    const int32_t* __restrict__ start, Elem* __restrict__ k, Elem* __restrict__ v, int L, int H,
    int blocks_per_stream, unsigned* status)
{
    grid_dep_wait();
    const int b = blockIdx.x / blocks_per_stream;
    const int r = (blockIdx.x - b * blocks_per_stream) * 64 + (threadIdx.x >> 2);
    const int l4 = threadIdx.x & 3;
    unsigned err = 0;
    if (r < H * L) {
        const int h = r / L, i = r - h * L;
        const int len = __ldg(cache_seqlens + b);
        const long long p = (start ? static_cast<long long>(__ldg(start + b)) : 0) + i;
        uint4 q[2] = {};
        float s[2] = {0.f, 0.f};
        if (p < 0 || len < 0) {
            err = kErrBounds;
        } else if (p < len) {
            int slot;                       // p < len <= 2^31 - 1
            const int lb = page_of(static_cast<int>(p), block_size, shift, slot);
            const int blk = lb < mbps ? __ldg(block_table + static_cast<long long>(b) * mbps + lb) : -1;
            if (blk < 0 || blk >= num_blocks) {
                err = kErrBounds;
            } else {
                const long long page = static_cast<long long>(blk) * H + h;
                const long long row = (page * block_size + slot) * kE4Row + 16 * l4;
                q[0] = __ldg(reinterpret_cast<const uint4*>(k_pool + row));
                q[1] = __ldg(reinterpret_cast<const uint4*>(v_pool + row));
                s[0] = e4m3_scale(__ldg(kv_scale + 2 * page * block_size + slot));
                s[1] = e4m3_scale(__ldg(kv_scale + (2 * page + 1) * block_size + slot));
            }
        }
        const long long dst = ((static_cast<long long>(b) * L + i) * H + h) * kE4Row + 16 * l4;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const uint32_t w[4] = {q[kv].x, q[kv].y, q[kv].z, q[kv].w};
            float x[16];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 lo = e4m3_unpack2(w[e]), hi = e4m3_unpack2(w[e] >> 16);
                x[4 * e] = lo.x * s[kv];
                x[4 * e + 1] = lo.y * s[kv];
                x[4 * e + 2] = hi.x * s[kv];
                x[4 * e + 3] = hi.y * s[kv];
            }
            store16((kv ? v : k) + dst, x);
        }
    }
    grid_dep_trigger();
    if (err && l4 == 0) atomicOr(status, err);
}

// log2 of a power of two, else -1
int shift_of(int block_size) { return block_size & (block_size - 1) ? -1 : __builtin_ctz(static_cast<unsigned>(block_size)); }

}  // namespace
}  // namespace oasr

extern "C" oasr_status oasr_paged_append_e4m3(const void* k_new, const void* v_new, void* k_pool,
                                              void* v_pool, void* kv_scale, int num_blocks,
                                              int block_size, const int32_t* block_table,
                                              int max_blocks_per_seq, const int32_t* cache_seqlens,
                                              int B, int T, int H, int D, oasr_dtype dt,
                                              cudaStream_t stream)
{
    using namespace oasr;
    if (!k_new || !v_new || !k_pool || !v_pool || !kv_scale || !block_table || !cache_seqlens)
        return OASR_ERR_INVALID_ARG;
    if (num_blocks <= 0 || block_size <= 0 || max_blocks_per_seq <= 0 || B <= 0 || T <= 0 ||
        H <= 0 || D <= 0)
        return OASR_ERR_INVALID_ARG;
    if ((dt != OASR_F32 && dt != OASR_BF16) || D != kE4Row) return OASR_ERR_UNSUPPORTED;
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pool) || !aligned16(v_pool) ||
        !aligned16(kv_scale))
        return OASR_ERR_INVALID_ARG;
    const long long rows = 2LL * H * T;
    const long long per_stream = (rows + 63) / 64;
    if (rows > 0x3fffffffLL || per_stream * B > 0x7fffffffLL) return OASR_ERR_UNSUPPORTED;
    unsigned* status = status_word();
    if (!status) return OASR_ERR_CUDA;
    const uint32_t over_T = T == 1 ? 0xffffffffu : static_cast<uint32_t>((1ull << 32) / T);
    auto go = [&](auto* kn, auto* vn, auto kern) {
        return launch_pdl(kern, dim3(static_cast<unsigned>(per_stream * B)), dim3(256), 0, stream, kn, vn,
                          static_cast<uint8_t*>(k_pool), static_cast<uint8_t*>(v_pool),
                          static_cast<uint8_t*>(kv_scale), num_blocks, block_size, shift_of(block_size), block_table,
                          max_blocks_per_seq, cache_seqlens, T, H, over_T, static_cast<int>(per_stream), status);
    };
    if (dt == OASR_F32)
        return go(static_cast<const float*>(k_new), static_cast<const float*>(v_new), append_e4m3_kernel<float>);
    return go(static_cast<const __nv_bfloat16*>(k_new), static_cast<const __nv_bfloat16*>(v_new),
              append_e4m3_kernel<__nv_bfloat16>);
}

extern "C" oasr_status oasr_paged_read_e4m3(const void* k_pool, const void* v_pool,
                                            const void* kv_scale, int num_blocks, int block_size,
                                            const int32_t* block_table, int max_blocks_per_seq,
                                            const int32_t* cache_seqlens, const int32_t* start,
                                            void* k, void* v, int B, int L, int H, int D,
                                            oasr_dtype dt, cudaStream_t stream)
{
    using namespace oasr;
    if (!k_pool || !v_pool || !kv_scale || !block_table || !cache_seqlens || !k || !v)
        return OASR_ERR_INVALID_ARG;
    if (num_blocks <= 0 || block_size <= 0 || max_blocks_per_seq <= 0 || B <= 0 || L <= 0 ||
        H <= 0 || D <= 0)
        return OASR_ERR_INVALID_ARG;
    if ((dt != OASR_F32 && dt != OASR_BF16) || D != kE4Row) return OASR_ERR_UNSUPPORTED;
    if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned16(kv_scale) || !aligned16(k) || !aligned16(v))
        return OASR_ERR_INVALID_ARG;
    const long long rows = static_cast<long long>(H) * L;
    const long long per_stream = (rows + 63) / 64;
    if (rows > 0x3fffffffLL || per_stream * B > 0x7fffffffLL) return OASR_ERR_UNSUPPORTED;
    unsigned* status = status_word();
    if (!status) return OASR_ERR_CUDA;
    auto go = [&](auto* kd, auto* vd, auto kern) {
        return launch_pdl(kern, dim3(static_cast<unsigned>(per_stream * B)), dim3(256), 0, stream,
                          static_cast<const uint8_t*>(k_pool), static_cast<const uint8_t*>(v_pool),
                          static_cast<const uint8_t*>(kv_scale), num_blocks, block_size, shift_of(block_size), block_table,
                          max_blocks_per_seq, cache_seqlens, start, kd, vd, L, H,
                          static_cast<int>(per_stream), status);
    };
    if (dt == OASR_F32) return go(static_cast<float*>(k), static_cast<float*>(v), read_e4m3_kernel<float>);
    return go(static_cast<__nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(v), read_e4m3_kernel<__nv_bfloat16>);
}
