// oasr_paged_append_e4m3 and oasr_paged_read_e4m3: the chunk's K/V rows quantised into the
// 8-bit pools, and cached rows read back dense (format: e4m3.cuh).
//
// The 8-bit pools are [num_blocks][H][block_size][64] and the scales [num_blocks][H][K, V][block_size]:
// one head's rows of a page are one contiguous run (1 KB for 16 frames), and so are its scales
// (32 bytes), because an attention program reads one head of a stream.
//
// Both calls are bound by HBM: a row costs 64 + 1 bytes on the 8-bit side and 128 (bf16) or 256
// (fp32) on the other, against some 60 instructions per 4 rows.
#include "e4m3.cuh"
#include "host_common.h"

namespace oasr {
namespace {

constexpr int kRowsPerGroup = 2;   // rows of one 8-lane group, loaded before either is reduced (1, 4, 8: slower)

// Page of position p (below 2^31) and its place there: a shift where block_size is a power of two (shift
// >= 0), else a 32-bit division (64-bit ones took half of the append's time).
__device__ __forceinline__ int page_of(int p, int block_size, int shift, int& slot)
{
    const int lb = shift >= 0 ? p >> shift : static_cast<int>(static_cast<unsigned>(p) / static_cast<unsigned>(block_size));
    slot = p - lb * block_size;
    return lb;
}

// Eight lanes per row, four rows per warp and step; rows of one stream in the order (K or V,
// head, frame), so neighbouring groups write neighbouring rows and scale bytes of a page.
// grid: blocks_per_stream blocks of 64 rows for each stream.
template <typename Elem>
__global__ void __launch_bounds__(256) append_e4m3_kernel(
    const Elem* __restrict__ k_new, const Elem* __restrict__ v_new, uint8_t* __restrict__ k_pool,
    uint8_t* __restrict__ v_pool, uint8_t* __restrict__ kv_scale, int num_blocks, int block_size, int shift,
    const int32_t* __restrict__ block_table, int mbps, const int32_t* __restrict__ cache_seqlens,
    int T, int H, int blocks_per_stream, unsigned* status)
{
    grid_dep_wait();     // the previous grid on the stream has finished (programmatic launch)
    const int b = blockIdx.x / blocks_per_stream;
    const int r0 = (blockIdx.x - b * blocks_per_stream) * (32 * kRowsPerGroup) +
                   (threadIdx.x >> 5) * (4 * kRowsPerGroup) + ((threadIdx.x & 31) >> 3);
    const int l8 = threadIdx.x & 7, rows = 2 * H * T;
    unsigned err = 0;
    float x[kRowsPerGroup][8];
    int kv[kRowsPerGroup], h[kRowsPerGroup], t[kRowsPerGroup];
#pragma unroll
    for (int u = 0; u < kRowsPerGroup; ++u) {
        const int r = min(r0 + 4 * u, rows - 1);    // surplus groups redo the last row and store nothing
        const int rh = r / T;
        t[u] = r - rh * T;
        kv[u] = rh >= H;
        h[u] = rh - (kv[u] ? H : 0);
        load8((kv[u] ? v_new : k_new) + ((static_cast<long long>(b) * T + t[u]) * H + h[u]) * kE4Row + 8 * l8, x[u]);
    }
    const int C = __ldg(cache_seqlens + b);
#pragma unroll
    for (int u = 0; u < kRowsPerGroup; ++u) {
        uint2 q;
        const uint32_t byte = e4m3_quantise8(x[u], 0xffffffffu, q);
        if (r0 + 4 * u < rows) {
            const int p = static_cast<int>(static_cast<unsigned>(C) + t[u]);   // negative when it passes 2^31 too
            int slot, blk = -1;
            const int lb = page_of(p, block_size, shift, slot);
            if (p >= 0 && lb < mbps) blk = __ldg(block_table + static_cast<long long>(b) * mbps + lb);
            if (blk < 0 || blk >= num_blocks) {
                err = kErrBounds;
            } else {
                const long long page = static_cast<long long>(blk) * H + h[u];
                *reinterpret_cast<uint2*>((kv[u] ? v_pool : k_pool) + (page * block_size + slot) * kE4Row + 8 * l8) = q;
                if (l8 == 0) kv_scale[(2 * page + kv[u]) * block_size + slot] = static_cast<uint8_t>(byte);
            }
        }
    }
    grid_dep_trigger();
    if (err && l8 == 0) atomicOr(status, err);
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
    const long long per_stream = (rows + 32 * kRowsPerGroup - 1) / (32 * kRowsPerGroup);
    if (rows > 0x3fffffffLL || per_stream * B > 0x7fffffffLL) return OASR_ERR_UNSUPPORTED;
    unsigned* status = status_word();
    if (!status) return OASR_ERR_CUDA;
    auto go = [&](auto* kn, auto* vn, auto kern) {
        return launch_pdl(kern, dim3(static_cast<unsigned>(per_stream * B)), dim3(256), 0, stream, kn, vn,
                          static_cast<uint8_t*>(k_pool), static_cast<uint8_t*>(v_pool),
                          static_cast<uint8_t*>(kv_scale), num_blocks, block_size, shift_of(block_size), block_table,
                          max_blocks_per_seq, cache_seqlens, T, H, static_cast<int>(per_stream), status);
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
