// oasr_block_table_update and oasr_paged_append_slots: pages for requests of any lengths, taken and
// given back on the device, and rows of those requests into the pools by the slots they were given.
//
// A stream that grows from C to N rows needs pages ceil(C / bs) .. ceil(N / bs) - 1; they come from a
// ring of free block ids in the streams' order, so each stream's first place in the ring is a prefix sum
// over the streams before it.  Every CTA adds up all streams' lengths (8 bytes each, from L2) for its own
// prefix and the totals: one launch and no wait between CTAs, where a scan of its own would be another
// launch.  The ring is what keeps the CTAs apart: pages are taken at its head and given back behind its
// tail, so no CTA writes what another one still reads, and the last CTA to finish moves both ends.
//
// An entry given back may name no block: -1 where an earlier call was short and left the stream without the page, or took
// it back already.  Such entries must not enter the ring, and which places the ones behind them get is then known only once
// every entry has been read.  The places above count every entry; where one turns out to name none, the last CTA to finish
// closes the gaps, and where there are more entries than places (so some must name none), it alone does the taking back.
#include "host_common.h"
#include "ptx.cuh"

namespace oasr {
namespace {

constexpr int kTabThreads = 256, kTabMaxStreams = 4096;
constexpr int kTabItems = 8;              // entries a thread sorts out at a time
constexpr unsigned kTabGap = 1u << 16;    // in the count of finished CTAs (at most 1024): one that found such an entry

// What a stream's change of length asks for.
struct Change {
    int C, N, P0, P1;
    bool bad;
    __device__ __forceinline__ Change(int c, int n, int cap, int bs)
    {
        C = min(max(c, 0), cap);
        N = min(max(n, 0), cap);
        bad = C != c || N != n;
        P0 = (C + bs - 1) / bs;
        P1 = (N + bs - 1) / bs;
    }
    __device__ __forceinline__ int need() const { return max(P1 - P0, 0); }
    __device__ __forceinline__ int give() const { return max(P0 - P1, 0); }
    __device__ __forceinline__ int rows() const { return max(N - C, 0); }
};

struct TableArgs {
    int32_t* table;
    const int32_t *lens, *news;
    int B, mbps, bs;
    int32_t* ring;
    int nb;
    int32_t* state;   // head, count, short, CTAs that have finished (and kTabGap for each that found gaps)
    int32_t* slots;
    int total;
    int32_t* cu;
    unsigned* status;
};

// STREAMS to a CTA: one, so that a stream's slots have 256 threads, while the CTAs' sums over all streams cost less
// than that gains (256 streams of up to 1500 new rows: 4.8 us against 7.7 with four, 512 6.8 and 8.6, of up to 16 new rows
// 5.2 and 4.8), else four (1024 streams of up to 1500: 9.3 us against 10.2 with one).
template <int STREAMS>
__global__ void __launch_bounds__(kTabThreads) block_table_kernel(const TableArgs a)
{
    constexpr int kTabGroup = kTabThreads / STREAMS;   // threads of a stream
    grid_dep_wait();     // the previous grid on the stream has finished (programmatic launch)
    grid_dep_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b0 = blockIdx.x * STREAMS, cap = a.mbps * a.bs;
    unsigned err = 0;

    // pages and rows of all streams, and of those before this CTA's
    int need = 0, give = 0, need0 = 0, give0 = 0;
    unsigned long long rows = 0, rows0 = 0;
    for (int b = tid; b < a.B; b += kTabThreads) {
        const Change c(__ldg(a.lens + b), __ldg(a.news + b), cap, a.bs);
        need += c.need();
        give += c.give();
        rows += c.rows();
        if (b < b0) {
            need0 += c.need();
            give0 += c.give();
            rows0 += c.rows();
        }
    }
    __shared__ int s_sum[4][kTabThreads / 32];
    __shared__ unsigned long long s_rows[2][kTabThreads / 32];
    need = __reduce_add_sync(0xffffffffu, need);
    give = __reduce_add_sync(0xffffffffu, give);
    need0 = __reduce_add_sync(0xffffffffu, need0);
    give0 = __reduce_add_sync(0xffffffffu, give0);
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        rows += __shfl_xor_sync(0xffffffffu, rows, o);
        rows0 += __shfl_xor_sync(0xffffffffu, rows0, o);
    }
    if (lane == 0) {
        s_sum[0][warp] = need, s_sum[1][warp] = give, s_sum[2][warp] = need0, s_sum[3][warp] = give0;
        s_rows[0][warp] = rows, s_rows[1][warp] = rows0;
    }
    __syncthreads();
    need = give = need0 = give0 = 0;
    rows = rows0 = 0;
#pragma unroll
    for (int w = 0; w < kTabThreads / 32; ++w) {
        need += s_sum[0][w], give += s_sum[1][w], need0 += s_sum[2][w], give0 += s_sum[3][w];
        rows += s_rows[0][w], rows0 += s_rows[1][w];
    }

    // a state that no call of the library has left: nothing is handed out or taken back, and it stays as it is
    int head = a.state[0], count = a.state[1];
    const bool sane = head >= 0 && head < a.nb && count >= 0 && count <= a.nb;
    if (!sane) {
        err = kErrBounds;
        head = count = 0;
        give = 0;
    }
    const int room = a.nb - count;
    const unsigned tail = static_cast<unsigned>(head) + count;
    const bool granted = need <= count;
    auto place = [&](unsigned i) { return i >= static_cast<unsigned>(a.nb) ? i - a.nb : i; };   // i < 2 nb

    auto names_block = [&](int id) { return id >= 0 && id < a.nb; };
    int gaps = 0;
    const int b = b0 + tid / kTabGroup, t0 = tid % kTabGroup;
    if (b < a.B) {
        for (int i = b0; i < b; ++i) {
            const Change c(__ldg(a.lens + i), __ldg(a.news + i), cap, a.bs);
            need0 += c.need();
            give0 += c.give();
            rows0 += c.rows();
        }
        const Change c(__ldg(a.lens + b), __ldg(a.news + b), cap, a.bs);
        if (c.bad) err = kErrBounds;
        int32_t* row = a.table + static_cast<long long>(b) * a.mbps;
        const unsigned from = static_cast<unsigned>(head) + need0;
        auto fresh = [&](int i) {   // the i-th page handed to this stream
            const int id = a.ring[place(from + i)];
            return names_block(id) ? id : -1;
        };
        if (granted)
            for (int i = t0; i < c.need(); i += kTabGroup) row[c.P0 + i] = fresh(i);
        for (int i = t0; sane && give <= room && i < c.give(); i += kTabGroup) {
            const int id = row[c.P1 + i];
            row[c.P1 + i] = -1;
            a.ring[place(tail + (give0 + i))] = names_block(id) ? id : -1;
            if (!names_block(id)) {
                gaps = 1;
                if (id != -1) err = kErrBounds;
            }
        }
        for (int t = t0; t < c.rows(); t += kTabGroup) {
            if (rows0 + t >= static_cast<unsigned long long>(a.total)) {
                err = kErrBounds;
                break;
            }
            int slot = -1;
            if (granted) {
                const int p = c.C + t, page = static_cast<unsigned>(p) / static_cast<unsigned>(a.bs);
                const int id = page < c.P0 ? row[page] : fresh(page - c.P0);
                if (names_block(id))
                    slot = id * a.bs + (p - page * a.bs);
                else
                    err = kErrBounds;
            }
            a.slots[rows0 + t] = slot;
        }
        if (t0 == 0) {
            a.cu[b] = static_cast<int32_t>(min(rows0, 0x7fffffffull));
            if (b == a.B - 1) a.cu[a.B] = static_cast<int32_t>(min(rows, 0x7fffffffull));
        }
    }
    // slots behind the last row
    for (unsigned long long i = rows + blockIdx.x * kTabThreads + tid; i < static_cast<unsigned long long>(a.total);
         i += static_cast<unsigned long long>(gridDim.x) * kTabThreads)
        a.slots[i] = -1;
    auto finish = [&](int back) {
        if (sane) {
            a.state[0] = static_cast<int32_t>(place(static_cast<unsigned>(head) + (granted ? need : 0)));
            a.state[1] = count - (granted ? need : 0) + back;
        }
        a.state[2] = granted ? 0 : need - count;
        a.state[3] = 0;
    };
    gaps = __syncthreads_or(gaps);   // and head and count have been read
    __shared__ bool s_sort;          // the last CTA to finish, and there are gaps
    if (tid == 0) {
        __threadfence();
        const unsigned seen = atomicAdd(reinterpret_cast<unsigned*>(a.state) + 3, gaps ? kTabGap + 1 : 1u) + (gaps ? kTabGap : 0u);
        const bool last = seen % kTabGap == gridDim.x - 1;
        s_sort = last && (seen >= kTabGap || give > room);
        if (s_sort)
            __threadfence();
        else if (last)
            finish(give);
    }
    __syncthreads();
    if (s_sort) {
        int back = 0;
        __shared__ int s_warp[kTabThreads / 32];
        // those of n entries that name a block go behind the ones before them, in their order
        auto take_back = [&](int n, auto&& entry) {
            for (unsigned i0 = 0; i0 < static_cast<unsigned>(n); i0 += kTabThreads * kTabItems) {
                const unsigned i = i0 + tid * kTabItems;
                int id[kTabItems], own = 0;
#pragma unroll
                for (int u = 0; u < kTabItems; ++u) {
                    id[u] = i + u < static_cast<unsigned>(n) ? entry(i + u) : -1;
                    own += names_block(id[u]);
                }
                int upto = own;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += v;
                }
                if (lane == 31) s_warp[warp] = upto;
                __syncthreads();   // every entry of this step has been read
                int at = back + upto - own;
#pragma unroll
                for (int w = 0; w < kTabThreads / 32; ++w) {
                    if (w < warp) at += s_warp[w];
                    back += s_warp[w];
                }
#pragma unroll
                for (int u = 0; u < kTabItems; ++u)
                    if (names_block(id[u])) {
                        if (at < room)
                            a.ring[place(tail + at)] = id[u];
                        else
                            err = kErrBounds;   // more pages come back than were ever out
                        ++at;
                    }
                __syncthreads();
            }
        };
        if (give <= room) {
            take_back(give, [&](unsigned i) { return __ldcg(a.ring + place(tail + i)); });
        } else {
            for (int i = 0; i < a.B; ++i) {
                const Change c(__ldg(a.lens + i), __ldg(a.news + i), cap, a.bs);
                int32_t* row = a.table + static_cast<long long>(i) * a.mbps + c.P1;
                take_back(c.give(), [&](unsigned p) {
                    const int id = row[p];
                    row[p] = -1;
                    if (id < -1 || id >= a.nb) err = kErrBounds;
                    return id;
                });
            }
        }
        if (tid == 0) finish(min(back, room));
    }
    if (err) atomicOr(a.status, err);
}

// A warp moves two rows of K and of V, every load of them ahead of the first store.
constexpr int kSlotRows = 2;

__global__ void __launch_bounds__(256) append_slots_kernel(const uint4* __restrict__ k_new, const uint4* __restrict__ v_new,
                                                           long long k_stride, long long v_stride,
                                                           uint4* __restrict__ k_pool, uint4* __restrict__ v_pool, int slots,
                                                           const int32_t* __restrict__ slot_map, int total, int row_vecs,
                                                           unsigned* status)
{
    grid_dep_wait();
    const int lane = threadIdx.x & 31;
    const int r0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * kSlotRows;
    int slot[kSlotRows];
    unsigned err = 0;
#pragma unroll
    for (int r = 0; r < kSlotRows; ++r) {
        slot[r] = r0 + r < total ? __ldg(slot_map + r0 + r) : -1;
        if (slot[r] < -1 || slot[r] >= slots) {
            err = kErrBounds;
            slot[r] = -1;
        }
    }
    for (int c0 = 0; c0 < row_vecs; c0 += 64) {
        uint4 k[kSlotRows][2], v[kSlotRows][2];
#pragma unroll
        for (int r = 0; r < kSlotRows; ++r)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int c = c0 + 32 * u + lane;
                if (slot[r] >= 0 && c < row_vecs) {
                    k[r][u] = __ldcs(k_new + (r0 + r) * k_stride + c);
                    v[r][u] = __ldcs(v_new + (r0 + r) * v_stride + c);
                }
            }
#pragma unroll
        for (int r = 0; r < kSlotRows; ++r)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int c = c0 + 32 * u + lane;
                if (slot[r] >= 0 && c < row_vecs) {
                    k_pool[static_cast<long long>(slot[r]) * row_vecs + c] = k[r][u];
                    v_pool[static_cast<long long>(slot[r]) * row_vecs + c] = v[r][u];
                }
            }
    }
    grid_dep_trigger();
    if (err && lane == 0) atomicOr(status, err);
}

}  // namespace
}  // namespace oasr

extern "C" oasr_status oasr_block_table_update(int32_t* block_table, const int32_t* cache_seqlens,
                                               const int32_t* new_seqlens, int B, int max_blocks_per_seq, int block_size,
                                               int32_t* free_blocks, int num_blocks, int32_t* free_state,
                                               int32_t* slot_map, int total, int32_t* cu_seqlens, cudaStream_t stream)
{
    using namespace oasr;
    if (!block_table || !cache_seqlens || !new_seqlens || !free_blocks || !free_state || !cu_seqlens ||
        (!slot_map && total > 0))
        return OASR_ERR_INVALID_ARG;
    if (B <= 0 || max_blocks_per_seq <= 0 || block_size <= 0 || num_blocks <= 0 || total < 0) return OASR_ERR_INVALID_ARG;
    constexpr long long kInt = 0x7fffffff;
    if (B > kTabMaxStreams || static_cast<long long>(B) * max_blocks_per_seq > kInt ||
        static_cast<long long>(max_blocks_per_seq) * block_size > kInt - kTabThreads - block_size ||   // loops step past it
        static_cast<long long>(num_blocks) * block_size > kInt)
        return OASR_ERR_UNSUPPORTED;
    const TableArgs a = {block_table, cache_seqlens, new_seqlens, B,     max_blocks_per_seq, block_size,   free_blocks,
                         num_blocks,  free_state,    slot_map,    total, cu_seqlens,         status_word()};
    if (!a.status) return OASR_ERR_CUDA;
    if (B <= 512) return launch_pdl(block_table_kernel<1>, dim3(B), dim3(kTabThreads), 0, stream, a);
    return launch_pdl(block_table_kernel<4>, dim3((B + 3) / 4), dim3(kTabThreads), 0, stream, a);
}

extern "C" oasr_status oasr_paged_append_slots(const void* k_new, const void* v_new, int64_t k_stride, int64_t v_stride,
                                               void* k_pool, void* v_pool, int num_blocks, int block_size,
                                               const int32_t* slot_map, int total, int H, int D, oasr_dtype dt,
                                               cudaStream_t stream)
{
    using namespace oasr;
    if (!k_new || !v_new || !k_pool || !v_pool || !slot_map) return OASR_ERR_INVALID_ARG;
    if (num_blocks <= 0 || block_size <= 0 || total <= 0 || H <= 0 || D <= 0) return OASR_ERR_INVALID_ARG;
    if (dt != OASR_F32 && dt != OASR_BF16) return OASR_ERR_UNSUPPORTED;
    const long long es = dt == OASR_F32 ? 4 : 2, row = static_cast<long long>(H) * D;
    if ((D * es) % 16 || row * es > 0x7fffffffLL || static_cast<long long>(num_blocks) * block_size > 0x7fffffffLL)
        return OASR_ERR_UNSUPPORTED;
    if (k_stride < row || v_stride < row || (k_stride * es) % 16 || (v_stride * es) % 16) return OASR_ERR_INVALID_ARG;
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pool) || !aligned16(v_pool)) return OASR_ERR_INVALID_ARG;
    unsigned* status = status_word();
    if (!status) return OASR_ERR_CUDA;
    const unsigned warps = (static_cast<unsigned>(total) + kSlotRows - 1) / kSlotRows;
    return launch_pdl(append_slots_kernel, dim3((warps + 7) / 8), dim3(256), 0, stream, static_cast<const uint4*>(k_new),
                      static_cast<const uint4*>(v_new), static_cast<long long>(k_stride * es / 16),
                      static_cast<long long>(v_stride * es / 16), static_cast<uint4*>(k_pool), static_cast<uint4*>(v_pool),
                      num_blocks * block_size, slot_map, total, static_cast<int>(row * es / 16), status);
}
