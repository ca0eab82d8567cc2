// Cross attention for many rows a sequence (whole transcripts, rescored hypotheses), bf16, on tcgen05.
//
// A CTA takes tiles of up to 128 rows (queries times the heads of a group, cross.cuh) against all keys of their
// sequence, 128 at a time:
//
//   S = Q . K^T    tcgen05, 128 x 128 in tensor memory
//   P = 2^(c S - m), m the row's running maximum, its sum in fp32      a softmax thread per row
//   O += P . V     tcgen05, P bf16 in tensor memory, O 128 x 64
//
// S, P and O have columns of their own (128 + 64 + 64 of 256), so the next stage's S is computed while this one's
// exponentials are, and two CTAs share an SM: one's softmax runs beside the other's products.  O is rescaled
// only when a row's maximum has grown by more than 2^8 (P then stays below 2^8, the same relative
// rounding).  P is rounded to bf16, as the product takes both operands in one type: 0.0022 of the result in rms against 64 bits,
// 0.0017 by the result's own rounding; its other half in bf16 would need 64 more columns, or a stage of 96 keys.  P . V stops at the 16 keys that hold the last one; V rows behind it within those are zeroed.
//
// The grid has a CTA for every tile; those that run take over the ones that have not started (cluster launch control), so
// that a tile's start-up (2.7 us of a CTA) passes while the one before it is worked on: 256 transcripts of 20 to
// 448 rows over up to 1500 states 225 -> 149 us.
//
// What bounds it: the chain of a stage (128 keys), about 1830 cycles of a CTA alone: S read 240, maxima 200, exponentials
// 820 (the exponential unit would need 512), the hand-overs between roles 110 to 400 each.  Two CTAs an SM take some 2500
// cycles each for one of theirs, so an SM finishes a stage every 1270.
// 304 sequences of 512 rows over 1280 keys, 8 heads: 428 us, 0.95 PFLOP/s, the tensor pipe 31 % active in the rescoring
// of 64 utterances (51.6 us).  Right and slower there: eight softmax warps (rows in halves, joined through shared memory, or
// four lanes to a row), 96 keys a stage with two P, issuers of their own for S and P . V (the registers then leave 128 a
// thread), rows written during the next tile's first stage, polling instead of suspended waits.
#include "cluster.cuh"
#include "cross.cuh"

namespace oasr {
namespace {

constexpr int kCRows = 128, kCKeys = 128, kCRowBytes = 128;
constexpr int kCSoftWarps = 4, kCProducer = kCSoftWarps, kCIssuer = kCSoftWarps + 1, kCThreads = 32 * (kCIssuer + 1);
constexpr int kCColS = 0, kCColP = 128, kCColO = 192, kCCols = 256;

// Out of line: the kernel's roles run different code at once, and instruction fetch stalls them otherwise.
__device__ __noinline__ bool c_wait_slow(uint32_t bar, uint32_t parity, volatile int* abort)
{
    return sleep_or_abort(bar, parity, abort);
}
__device__ __forceinline__ bool c_wait(uint32_t bar, uint32_t parity, volatile int* abort)
{
    return mbar_try_wait(bar, parity) || c_wait_slow(bar, parity, abort);
}

// A row tile of one sequence and key head, as the producer hands it to the other roles.
struct CItem {
    int q0, r0, live;   // the sequence's first query; the tile's first row and its rows (0: no more items)
    int h, nk;          // key head, keys
};
constexpr int kCItems = 4;   // handed over and not yet finished

// The grid counts row tiles of all sequences, one after the other, with their key heads: the producer finds a tile's
// sequence from the tiles before every kCIndex-th part of them.
constexpr int kCIndex = 1024;

struct CSmem {
    static constexpr int tile = kCKeys * kCRowBytes, ks = 3, vs = 2;
    static constexpr int off_q = 0, off_k = tile, off_v = off_k + ks * tile;
    static constexpr int off_bar = off_v + vs * tile;   // k full[3], empty[3], v full[2], empty[2], q full, q free, s full, s free, p full, pv done, drain
    static constexpr int off_item_bar = off_bar + (2 * ks + 2 * vs + 7) * 8;   // item full[4], free[4], the answer's
    static constexpr int off_next = (off_item_bar + (2 * kCItems + 1) * 8 + 15) / 16 * 16;
    static constexpr int off_item = off_next + 16;
    static constexpr int off_misc = off_item + kCItems * static_cast<int>(sizeof(CItem));
    static constexpr int off_index = off_misc + 16;
    static constexpr int bytes = off_index + kCIndex * 4 + 1024;
};

template <bool PAGED>
__global__ void __launch_bounds__(kCThreads, 2) cross_tc_kernel(const __grid_constant__ CUtensorMap tm_q,
                                                                const __grid_constant__ CUtensorMap tm_k,
                                                                const __grid_constant__ CUtensorMap tm_v, const CrossArgs a)
{
    using SP = CSmem;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_addr(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(sm + SP::off_misc);
    volatile int* s_abort = reinterpret_cast<volatile int*>(sm + SP::off_misc + 4);
    const uint32_t bar_k = sb + SP::off_bar, bar_k_free = bar_k + 8 * SP::ks;
    const uint32_t bar_v = bar_k_free + 8 * SP::ks, bar_v_free = bar_v + 8 * SP::vs;
    const uint32_t bar_q = bar_v_free + 8 * SP::vs, bar_q_free = bar_q + 8, bar_s = bar_q_free + 8, bar_s_free = bar_s + 8;
    const uint32_t bar_p = bar_s_free + 8, bar_pv = bar_p + 8, bar_drain = bar_pv + 8;
    const uint32_t bar_item = sb + SP::off_item_bar, bar_item_free = bar_item + 8 * kCItems, bar_next = bar_item_free + 8 * kCItems;
    volatile CItem* items = reinterpret_cast<volatile CItem*>(sm + SP::off_item);
    unsigned err = 0;
    if (tid == 0) {
        for (int i = 0; i < SP::ks; ++i) {
            mbar_init(bar_k + 8 * i, 1);
            mbar_init(bar_k_free + 8 * i, 1);
        }
        for (int i = 0; i < SP::vs; ++i) {
            mbar_init(bar_v + 8 * i, 1);
            mbar_init(bar_v_free + 8 * i, 1);
        }
        mbar_init(bar_q, 1);
        mbar_init(bar_q_free, 1);
        mbar_init(bar_s, 1);
        mbar_init(bar_s_free, kCSoftWarps);
        mbar_init(bar_p, kCSoftWarps);
        mbar_init(bar_pv, 1);
        mbar_init(bar_drain, 1);
        for (int i = 0; i < kCItems; ++i) {
            mbar_init(bar_item + 8 * i, 1);
            mbar_init(bar_item_free + 8 * i, kCSoftWarps + 1);
        }
        mbar_init(bar_next, 1);
        fence_mbar_init();
        *s_abort = 0;
    }
    if (warp == kCProducer && lane == 0) {
        prefetch_tensormap(&tm_q);
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
    }
    if (warp == kCIssuer) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(s_tmem)), "r"(kCCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    grid_dep_wait();

    const int qpt = kCRows / a.G, rpt = qpt * a.G;   // queries and rows of a tile

    if (warp == kCProducer) {
        // ------------------------------------------------------------ TMA producer
        // It takes the grid's work items one after the other, hands each to the other roles and requests its tiles: K two
        // stages ahead of V, whose slots are free only once their weights are through.
        // paged: lane i brings the i-th page of a stage (its part of one, for pages over 128)
        const int bs = min(a.bs, kCKeys), boxes = PAGED ? kCKeys / bs : 1;
        int g = 0, nv = 0, nq = 0, ni = 0;   // K stages, V stages, Q tiles requested; items handed over
        bool ok = true;
        auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, c_wait(bar, parity, s_abort)); };
        auto hand_over = [&](const CItem& it) {
            const int slot = ni % kCItems;
            if (ni >= kCItems && !wait(bar_item_free + 8 * slot, ((ni / kCItems) - 1) & 1)) return false;
            if (lane == 0) {
                items[slot].q0 = it.q0, items[slot].r0 = it.r0, items[slot].live = it.live, items[slot].h = it.h, items[slot].nk = it.nk;
                mbar_arrive_release(bar_item + 8 * slot);
            }
            ++ni;
            return true;
        };
        auto bring = [&](const CUtensorMap* tm, uint32_t dst, uint32_t bar, int h, int row) {
            const int n = __popc(__ballot_sync(0xffffffffu, row >= 0));
            if (lane == 0) mbar_arrive_expect_tx(bar, PAGED ? n * bs * kCRowBytes : SP::tile);
            __syncwarp();
            if (row >= 0) tma_load_3d(dst + lane * bs * kCRowBytes, tm, bar, 0, h, row);
        };
        if (lane == 0) ask_next(sb + SP::off_next, bar_next);
        int asked = 1;
        // tiles before sequence i * per
        int* index = reinterpret_cast<int*>(sm + SP::off_index);
        const int per = (a.N + kCIndex - 1) / kCIndex;
        auto tiles_of = [&](int s) {
            int q0 = __ldg(a.cu_q + s), q1 = __ldg(a.cu_q + s + 1);
            CrossSeq::clamp(q0, q1, a.total_q, err);
            return ((q1 - q0) * a.G + rpt - 1) / rpt;
        };
        constexpr long long kMost = 0x3fffffff;   // offsets that run wild may add up to more; they are flagged already
        long long all = 0;
        for (int i0 = 0; i0 * per < a.N; i0 += 32) {
            long long n = 0;
            for (int s = (i0 + lane) * per; s < min((i0 + lane + 1) * per, a.N); ++s) n += tiles_of(s);
            long long sum = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long v = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += v;
            }
            index[i0 + lane] = static_cast<int>(min(all + sum - n, kMost));
            all = min(all + __shfl_sync(0xffffffffu, sum, 31), kMost);
        }
        __syncwarp();
        struct Work {
            int s, h, tile;   // s < 0: past the last tile
            CrossSeq t;
        };
        auto look_up = [&](int x) {
            Work w = {-1, x % a.Hkv, x / a.Hkv, {}};
            if (w.tile >= all) return w;
            const int parts = (a.N + per - 1) / per;
            // the last part that begins at or before the tile
            int lo = 0;
            for (int step = kCIndex / 32; step; step >>= 5) {
                const int i = lo + step * lane;
                lo += step * (__popc(__ballot_sync(0xffffffffu, i < parts && index[min(i, parts - 1)] <= w.tile)) - 1);
            }
            w.tile -= index[lo];
            w.s = lo * per;
            if (per > 1)
                for (int n; w.tile >= (n = tiles_of(w.s)); ++w.s) w.tile -= n;
            w.t = CrossSeq(a, w.s, err);
            return w;
        };
        int x = blockIdx.x;
        Work w = look_up(x);
        while (ok) {
            const CrossSeq t = w.t;
            const int h = w.h, s = w.s, tile = w.tile;
            if (s >= 0) {
                const int rows = t.nq * a.G, stages = (t.nk + kCKeys - 1) / kCKeys;
                auto page_of = [&](int j0) {   // row of the lane's box; -1: past the last key
                    const int j = j0 + lane * bs;
                    if (!PAGED) return lane == 0 ? t.k0 + j0 : -1;
                    if (lane >= boxes || j >= t.nk) return -1;
                    const int r = cross_row<true>(a, t, s, j, err);
                    return r < 0 ? a.num_blocks * a.bs : r;   // outside the pools: comes as zeros
                };
                int krow = page_of(0), vrow = krow;
                if (!(ok = hand_over({t.q0, tile * rpt, min(rpt, rows - tile * rpt), h, t.nk}))) break;
                if (stages) {
                    // the Q tile is free once the last item's scores are, which wait for no V but the ones requested
                    if (nq > 0 && !(ok = wait(bar_q_free, (nq - 1) & 1))) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(bar_q, rpt * kCRowBytes);
                        tma_load_3d(sb + SP::off_q, &tm_q, bar_q, 0, h * a.G, t.q0 + tile * qpt);
                    }
                    ++nq;
                }
                for (int i = 0, v = 0; stages && i <= stages && ok; ++i) {
                    for (; v < (i == stages ? i : i - 2); ++v) {
                        const int vs = nv % SP::vs;
                        if (nv >= SP::vs && !(ok = wait(bar_v_free + 8 * vs, ((nv / SP::vs) - 1) & 1))) break;
                        bring(&tm_v, sb + SP::off_v + vs * SP::tile, bar_v + 8 * vs, h, vrow);
                        ++nv;
                        vrow = page_of((v + 1) * kCKeys);
                    }
                    if (i == stages || !ok) break;
                    const int ks = g % SP::ks;
                    if (g >= SP::ks && !(ok = wait(bar_k_free + 8 * ks, ((g / SP::ks) - 1) & 1))) break;
                    bring(&tm_k, sb + SP::off_k + ks * SP::tile, bar_k + 8 * ks, h, krow);
                    ++g;
                    krow = page_of((i + 1) * kCKeys);
                }
            }
            if (!ok) break;
            // sequences longer than announced have tiles past the grid
            if (x + static_cast<long long>(gridDim.x) < all * a.Hkv && x + static_cast<long long>(gridDim.x) <= 0x7fffffff) {
                x += gridDim.x;
                w = look_up(x);
                continue;
            }
            if (!(ok = wait(bar_next, (asked - 1) & 1))) break;
            x = next_cta(sb + SP::off_next);
            if (x < 0) break;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ask_next(sb + SP::off_next, bar_next);
            ++asked;
            w = look_up(x);
        }
        if (ok) hand_over({0, 0, 0, 0, 0});
        // no copy may still be landing when the CTA exits
        if (lane == 0) {
            for (int u = g - SP::ks; u < g; ++u)
                if (u >= 0 && !mbar_wait(bar_k + 8 * (u % SP::ks), (u / SP::ks) & 1)) *s_abort = 1;
            for (int u = nv - SP::vs; u < nv; ++u)
                if (u >= 0 && !mbar_wait(bar_v + 8 * (u % SP::vs), (u / SP::vs) & 1)) *s_abort = 1;
            if (nq && !mbar_wait(bar_q, (nq - 1) & 1)) *s_abort = 1;
            if (!mbar_wait(bar_next, (asked - 1) & 1)) *s_abort = 1;
        }
    } else if (warp == kCIssuer) {
        // ------------------------------------------------------------- MMA issuer
        if (lane == 0) {
            constexpr uint32_t id_s = idesc(kCRows, kCKeys, 0), id_o = idesc(kCRows, 64, 1);
            int gs = 0, g = 0, nq = 0;   // S issued, P . V issued, Q tiles
            bool ok = true;
            for (int ni = 0; ok; ++ni) {
                const int slot = ni % kCItems;
                if (!c_wait(bar_item + 8 * slot, (ni / kCItems) & 1, s_abort)) break;
                const int live = items[slot].live, nk = items[slot].nk, stages = (nk + kCKeys - 1) / kCKeys;
                mbar_arrive_release(bar_item_free + 8 * slot);
                if (!live) break;
                if (!stages) continue;
                if (!c_wait(bar_q, nq & 1, s_abort)) break;
                ++nq;
                auto issue_s = [&](bool last) {
                    const int ks = gs % SP::ks;
                    if (!c_wait(bar_k + 8 * ks, (gs / SP::ks) & 1, s_abort) ||
                        (gs > 0 && !c_wait(bar_s_free, (gs - 1) & 1, s_abort)))
                        return false;
                    tc_fence_after();
                    const uint32_t kb = sb + SP::off_k + ks * SP::tile;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_ss(tmem + kCColS, sdesc(sb + SP::off_q + 32 * k), sdesc(kb + 32 * k), id_s, k > 0);
                    umma_commit(bar_s);
                    umma_commit(bar_k_free + 8 * ks);
                    if (last) umma_commit(bar_q_free);
                    ++gs;
                    return true;
                };
                ok = issue_s(stages == 1);
                for (int st = 0; st < stages && ok; ++st, ++g) {
                    if (st + 1 < stages && !(ok = issue_s(st + 2 == stages))) break;
                    const int vs = g % SP::vs;
                    if (!c_wait(bar_p, g & 1, s_abort) || !c_wait(bar_v + 8 * vs, (g / SP::vs) & 1, s_abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t vb = sb + SP::off_v + vs * SP::tile;
                    const int steps = min((nk - st * kCKeys + 15) >> 4, kCKeys / 16);
#pragma unroll
                    for (int k = 0; k < kCKeys / 16; ++k)
                        if (k < steps) umma_ts(tmem + kCColO, tmem + kCColP + 8 * k, sdesc(vb + 2048 * k), id_o, st > 0 || k > 0);
                    umma_commit(bar_pv);
                    umma_commit(bar_v_free + 8 * vs);
                }
            }
            // drain: every product issued has finished and its arrivals have landed
            umma_commit(bar_drain);
            if (!mbar_wait(bar_drain, 0)) *s_abort = 1;
        }
    } else {
        // ---------------------------------------------------------------- softmax
        const uint32_t tl = tmem + (static_cast<uint32_t>(32 * warp) << 16);
        const int r = tid;   // the thread's row of the tile
        int g = 0;
        bool ok = true;
        auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, c_wait(bar, parity, s_abort)); };
        for (int ni = 0; ok; ++ni) {
            const int slot = ni % kCItems;
            if (!wait(bar_item + 8 * slot, (ni / kCItems) & 1)) break;
            const int q0 = items[slot].q0, R = items[slot].r0 + r, live = items[slot].live, h = items[slot].h, nk = items[slot].nk;
            const int stages = (nk + kCKeys - 1) / kCKeys;
            __syncwarp();
            if (lane == 0) mbar_arrive_release(bar_item_free + 8 * slot);
            if (!live) break;
            const int qi = R / a.G;
            __nv_bfloat16* to = static_cast<__nv_bfloat16*>(a.out) +
                                (static_cast<long long>(q0 + qi) * a.H + h * a.G + R - qi * a.G) * 64;
            if (!stages) {   // no keys: zeros
                if (r < live)
                    for (int j = 0; j < 8; ++j) reinterpret_cast<uint4*>(to)[j] = make_uint4(0, 0, 0, 0);
                continue;
            }
            float m = -INFINITY, l = 0.f;
            for (int st = 0; st < stages; ++st, ++g) {
                if (!(ok = wait(bar_s, g & 1))) break;
                tc_fence_after();
                const int left = nk - st * kCKeys;   // keys of this stage and later ones
                if (32 * warp < live) {
                    uint32_t s0[32], s1[32], s2[32], s3[32];
                    OASR_TMEM_LD32(tl + kCColS, s0);
                    OASR_TMEM_LD32(tl + kCColS + 32, s1);
                    OASR_TMEM_LD32(tl + kCColS + 64, s2);
                    OASR_TMEM_LD32(tl + kCColS + 96, s3);
                    tmem_wait_ld();   // of the whole warp
                    tc_fence_before();
                    if (lane == 0) mbar_arrive_release(bar_s_free);
                    if (left < kCKeys) {   // keys past the last one
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            if (j >= left) s0[j] = 0xff800000u;
                            if (32 + j >= left) s1[j] = 0xff800000u;
                            if (64 + j >= left) s2[j] = 0xff800000u;
                            if (96 + j >= left) s3[j] = 0xff800000u;
                        }
                    }
                    // eight maxima side by side
                    float y[8];
                    auto f32 = [](uint32_t w) { return __uint_as_float(w); };
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        y[q] = fmax3(f32(s0[q]), f32(s0[q + 8]), f32(s0[q + 16]));
                        y[q] = fmax3(y[q], f32(s0[q + 24]), f32(s1[q]));
                        y[q] = fmax3(y[q], f32(s1[q + 8]), f32(s1[q + 16]));
                        y[q] = fmax3(y[q], f32(s1[q + 24]), f32(s2[q]));
                        y[q] = fmax3(y[q], f32(s2[q + 8]), f32(s2[q + 16]));
                        y[q] = fmax3(y[q], f32(s2[q + 24]), f32(s3[q]));
                        y[q] = fmax3(y[q], f32(s3[q + 8]), f32(s3[q + 16]));
                        y[q] = fmaxf(y[q], f32(s3[q + 24]));
                    }
                    const float top = fmax3(fmax3(y[0], y[1], y[2]), fmax3(y[3], y[4], y[5]), fmaxf(y[6], y[7])) * a.c;
                    if (st == 0) {
                        m = fmaxf(top, kLowest);
                    } else {
                        const bool grown = top > m + 8.f;
                        if (__any_sync(0xffffffffu, grown)) {
                            if (!(ok = wait(bar_pv, (g - 1) & 1))) break;
                            tc_fence_after();
                            const float f = grown ? ex2_approx(m - top) : 1.f;
                            if (grown) m = top;
                            l *= f;
#pragma unroll 1
                            for (int q = 0; q < 8; ++q) {
                                uint32_t w[8];
                                OASR_TMEM_LD8(tl + kCColO + 8 * q, w);
                                tmem_wait_ld();
#pragma unroll
                                for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(__uint_as_float(w[j]) * f);
                                OASR_TMEM_ST8(tl + kCColO + 8 * q, w);
                            }
                        }
                    }
                    float2 sum[4] = {};
                    const float2 c2 = make_float2(a.c, a.c), m2 = make_float2(-m, -m);
                    auto weights = [&](const uint32_t (&w)[32], uint32_t (&pk)[16]) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float2 e = __ffma2_rn(make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1])), c2, m2);
                            const float2 p = make_float2(ex2_approx(e.x), ex2_approx(e.y));
                            sum[j & 3] = __fadd2_rn(sum[j & 3], p);
                            pk[j] = pack_bf16(p.x, p.y);
                        }
                    };
                    uint32_t pk[16];
                    weights(s0, pk);
                    if (g > 0) {   // the last P . V has read P
                        if (!(ok = wait(bar_pv, (g - 1) & 1))) break;
                        tc_fence_after();
                    }
                    OASR_TMEM_ST16(tl + kCColP, pk);
                    weights(s1, pk);
                    OASR_TMEM_ST16(tl + kCColP + 16, pk);
                    weights(s2, pk);
                    OASR_TMEM_ST16(tl + kCColP + 32, pk);
                    weights(s3, pk);
                    OASR_TMEM_ST16(tl + kCColP + 48, pk);
                    sum[0] = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
                    l += sum[0].x + sum[0].y;
                    tmem_wait_st();
                    tc_fence_before();
                } else {
                    // no rows of this warp's lanes: what their P holds reaches no other row
                    if (lane == 0) mbar_arrive_release(bar_s_free);
                    if (g > 0 && !(ok = wait(bar_pv, (g - 1) & 1))) break;
                }
                // V rows past the last key: P is 0 there, and must not meet what they hold
                const int end = (left + 15) & ~15;
                if (left < end && end <= kCKeys && 32 * warp < end && 32 * warp + 32 > left) {
                    if (!(ok = wait(bar_v + 8 * (g % SP::vs), (g / SP::vs) & 1))) break;
                    if (r >= left && r < end) {
                        uint4* row = reinterpret_cast<uint4*>(sm + SP::off_v + (g % SP::vs) * SP::tile + r * kCRowBytes);
#pragma unroll
                        for (int c = 0; c < 8; ++c) row[c] = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive_release(bar_p);
            }
            if (!ok || !(ok = wait(bar_pv, (g - 1) & 1))) break;
            tc_fence_after();
            if (32 * warp < live) {
                const float f = l == 0.f ? 0.f : 1.f / l;   // scores of -inf alone
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t w[32];
                    OASR_TMEM_LD32(tl + kCColO + 32 * q, w);
                    tmem_wait_ld();
                    if (r < live) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t o[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                o[e] = pack_bf16(__uint_as_float(w[8 * j + 2 * e]) * f, __uint_as_float(w[8 * j + 2 * e + 1]) * f);
                            reinterpret_cast<uint4*>(to)[4 * q + j] = make_uint4(o[0], o[1], o[2], o[3]);
                        }
                    }
                }
            }
            tc_fence_before();
        }
    }
    grid_dep_trigger();
    tc_fence_before();
    __syncthreads();
    if (warp == kCIssuer) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCCols));
    }
    if (tid == 0 && *s_abort) err |= kErrTimeout;
    if (err) atomicOr(a.status, err);
}

int g_smem_done_xtc[2][64];

}  // namespace

bool cross_tc_takes(const CrossArgs& a)
{
    // Pages that tile a stage of 128 keys, as a stage's boxes lie one behind the other.  Others (of 24 frames, say), and groups of
    // more than 128 heads, stay with tiles of 16 rows: 256 transcripts 760 us in pages of 24, 150 in pages of 32 and 205 in
    // pages of 8, whose boxes are the smallest.
    return a.G <= kCRows && (!a.table || (a.bs >= 8 && a.bs <= 32768 && !(a.bs & (a.bs - 1))));
}

oasr_status cross_tc(const CrossArgs& a, int max_q, cudaStream_t stream)
{
    const bool paged = a.table != nullptr;
    const int qpt = kCRows / a.G;
    CUtensorMap tm_q, tm_k, tm_v;
    const long long keys = paged ? static_cast<long long>(a.num_blocks) * a.bs : a.total_k;
    const int box = paged && a.bs < kCKeys ? a.bs : kCKeys;
    if (!encode_head_rows_bf16(&tm_q, a.q, a.total_q, a.H, a.q_stride, a.G, qpt) ||
        !encode_head_rows_bf16(&tm_k, a.k, keys, a.Hkv, a.k_stride, 1, box) ||
        !encode_head_rows_bf16(&tm_v, a.v, keys, a.Hkv, a.v_stride, 1, box))
        return OASR_ERR_INVALID_ARG;
    auto kern = paged ? cross_tc_kernel<true> : cross_tc_kernel<false>;
    if (!ensure_smem(kern, CSmem::bytes, g_smem_done_xtc[paged])) return OASR_ERR_CUDA;
    // a CTA for each tile there can be: no more than the longest sequence has for all, or than all queries and a
    // partly filled tile of each sequence make (CTAs without one would only crowd those that have)
    const long long most = static_cast<long long>(a.total_q) / qpt + a.N, each = (static_cast<long long>(max_q) + qpt - 1) / qpt * a.N;
    const long long tiles = most < each ? most : each;
    if (most * a.Hkv > 0x7fffffffLL) return OASR_ERR_UNSUPPORTED;
    return launch_pdl(kern, dim3(static_cast<unsigned>(tiles * a.Hkv)), dim3(kCThreads), CSmem::bytes, stream, tm_q, tm_k, tm_v, a);
}

}  // namespace oasr
