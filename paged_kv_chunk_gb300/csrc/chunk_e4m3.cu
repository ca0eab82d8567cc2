// Streaming chunk attention over the 8-bit paged cache (oasr_chunk_relattn_paged_e4m3) and the
// fused append + attention step (oasr_chunk_step_paged_e4m3).  Score, masking and table index
// are those of the 16-bit calls (chunk_attn.cu); the keys and values are what the pool's e4m3
// rows and their power-of-two scales stand for (e4m3.cuh).
//
//   s_ij = scale * (2^ek_j (q_i + u) . k8_j + (q_i + v) . rel[R - T - C + j - i])
//   out_i = sum_j softmax(s_i)_j 2^ev_j v8_j
//
// The scales stay out of the products: 2^ek multiplies the accumulated score of its key (one fused
// multiply-add with the position term) and 2^ev adds ev to the exponent of its key's weight; both are
// exact.  k8 and v8 go into fp16 matrix instructions (e4m3 is exact in fp16).  fp16 holds q + u (each
// query row scaled by a power of two) and the weights with three bits more than bf16 would: rms error
// against 64 bits 0.0021 of the output's on random data, 0.0031 with bf16 (0.0017 is the rounding of
// the output itself).
//
// A CTA takes items (stream, head, tile of 16 or 32 queries) in turn: four consumer warps and a producer
// warp.  The producer brings stages of 64 keys by TMA (boxes of K and V rows, two 64-byte rows to a
// 128-byte swizzled line, and one bulk copy of each page's scales) and tiles of 64 rel rows into a ring;
// consumer warp w takes keys 16w .. 16w+15 of each stage for all the item's queries.  The position term
// is computed beside the stages into a skewed bf16 table that is a window of 256 of its columns, so its
// shared memory does not grow with the history.  In the fused step (T <= 16) the chunk itself never comes
// through the pool: the consumer warps quantise k_new's and v_new's rows into a region of their own, from
// which they are attended to, and store the same bytes into the pool.
//
// When the (stream, head) pairs are too few to fill the GPU the keys of each are divided over a cluster
// of up to 16 CTAs, whose partial sums meet through distributed shared memory.
//
// What bounds it: per 16 keys and 16 queries a warp converts 24 words, multiplies, adds the position term,
// exponentiates and rounds, 405 warp instructions in all, at half of the issue rate because registers leave too
// few warps to cover the chains' latencies; HBM is at a tenth to a third of its rate.  Device times: the
// Conformer-large step (256 streams, 8 heads, 16 frames, window 512) 63.5 us, one stream and one frame over 8000
// keys 14.4, 128 streams of 64 frames over 0 to 1024 keys 125.
#include "attn_core.cuh"
#include "cluster.cuh"
#include "e4m3.cuh"
#include "host_common.h"

namespace oasr {

namespace {

constexpr int kE4MaxPages = 512;                    // block-table entries a CTA caches
constexpr int kE4Stage = 2 * kStageKeys * kE4Row;   // a ring slot: K and V rows of a stage, or 64 rel rows
constexpr int kSlots = 4;                           // of the ring: 3 and 6 were 1% slower over 1984 keys
constexpr int kE4MaxT = 64;
constexpr int kChunkRows = 16;                      // rows of the chunk region (fused: T <= 16)
constexpr int kE4Consumers = 32 * kConsumerWarps;
constexpr int kTableW = 256;                        // columns of the position table's window
constexpr int kTableStride = kTableW + 16;          // 8 mod 32 words: 8-byte reads without conflicts
constexpr int kOrderMax = 512;                      // streams of a cohort whose items are sorted by length
constexpr int kMaxRowExp = 120;
constexpr uint32_t kRowRoom = 30;                   // octaves a row's |q + v| may lie above its |q + u|, scaled as one
constexpr float kNoMax = -3.0e38f;                  // the running maximum before any key

struct E4Args {
    uint8_t* k_pool;
    uint8_t* v_pool;
    uint8_t* kv_scale;
    const int32_t* block_table;
    const int32_t* cache_seqlens;
    const uint16_t* pos_bias_u;
    const uint16_t* pos_bias_v;
    uint16_t* out;
    unsigned* status;
    int num_blocks, block_size, bs_shift, mbps, T, H, R;
    int items;        // (stream, head, query tile)
    int B, sorted;    // sorted: items of unequal streams go to the CTAs longest first
    int q_tiles, splits;
    float scale, scale_log2;   // the latter times log2(e)
    uint32_t zero;             // 0, which the compiler does not know (mbar_arrive_after)
};

// Shared memory (byte offsets from a 1024-aligned base).
template <int MT, int NS, bool FUSED>
struct E4Smem {
    static constexpr int Tp = 16 * MT;
    static constexpr int off_ring = 0;
    static constexpr int off_q = off_ring + NS * kE4Stage;            // q as it comes
    static constexpr int off_qv = off_q + Tp * kRowBytes;             // bf16((q + v) 2^-x)
    static constexpr int off_qu = off_qv + Tp * kRowBytes;            // fp16((q + u) 2^-x)
    static constexpr int off_cn = off_qu + Tp * kRowBytes;            // the chunk's K and V rows as they come ...
    static constexpr int off_ck = off_cn + (FUSED ? 2 * kChunkRows * kRowBytes : 0);   // ... and quantised
    static constexpr int off_gt = off_ck + (FUSED ? 2 * kChunkRows * kE4Row : 0);      // the position table's window;
    static constexpr int off_co = off_gt;                             // after the keys: two shares' rows, m, lambda
    static constexpr int off_cm = off_co + 2 * Tp * kOW * 4;
    static constexpr int off_cl = off_cm + 2 * Tp * 4;
    static constexpr int gt_bytes = Tp * kTableStride * 2, comb_bytes = off_cl + 2 * Tp * 4 - off_co;
    static constexpr int off_sc = off_gt + (gt_bytes > comb_bytes ? gt_bytes : comb_bytes);   // scales [NS][2 * 64]
    static constexpr int off_csc = off_sc + NS * 2 * kStageKeys;      // the chunk's [2][16]
    static constexpr int off_re = off_csc + 2 * kChunkRows;           // 2^x of the query rows
    static constexpr int off_item = off_re + Tp * 4;                  // cache length of the item, two of them; failed
    static constexpr int off_bar = off_item + 16;                     // full[NS], empty[NS], q full, q free
    static constexpr int off_order = off_bar + (2 * NS + 2) * 8;      // streams by length (16 bits each)
    static constexpr int off_bt = off_order + 2 * kOrderMax;          // block-table row, two of them
    static constexpr int bytes = off_bt;                              // + 2 * mbps * 4
    // clusters (one item each): the CTA's share, in the ring's memory
    static constexpr int part_o = 0;
    static constexpr int part_m = part_o + Tp * kHeadDim * 4;
    static constexpr int part_l = part_m + Tp * 4;
    static_assert(part_l + Tp * 4 <= NS * kE4Stage, "share area");
    static_assert(off_ck % 1024 == 0 && off_gt % 16 == 0 && off_sc % 16 == 0 && off_bar % 8 == 0, "alignment");
};

// Byte offset of 16-byte chunk c (0..3) of key r in a tile of 64-byte rows, two to a 128-byte line,
// written by TMA with 128-byte swizzling (tile base 1024-byte aligned).
__device__ __forceinline__ uint32_t swz_key(int r, int c) { return swz128(r >> 1, 4 * (r & 1) + c); }

// Bytes 0, 1 (lo) and 2, 3 (hi) of w, e4m3, as pairs of fp16 (exact).
__device__ __forceinline__ void e4m3_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi)
{
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// D += A (16x16 fp16, row) * B (16x8 fp16, col), fp32 accumulators.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same without an addend.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ void mma_bf16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Two 16 x 16 byte matrices, transposed: lane (g4, t4) gets bytes 4 t4 .. 4 t4 + 3 of columns g4
// (r0, r2) and 8 + g4 (r1, r3), a byte index being a row.
__device__ __forceinline__ void ldsm8_x2_t(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3)
{
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

// Arrives on `bar` once the loads that `words` came from have returned: the arrival's address depends on them
// (zero is 0).  A slot may only be released then: loads wait in another unit's queue than the arrival, which can
// overtake them, and a copy then lands under them.  One word of a load is enough, its words come together.
__device__ __forceinline__ void mbar_arrive_after(uint32_t bar, uint32_t words, uint32_t zero)
{
    mbar_arrive_release(bar + words * zero);
}

// A slice of 16 keys in registers: raw K and V words and scale bytes.  A lane's four keys are
// neighbours, 4 t4 .. 4 t4 + 3: as columns of the scores they are columns 2 t4, 2 t4 + 1 of two 8-key tiles
// (tile n holds keys 4 i + 2 n and 4 i + 2 n + 1), as rows of V the bytes of a transposed word.
struct E4Slice {
    uint4 k[2];         // key 4 (g4 / 2) + 2 n + g4 % 2, dims 16 t4 ..
    uint32_t v[8];      // dim 8 i + g4 of keys 4 t4 ..
    uint32_t ks, vs;    // scale bytes of keys 4 t4 ..
};

// k_s, v_s: shared addresses of the slice's first rows; sc: its first K scale, v_off bytes before its first
// V scale; far_off: bytes from the scales of keys 0 .. 7 to those of keys 8 .. 15 (pages of eight keys
// hold 16 scales each).
// The lane's part of the addresses is computed once (E4Lane); the other rows and chunks it reads differ from
// it in single bits of the swizzled offset.
struct E4Lane {
    uint32_t k, v, sc;
};

__device__ __forceinline__ E4Lane e4_lane(int lane, int far_off)
{
    const int g4 = lane >> 2, t4 = lane & 3;
    E4Lane l;
    l.k = swz_key(4 * (g4 >> 1) + (g4 & 1), t4);
    l.v = swz_key(lane & 15, lane >> 4);
    l.sc = 4 * (t4 & 1) + (t4 >> 1) * far_off;
    return l;
}

__device__ __forceinline__ void load_slice(E4Slice& x, const E4Lane& l, uint32_t k_s, uint32_t v_s, uint32_t sc, uint32_t v_off)
{
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x.ks) : "r"(sc + l.sc));
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x.vs) : "r"(sc + l.sc + v_off));
#pragma unroll
    for (int dp = 0; dp < 2; ++dp)   // two chunks on
        ldsm8_x2_t((v_s + l.v) ^ (32u * dp), x.v[4 * dp], x.v[4 * dp + 1], x.v[4 * dp + 2], x.v[4 * dp + 3]);
#pragma unroll
    for (int n = 0; n < 2; ++n)   // two keys on: the next line, its swizzle's lowest bit flipped
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x.k[n].x), "=r"(x.k[n].y), "=r"(x.k[n].z), "=r"(x.k[n].w)
                     : "r"((k_s + l.k) ^ (144u * n)));
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Eight dims (chunk l8) of one query row, by eight neighbouring lanes: bf16(q + v) into the swizzled
// tile qv and fp16(q + u) into qu, both times a power of two 2^-x, and 2^x into row_pow.  u, v: the head's
// biases.  x brings the row's largest |q + u| into [1, 2), but the largest |q + v| no further up than 2^31: where
// q + u vanishes beside it (a padded frame, q = -u), 2^-x alone would take the position term past fp32's range.  Where
// that holds x back, fp16 loses bits of q + u only if it is below 2^-44 of q + v.
__device__ __forceinline__ void prepare_row(const uint8_t* q_tile, uint8_t* qv, uint8_t* qu, float* row_pow,
                                            const uint16_t* u, const uint16_t* v, int row, int l8)
{
    const uint4 qw = *reinterpret_cast<const uint4*>(q_tile + swz128(row, l8));
    const uint4 uw = __ldg(reinterpret_cast<const uint4*>(u) + l8), vw = __ldg(reinterpret_cast<const uint4*>(v) + l8);
    const uint32_t q[4] = {qw.x, qw.y, qw.z, qw.w}, un[4] = {uw.x, uw.y, uw.z, uw.w}, vn[4] = {vw.x, vw.y, vw.z, vw.w};
    float a[8], p[8];
    float m = 0.f, mp = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[2 * i] = bf16_lo(q[i]) + bf16_lo(un[i]);
        a[2 * i + 1] = bf16_hi(q[i]) + bf16_hi(un[i]);
        p[2 * i] = bf16_lo(q[i]) + bf16_lo(vn[i]);
        p[2 * i + 1] = bf16_hi(q[i]) + bf16_hi(vn[i]);
        m = fmax3(m, fabsf(a[2 * i]), fabsf(a[2 * i + 1]));
        mp = fmax3(mp, fabsf(p[2 * i]), fabsf(p[2 * i + 1]));
    }
    // the exponents' maximum is that of m and 2^-30 mp (signs are clear, so bits order as the values do)
    uint32_t e = max(__float_as_uint(m), max(__float_as_uint(mp), kRowRoom << 23) - (kRowRoom << 23));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) e = max(e, __shfl_xor_sync(0xffffffffu, e, o));
    const int x = max(-kMaxRowExp, min(kMaxRowExp, static_cast<int>(e >> 23) - 127));
    const float f = pow2(-x);
    uint32_t pu[4], pv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        pu[i] = pack_f16(a[2 * i] * f, a[2 * i + 1] * f);
        pv[i] = pack_bf16(p[2 * i] * f, p[2 * i + 1] * f);
    }
    *reinterpret_cast<uint4*>(qu + swz128(row, l8)) = make_uint4(pu[0], pu[1], pu[2], pu[3]);
    *reinterpret_cast<uint4*>(qv + swz128(row, l8)) = make_uint4(pv[0], pv[1], pv[2], pv[3]);
    if (l8 == 0) row_pow[row] = pow2(x);
}

// A fragments of 16 rows of a prepared tile, the head dimension in the order of the e4m3 words: quad
// position t4 holds dims 16 t4 .., k-step ks the dims 4 ks .. 4 ks + 3 of them.
__device__ __forceinline__ void load_a(uint32_t (&f)[4][4], const uint8_t* tile, int mt, int lane)
{
    const uint32_t at = smem_addr(tile) + swz128(lane >> 2, 2 * (lane & 3));
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            uint4 w;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                         : "r"((at ^ (16u * c)) + (2 * mt + half) * 1024));
            f[2 * c][half] = w.x;
            f[2 * c][half + 2] = w.y;
            f[2 * c + 1][half] = w.z;
            f[2 * c + 1][half + 2] = w.w;
        }
    }
}

// A warp's column tiles of the position term: the CTA's Tp query rows (qv tile) against two eights of the
// 64 rel rows in the ring slot `rows` (128-byte swizzled), which are columns col0 .. col0 + 63 of the item's
// table G[i][c], c counting rel rows from the one of the last query's first key.  G[i][c] goes to
// gs[i * kTableStride + (c + i + 1) % kTableW] rounded to bf16 (a relative 2^-8 of the position term, the
// size of the rounding of q + v), so that query i and key j read column (j + Tp) % kTableW of row i.
// Every lane arrives on release_bar once it has read its rows (zero: see mbar_arrive_after).
template <int MT>
__device__ __forceinline__ void table_tiles(uint16_t* gs, const uint8_t* qv, const uint8_t* rows, int col0, int warp,
                                            int lane, uint32_t release_bar, uint32_t zero)
{
    const int g4 = lane >> 2, t4 = lane & 3;
    uint4 bl[2], bh[2];
    const uint32_t at = smem_addr(rows) + swz128(g4, 2 * t4) + warp * 1024;   // eight rows a kilobyte
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(bl[u].x), "=r"(bl[u].y), "=r"(bl[u].z), "=r"(bl[u].w)
                     : "r"(at + 4096 * u));
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(bh[u].x), "=r"(bh[u].y), "=r"(bh[u].z), "=r"(bh[u].w)
                     : "r"((at ^ 16u) + 4096 * u));
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        uint32_t qa[4][4];
        load_a(qa, qv, mt, lane);
        uint16_t* r0 = gs + (16 * mt + g4) * kTableStride;
        uint16_t* r1 = r0 + 8 * kTableStride;
        float c[2][4];
        mma_bf16_first(c[0], qa[0], bl[0].x, bl[0].y);
        mma_bf16_first(c[1], qa[0], bl[1].x, bl[1].y);
        mma_bf16_16816(c[0], qa[1], bl[0].z, bl[0].w);
        mma_bf16_16816(c[1], qa[1], bl[1].z, bl[1].w);
        mma_bf16_16816(c[0], qa[2], bh[0].x, bh[0].y);
        mma_bf16_16816(c[1], qa[2], bh[1].x, bh[1].y);
        mma_bf16_16816(c[0], qa[3], bh[0].z, bh[0].w);
        mma_bf16_16816(c[1], qa[3], bh[1].z, bh[1].w);
        if (mt == 0) mbar_arrive_after(release_bar, __float_as_uint(c[0][0]) ^ __float_as_uint(c[1][0]), zero);
        // only the window's last slot can run over its end
        const int x = (col0 & (kTableW - 1)) + 8 * warp + 2 * t4 + 16 * mt + g4 + 1;
        const uint32_t w[4] = {pack_bf16(c[0][0], c[0][1]), pack_bf16(c[0][2], c[0][3]), pack_bf16(c[1][0], c[1][1]),
                               pack_bf16(c[1][2], c[1][3])};
        if ((col0 & (kTableW - 1)) != kTableW - kStageKeys) {
            uint16_t* d = r0 + x;
            d[0] = static_cast<uint16_t>(w[0]);
            d[1] = static_cast<uint16_t>(w[0] >> 16);
            d[8 * kTableStride + 8] = static_cast<uint16_t>(w[1]);
            d[8 * kTableStride + 9] = static_cast<uint16_t>(w[1] >> 16);
            d[32] = static_cast<uint16_t>(w[2]);
            d[33] = static_cast<uint16_t>(w[2] >> 16);
            d[8 * kTableStride + 40] = static_cast<uint16_t>(w[3]);
            d[8 * kTableStride + 41] = static_cast<uint16_t>(w[3] >> 16);
        } else {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int y = x + 8 * kConsumerWarps * u;
                r0[y & (kTableW - 1)] = static_cast<uint16_t>(w[2 * u]);
                r0[(y + 1) & (kTableW - 1)] = static_cast<uint16_t>(w[2 * u] >> 16);
                r1[(y + 8) & (kTableW - 1)] = static_cast<uint16_t>(w[2 * u + 1]);
                r1[(y + 9) & (kTableW - 1)] = static_cast<uint16_t>(w[2 * u + 1] >> 16);
            }
        }
    }
}

// Running state of 16 query rows of one warp.  With t_ij = s_ij + ev_j (log2 units: the size of key j's
// contribution to the output), m is the running maximum of t, o the sum of 2^(t - m) v8 and l the
// sum of 2^(s - m + E - kSumRoom), where E is within 7 of the largest V scale exponent so far.
constexpr int kSumRoom = 70;
struct E4Acc {
    float o[8][4];   // o[d]: dims 8 d + 2 t4, 8 d + 2 t4 + 1 of row g4, then of row g4 + 8
    float m[2];
    float2 l[2];     // a share of the even keys, one of the odd; lambda (in .x) from the join on
};

// One warp, 16 MT query rows against one slice.  x0: the position table's column of the slice's first key
// (aligned: a multiple of 16, so that a lane's four keys are eight bytes of one row); keys [0, kvalid) of
// the slice exist; sc: scale * log2(e) * 2^x of rows g4 and g4 + 8 of each m-tile.  Every lane arrives on
// release_bar (unless 0) when the slice has been read (zero: see mbar_arrive_after).
//
// P is 2^(t - m), at most one, and goes into the product as fp16: its rounding is 2^-11 of each
// weight and never more than 2^-25 of the row's largest contribution, whatever the scales.  The
// row sum takes p back out of it, l += P 2^(E - ev - kSumRoom); a slice with a scale below 2^(E - 40) (a row of
// zeros has 2^-100), where that could underflow, sums 2^(s - m + E - kSumRoom) of its own.  A key of far smaller
// scale can have a score far above m - E; its term and the sum then stop at 2^90 and 2^100, of which the terms
// of the largest contributions, 2^-kSumRoom, are less than 2^-150: no more than fp32 weights can tell from nothing.
template <int MT>
__device__ __forceinline__ void slice_e4m3(E4Acc (&acc)[MT], const uint8_t* qu_tile, E4Slice& x,
                                           const uint16_t* gs, int x0, bool aligned, int kvalid,
                                           const float (&sc)[MT][2], int& E, int lane, uint32_t release_bar,
                                           uint32_t zero)
{
    const int g4 = lane >> 2, t4 = lane & 3;
    float s[MT][2][4];
    {
        // (q + u) from shared memory again for each slice: kept in registers it costs more in spilled addresses
        uint32_t qu[MT][4][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) load_a(qu[mt], qu_tile, mt, lane);
        const uint32_t w[2][4] = {{x.k[0].x, x.k[0].y, x.k[0].z, x.k[0].w}, {x.k[1].x, x.k[1].y, x.k[1].z, x.k[1].w}};
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {   // the tiles in turn: independent products back to back
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                uint32_t b0, b1;
                e4m3_to_f16(w[n][ks], b0, b1);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    if (ks == 0)
                        mma_f16_first(s[mt][n], qu[mt][ks], b0, b1);
                    else
                        mma_f16_16816(s[mt][n], qu[mt][ks], b0, b1);
                }
            }
        }
    }
    const bool tail = kvalid < 16;
    if (tail) {   // rows past the last key may hold anything: V bytes and scales (their scores are replaced below)
        const int have = max(0, min(4, kvalid - 4 * t4));
        const uint32_t mask = have == 4 ? 0xffffffffu : (1u << (8 * have)) - 1u;
#pragma unroll
        for (int i = 0; i < 8; ++i) x.v[i] &= mask;
        x.vs = (x.vs & mask) | (static_cast<uint32_t>(E + 127) * 0x01010101u & ~mask);
    }
    // keys 4 t4 ..: 2^ek, ev and 2^(E - ev - kSumRoom), from the scale bytes in place
    // (0x4b000000 | byte is 2^23 + byte)
    bool far = false;
    float dE = 0.f;
    {
        const int mine = static_cast<int>((x.vs >> (8 * (g4 & 3))) & 255u) - 127;   // each key by some lane
        if (__any_sync(0xffffffffu, static_cast<unsigned>(mine - E + 40) > 47u)) {
            const int top = __reduce_max_sync(0xffffffffu, mine);
            if (top > E + 7) {
                dE = static_cast<float>(top - E);
                E = top;
            }
            far = __any_sync(0xffffffffu, mine < E - 40);
        }
    }
    float2 ks[2], ev[2], back[2];   // by pairs of keys: two operations an instruction
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        auto kscale = [&](int e) { return __uint_as_float(__byte_perm(x.ks, 0u, 0x0444 | (e << 12)) >> 1); };
        const uint32_t w0 = __byte_perm(x.vs, 0x4b000000u, 0x7440 | (2 * n)), w1 = __byte_perm(x.vs, 0x4b000000u, 0x7441 | (2 * n));
        auto to_E = [&](uint32_t w) { return __uint_as_float(static_cast<uint32_t>(E + 254 - kSumRoom) * 0x00800000u - w * 0x00800000u); };
        ks[n] = make_float2(kscale(2 * n), kscale(2 * n + 1));
        ev[n] = __fadd2_rn(make_float2(__uint_as_float(w0), __uint_as_float(w1)), make_float2(-8388735.f, -8388735.f));   // 2^23 + 127
        back[n] = make_float2(to_E(w0), to_E(w1));
    }
    uint32_t pa[MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        E4Acc& a = acc[mt];
        float mx0 = a.m[0], mx1 = a.m[1];
        const uint16_t* r0 = gs + (16 * mt + g4) * kTableStride;
        const uint16_t* r1 = r0 + 8 * kTableStride;
        uint32_t y0[2], y1[2];
        if (aligned) {
            const int c = (x0 & (kTableW - 1)) + 4 * t4;
            const uint2 p0 = *reinterpret_cast<const uint2*>(r0 + c), p1 = *reinterpret_cast<const uint2*>(r1 + c);
            y0[0] = p0.x; y0[1] = p0.y;
            y1[0] = p1.x; y1[1] = p1.y;
        } else {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int c = (x0 + 4 * t4 + 2 * n) & (kTableW - 1), d = (x0 + 4 * t4 + 2 * n + 1) & (kTableW - 1);
                y0[n] = r0[c] | static_cast<uint32_t>(r0[d]) << 16;
                y1[n] = r1[c] | static_cast<uint32_t>(r1[d]) << 16;
            }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            auto score = [&](int e, uint32_t g, float sc1) {
                const float2 t = __ffma2_rn(__ffma2_rn(make_float2(s[mt][n][e], s[mt][n][e + 1]), ks[n], make_float2(bf16_lo(g), bf16_hi(g))),
                                            make_float2(sc1, sc1), ev[n]);
                s[mt][n][e] = tail && 4 * t4 + 2 * n >= kvalid ? -INFINITY : t.x;
                s[mt][n][e + 1] = tail && 4 * t4 + 2 * n + 1 >= kvalid ? -INFINITY : t.y;
            };
            score(0, y0[n], sc[mt][0]);
            score(2, y1[n], sc[mt][1]);
            mx0 = fmax3(mx0, s[mt][n][0], s[mt][n][1]);
            mx1 = fmax3(mx1, s[mt][n][2], s[mt][n][3]);
        }
        // the maximum has come of both K loads and both scale loads
        if (mt == 0 && release_bar) mbar_arrive_after(release_bar, __float_as_uint(mx0) ^ x.v[0] ^ x.v[4], zero);
        // the reference only moves when a weight would pass 2^8 (fp16 holds 2^15)
        if (__any_sync(0xffffffffu, mx0 > a.m[0] + 8.f || mx1 > a.m[1] + 8.f) || dE != 0.f) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
            const float d0 = a.m[0] - mx0, d1 = a.m[1] - mx1;
            const float alpha0 = ex2_approx(d0), alpha1 = ex2_approx(d1);
            // l by halves: the factor may pass fp32's range where l is small
            const float h0 = ex2_approx(0.5f * (d0 + dE)), h1 = ex2_approx(0.5f * (d1 + dE));
            a.l[0] = make_float2(fminf(a.l[0].x * h0 * h0, 0x1p100f), fminf(a.l[0].y * h0 * h0, 0x1p100f));
            a.l[1] = make_float2(fminf(a.l[1].x * h1 * h1, 0x1p100f), fminf(a.l[1].y * h1 * h1, 0x1p100f));
#pragma unroll
            for (int d = 0; d < 8; ++d) {
                a.o[d][0] *= alpha0;
                a.o[d][1] *= alpha0;
                a.o[d][2] *= alpha1;
                a.o[d][3] *= alpha1;
            }
            a.m[0] = mx0;
            a.m[1] = mx1;
        }
        const float base0 = a.m[0], base1 = a.m[1];
        if (far) {
            const float off = static_cast<float>(E - kSumRoom);
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float v = e ? ev[n].y : ev[n].x;
                    a.l[0].x += ex2_approx(fminf(s[mt][n][e] - v - base0 + off, 90.f));
                    a.l[1].x += ex2_approx(fminf(s[mt][n][2 + e] - v - base1 + off, 90.f));
                }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const float2 t0 = __fadd2_rn(make_float2(s[mt][n][0], s[mt][n][1]), make_float2(-base0, -base0));
            const float2 t1 = __fadd2_rn(make_float2(s[mt][n][2], s[mt][n][3]), make_float2(-base1, -base1));
            const float2 p0 = make_float2(ex2_approx(t0.x), ex2_approx(t0.y)), p1 = make_float2(ex2_approx(t1.x), ex2_approx(t1.y));
            if (!far) {
                a.l[0] = __ffma2_rn(p0, back[n], a.l[0]);
                a.l[1] = __ffma2_rn(p1, back[n], a.l[1]);
            }
            pa[mt][2 * n] = pack_f16(p0.x, p0.y);
            pa[mt][2 * n + 1] = pack_f16(p1.x, p1.y);
        }
    }
#pragma unroll
    for (int d = 0; d < 8; ++d) {
        uint32_t b0, b1;
        e4m3_to_f16(x.v[d], b0, b1);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) mma_f16_16816(acc[mt].o[d], pa[mt], b0, b1);
    }
}

// Bounded wait, inline: a call would spill the registers that live across it.
__device__ __forceinline__ bool e4_wait(uint32_t bar, uint32_t parity)
{
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (;;) {
        for (int k = 0; k < 16; ++k)
            if (mbar_try_wait(bar, parity)) return true;
        if (global_timer_ns() - t0 > kWaitLimitNs) return false;
    }
}

// 2-D tiled bulk load with an L2 hint, and an untiled bulk copy; both count bytes on `bar`.
__device__ __forceinline__ void tma_load_2d_hint(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y,
                                                 uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
        : "memory");
}

__device__ __forceinline__ float ld_cluster(uint32_t addr, uint32_t rank)
{
    float v;
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// Weight of a share whose maximum (log2) is `x` against the largest, `top`; a share without keys has
// kNoMax (or -inf) and weight 0.
//
// Shares of a row are joined from o, m and lambda = log2(sum of 2^s) = m - E + kSumRoom + log2(l): the V scales
// move m away from the scores (a share of zero rows has an m of s - 100), so the row sum has a
// maximum of its own.  out = sum(o 2^(m - m*)) 2^(m* - lambda*) / sum(2^(lambda - lambda*)).
__device__ __forceinline__ float part_weight(float x, float top) { return x <= kNoMax ? 0.f : ex2_approx(x - top); }

// What a CTA does with one item: keys, ring slots and the position table, from the stream's cache length.
struct E4Item {
    int C, K;          // cached frames; keys (frames and chunk, as far as the table reaches)
    int p0;            // position of the chunk's first row: C, or below zero where the length is (no row there)
    int kc, nc;        // keys from the pool, from the chunk region
    int st0, st1;      // stages of this CTA's share
    int nrel;          // rel slots: the table has a column for each distance of the share's keys
    int off;           // rel row of query i and key j: off + j - i
    unsigned err;
};

template <int MT, bool FUSED>
__device__ __forceinline__ E4Item e4_item(const E4Args& a, int C, int split)
{
    E4Item t;
    t.err = 0;
    const int cap = a.mbps << a.bs_shift;                 // keys the block table holds (at most 2^17)
    t.p0 = max(C, -kE4MaxT);
    if (C < 0) { C = 0; t.err = kErrBounds; }
    if (C > cap) { C = cap; t.err = kErrBounds; }
    t.C = C;
    t.K = C + a.T;
    if (t.K > cap) { t.K = cap; t.err = kErrBounds; }
    if (C + 2 * a.T - 1 > a.R) t.err = kErrBounds;        // distances the rel table does not hold
    t.off = a.R - a.T - C;
    t.kc = FUSED ? C : t.K;
    const int n = (t.kc + kStageKeys - 1) / kStageKeys;
    t.st0 = n * split / a.splits;                         // n <= 2^11
    t.st1 = n * (split + 1) / a.splits;
    const bool last = split == a.splits - 1;              // the chunk follows the last pool keys
    t.nc = FUSED && last ? t.K - t.kc : 0;
    const int nkeys = (last ? t.K : t.st1 * kStageKeys) - t.st0 * kStageKeys;
    t.nrel = nkeys > 0 ? (nkeys + 16 * MT - 1 + 63) >> 6 : 0;
    return t;
}

// The items of CTA x in turn: x, grid + x, ... of the items in order, or, with the streams sorted by
// length, alternately from both ends of each round of `grid` items (longest first: every CTA gets about the
// same number of keys; streams of 0 to 1024 keys, seven items a CTA: 144 -> 124 us).
struct E4Walk {
    int items, grid, x, round;
    const uint16_t* order;   // streams by length, or null

    __device__ __forceinline__ int at(int r) const { return order && (r & 1) ? (r + 1) * grid - 1 - x : r * grid + x; }
    // the round of the first item from round r on (a reversed last round may leave a CTA out), or -1
    __device__ __forceinline__ int from(int r) const
    {
        for (; r * static_cast<long long>(grid) < items; ++r)
            if (at(r) < items) return r;
        return -1;
    }
    __device__ __forceinline__ void decode(int r, int H, int q_tiles, int& b, int& h, int& qt) const
    {
        const int i = at(r), bh = i / q_tiles;
        qt = i - bh * q_tiles;
        b = bh / H;
        h = bh - b * H;
        if (order) b = order[b];
    }
};

// Persistent: CTA x takes the items of its E4Walk.  The producer warp runs ahead of the consumers by the
// ring's slots, across items, so the next item's rows arrive while this one's are multiplied and joined.
// Ring order of an item with stages s = 0, 1, ..: rel slots 0 and 1, stage 0, rel slot 2, stage 1, ...
// (stage s needs the table's columns up to rel slot s + 1).
template <int MT, int NS, int CTAS, bool FUSED>
__global__ void __launch_bounds__(kThreads, CTAS) chunk_e4m3_kernel(
    const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_r,
    const __grid_constant__ CUtensorMap tm_kn, const __grid_constant__ CUtensorMap tm_vn, const E4Args a)
{
    static_assert(!FUSED || MT == 1, "the chunk region holds one m-tile's rows");
    using SP = E4Smem<MT, NS, FUSED>;
    constexpr int Tp = SP::Tp;
    extern __shared__ __align__(1024) uint8_t sm[];   // the only shared memory: its base is aligned
    const uint32_t sb = smem_addr(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = a.splits, T = a.T, H = a.H, sh = a.bs_shift, bs = a.block_size;
    const int split = blockIdx.x % S;
    const uint32_t bar_full = sb + SP::off_bar;
    const uint32_t bar_empty = bar_full + NS * 8;
    const uint32_t bar_q = bar_empty + NS * 8;    // an item's q, chunk rows, cache length and block-table row are in
    const uint32_t bar_qfree = bar_q + 8;         // ... and have been read
    int* s_len = reinterpret_cast<int*>(sm + SP::off_item);
    int* s_bt = reinterpret_cast<int*>(sm + SP::off_bt);
    volatile int& s_failed = s_len[2];
    unsigned err = 0;

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(bar_full + 8 * i, 1);
            mbar_init(bar_empty + 8 * i, kE4Consumers);
        }
        mbar_init(bar_q, 1);
        mbar_init(bar_qfree, kE4Consumers);
        fence_mbar_init();
        s_failed = 0;
    }
    if (warp == kConsumerWarps && lane == 0) {
        prefetch_tensormap(&tm_q);
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
        prefetch_tensormap(&tm_r);
    }
    __syncthreads();
    grid_dep_wait();   // the previous grid on the stream has finished (programmatic launch)

    E4Walk walk = {a.items, static_cast<int>(gridDim.x) / S, static_cast<int>(blockIdx.x) / S, 0, nullptr};
    if (a.sorted) {
        // streams by length, longest first: each counts the longer ones (and, of its own length, the earlier)
        int* len = reinterpret_cast<int*>(sm + SP::off_gt);
        uint16_t* order = reinterpret_cast<uint16_t*>(sm + SP::off_order);
        const int len0 = __ldg(a.cache_seqlens);
        int differ = 0;
        for (int i = tid; i < a.B; i += kThreads) {
            len[i] = __ldg(a.cache_seqlens + i);
            differ |= len[i] != len0;
        }
        if (__syncthreads_or(differ)) {
            for (int i = tid; i < a.B; i += kThreads) {
                const int mine = len[i];
                int rank = 0;
                for (int j = 0; j < a.B; ++j) rank += len[j] > mine || (len[j] == mine && j < i);
                order[rank] = static_cast<uint16_t>(i);
            }
            walk.order = order;
        }
        __syncthreads();
    }

    if (warp == kConsumerWarps) {
        // ------------------------------------------------------------ producer
        const uint64_t pol = policy_evict_first();
        const int box = min(bs, kStageKeys), box_sh = min(sh, 6);
        int n_issued = 0, n_items = 0;
        bool ok = true;
        auto acquire = [&]() {   // the next slot is free
            ok = ok && __all_sync(0xffffffffu, n_issued < NS ||
                                                   e4_wait(bar_empty + 8 * (n_issued % NS), ((n_issued / NS) - 1) & 1));
            return ok;
        };
        constexpr int kRowRegs = 4;   // entries of a lane loaded ahead (128 pages); the rest of a longer row later
        int C = 0, row[kRowRegs];
        auto request = [&](int r) {
            int b, h, qt;
            walk.decode(r, H, a.q_tiles, b, h, qt);
            C = __ldg(a.cache_seqlens + b);
#pragma unroll
            for (int k = 0; k < kRowRegs; ++k)
                if (lane + 32 * k < a.mbps) row[k] = __ldg(a.block_table + static_cast<long long>(b) * a.mbps + lane + 32 * k);
        };
        int next = walk.from(0);
        if (next >= 0) request(next);
        for (int round = next; round >= 0 && ok; round = next, ++n_items) {
            int b, h, qt;
            walk.decode(round, H, a.q_tiles, b, h, qt);
            const int i0 = qt * Tp;
            // the item's cache length and block-table row, into the buffers of the item before last
            if (n_items >= 1) {
                ok = __all_sync(0xffffffffu, e4_wait(bar_qfree, (n_items - 1) & 1));
                if (!ok) break;
            }
            int* bt = s_bt + (n_items & 1) * a.mbps;
#pragma unroll
            for (int k = 0; k < kRowRegs; ++k)
                if (lane + 32 * k < a.mbps) bt[lane + 32 * k] = row[k];
            for (int i = lane + 32 * kRowRegs; i < a.mbps; i += 32)
                bt[i] = __ldg(a.block_table + static_cast<long long>(b) * a.mbps + i);
            if (lane == 0) s_len[n_items & 1] = C;
            const E4Item t = e4_item<MT, FUSED>(a, C, split);
            __syncwarp();
            if (lane == 0) {
                mbar_arrive_expect_tx(bar_q, Tp * kRowBytes + (FUSED ? 2 * kChunkRows * kRowBytes : 0));
                tma_load_3d(sb + SP::off_q, &tm_q, bar_q, 0, h, b * T + i0);
                if (FUSED) {
                    tma_load_3d(sb + SP::off_cn, &tm_kn, bar_q, 0, h, b * T);
                    tma_load_3d(sb + SP::off_cn + kChunkRows * kRowBytes, &tm_vn, bar_q, 0, h, b * T);
                }
            }
            next = walk.from(round + 1);
            if (next >= 0) request(next);
            auto issue_rel = [&](int r) {
                if (!acquire()) return;
                if (lane == 0) {
                    const uint32_t bar = bar_full + 8 * (n_issued % NS);
                    mbar_arrive_expect_tx(bar, kE4Stage);
                    tma_load_3d(sb + (n_issued % NS) * kE4Stage, &tm_r, bar, 0, h,
                                t.off + (t.st0 + r) * kStageKeys - i0 - (Tp - 1));
                }
                ++n_issued;
            };
            if (t.nrel > 0) issue_rel(0);
            for (int s = t.st0; s < t.st1 && ok; ++s) {
                if (s - t.st0 + 1 < t.nrel) issue_rel(s - t.st0 + 1);
                if (!acquire()) break;
                const int slot = n_issued % NS;
                const uint32_t bar = bar_full + 8 * slot;
                const int j0 = s * kStageKeys;
                const int nbox = min(kStageKeys >> box_sh, (t.kc - j0 + box - 1) >> box_sh);
                // lane q: K box of page piece q and its scales, lane 16 + q: its V box
                const int q = lane & 15;
                const int j = j0 + q * box;
                const int blk = q < nbox ? bt[j >> sh] : -1;
                const bool valid = blk >= 0 && blk < a.num_blocks;
                const uint32_t sc_dst = SP::off_sc + slot * 2 * kStageKeys + q * 2 * box;
                if (q < nbox && !valid) {   // no such block: its rows read as zeros, with scales of zero
                    err |= kErrBounds;
                    if (lane < 16) {
                        for (int i = 0; i < box / 2; ++i) *reinterpret_cast<uint32_t*>(sm + sc_dst + 4 * i) = 0u;
                        fence_proxy_async_smem();
                    }
                }
                const int nvalid = __popc(__ballot_sync(0xffffffffu, valid) & 0xffffu);
                __syncwarp();   // the zeros are written before the arrival (a ballot orders no memory)
                if (lane == 0)
                    mbar_arrive_expect_tx(bar, static_cast<uint32_t>(nbox * box * 2 * kE4Row + nvalid * 2 * box));
                __syncwarp();
                if (q < nbox) {
                    const int in_page = j & (bs - 1);
                    // rows of the pools are below 2^31; an invalid block's box lies outside and reads zeros
                    const int row = valid ? (((blk * H + h) << sh) + in_page) : -4 * box;
                    const int line = row >> 1;
                    const uint32_t dst = sb + slot * kE4Stage + q * box * kE4Row;
                    if (lane < 16) {
                        tma_load_2d_hint(dst, &tm_k, bar, 0, line, pol);
                        if (valid) {
                            const uint8_t* src = a.kv_scale + 2 * static_cast<long long>(row - in_page) + in_page;
                            if (bs <= kStageKeys) {
                                bulk_load(sb + sc_dst, src, 2 * box, bar);   // K and V scales of the page are adjacent
                            } else {
                                bulk_load(sb + sc_dst, src, box, bar);
                                bulk_load(sb + sc_dst + box, src + bs, box, bar);
                            }
                        }
                    } else {
                        tma_load_2d_hint(dst + kStageKeys * kE4Row, &tm_v, bar, 0, line, pol);
                    }
                }
                ++n_issued;
            }
        }
        if (!ok) err |= kErrTimeout;
        // every copy this CTA requested lands before it ends
        for (int x = n_issued > NS ? n_issued - NS : 0; x < n_issued; ++x)
            if (!mbar_wait_idle(bar_full + 8 * (x % NS), (x / NS) & 1)) err |= kErrTimeout;
        if (n_items > 0 && !mbar_wait_idle(bar_q, (n_items - 1) & 1)) err |= kErrTimeout;
        if (err) atomicOr(a.status, err);
        if (S > 1) {
            cluster_sync();
            cluster_sync();
        }
        return;
    }

    // ---------------------------------------------------------------- consumers
    const int g4 = lane >> 2, t4 = lane & 3;
    const int box_sh = min(sh, 6), box = 1 << box_sh;
    const int jl = 16 * warp;   // this warp's keys of a stage
    const int far_off = box == 8 ? 16 : 8;   // scales of keys 8 .. 15 of a slice, from those of keys 0 .. 7
    const int sc_off = SP::off_sc + ((jl >> box_sh) << (box_sh + 1)) + (jl & (box - 1));
    const E4Lane ll = e4_lane(lane, far_off);
    uint16_t* gs = reinterpret_cast<uint16_t*>(sm + SP::off_gt);
    float* s_pow = reinterpret_cast<float*>(sm + SP::off_re);
    float* comb_o = reinterpret_cast<float*>(sm + SP::off_co);
    float* comb_m = reinterpret_cast<float*>(sm + SP::off_cm);
    float* comb_l = reinterpret_cast<float*>(sm + SP::off_cl);
    bool failed = false;
    int it = 0, n_items = 0;   // ring slots read, items begun
#pragma unroll 1
    for (int round = walk.from(0), next; round >= 0; round = next, ++n_items) {
        next = walk.from(round + 1);
        int b, h, qt;
        walk.decode(round, H, a.q_tiles, b, h, qt);
        const int i0 = qt * Tp;
        if (!failed && !e4_wait(bar_q, n_items & 1)) failed = true;
        const E4Item t = e4_item<MT, FUSED>(a, failed ? 0 : s_len[n_items & 1], split);
        err |= t.err;
        if (FUSED && t.nc > 0 && !failed) {
            // the chunk's rows, eight lanes each: quantised into the chunk region (rows past T zero) and the pool
            const int r = tid >> 3, l8 = lane & 7;
            const int p = t.p0 + r;
            const int blk = r < t.nc && p >= 0 ? s_bt[(n_items & 1) * a.mbps + (p >> sh)] : -1;
            const bool valid = blk >= 0 && blk < a.num_blocks;
            if (r < t.nc && !valid) err |= kErrBounds;   // dropped by the append: reads as zeros
            const long long page = static_cast<long long>(valid ? blk : 0) * H + h;
            const int slot = p & (bs - 1);
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                float x[8];
                unpack8(*reinterpret_cast<const uint4*>(sm + SP::off_cn + kv * kChunkRows * kRowBytes + swz128(r, l8)), x);
                uint2 q;
                uint32_t byte = e4m3_quantise8(x, 0xffffffffu, q);
                if (valid) {
                    *reinterpret_cast<uint2*>((kv ? a.v_pool : a.k_pool) + (page * bs + slot) * kE4Row + 8 * l8) = q;
                    if (l8 == 0) a.kv_scale[(2 * page + kv) * bs + slot] = static_cast<uint8_t>(byte);
                } else {
                    q = make_uint2(0u, 0u);
                    byte = 0;
                }
                *reinterpret_cast<uint2*>(sm + SP::off_ck + kv * kChunkRows * kE4Row + swz_key(r, l8 >> 1) + 8 * (l8 & 1)) = q;
                if (l8 == 0) sm[SP::off_csc + kv * kChunkRows + r] = static_cast<uint8_t>(byte);
            }
        }
#pragma unroll
        for (int r = 0; r < Tp; r += 4 * kConsumerWarps)
            prepare_row(sm + SP::off_q, sm + SP::off_qv, sm + SP::off_qu, s_pow, a.pos_bias_u + h * kHeadDim,
                        a.pos_bias_v + h * kHeadDim, r + (tid >> 3), lane & 7);
        fence_proxy_async_smem();   // the next item's q and chunk rows overwrite what was read here
        mbar_arrive_release(bar_qfree);
        named_bar_sync(1, kE4Consumers);   // the query tiles and the chunk region are complete

        float sc[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            sc[mt][0] = a.scale_log2 * s_pow[16 * mt + g4];
            sc[mt][1] = a.scale_log2 * s_pow[16 * mt + g4 + 8];
        }
        E4Acc acc[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int d = 0; d < 8; ++d) acc[mt].o[d][0] = acc[mt].o[d][1] = acc[mt].o[d][2] = acc[mt].o[d][3] = 0.f;
            acc[mt].m[0] = acc[mt].m[1] = kNoMax;
            acc[mt].l[0] = acc[mt].l[1] = make_float2(0.f, 0.f);
        }
        int E = -127;   // the smallest a scale byte says; the first keys raise it
        const int n = t.st1 - t.st0;
        // rel slots 0 and 1, then a stage and the next rel slot at a time; after the stages the chunk
        int r = 0;
        auto next_rel = [&]() {
            if (!failed && !e4_wait(bar_full + 8 * (it % NS), (it / NS) & 1)) failed = true;
            if (!failed)
                table_tiles<MT>(gs, sm + SP::off_qv, sm + (it % NS) * kE4Stage, kStageKeys * r, warp, lane,
                                bar_empty + 8 * (it % NS), a.zero);
            ++it;
            ++r;
        };
        if (t.nrel > 0) next_rel();
#pragma unroll 1
        for (int s = 0; s < n; ++s) {
            if (r < t.nrel) next_rel();
            named_bar_sync(1, kE4Consumers);   // the columns of this stage's keys are complete
            const int slot = it % NS;
            if (!failed && !e4_wait(bar_full + 8 * slot, (it / NS) & 1)) failed = true;
            ++it;
            if (failed) continue;
            const int kv = min(t.kc - (t.st0 + s) * kStageKeys, kStageKeys) - jl;
            E4Slice x;
            if (kv > 0)
                load_slice(x, ll, sb + slot * kE4Stage + jl * kE4Row, sb + slot * kE4Stage + (kStageKeys + jl) * kE4Row,
                           sb + sc_off + slot * 2 * kStageKeys, box);
            if (kv > 0)
                slice_e4m3<MT>(acc, sm + SP::off_qu, x, gs, s * kStageKeys + jl + Tp, true, kv, sc, E, lane, bar_empty + 8 * slot,
                               a.zero);
            else
                mbar_arrive_release(bar_empty + 8 * slot);
        }
        if (FUSED && t.nc > 0) {
            if (n == 0) named_bar_sync(1, kE4Consumers);
            if (warp == kConsumerWarps - 1 && !failed) {   // one slice
                E4Slice x;
                load_slice(x, e4_lane(lane, 8), sb + SP::off_ck, sb + SP::off_ck + kChunkRows * kE4Row, sb + SP::off_csc, kChunkRows);
                const int x0 = t.C - t.st0 * kStageKeys + Tp;
                slice_e4m3<MT>(acc, sm + SP::off_qu, x, gs, x0, (x0 & 15) == 0, t.nc, sc, E, lane, 0u, 0u);
            }
        }

        // the warps' shares of each row: two warps write, two add theirs and write, all finish
        auto put = [&](int part) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int row = part * Tp + 16 * mt + g4 + 8 * half;
#pragma unroll
                    for (int d = 0; d < 8; ++d)
                        *reinterpret_cast<float2*>(comb_o + row * kOW + 8 * d + 2 * t4) =
                            make_float2(acc[mt].o[d][2 * half], acc[mt].o[d][2 * half + 1]);
                    if (t4 == 0) {
                        comb_m[row] = acc[mt].m[half];
                        comb_l[row] = acc[mt].l[half].x;
                    }
                }
        };
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float l = acc[mt].l[half].x + acc[mt].l[half].y;
                l += __shfl_xor_sync(0xffffffffu, l, 1);
                l += __shfl_xor_sync(0xffffffffu, l, 2);
                acc[mt].l[half].x = acc[mt].m[half] - static_cast<float>(E - kSumRoom) + log2f(l);   // lambda from here on
            }
        named_bar_sync(1, kE4Consumers);   // every warp is done with the table
        if (warp >= 2) put(warp - 2);
        if (failed) s_failed = 1;
        named_bar_sync(1, kE4Consumers);
        if (warp < 2) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int row = warp * Tp + 16 * mt + g4 + 8 * half;
                    const float m2 = comb_m[row], l2 = comb_l[row];
                    const float m = fmaxf(acc[mt].m[half], m2), l = fmaxf(acc[mt].l[half].x, l2);
                    const float w1 = part_weight(acc[mt].m[half], m), w2 = part_weight(m2, m);
                    acc[mt].l[half].x = l + log2f(part_weight(acc[mt].l[half].x, l) + part_weight(l2, l));
                    acc[mt].m[half] = m;
#pragma unroll
                    for (int d = 0; d < 8; ++d) {
                        const float2 o = *reinterpret_cast<const float2*>(comb_o + row * kOW + 8 * d + 2 * t4);
                        acc[mt].o[d][2 * half] = acc[mt].o[d][2 * half] * w1 + o.x * w2;
                        acc[mt].o[d][2 * half + 1] = acc[mt].o[d][2 * half + 1] * w1 + o.y * w2;
                    }
                }
            __syncwarp();
            put(warp);
        }
        if (next < 0) grid_dep_trigger();   // the next grid may schedule (it waits for this one)
        named_bar_sync(1, kE4Consumers);
        if (s_failed) {
            failed = true;
            if (S == 1) break;
        }
        const int Tq = min(Tp, T - i0);
        if (S == 1) {
            for (int i = tid; i < Tq * 8; i += kE4Consumers) {
                const int row = i >> 3, d0 = (i & 7) * 8;
                const float m0 = comb_m[row], m1 = comb_m[Tp + row], l0 = comb_l[row], l1 = comb_l[Tp + row];
                const float m = fmaxf(m0, m1), l = fmaxf(l0, l1);
                const float f = exp2f(m - l) / (part_weight(l0, l) + part_weight(l1, l));
                const float w0 = part_weight(m0, m) * f, w1 = part_weight(m1, m) * f;
                const float4* p0 = reinterpret_cast<const float4*>(comb_o + row * kOW + d0);
                const float4* p1 = reinterpret_cast<const float4*>(comb_o + (Tp + row) * kOW + d0);
                uint32_t o[4];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float4 x = p0[c], y = p1[c];
                    o[2 * c] = pack_bf16(x.x * w0 + y.x * w1, x.y * w0 + y.y * w1);
                    o[2 * c + 1] = pack_bf16(x.z * w0 + y.z * w1, x.w * w0 + y.w * w1);
                }
                *reinterpret_cast<uint4*>(a.out + ((static_cast<long long>(b) * T + i0 + row) * H + h) * kHeadDim + d0) =
                    make_uint4(o[0], o[1], o[2], o[3]);
            }
            continue;
        }
        // a cluster's only item: the CTA's share into the ring's memory (every slot has been read)
        float* part_o = reinterpret_cast<float*>(sm + SP::part_o);
        float* part_m = reinterpret_cast<float*>(sm + SP::part_m);
        float* part_l = reinterpret_cast<float*>(sm + SP::part_l);
        for (int i = tid; i < Tq * kHeadDim; i += kE4Consumers) {
            const int row = i / kHeadDim, d = i % kHeadDim;
            const float m0 = comb_m[row], m1 = comb_m[Tp + row], l0 = comb_l[row], l1 = comb_l[Tp + row];
            const float m = failed ? kNoMax : fmaxf(m0, m1), l = failed ? -INFINITY : fmaxf(l0, l1);
            part_o[i] = failed ? 0.f : part_weight(m0, m) * comb_o[row * kOW + d] + part_weight(m1, m) * comb_o[(Tp + row) * kOW + d];
            if (d == 0) {
                part_m[row] = m;
                part_l[row] = failed ? l : l + log2f(part_weight(l0, l) + part_weight(l1, l));
            }
        }
        cluster_sync();
        // rows split, split + S, ... of the cluster's queries are finished here
        for (int row = split + S * warp; row < Tq; row += S * kConsumerWarps) {
            float m = kNoMax, l = -INFINITY;
            for (int k = 0; k < S; ++k) {
                m = fmaxf(m, ld_cluster(sb + SP::part_m + 4 * row, k));
                l = fmaxf(l, ld_cluster(sb + SP::part_l + 4 * row, k));
            }
            float o0 = 0.f, o1 = 0.f, sum = 0.f;
            for (int k = 0; k < S; ++k) {
                const float w = part_weight(ld_cluster(sb + SP::part_m + 4 * row, k), m);
                sum += part_weight(ld_cluster(sb + SP::part_l + 4 * row, k), l);
                o0 += w * ld_cluster(sb + SP::part_o + 4 * (row * kHeadDim + 2 * lane), k);
                o1 += w * ld_cluster(sb + SP::part_o + 4 * (row * kHeadDim + 2 * lane + 1), k);
            }
            const float f = exp2f(m - l) / sum;
            reinterpret_cast<uint32_t*>(a.out + ((static_cast<long long>(b) * T + i0 + row) * H + h) * kHeadDim)[lane] =
                pack_bf16(o0 * f, o1 * f);
        }
        cluster_sync();   // no CTA ends while another may still read its share
    }
    if (s_failed) err |= kErrTimeout;
    if (err) atomicOr(a.status, err);
}

// ----------------------------------------------------------------------------- fp32

// fp32 throughout (no TF32), the chunk already in the pool.  One CTA per (stream, head, 16 queries, share
// of the keys); tiles of 64 keys, K and V decoded to fp32 on their way into shared memory (exact), the
// rel rows the tile's distances need (79 of them) copied beside them a tile ahead.  Content and position
// products are register tiles of 2 rows by 4 keys or 5 distances, summed apart (their sum is rounded
// once); the position term is skewed through shared memory.  The operands of a tile's 16 * 64 *
// (64 + 80 + 64) FMAs come through shared memory: its wavefronts are at 65% of their peak, the FMA pipe at 31% (64
// streams of 16 frames over 512 keys, 8 heads: 112 us; the Conformer-large step 380).
constexpr int kFRows = 16, kFKeys = 64, kFRel = 80;
constexpr int kFStride = 68;      // floats of a 64-value row: rows apart by four banks
constexpr int kFThreads = 128;

struct F32Smem {
    float qu[kFRows][kFStride], qv[kFRows][kFStride];
    float k[kFKeys][kFStride], v[kFKeys][kFStride];
    float rel[2][kFRel][kFStride];
    float g[kFRows][kFRel + 4];
    float p[kFRows][kFStride];
    float part_o[kFRows][kHeadDim], part_m[kFRows], part_l[kFRows];
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}

__global__ void __launch_bounds__(kFThreads) chunk_e4m3_f32_kernel(
    const float* __restrict__ q, const uint8_t* __restrict__ k_pool, const uint8_t* __restrict__ v_pool,
    const uint8_t* __restrict__ kv_scale, const float* __restrict__ u, const float* __restrict__ vb,
    const float* __restrict__ rel, float* __restrict__ out, const E4Args a)
{
    extern __shared__ __align__(16) uint8_t smem_raw[];
    F32Smem& sm = *reinterpret_cast<F32Smem*>(smem_raw);
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int S = a.splits, T = a.T, H = a.H, bs = a.block_size;
    int idx = blockIdx.x;
    const int split = idx % S;
    idx /= S;
    const int i0 = (idx % a.q_tiles) * kFRows;
    idx /= a.q_tiles;
    const int b = idx / H, h = idx - b * H;
    grid_dep_wait();
    const E4Item t = e4_item<1, false>(a, __ldg(a.cache_seqlens + b), split);
    unsigned err = t.err;
    // query rows past T are zero
    for (int i = tid; i < kFRows * 16; i += kFThreads) {
        const int r = i >> 4, d = 4 * (i & 15);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i0 + r < T) x = __ldg(reinterpret_cast<const float4*>(q + ((static_cast<long long>(b) * T + i0 + r) * H + h) * kHeadDim + d));
        const float4 y = __ldg(reinterpret_cast<const float4*>(u + h * kHeadDim + d));
        const float4 z = __ldg(reinterpret_cast<const float4*>(vb + h * kHeadDim + d));
        *reinterpret_cast<float4*>(&sm.qu[r][d]) = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
        *reinterpret_cast<float4*>(&sm.qv[r][d]) = make_float4(x.x + z.x, x.y + z.y, x.z + z.z, x.w + z.w);
    }
    // this thread's 32 bytes of a key's K and V rows
    const int kr = tid >> 1, kd = 32 * (tid & 1);
    uint4 raw[4];
    float ks = 0.f, vs = 0.f;
    auto request = [&](int s) {
        const int j = s * kFKeys + kr;
        ks = vs = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) raw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (j < t.K) {
            const int lb = j >> a.bs_shift;
            const int blk = __ldg(a.block_table + static_cast<long long>(b) * a.mbps + lb);
            if (blk >= 0 && blk < a.num_blocks) {
                const long long page = static_cast<long long>(blk) * H + h;
                const int slot = j & (bs - 1);
                const uint4* kp = reinterpret_cast<const uint4*>(k_pool + (page * bs + slot) * kE4Row + kd);
                const uint4* vp = reinterpret_cast<const uint4*>(v_pool + (page * bs + slot) * kE4Row + kd);
                raw[0] = kp[0];
                raw[1] = kp[1];
                raw[2] = vp[0];
                raw[3] = vp[1];
                ks = e4m3_scale(kv_scale[2 * page * bs + slot]);
                vs = e4m3_scale(kv_scale[(2 * page + 1) * bs + slot]);
            } else {
                err |= kErrBounds;
            }
        }
    };
    auto request_rel = [&](int s, int buf) {   // table rows of the distances of keys 64 s .. and the queries
        for (int i = tid; i < (kFRel - 1) * 16; i += kFThreads) {
            const int r = i >> 4, d = 4 * (i & 15);
            const int rho = t.off + s * kFKeys - i0 - (kFRows - 1) + r;
            const bool on = rho >= 0 && rho < a.R;
            cp_async16(smem_addr(&sm.rel[buf][r][d]), rel + (static_cast<long long>(on ? rho : 0) * H + h) * kHeadDim + d, on);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[2][4] = {};
    if (t.st0 < t.st1) {
        request(t.st0);
        request_rel(t.st0, 0);
    }
    for (int s = t.st0; s < t.st1; ++s) {
        const int buf = (s - t.st0) & 1;
        __syncthreads();   // the previous tile has been read
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
            float* dst = (i < 2 ? sm.k : sm.v)[kr] + kd + 16 * (i & 1);
            const float sc = i < 2 ? ks : vs;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 lo = e4m3_unpack2(w[e]), hi = e4m3_unpack2(w[e] >> 16);
                *reinterpret_cast<float4*>(dst + 4 * e) = make_float4(lo.x * sc, lo.y * sc, hi.x * sc, hi.y * sc);
            }
        }
        if (s + 1 < t.st1) {
            request(s + 1);
            request_rel(s + 1, buf ^ 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncthreads();
        float sc[2][4] = {}, gc[2][5] = {};
#pragma unroll 4
        for (int d = 0; d < kHeadDim; d += 4) {
            const float4 q0 = *reinterpret_cast<const float4*>(&sm.qu[ty][d]), q1 = *reinterpret_cast<const float4*>(&sm.qu[ty + 8][d]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float4 kk = *reinterpret_cast<const float4*>(&sm.k[tx + 16 * c][d]);
                sc[0][c] = fmaf(q0.w, kk.w, fmaf(q0.z, kk.z, fmaf(q0.y, kk.y, fmaf(q0.x, kk.x, sc[0][c]))));
                sc[1][c] = fmaf(q1.w, kk.w, fmaf(q1.z, kk.z, fmaf(q1.y, kk.y, fmaf(q1.x, kk.x, sc[1][c]))));
            }
        }
#pragma unroll 4
        for (int d = 0; d < kHeadDim; d += 4) {
            const float4 q0 = *reinterpret_cast<const float4*>(&sm.qv[ty][d]), q1 = *reinterpret_cast<const float4*>(&sm.qv[ty + 8][d]);
#pragma unroll
            for (int c = 0; c < 5; ++c) {
                const float4 rr = *reinterpret_cast<const float4*>(&sm.rel[buf][tx + 16 * c][d]);
                gc[0][c] = fmaf(q0.w, rr.w, fmaf(q0.z, rr.z, fmaf(q0.y, rr.y, fmaf(q0.x, rr.x, gc[0][c]))));
                gc[1][c] = fmaf(q1.w, rr.w, fmaf(q1.z, rr.z, fmaf(q1.y, rr.y, fmaf(q1.x, rr.x, gc[1][c]))));
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int c = 0; c < 5; ++c) sm.g[ty + 8 * r][tx + 16 * c] = gc[r][c];
        __syncwarp();      // a row's 16 threads are half a warp
        const int left = t.K - s * kFKeys;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = ty + 8 * r;
            float mx = m[r];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int j = tx + 16 * c;
                sc[r][c] = j < left ? (sc[r][c] + sm.g[row][j + kFRows - 1 - row]) * a.scale : -INFINITY;
                mx = fmaxf(mx, sc[r][c]);
            }
#pragma unroll
            for (int x = 8; x; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
            const float base = mx == -INFINITY ? 0.f : mx;
            const float alpha = expf(m[r] - base);
            m[r] = mx;
            float sum = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float e = expf(sc[r][c] - base);
                sum += e;
                sm.p[row][tx + 16 * c] = e;
            }
            l[r] = fmaf(l[r], alpha, sum);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[r][e] *= alpha;
        }
        __syncwarp();
        float acc[2][4] = {};   // the tile's own sum, added to the running one once
#pragma unroll 4
        for (int j = 0; j < kFKeys; j += 4) {
            const float4 p0 = *reinterpret_cast<const float4*>(&sm.p[ty][j]), p1 = *reinterpret_cast<const float4*>(&sm.p[ty + 8][j]);
            const float w0[4] = {p0.x, p0.y, p0.z, p0.w}, w1[4] = {p1.x, p1.y, p1.z, p1.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 vv = *reinterpret_cast<const float4*>(&sm.v[j + e][4 * tx]);
                acc[0][0] = fmaf(w0[e], vv.x, acc[0][0]);
                acc[0][1] = fmaf(w0[e], vv.y, acc[0][1]);
                acc[0][2] = fmaf(w0[e], vv.z, acc[0][2]);
                acc[0][3] = fmaf(w0[e], vv.w, acc[0][3]);
                acc[1][0] = fmaf(w1[e], vv.x, acc[1][0]);
                acc[1][1] = fmaf(w1[e], vv.y, acc[1][1]);
                acc[1][2] = fmaf(w1[e], vv.z, acc[1][2]);
                acc[1][3] = fmaf(w1[e], vv.w, acc[1][3]);
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[r][e] += acc[r][e];
    }
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int x = 8; x; x >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], x);
    grid_dep_trigger();
    if (err) atomicOr(a.status, err);
    if (S == 1) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = i0 + ty + 8 * r;
            if (row < T)
                *reinterpret_cast<float4*>(out + ((static_cast<long long>(b) * T + row) * H + h) * kHeadDim + 4 * tx) =
                    make_float4(o[r][0] / l[r], o[r][1] / l[r], o[r][2] / l[r], o[r][3] / l[r]);
        }
        return;
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        *reinterpret_cast<float4*>(&sm.part_o[ty + 8 * r][4 * tx]) = make_float4(o[r][0], o[r][1], o[r][2], o[r][3]);
        if (tx == 0) {
            sm.part_m[ty + 8 * r] = m[r];
            sm.part_l[ty + 8 * r] = l[r];
        }
    }
    cluster_sync();
    // rows split, split + S, ... of the cluster's queries are finished here, a warp each
    const uint32_t po = smem_addr(&sm.part_o[0][0]), pm = smem_addr(&sm.part_m[0]), pl = smem_addr(&sm.part_l[0]);
    const int lane = tid & 31;
    for (int row = split + S * (tid >> 5); row < min(kFRows, T - i0); row += S * (kFThreads / 32)) {
        float mx = -INFINITY;
        for (int k = 0; k < S; ++k) mx = fmaxf(mx, ld_cluster(pm + 4 * row, k));
        float o0 = 0.f, o1 = 0.f, sum = 0.f;
        for (int k = 0; k < S; ++k) {
            const float mk = ld_cluster(pm + 4 * row, k);
            const float w = mk == -INFINITY ? 0.f : expf(mk - mx);   // a share without keys
            sum = fmaf(w, ld_cluster(pl + 4 * row, k), sum);
            o0 = fmaf(w, ld_cluster(po + 4 * (row * kHeadDim + 2 * lane), k), o0);
            o1 = fmaf(w, ld_cluster(po + 4 * (row * kHeadDim + 2 * lane + 1), k), o1);
        }
        reinterpret_cast<float2*>(out + ((static_cast<long long>(b) * T + i0 + row) * H + h) * kHeadDim)[lane] = make_float2(o0 / sum, o1 / sum);
    }
    cluster_sync();
}

// --------------------------------------------------------------------------- host

int g_smem_done_e4[4][64];
bool g_clusters_e4[4][64];

// Allow clusters of more than eight CTAs of `func`, once per device.
template <typename F>
bool ensure_clusters(F* func, bool (&done)[64])
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    if (!done[dev] && cudaFuncSetAttribute(reinterpret_cast<const void*>(func), cudaFuncAttributeNonPortableClusterSizeAllowed,
                                           1) != cudaSuccess)
        return false;
    done[dev] = true;
    return true;
}

constexpr int kMaxShares = 16;   // CTAs of a cluster (over the portable eight: enabled per kernel)

// Query tiles of Tp rows, and shares of the keys while the (stream, head, tile) triples leave half of the
// SMs idle and every share keeps two stages of the keys a well-formed stream can have; the number of triples.
long long e4_splits(E4Args& a, int B, int Tp, int k_max)
{
    a.q_tiles = (a.T + Tp - 1) / Tp;
    const long long pairs = static_cast<long long>(B) * a.H * a.q_tiles;
    const int stages = (k_max + kStageKeys - 1) / kStageKeys, sms = sm_count();
    a.splits = 1;
    while (a.splits < kMaxShares && pairs * a.splits * 2 <= sms && stages >= 2 * a.splits) a.splits *= 2;
    return pairs;
}

// first: enqueues what goes before the kernel, once nothing but the launch itself can fail.
template <int MT, int NS, int CTAS, bool FUSED, typename First>
oasr_status launch_e4(const void* q, const void* k_new, const void* v_new, const void* rel, E4Args& a, int k_max, int B,
                      int slot, cudaStream_t stream, First first)
{
    using SP = E4Smem<MT, NS, FUSED>;
    CUtensorMap tm_q, tm_k, tm_v, tm_r, tm_kn, tm_vn;
    const int box = a.block_size < kStageKeys ? a.block_size : kStageKeys;
    const long long rows = static_cast<long long>(a.num_blocks) * a.H * a.block_size, frames = static_cast<long long>(B) * a.T;
    if (!encode_rows_bf16(&tm_q, q, frames, a.H, SP::Tp) || !encode_rows_bf16(&tm_r, rel, a.R, a.H, kStageKeys) ||
        !encode_rows_e4m3(&tm_k, a.k_pool, rows, box) || !encode_rows_e4m3(&tm_v, a.v_pool, rows, box))
        return OASR_ERR_INVALID_ARG;
    tm_kn = tm_vn = tm_q;   // unused without the chunk
    if (FUSED && (!encode_rows_bf16(&tm_kn, k_new, frames, a.H, kChunkRows) ||
                  !encode_rows_bf16(&tm_vn, v_new, frames, a.H, kChunkRows)))
        return OASR_ERR_INVALID_ARG;
    auto kern = chunk_e4m3_kernel<MT, NS, CTAS, FUSED>;
    const int smem = SP::bytes + 2 * a.mbps * 4;
    if (!ensure_smem(kern, smem, g_smem_done_e4[slot]) || !ensure_clusters(kern, g_clusters_e4[slot])) return OASR_ERR_CUDA;
    const long long pairs = e4_splits(a, B, SP::Tp, k_max);
    a.items = static_cast<int>(pairs);
    a.B = B;
    const long long most = static_cast<long long>(CTAS) * sm_count();
    const long long ctas = a.splits > 1 ? pairs * a.splits : pairs < most ? pairs : most;
    a.sorted = a.splits == 1 && pairs > ctas && B <= kOrderMax;
    if (const oasr_status st = first(); st != OASR_OK) return st;
    return launch_pdl_cluster(kern, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), smem, a.splits, stream, tm_q, tm_k, tm_v,
                              tm_r, tm_kn, tm_vn, static_cast<const E4Args>(a));
}

template <bool FUSED>
oasr_status dispatch_e4(const void* q, const void* k_new, const void* v_new, void* k_pool, void* v_pool,
                        void* kv_scale, int num_blocks, int block_size, const int32_t* bt, int mbps,
                        const int32_t* cs, const void* u, const void* vb, const void* rel, int R, void* out, int B,
                        int T, int H, int D, float scale, oasr_dtype dt, cudaStream_t stream)
{
    if (!q || !k_pool || !v_pool || !kv_scale || !bt || !cs || !u || !vb || !rel || !out)
        return OASR_ERR_INVALID_ARG;
    if (FUSED && (!k_new || !v_new)) return OASR_ERR_INVALID_ARG;
    if (num_blocks <= 0 || block_size <= 0 || mbps <= 0 || R <= 0 || B <= 0 || T <= 0 || H <= 0 || D <= 0)
        return OASR_ERR_INVALID_ARG;
    if (dt != OASR_F32 && dt != OASR_BF16) return OASR_ERR_UNSUPPORTED;
    if (D != kHeadDim || T > kE4MaxT) return OASR_ERR_UNSUPPORTED;
    if (block_size < 8 || block_size > 256 || (block_size & (block_size - 1))) return OASR_ERR_UNSUPPORTED;
    if (mbps > kE4MaxPages) return OASR_ERR_UNSUPPORTED;
    // pool rows and query rows are 32-bit copy coordinates
    if (static_cast<long long>(num_blocks) * H > 0x7fffffffLL / block_size ||
        static_cast<long long>(B) * T > 0x7fffffffLL - 64 || static_cast<long long>(B) * H > 0x7fffffffLL)
        return OASR_ERR_UNSUPPORTED;
    const void* ptrs[] = {q, k_pool, v_pool, kv_scale, u, vb, rel, out, FUSED ? k_new : q, FUSED ? v_new : q};
    for (const void* p : ptrs)
        if (!aligned16(p)) return OASR_ERR_INVALID_ARG;
    // (stream, head, query tile) items are 32-bit numbers; fp32 has a CTA for each
    const int Tp = dt == OASR_F32 || T <= 16 ? 16 : 32;
    if (static_cast<long long>(B) * H * ((T + Tp - 1) / Tp) > (dt == OASR_F32 ? 0x7fffffffLL : 0x7fffffffLL / 2))
        return OASR_ERR_UNSUPPORTED;
    unsigned* status = status_word();
    if (!status || !sm_count()) return OASR_ERR_CUDA;
    // more than one m-tile of queries (and fp32): the append first, then the attention over the pool
    auto append = [&] {
        if (!FUSED || (dt == OASR_BF16 && T <= 16)) return OASR_OK;
        return oasr_paged_append_e4m3(k_new, v_new, k_pool, v_pool, kv_scale, num_blocks, block_size, bt, mbps, cs, B, T,
                                      H, D, dt, stream);
    };
    E4Args a = {};
    a.k_pool = static_cast<uint8_t*>(k_pool);
    a.v_pool = static_cast<uint8_t*>(v_pool);
    a.kv_scale = static_cast<uint8_t*>(kv_scale);
    a.block_table = bt;
    a.cache_seqlens = cs;
    a.pos_bias_u = static_cast<const uint16_t*>(u);
    a.pos_bias_v = static_cast<const uint16_t*>(vb);
    a.out = static_cast<uint16_t*>(out);
    a.status = status;
    a.num_blocks = num_blocks;
    a.block_size = block_size;
    a.bs_shift = __builtin_ctz(static_cast<unsigned>(block_size));
    a.mbps = mbps;
    a.T = T;
    a.H = H;
    a.R = R;
    a.scale = scale;
    a.scale_log2 = scale * 1.4426950408889634f;
    // keys a well-formed stream of the call can have
    const long long pages = static_cast<long long>(mbps) * block_size, dist = static_cast<long long>(R) - T + 1;
    const long long k_max = pages < dist ? pages : dist;
    const int km = static_cast<int>(k_max < T ? T : k_max);
    if (dt == OASR_F32) {
        const long long pairs = e4_splits(a, B, kFRows, km);
        if (!ensure_smem(chunk_e4m3_f32_kernel, sizeof(F32Smem), g_smem_done_e4[3]) ||
            !ensure_clusters(chunk_e4m3_f32_kernel, g_clusters_e4[3]))
            return OASR_ERR_CUDA;
        if (const oasr_status st = append(); st != OASR_OK) return st;
        return launch_pdl_cluster(chunk_e4m3_f32_kernel, dim3(static_cast<unsigned>(pairs * a.splits)), dim3(kFThreads),
                                  static_cast<int>(sizeof(F32Smem)), a.splits, stream, static_cast<const float*>(q),
                                  static_cast<const uint8_t*>(a.k_pool), static_cast<const uint8_t*>(a.v_pool),
                                  static_cast<const uint8_t*>(a.kv_scale), static_cast<const float*>(u),
                                  static_cast<const float*>(vb), static_cast<const float*>(rel), static_cast<float*>(out),
                                  static_cast<const E4Args>(a));
    }
    // 32 queries a CTA convert each key once for both m-tiles, and two CTAs fit an SM's registers: 76 streams of 64
    // queries over 960 keys take 102 us, 112 with tiles of 16 (three CTAs), 108 with three CTAs and spills
    if (T <= 16) return launch_e4<1, kSlots, 3, FUSED>(q, k_new, v_new, rel, a, km, B, FUSED ? 1 : 0, stream, append);
    return launch_e4<2, kSlots, 2, false>(q, k_new, v_new, rel, a, km, B, 2, stream, append);
}

}  // namespace
}  // namespace oasr

extern "C" oasr_status oasr_chunk_relattn_paged_e4m3(
    const void* q, const void* k_pool, const void* v_pool, const void* kv_scale, int num_blocks, int block_size,
    const int32_t* block_table, int max_blocks_per_seq, const int32_t* cache_seqlens, const void* pos_bias_u,
    const void* pos_bias_v, const void* rel, int R, void* out, int B, int T, int H, int D, float scale,
    oasr_dtype dt, cudaStream_t stream)
{
    return oasr::dispatch_e4<false>(q, nullptr, nullptr, const_cast<void*>(k_pool), const_cast<void*>(v_pool),
                                    const_cast<void*>(kv_scale), num_blocks, block_size, block_table,
                                    max_blocks_per_seq, cache_seqlens, pos_bias_u, pos_bias_v, rel, R, out, B, T, H,
                                    D, scale, dt, stream);
}

extern "C" oasr_status oasr_chunk_step_paged_e4m3(
    const void* q, const void* k_new, const void* v_new, void* k_pool, void* v_pool, void* kv_scale, int num_blocks,
    int block_size, const int32_t* block_table, int max_blocks_per_seq, const int32_t* cache_seqlens,
    const void* pos_bias_u, const void* pos_bias_v, const void* rel, int R, void* out, int B, int T, int H, int D,
    float scale, oasr_dtype dt, cudaStream_t stream)
{
    return oasr::dispatch_e4<true>(q, k_new, v_new, k_pool, v_pool, kv_scale, num_blocks, block_size, block_table,
                                   max_blocks_per_seq, cache_seqlens, pos_bias_u, pos_bias_v, rel, R, out, B, T, H, D,
                                   scale, dt, stream);
}
