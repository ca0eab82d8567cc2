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
// exact.  k8 and v8 go into fp16 matrix instructions: e4m3's exponent and fraction, shifted into an
// fp16's, are the value times 2^-8, subnormals included, for three or four integer instructions per
// two values.  fp16 holds q + u (each query row scaled by a power of two) and the weights with three
// bits more than bf16 would: rms error against 64 bits 0.0021 of the output's on random data, 0.0031
// with bf16 (0.0017 is the rounding of the output itself).
//
// One CTA per (stream, head, block of up to 32 queries, share of the keys): four consumer warps and
// a producer warp.  The producer brings stages of 64 keys by TMA (a box of K and one of V per page,
// 64-byte rows, 64-byte swizzle, and one bulk copy of the page's scales) into a ring; consumer warp
// w takes keys 16w .. 16w+15 of each stage for all the CTA's queries.  The position term is computed
// per segment of the keys into a pre-skewed bf16 table (PosTable, attn_core.cuh), so its shared
// memory does not grow with the history.  The chunk itself never comes through the pool: the
// consumer warps quantise it from k_new / v_new into a region of its own, from which it is attended
// to, and store the same bytes into the pool.
//
// When the (stream, head) pairs are too few to fill the GPU the keys of each are divided over a
// cluster of up to eight CTAs, whose partial sums meet through distributed shared memory.
#include "attn_core.cuh"
#include "e4m3.cuh"
#include "host_common.h"
#include "tcgen05.cuh"

namespace oasr {

namespace {

#ifndef E4NS
#define E4NS 3
#define E4CTAS 5
#define E4SEG 2
#define E4NW 2
#define E4NS2 4
#define E4CTAS2 3
#define E4SEG2 2
#define E4NW2 2
#endif
constexpr int kE4MaxPages = 512;              // block-table entries a CTA caches
constexpr int kE4Stage = 2 * kStageKeys * kE4Row;   // K and V rows of a stage
constexpr int kE4MaxT = 64;
constexpr int kMaxRowExp = 120;
constexpr float kNoMax = -3.0e38f;   // the running maximum before any key

struct E4Args {
    const __nv_bfloat16* k_new;   // fused only
    const __nv_bfloat16* v_new;   // fused only
    uint8_t* k_pool;
    uint8_t* v_pool;
    uint8_t* kv_scale;
    const int32_t* block_table;
    const int32_t* cache_seqlens;
    const uint16_t* pos_bias_u;
    const uint16_t* pos_bias_v;
    const uint16_t* rel;
    uint16_t* out;
    unsigned* status;
    int num_blocks, block_size, bs_shift, mbps, T, H, R;
    int q_tiles, splits;
    int seg;          // stages per segment of the position table
    int gt_w;         // row stride of the table (bf16 elements)
    float scale_log2; // scale * log2(e)
};

// Shared memory (byte offsets from a 1024-aligned base).  The ring's rows are reused by the
// combine once the key loop is over.
template <int MT, int NW, int NS>
struct E4Smem {
    static constexpr int Tp = 16 * MT;
    static constexpr int Tc = 16;                                     // rows of the chunk region (one m-tile)
    static constexpr int off_q = NS * kE4Stage;                       // q, then bf16((q + v) 2^-x)
    static constexpr int off_qu = off_q + Tp * kRowBytes;             // fp16((q + u) 2^-x)
    static constexpr int off_ck = off_qu + Tp * kRowBytes;            // the chunk's K and V rows
    static constexpr int off_sc = off_ck + 2 * Tc * kE4Row;           // scales [NS][2 * 64]
    static constexpr int off_csc = off_sc + NS * 2 * kStageKeys;      // the chunk's [2][Tc]
    static constexpr int off_re = off_csc + 2 * Tc;                   // 2^x of the query rows
    static constexpr int off_bt = off_re + Tp * 4;
    static constexpr int off_bar = off_bt + kE4MaxPages * 4;          // full[NS], empty[NS], q
    static constexpr int off_gt = (off_bar + (2 * NS + 1) * 8 + 15) & ~15;
    static constexpr int bytes = off_gt + 1024;                       // + Tp * gt_w * 2
    // combine: the warps' partials, then the CTA's own for its cluster
    static constexpr int comb_o = 0;
    static constexpr int comb_m = comb_o + NW * Tp * kOW * 4;
    static constexpr int comb_l = comb_m + NW * Tp * 4;
    static constexpr int part_o = comb_l + NW * Tp * 4;
    static constexpr int part_m = part_o + Tp * kHeadDim * 4;
    static constexpr int part_l = part_m + Tp * 4;
    static_assert(part_l + Tp * 4 <= NS * kE4Stage, "combine area");
    static_assert(off_q % 1024 == 0 && off_ck % 1024 == 0 && off_sc % 16 == 0, "TMA alignment");
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
__device__ __forceinline__ void load_slice(E4Slice& x, uint32_t k_s, uint32_t v_s, const uint8_t* sc, int far_off,
                                           int v_off, int lane)
{
    const int g4 = lane >> 2, t4 = lane & 3;
#pragma unroll
    for (int n = 0; n < 2; ++n)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x.k[n].x), "=r"(x.k[n].y), "=r"(x.k[n].z), "=r"(x.k[n].w)
                     : "r"(k_s + swz_key(4 * (g4 >> 1) + 2 * n + (g4 & 1), t4)));
#pragma unroll
    for (int dp = 0; dp < 2; ++dp)
        ldsm8_x2_t(v_s + swz_key(lane & 15, 2 * dp + (lane >> 4)), x.v[4 * dp], x.v[4 * dp + 1], x.v[4 * dp + 2], x.v[4 * dp + 3]);
    const uint8_t* p = sc + 4 * (t4 & 1) + (t4 >> 1) * far_off;
    x.ks = *reinterpret_cast<const uint32_t*>(p);
    x.vs = *reinterpret_cast<const uint32_t*>(p + v_off);
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Eight dims (chunk l8) of one query row, by eight neighbouring lanes: bf16(q + v) over q's own place in
// the swizzled tile and fp16(q + u) into qu, both times the power of two that brings the row's largest
// |q + u| into [1, 2), and its inverse into row_pow.  u, v: the head's biases.
__device__ __forceinline__ void prepare_row(uint8_t* q_tile, uint8_t* qu, float* row_pow, const uint16_t* u,
                                            const uint16_t* v, int row, int l8)
{
    const uint4 qw = *reinterpret_cast<const uint4*>(q_tile + swz128(row, l8));
    const uint4 uw = __ldg(reinterpret_cast<const uint4*>(u) + l8), vw = __ldg(reinterpret_cast<const uint4*>(v) + l8);
    const uint32_t q[4] = {qw.x, qw.y, qw.z, qw.w}, un[4] = {uw.x, uw.y, uw.z, uw.w}, vn[4] = {vw.x, vw.y, vw.z, vw.w};
    float a[8];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[2 * i] = bf16_lo(q[i]) + bf16_lo(un[i]);
        a[2 * i + 1] = bf16_hi(q[i]) + bf16_hi(un[i]);
        m = fmax3(m, fabsf(a[2 * i]), fabsf(a[2 * i + 1]));
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const int x = max(-kMaxRowExp, min(kMaxRowExp, static_cast<int>(__float_as_uint(m) >> 23) - 127));
    const float f = pow2(-x);
    uint32_t pu[4], pv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        pu[i] = pack_f16(a[2 * i] * f, a[2 * i + 1] * f);
        pv[i] = pack_bf16((bf16_lo(q[i]) + bf16_lo(vn[i])) * f, (bf16_hi(q[i]) + bf16_hi(vn[i])) * f);
    }
    *reinterpret_cast<uint4*>(qu + swz128(row, l8)) = make_uint4(pu[0], pu[1], pu[2], pu[3]);
    *reinterpret_cast<uint4*>(q_tile + swz128(row, l8)) = make_uint4(pv[0], pv[1], pv[2], pv[3]);
    if (l8 == 0) row_pow[row] = pow2(x);
}

// A fragments of 16 rows of a prepared tile, the head dimension in the order of the e4m3 words: quad
// position t4 holds dims 16 t4 .., k-step ks the dims 4 ks .. 4 ks + 3 of them.
__device__ __forceinline__ void load_a(uint32_t (&f)[4][4], const uint8_t* tile, int mt, int lane)
{
    const int g4 = lane >> 2, t4 = lane & 3;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int row = 16 * mt + g4 + 8 * half;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint4 w = *reinterpret_cast<const uint4*>(tile + swz128(row, 2 * t4 + c));
            f[2 * c][half] = w.x;
            f[2 * c][half + 2] = w.y;
            f[2 * c + 1][half] = w.z;
            f[2 * c + 1][half + 2] = w.w;
        }
    }
}

// A warp's column tiles of the position table (PosTable in attn_core.cuh; each row times its 2^-x): the CTA's
// Tp query rows (qa: bf16((q + v) 2^-x)) against every NW-th eight of the 64 rel rows in the ring slot `rows`
// (128-byte swizzled), table columns col0 ...  G[i][c] goes to gs[i * W + c + i + 1], so that query i and the
// segment's key j read gs[i * W + j + Tp].  Every lane arrives on release_bar once it has read its rows.
template <int MT, int NW>
__device__ __forceinline__ void table_tiles(uint16_t* gs, int W, const uint32_t (&qa)[MT][4][4], const uint8_t* rows,
                                            int col0, int ntiles, int warp, int lane, uint32_t release_bar)
{
    const int g4 = lane >> 2, t4 = lane & 3;
    constexpr int N = 8 / NW;
    uint4 bl[N], bh[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const int r = 8 * (warp + NW * u) + g4;
        bl[u] = *reinterpret_cast<const uint4*>(rows + swz128(r, 2 * t4));
        bh[u] = *reinterpret_cast<const uint4*>(rows + swz128(r, 2 * t4 + 1));
    }
    mbar_arrive_release(release_bar);
#pragma unroll
    for (int u = 0; u < N; ++u) {
        if (warp + NW * u >= ntiles) break;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            float c[4];
            mma_bf16_first(c, qa[mt][0], bl[u].x, bl[u].y);
            mma_bf16_16816(c, qa[mt][1], bl[u].z, bl[u].w);
            mma_bf16_16816(c, qa[mt][2], bh[u].x, bh[u].y);
            mma_bf16_16816(c, qa[mt][3], bh[u].z, bh[u].w);
            // columns past the last stay within their row (its stride leaves room for a tile)
            uint16_t* d = gs + (16 * mt + g4) * (W + 1) + 1 + 2 * t4 + col0 + 8 * (warp + NW * u);
            const uint32_t w0 = pack_bf16(c[0], c[1]), w1 = pack_bf16(c[2], c[3]);
            d[0] = static_cast<uint16_t>(w0);
            d[1] = static_cast<uint16_t>(w0 >> 16);
            d[8 * W + 8] = static_cast<uint16_t>(w1);
            d[8 * W + 9] = static_cast<uint16_t>(w1 >> 16);
        }
    }
}

// Running state of 16 query rows of one warp.  With t_ij = s_ij + ev_j (log2 units: the size of key j's
// contribution to the output), m is the running maximum of t, o the sum of 2^(t - m) v8 and l the
// sum of 2^(s - m + E), where E is within 7 of the largest V scale exponent so far.
struct E4Acc {
    float o[8][4];   // o[d]: dims 8 d + 2 t4, 8 d + 2 t4 + 1 of row g4, then of row g4 + 8
    float m[2], l[2];
};

// One warp, 16 MT query rows against one slice.  gq: the position table at the slice's first key
// (key jl of query row i reads gq[i * W + jl], aligned: eight bytes at a time); keys [0, kvalid) of the slice exist; sc: scale * log2(e) * 2^x of
// rows g4 and g4 + 8 of each m-tile.
//
// P is 2^(t - m), at most one, and goes into the product as fp16: its rounding is 2^-11 of each
// weight and never more than 2^-25 of the row's largest contribution, whatever the scales.  The
// row sum takes p back out of it, l += P 2^(E - ev); a slice with a scale below 2^(E - 40) (a row of
// zeros has 2^-100), where that could underflow, sums 2^(s - m + E) of its own.
template <int MT>
__device__ __forceinline__ void slice_e4m3(E4Acc (&acc)[MT], const uint32_t (&qu)[MT][4][4], E4Slice& x,
                                           const uint16_t* gq, int W, bool aligned, int kvalid,
                                           const float (&sc)[MT][2], int& E, int lane)
{
    const int g4 = lane >> 2, t4 = lane & 3;
    float s[MT][2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const uint32_t w[4] = {x.k[n].x, x.k[n].y, x.k[n].z, x.k[n].w};
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            uint32_t b0, b1;
            e4m3_to_f16(w[ks], b0, b1);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if (ks == 0)
                    mma_f16_first(s[mt][n], qu[mt][ks], b0, b1);
                else
                    mma_f16_16816(s[mt][n], qu[mt][ks], b0, b1);
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
    // keys 4 t4 ..: 2^ek, ev and 2^(E - ev), from the scale bytes in place
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
    float ks[4], ev[4], back[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        ks[e] = __uint_as_float(__byte_perm(x.ks, 0u, 0x0444 | (e << 12)) >> 1);
        const uint32_t w = __byte_perm(x.vs, 0x4b000000u, 0x7440 | e);
        ev[e] = __uint_as_float(w) - 8388735.f;                    // 2^23 + 127
        back[e] = __uint_as_float(static_cast<uint32_t>(E + 254) * 0x00800000u - w * 0x00800000u);
    }
    uint32_t pa[MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        E4Acc& a = acc[mt];
        float mx0 = a.m[0], mx1 = a.m[1];
        const uint16_t* r0 = gq + (16 * mt + g4) * W + 4 * t4;
        const uint16_t* r1 = r0 + 8 * W;
        uint32_t y0[2], y1[2];
        if (aligned) {
            const uint2 p0 = *reinterpret_cast<const uint2*>(r0), p1 = *reinterpret_cast<const uint2*>(r1);
            y0[0] = p0.x; y0[1] = p0.y;
            y1[0] = p1.x; y1[1] = p1.y;
        } else {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                y0[n] = r0[2 * n] | static_cast<uint32_t>(r0[2 * n + 1]) << 16;
                y1[n] = r1[2 * n] | static_cast<uint32_t>(r1[2 * n + 1]) << 16;
            }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const float gb[4] = {bf16_lo(y0[n]), bf16_hi(y0[n]), bf16_lo(y1[n]), bf16_hi(y1[n])};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int k = 2 * n + (e & 1);
                s[mt][n][e] = fmaf(fmaf(s[mt][n][e], ks[k], gb[e]), sc[mt][e >> 1], ev[k]);
                if (tail && 4 * t4 + k >= kvalid) s[mt][n][e] = -INFINITY;
            }
            mx0 = fmax3(mx0, s[mt][n][0], s[mt][n][1]);
            mx1 = fmax3(mx1, s[mt][n][2], s[mt][n][3]);
        }
        // the reference only moves when a weight would pass 2^8 (fp16 holds 2^15)
        if (__any_sync(0xffffffffu, mx0 > a.m[0] + 8.f || mx1 > a.m[1] + 8.f) || dE != 0.f) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
            const float d0 = a.m[0] - mx0, d1 = a.m[1] - mx1;
            const float alpha0 = ex2_approx(d0), alpha1 = ex2_approx(d1);
            a.l[0] *= ex2_approx(fminf(d0 + dE, 126.f));
            a.l[1] *= ex2_approx(fminf(d1 + dE, 126.f));
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
            const float off = static_cast<float>(E);
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int k = 2 * n + e;
                    a.l[0] += ex2_approx(s[mt][n][e] - ev[k] - base0 + off);
                    a.l[1] += ex2_approx(s[mt][n][2 + e] - ev[k] - base1 + off);
                    back[k] = 0.f;
                }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            s[mt][n][0] = ex2_approx(s[mt][n][0] - base0);
            s[mt][n][1] = ex2_approx(s[mt][n][1] - base0);
            s[mt][n][2] = ex2_approx(s[mt][n][2] - base1);
            s[mt][n][3] = ex2_approx(s[mt][n][3] - base1);
            a.l[0] = fmaf(s[mt][n][0], back[2 * n], fmaf(s[mt][n][1], back[2 * n + 1], a.l[0]));
            a.l[1] = fmaf(s[mt][n][2], back[2 * n], fmaf(s[mt][n][3], back[2 * n + 1], a.l[1]));
            pa[mt][2 * n] = pack_f16(s[mt][n][0], s[mt][n][1]);
            pa[mt][2 * n + 1] = pack_f16(s[mt][n][2], s[mt][n][3]);
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
// Shares of a row are joined from o, m and lambda = log2(sum of 2^s) = m - E + log2(l): the V scales
// move m away from the scores (a share of zero rows has an m of s - 100), so the row sum has a
// maximum of its own.  out = sum(o 2^(m - m*)) 2^(m* - lambda*) / sum(2^(lambda - lambda*)).
__device__ __forceinline__ float part_weight(float x, float top) { return x <= kNoMax ? 0.f : ex2_approx(x - top); }

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

template <int MT, int NW, int NS, int CTAS, bool FUSED>
__global__ void __launch_bounds__(32 * (NW + 1), CTAS) chunk_e4m3_kernel(
    const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_r, const E4Args a)
{
    static_assert(!FUSED || MT == 1, "the chunk region holds one m-tile's rows");
    using SP = E4Smem<MT, NW, NS>;
    constexpr int Tp = SP::Tp, kCons = 32 * NW;   // consumer threads
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_addr(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = a.splits, T = a.T, H = a.H;
    int idx = blockIdx.x;
    const int split = idx % S;
    idx /= S;
    const int qt = idx % a.q_tiles;
    idx /= a.q_tiles;
    const int b = idx / H, h = idx - b * H;
    const int i0 = qt * Tp;                       // the CTA's first query
    const int Tq = min(Tp, T - i0);               // its queries
    unsigned err = 0;
    const bool producer = warp == NW;
    if (producer && lane == 0) {
        prefetch_tensormap(&tm_q);
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
        prefetch_tensormap(&tm_r);
    }
    grid_dep_wait();
    const uint32_t bar_full = sb + SP::off_bar;
    const uint32_t bar_empty = bar_full + NS * 8;
    const uint32_t bar_q = bar_empty + NS * 8;
    float* s_pow = reinterpret_cast<float*>(sm + SP::off_re);
    int* s_bt = reinterpret_cast<int*>(sm + SP::off_bt);
    __shared__ int s_failed;

    int C = __ldg(a.cache_seqlens + b);
    // consumers: the thread's chunk rows (eight lanes each), requested first of all
    constexpr int kRounds = 32 / (4 * NW);
    uint4 pre[kRounds] = {};
    if (FUSED && !producer && split == S - 1) {
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            const int r = (tid >> 3) + 4 * NW * i, t = r & 15;
            if (t < T)
                pre[i] = __ldg(reinterpret_cast<const uint4*>(
                    (r >= 16 ? a.v_new : a.k_new) + ((static_cast<long long>(b) * T + t) * H + h) * kE4Row) + (lane & 7));
        }
    }
    if (producer) {
        const int32_t* bt_row = a.block_table + static_cast<long long>(b) * a.mbps;
        constexpr int kRowRegs = 4;
        int row[kRowRegs];
#pragma unroll
        for (int k = 0; k < kRowRegs; ++k)
            if (lane + 32 * k < a.mbps) row[k] = __ldg(bt_row + lane + 32 * k);
        if (lane == 0) {
            for (int i = 0; i < NS; ++i) {
                mbar_init(bar_full + 8 * i, 1);
                mbar_init(bar_empty + 8 * i, kCons);
            }
            mbar_init(bar_q, 1);
            fence_mbar_init();
            s_failed = 0;
            mbar_arrive_expect_tx(bar_q, Tp * kRowBytes);
            tma_load_3d(sb + SP::off_q, &tm_q, bar_q, 0, h, b * T + i0);
        }
#pragma unroll
        for (int k = 0; k < kRowRegs; ++k)
            if (lane + 32 * k < a.mbps) s_bt[lane + 32 * k] = row[k];
        for (int i = lane + 32 * kRowRegs; i < a.mbps; i += 32) s_bt[i] = __ldg(bt_row + i);
        __syncwarp();
        named_bar_arrive(2, kCons + 32);
    } else {
        named_bar_sync(2, kCons + 32);
    }
    if (C < 0) { C = 0; err |= kErrBounds; }
    const int sh = a.bs_shift, bs = a.block_size;
    const int cap = a.mbps << sh;                 // keys the table's pages hold (at most 2^17)
    if (C > cap) { C = cap; err |= kErrBounds; }
    int K = C + T;
    if (K > cap) { K = cap; err |= kErrBounds; }
    if (C + 2 * T - 1 > a.R) err |= kErrBounds;   // distances the rel table does not hold
    const int off = a.R - T - C;                  // rel row of query i and key j: off + j - i
    const int kc = FUSED ? C : K;       // keys that come from the pool
    const int n_all = (kc + kStageKeys - 1) / kStageKeys;
    const int st0 = static_cast<int>(static_cast<long long>(n_all) * split / S);
    const int st1 = static_cast<int>(static_cast<long long>(n_all) * (split + 1) / S);
    const bool chunk_here = FUSED && split == S - 1;   // the chunk follows the last pool keys
    const int nc = chunk_here ? K - kc : 0;            // its keys (fewer when it runs past the table)
    const int box = min(bs, kStageKeys), box_sh = min(sh, 6);
    // keys of the segment of stages [seg0, seg1): the last one of the last split has the chunk's too
    auto segment_keys = [&](int seg0, int seg1) {
        return max(0, ((seg1 >= st1 && chunk_here) ? K : min(seg1 * kStageKeys, kc)) - seg0 * kStageKeys);
    };
    // its position table has a column for each distance: rel rows rho0 .., in ring slots of 64 rows
    auto segment_rel = [&](int nkeys) { return nkeys ? (nkeys + Tp - 1 + 63) >> 6 : 0; };

    if (producer) {
        const uint64_t pol = policy_evict_first();
        int n_issued = 0;
        bool ok = true;
        for (int seg0 = st0;;) {
            const int seg1 = min(seg0 + a.seg, st1);
            const int nrel = segment_rel(segment_keys(seg0, seg1));
            for (int r = 0; r < nrel && ok; ++r) {
                const int it = n_issued, slot = it % NS;
                ok = __all_sync(0xffffffffu, it < NS || e4_wait(bar_empty + 8 * slot, ((it / NS) - 1) & 1));
                if (!ok) break;
                if (lane == 0) {
                    const uint32_t bar = bar_full + 8 * slot;
                    mbar_arrive_expect_tx(bar, kE4Stage);
                    tma_load_3d(sb + slot * kE4Stage, &tm_r, bar, 0, h, off + (seg0 + r) * kStageKeys - i0 - (Tp - 1));
                }
                ++n_issued;
            }
            for (int s = seg0; s < seg1 && ok; ++s) {
            const int it = n_issued, slot = it % NS;
            ok = __all_sync(0xffffffffu, it < NS || e4_wait(bar_empty + 8 * slot, ((it / NS) - 1) & 1));
            if (!ok) break;
            const uint32_t bar = bar_full + 8 * slot;
            const int j0 = s * kStageKeys;
            const int nbox = min(kStageKeys >> box_sh, (kc - j0 + box - 1) >> box_sh);
            // lane q: K box of page piece q and its scales, lane 16 + q: its V box
            const int q = lane & 15;
            const int j = j0 + q * box;
            const int blk = q < nbox ? s_bt[j >> sh] : -1;
            const bool valid = blk >= 0 && blk < a.num_blocks;
            const uint32_t sc_dst = sb + SP::off_sc + slot * 2 * kStageKeys + q * 2 * box;
            if (q < nbox && !valid) {   // no such block: its rows read as zeros, with scales of zero
                err |= kErrBounds;
                if (lane < 16) {
                    for (int i = 0; i < box / 2; ++i)
                        *reinterpret_cast<uint32_t*>(sm + (sc_dst - sb) + 4 * i) = 0u;
                    fence_proxy_async_smem();
                }
            }
            const int nvalid = __popc(__ballot_sync(0xffffffffu, valid) & 0xffffu);
            if (lane == 0)
                mbar_arrive_expect_tx(bar, static_cast<uint32_t>(nbox * box * 2 * kE4Row + nvalid * 2 * box));
            __syncwarp();
            if (q < nbox) {
                const int in_page = j & (bs - 1);
                const long long page = static_cast<long long>(valid ? blk : 0) * H + h;
                // an invalid block's box lies outside the pool and reads zeros
                const int line = valid ? static_cast<int>((page * bs + in_page) >> 1) : -2 * box;
                const uint32_t dst = sb + slot * kE4Stage + q * box * kE4Row;
                if (lane < 16) {
                    tma_load_2d_hint(dst, &tm_k, bar, 0, line, pol);
                    if (valid) {
                        const uint8_t* src = a.kv_scale + 2 * page * bs + in_page;
                        if (bs <= kStageKeys) {
                            bulk_load(sc_dst, src, 2 * box, bar);   // K and V scales of the page are adjacent
                        } else {
                            bulk_load(sc_dst, src, box, bar);
                            bulk_load(sc_dst + box, src + bs, box, bar);
                        }
                    }
                } else {
                    tma_load_2d_hint(dst + kStageKeys * kE4Row, &tm_v, bar, 0, line, pol);
                }
            }
            ++n_issued;
            }
            seg0 = seg1;
            if (seg0 >= st1 || !ok) break;
        }
        if (!ok) err |= kErrTimeout;
        // every copy this CTA requested lands before it ends
        for (int x = n_issued > NS ? n_issued - NS : 0; x < n_issued; ++x)
            if (!mbar_wait_idle(bar_full + 8 * (x % NS), (x / NS) & 1)) err |= kErrTimeout;
        if (!mbar_wait_idle(bar_q, 0)) err |= kErrTimeout;
        if (err) atomicOr(a.status, err);
        if (S > 1) {
            cluster_sync();
            cluster_sync();
        }
        return;
    }

    // ---------------------------------------------------------------- consumers
    bool failed = false;
    uint16_t* gs = reinterpret_cast<uint16_t*>(sm + SP::off_gt);
    const int W = a.gt_w;
    if (FUSED && chunk_here) {
        // the chunk's rows: quantised into the chunk region (rows past T zero) and, by the first
        // query tile, into the pool.  Eight lanes per row.
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            const int r = (tid >> 3) + 4 * NW * i, kv = r >= 16, t = r & 15, l8 = lane & 7;
            uint2 q = make_uint2(0u, 0u);
            uint32_t byte = 0;
            if (t < nc) {
                float x[8];
                unpack8(pre[i], x);
                byte = e4m3_quantise8(x, 0xffu << (lane & 24), q);
                const int p = C + t;
                const int blk = s_bt[p >> sh];
                if (blk < 0 || blk >= a.num_blocks) {   // dropped by the append: reads as zeros
                    err |= kErrBounds;
                    q = make_uint2(0u, 0u);
                    byte = 0;
                } else if (qt == 0) {
                    const int slot = p & (bs - 1);
                    const long long page = static_cast<long long>(blk) * H + h;
                    *reinterpret_cast<uint2*>((kv ? a.v_pool : a.k_pool) + (page * bs + slot) * kE4Row + 8 * l8) = q;
                    if (l8 == 0) a.kv_scale[(2 * page + kv) * bs + slot] = static_cast<uint8_t>(byte);
                }
            }
            *reinterpret_cast<uint2*>(sm + SP::off_ck + kv * SP::Tc * kE4Row + swz_key(t, l8 >> 1) + 8 * (l8 & 1)) = q;
            if (l8 == 0) sm[SP::off_csc + kv * SP::Tc + t] = static_cast<uint8_t>(byte);
        }
    }
    if (!e4_wait(bar_q, 0)) failed = true;
#pragma unroll
    for (int r = 0; r < Tp; r += 4 * NW)
        prepare_row(sm + SP::off_q, sm + SP::off_qu, s_pow, a.pos_bias_u + h * kHeadDim, a.pos_bias_v + h * kHeadDim,
                    r + (tid >> 3), lane & 7);
    named_bar_sync(1, kCons);   // the query tiles and the chunk region are complete
    // this warp's keys of a stage: 16 from each of 16 (warp + NW u)
    const int far_off = box == 8 ? 16 : 8;   // scales of keys 8 .. 15 of a slice, from those of keys 0 .. 7
    auto scale_off = [&](int jl) { return ((jl >> box_sh) << (box_sh + 1)) + (jl & (box - 1)); };
    E4Acc acc[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int d = 0; d < 8; ++d) acc[mt].o[d][0] = acc[mt].o[d][1] = acc[mt].o[d][2] = acc[mt].o[d][3] = 0.f;
        acc[mt].m[0] = acc[mt].m[1] = kNoMax;
        acc[mt].l[0] = acc[mt].l[1] = 0.f;
    }
    int E = -127;   // the smallest a scale byte says; the first keys raise it
    int it = 0;   // ring slots read
#pragma unroll 1
    for (int seg0 = st0;; seg0 += a.seg) {
        const int seg1 = min(seg0 + a.seg, st1);
        const bool last = seg1 >= st1;
        const int jbase = seg0 * kStageKeys;
        const int nkeys = segment_keys(seg0, seg1);
        if (nkeys) {
            uint32_t qa[MT][4][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) load_a(qa[mt], sm + SP::off_q, mt, lane);
            const int ntiles = (nkeys + Tp - 1 + 7) >> 3, nrel = segment_rel(nkeys);
#pragma unroll 1
            for (int r = 0; r < nrel; ++r, ++it) {
                const int slot = it % NS;
                if (failed || !e4_wait(bar_full + 8 * slot, (it / NS) & 1)) { failed = true; break; }
                table_tiles<MT, NW>(gs, W, qa, sm + slot * kE4Stage, 64 * r, ntiles - 8 * r, warp, lane,
                                bar_empty + 8 * slot);
            }
            named_bar_sync(1, kCons);   // the table is complete
        }
        uint32_t qu[MT][4][4];
        float sc[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            load_a(qu[mt], sm + SP::off_qu, mt, lane);
            sc[mt][0] = a.scale_log2 * s_pow[16 * mt + (lane >> 2)];
            sc[mt][1] = a.scale_log2 * s_pow[16 * mt + (lane >> 2) + 8];
        }
#pragma unroll 1
        for (int s = seg0; s < seg1; ++s, ++it) {
            const int slot = it % NS;
            if (failed || !e4_wait(bar_full + 8 * slot, (it / NS) & 1)) { failed = true; break; }
            constexpr int N = 4 / NW;
            const int kv = min(kc - s * kStageKeys, kStageKeys);
            E4Slice x[N];
#pragma unroll
            for (int u = 0; u < N; ++u) {
                const int jl = 16 * (warp + NW * u);
                if (kv > jl)
                    load_slice(x[u], sb + slot * kE4Stage + jl * kE4Row, sb + slot * kE4Stage + (kStageKeys + jl) * kE4Row,
                               sm + SP::off_sc + slot * 2 * kStageKeys + scale_off(jl), far_off, box, lane);
            }
            mbar_arrive_release(bar_empty + 8 * slot);
#pragma unroll
            for (int u = 0; u < N; ++u) {
                const int jl = 16 * (warp + NW * u);
                if (kv > jl)
                    slice_e4m3<MT>(acc, qu, x[u], gs + (s - seg0) * kStageKeys + jl + Tp, W, true, kv - jl, sc, E, lane);
            }
        }
        if (last) {
            if (nc > 0 && warp == NW - 1 && !failed) {   // the chunk: one slice
                E4Slice x;
                load_slice(x, sb + SP::off_ck, sb + SP::off_ck + SP::Tc * kE4Row, sm + SP::off_csc, 8, SP::Tc, lane);
                const int x0 = C - jbase + Tp;
                slice_e4m3<MT>(acc, qu, x, gs + x0, W, (x0 & 3) == 0, nc, sc, E, lane);
            }
            break;
        }
        named_bar_sync(1, kCons);   // the table has been read
    }
    if (failed) s_failed = 1;
    grid_dep_trigger();
    named_bar_sync(1, kCons);
    if (s_failed) err |= kErrTimeout;
    if (err) atomicOr(a.status, err);
    if (s_failed && S == 1) return;
    // the warps' partials, in the ring's memory (every stage has been read)
    float* comb_o = reinterpret_cast<float*>(sm + SP::comb_o);
    float* comb_m = reinterpret_cast<float*>(sm + SP::comb_m);
    float* comb_l = reinterpret_cast<float*>(sm + SP::comb_l);
    if (!s_failed) {
        const int g4 = lane >> 2, t4 = lane & 3;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float l = acc[mt].l[half];
                l += __shfl_xor_sync(0xffffffffu, l, 1);
                l += __shfl_xor_sync(0xffffffffu, l, 2);
                const int r = warp * Tp + 16 * mt + g4 + 8 * half;
#pragma unroll
                for (int d = 0; d < 8; ++d)
                    *reinterpret_cast<float2*>(comb_o + r * kOW + 8 * d + 2 * t4) =
                        make_float2(acc[mt].o[d][2 * half], acc[mt].o[d][2 * half + 1]);
                if (t4 == 0) {
                    comb_m[r] = acc[mt].m[half];
                    comb_l[r] = acc[mt].m[half] - static_cast<float>(E) + log2f(l);
                }
            }
        }
    }
    named_bar_sync(1, kCons);
    if (S == 1) {
        for (int i = tid; i < Tq * 8; i += kCons) {
            const int row = i >> 3, d0 = (i & 7) * 8;
            float m = comb_m[row], l = comb_l[row];
#pragma unroll
            for (int k = 1; k < NW; ++k) {
                m = fmaxf(m, comb_m[k * Tp + row]);
                l = fmaxf(l, comb_l[k * Tp + row]);
            }
            float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, sum = 0.f;
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                const float w = part_weight(comb_m[k * Tp + row], m);
                sum += part_weight(comb_l[k * Tp + row], l);
                const float4* src = reinterpret_cast<const float4*>(comb_o + (k * Tp + row) * kOW + d0);
                const float4 x = src[0], y = src[1];
                o[0] += w * x.x; o[1] += w * x.y; o[2] += w * x.z; o[3] += w * x.w;
                o[4] += w * y.x; o[5] += w * y.y; o[6] += w * y.z; o[7] += w * y.w;
            }
            const float f = exp2f(m - l) / sum;
            *reinterpret_cast<uint4*>(a.out + ((static_cast<long long>(b) * T + i0 + row) * H + h) * kHeadDim + d0) =
                make_uint4(pack_bf16(o[0] * f, o[1] * f), pack_bf16(o[2] * f, o[3] * f), pack_bf16(o[4] * f, o[5] * f),
                           pack_bf16(o[6] * f, o[7] * f));
        }
        return;
    }
    // the CTA's share
    float* part_o = reinterpret_cast<float*>(sm + SP::part_o);
    float* part_m = reinterpret_cast<float*>(sm + SP::part_m);
    float* part_l = reinterpret_cast<float*>(sm + SP::part_l);
    for (int i = tid; i < Tq * kHeadDim; i += kCons) {
        const int row = i / kHeadDim, d = i % kHeadDim;
        float m = -INFINITY, l = -INFINITY, o = 0.f, sum = 0.f;
        if (!s_failed) {
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                m = fmaxf(m, comb_m[k * Tp + row]);
                l = fmaxf(l, comb_l[k * Tp + row]);
            }
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                o += part_weight(comb_m[k * Tp + row], m) * comb_o[(k * Tp + row) * kOW + d];
                sum += part_weight(comb_l[k * Tp + row], l);
            }
        }
        part_o[i] = o;
        if (d == 0) {
            part_m[row] = m;
            part_l[row] = l + log2f(sum);
        }
    }
    cluster_sync();
    // rows split, split + S, ... of the cluster's queries are finished here
    for (int row = split + S * warp; row < Tq; row += S * NW) {
        float m = -INFINITY, l = -INFINITY;
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

// ----------------------------------------------------------------------------- fp32

// One warp per query row, lanes over keys, fp32 throughout (the 16-bit pools' fp32 kernel with
// rows decoded on the way in).  The chunk is already in the pool.
__global__ void __launch_bounds__(128) chunk_e4m3_f32_kernel(
    const float* __restrict__ q, const uint8_t* __restrict__ k_pool, const uint8_t* __restrict__ v_pool,
    const uint8_t* __restrict__ kv_scale, int num_blocks, int block_size,
    const int32_t* __restrict__ block_table, int mbps, const int32_t* __restrict__ cache_seqlens,
    const float* __restrict__ u, const float* __restrict__ vb, const float* __restrict__ rel, int R,
    float* __restrict__ out, int T, int H, float scale, unsigned* status)
{
    __shared__ float s_qu[kE4MaxT][kHeadDim];
    __shared__ float s_qv[kE4MaxT][kHeadDim];
    const int b = blockIdx.x / H, h = blockIdx.x % H;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    unsigned err = 0;
    int C = cache_seqlens[b];
    if (C < 0) { C = 0; err |= kErrBounds; }
    const int cap = mbps * block_size;
    if (C > cap) { C = cap; err |= kErrBounds; }
    int K = C + T;
    if (K > cap) { K = cap; err |= kErrBounds; }
    if (C + 2 * T - 1 > R) err |= kErrBounds;
    const int off = R - T - C;
    for (int idx = tid; idx < T * kHeadDim; idx += blockDim.x) {
        const int t = idx / kHeadDim, d = idx % kHeadDim;
        const float qq = q[((static_cast<long long>(b) * T + t) * H + h) * kHeadDim + d];
        s_qu[t][d] = qq + u[h * kHeadDim + d];
        s_qv[t][d] = qq + vb[h * kHeadDim + d];
    }
    __syncthreads();
    for (int i = warp; i < T; i += 4) {
        float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f;
        for (int j0 = 0; j0 < K; j0 += 32) {
            const int j = j0 + lane;
            float sc = -INFINITY, vs = 0.f;
            long long row_off = -1;
            if (j < K) {
                const int lb = j / block_size;
                const int blk = block_table[static_cast<long long>(b) * mbps + lb];
                float acc = 0.f;
                if (blk >= 0 && blk < num_blocks) {
                    const long long page = static_cast<long long>(blk) * H + h;
                    const int slot = j - lb * block_size;
                    row_off = (page * block_size + slot) * kE4Row;
                    vs = e4m3_scale(kv_scale[(2 * page + 1) * block_size + slot]);
                    const uint4* kr = reinterpret_cast<const uint4*>(k_pool + row_off);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint4 w4 = kr[c];
                        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 lo = e4m3_unpack2(w[e]), hi = e4m3_unpack2(w[e] >> 16);
                            const float* qq = &s_qu[i][16 * c + 4 * e];
                            acc = fmaf(qq[0], lo.x, acc);
                            acc = fmaf(qq[1], lo.y, acc);
                            acc = fmaf(qq[2], hi.x, acc);
                            acc = fmaf(qq[3], hi.y, acc);
                        }
                    }
                    acc *= e4m3_scale(kv_scale[2 * page * block_size + slot]);
                } else {
                    err |= kErrBounds;
                }
                const int rho = off + j - i;
                if (rho >= 0 && rho < R) {
                    const float4* rr = reinterpret_cast<const float4*>(rel + (static_cast<long long>(rho) * H + h) * kHeadDim);
#pragma unroll 4
                    for (int d4 = 0; d4 < kHeadDim / 4; ++d4) {
                        const float4 r4 = rr[d4];
                        acc = fmaf(s_qv[i][4 * d4], r4.x, acc);
                        acc = fmaf(s_qv[i][4 * d4 + 1], r4.y, acc);
                        acc = fmaf(s_qv[i][4 * d4 + 2], r4.z, acc);
                        acc = fmaf(s_qv[i][4 * d4 + 3], r4.w, acc);
                    }
                }
                sc = acc * scale;
            }
            float mx = sc;
#pragma unroll
            for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float m_new = fmaxf(m, mx);
            const float alpha = (m == -INFINITY) ? 0.f : expf(m - m_new);
            const float p = (j < K) ? expf(sc - m_new) : 0.f;
            float psum = p;
#pragma unroll
            for (int o = 16; o; o >>= 1) psum += __shfl_xor_sync(0xffffffffu, psum, o);
            l = l * alpha + psum;
            o0 *= alpha;
            o1 *= alpha;
            const float pv = p * vs;
            const int nj = min(32, K - j0);
            for (int jj = 0; jj < nj; ++jj) {
                const float pj = __shfl_sync(0xffffffffu, pv, jj);
                const long long ro = __shfl_sync(0xffffffffu, row_off, jj);
                if (ro >= 0) {
                    const float2 v2 = e4m3_unpack2(*reinterpret_cast<const uint16_t*>(v_pool + ro + 2 * lane));
                    o0 = fmaf(pj, v2.x, o0);
                    o1 = fmaf(pj, v2.y, o1);
                }
            }
            m = m_new;
        }
        float2* dst = reinterpret_cast<float2*>(out + ((static_cast<long long>(b) * T + i) * H + h) * kHeadDim);
        dst[lane] = make_float2(o0 / l, o1 / l);
    }
    if (err) atomicOr(status, err);
}

// --------------------------------------------------------------------------- host

int g_smem_done_e4[8][64];

// Row stride (bf16 elements) of the position table: every access stays below nkeys + 2 Tp + 8, and a
// stride of 16 mod 64 elements (8 mod 32 words) keeps the 8-byte reads of a slice conflict-free.
inline int e4_table_stride(int nkeys, int Tp) { return ((nkeys + 2 * Tp + 63) & ~63) + 16; }

template <int MT, int NW, int NS, int CTAS, bool FUSED>
oasr_status launch_e4(const void* q, E4Args& a, int k_max, int B, int seg, int slot, cudaStream_t stream)
{
    using SP = E4Smem<MT, NW, NS>;
    CUtensorMap tm_q, tm_k, tm_v, tm_r;
    const int box = a.block_size < kStageKeys ? a.block_size : kStageKeys;
    const long long rows = static_cast<long long>(a.num_blocks) * a.H * a.block_size;
    if (!encode_rows_bf16(&tm_q, q, static_cast<long long>(B) * a.T, a.H, SP::Tp) ||
        !encode_rows_bf16(&tm_r, a.rel, a.R, a.H, kStageKeys) || !encode_rows_e4m3(&tm_k, a.k_pool, rows, box) || !encode_rows_e4m3(&tm_v, a.v_pool, rows, box))
        return OASR_ERR_INVALID_ARG;
    auto kern = chunk_e4m3_kernel<MT, NW, NS, CTAS, FUSED>;
    // segments of at most eight stages and a part of one, sized for the keys a call can have
    const int stages = (k_max + kStageKeys - 1) / kStageKeys;
    a.seg = stages < seg ? stages : seg;
    a.gt_w = e4_table_stride(a.seg * kStageKeys + (FUSED ? 16 : 0), SP::Tp);
    const int smem = SP::bytes + SP::Tp * a.gt_w * 2;
    if (!ensure_smem(kern, smem, g_smem_done_e4[slot])) return OASR_ERR_CUDA;
    a.q_tiles = (a.T + SP::Tp - 1) / SP::Tp;
    const long long pairs = static_cast<long long>(B) * a.H * a.q_tiles;
    const int sms = sm_count();
    a.splits = 1;
    while (a.splits < 8 && pairs * a.splits * 2 <= sms && stages >= 2 * a.splits) a.splits *= 2;
    if (pairs * a.splits > 0x7fffffffLL) return OASR_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(pairs * a.splits));
    cfg.blockDim = dim3(32 * (NW + 1));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kern, tm_q, tm_k, tm_v, tm_r, static_cast<const E4Args>(a)) != cudaSuccess)
        return OASR_ERR_CUDA;
    return launch_status();
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
    unsigned* status = status_word();
    if (!status || !sm_count()) return OASR_ERR_CUDA;
    // more than one m-tile of queries (and fp32): the append first, then the attention over the pool
    if (FUSED && (dt == OASR_F32 || T > 16)) {
        const oasr_status st = oasr_paged_append_e4m3(k_new, v_new, k_pool, v_pool, kv_scale, num_blocks, block_size,
                                                      bt, mbps, cs, B, T, H, D, dt, stream);
        if (st != OASR_OK) return st;
    }
    if (dt == OASR_F32) {
        chunk_e4m3_f32_kernel<<<static_cast<unsigned>(B) * H, 128, 0, stream>>>(
            static_cast<const float*>(q), static_cast<const uint8_t*>(k_pool), static_cast<const uint8_t*>(v_pool),
            static_cast<const uint8_t*>(kv_scale), num_blocks, block_size, bt, mbps, cs,
            static_cast<const float*>(u), static_cast<const float*>(vb), static_cast<const float*>(rel), R,
            static_cast<float*>(out), T, H, scale, status);
        return launch_status();
    }
    E4Args a = {};
    a.k_new = static_cast<const __nv_bfloat16*>(k_new);
    a.v_new = static_cast<const __nv_bfloat16*>(v_new);
    a.k_pool = static_cast<uint8_t*>(k_pool);
    a.v_pool = static_cast<uint8_t*>(v_pool);
    a.kv_scale = static_cast<uint8_t*>(kv_scale);
    a.block_table = bt;
    a.cache_seqlens = cs;
    a.pos_bias_u = static_cast<const uint16_t*>(u);
    a.pos_bias_v = static_cast<const uint16_t*>(vb);
    a.rel = static_cast<const uint16_t*>(rel);
    a.out = static_cast<uint16_t*>(out);
    a.status = status;
    a.num_blocks = num_blocks;
    a.block_size = block_size;
    a.bs_shift = __builtin_ctz(static_cast<unsigned>(block_size));
    a.mbps = mbps;
    a.T = T;
    a.H = H;
    a.R = R;
    a.scale_log2 = scale * 1.4426950408889634f;
    // keys a well-formed stream of the call can have
    const long long pages = static_cast<long long>(mbps) * block_size, dist = static_cast<long long>(R) - T + 1;
    const long long k_max = pages < dist ? pages : dist;
    const int km = static_cast<int>(k_max < T ? T : k_max);
    if (T <= 16) return launch_e4<1, E4NW, E4NS, E4CTAS, FUSED>(q, a, km, B, E4SEG, FUSED ? 1 : 0, stream);
    return launch_e4<2, E4NW2, E4NS2, E4CTAS2, false>(q, a, km, B, E4SEG2, 2, stream);
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
