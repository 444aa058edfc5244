// Attention of few query rows over rows of the paged cache, on the matrix
// units a warp drives by itself (mma.sync, m16n8k16, bf16): single tokens,
// the union of the scan's winners, and what kvchunk.cu does not take (fp32
// queries, widths other than 64 and 128).
//
// The work is bound by reading K and V, so the products are turned round to
// have the cached rows as the 16-row operand and the (few) query rows as the
// 8-column one, and no cached byte passes through shared memory:
//   S^T [16 keys x 8 rows] = K [16 x D] Q^T,  O^T [D x 8] += V^T [D x 16] P^T.
// A dot product may run over the channels in any order, so a lane's operand
// registers for K are simply consecutive bytes of one row (16-byte loads,
// whole sectors), and Q is laid out in shared memory to match.  For V a lane
// holds the same channels of the keys 2c, 2c+1, 2c+8, 2c+9 and pairs the keys
// with byte permutes.  P^T comes out of S^T's registers by transposing 8x8
// tiles in registers (movmatrix).  8-bit codes become bf16 in a lane's
// registers, exactly: INT8 as 128 + low bits minus 128 or 256, E4M3 by moving
// its fields, then times the block's power of two.
//
// A CTA takes 8*NT query rows of one sequence and group and one stretch of
// its tokens; its four warps take 16-key tiles in turn, each with its own
// running maximum and sums, joined in shared memory.  Stretches are joined
// by kv_join_kernel in a fixed order, so results do not depend on timing.
#pragma once

#include "kv.cuh"

namespace fathom {

constexpr int kRowsWarps = 4;
constexpr int kRowsThreads = 32 * kRowsWarps;

// Query row tiles of a call and their split over the tokens.
struct KvSplit {
    int32_t nt;          // 8-row tiles per CTA, or 0: kvchunk.cuh takes the call
    int32_t tile_rows;   // query rows per CTA
    int32_t row_tiles;   // CTAs along a sequence's query rows
    int32_t splits;      // CTAs along its tokens, at most
    int32_t chunk;       // tokens of a stretch
};

struct KvRowsArgs {
    KvAttend a;
    KvSplit s;
    float* po;   // [splits][rows*H*G][D] value sums of a stretch
    float* pm;   // [splits][rows*H*G] maxima (in powers of two)
    float* pl;   // [splits][rows*H*G] weight sums
    int64_t heads;   // rows*H*G
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8x8 tile of 16-bit values held two to a lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(x));
    return r;
}

// 2^x to 2 ulp; below 2^-126 it is 0.
__device__ __forceinline__ float exp2_fast(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
    return r;
}

// NW words of a row, read once.
template <int NW>
__device__ __forceinline__ void load_words(const unsigned char* p, uint32_t* w)
{
    if (NW == 4)
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
    else if (NW == 2)
        asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];\n" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    else
        asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];\n" : "=r"(w[0]) : "l"(p));
}

__device__ __forceinline__ uint32_t bmul2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t bsub2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Bytes BLO of x and BHI of y as bf16 values times the powers `f` (bf16x2).
template <int FMT, int BLO, int BHI>
__device__ __forceinline__ uint32_t decode2(uint32_t x, uint32_t y, uint32_t f)
{
    if (FMT == FATHOM_KV_INT8) {
        // the byte in the low half of each 16 bits (the byte above it is cut off)
        const uint32_t t = __byte_perm(x, y, BLO | (BLO << 4) | ((4 + BHI) << 8) | ((4 + BHI) << 12));
        const uint32_t low = (t & 0x007f007fu) | 0x43004300u;    // 128 + low 7 bits
        const uint32_t off = (t & 0x00800080u) | 0x43004300u;    // 128, or 256 for a negative code
        return bmul2(bsub2(low, off), f);
    }
    // the byte on top: sign in place, exponent and mantissa 4 below; 2^120 of the power makes up for the bias
    const uint32_t t = __byte_perm(x, y, (BLO << 4) | BLO | ((4 + BHI) << 12) | ((4 + BHI) << 8));
    return bmul2(((t >> 4) & 0x07f007f0u) | (t & 0x80008000u), f);
}

// The 16 bits that decode2 multiplies with, from the exponent byte.
template <int FMT>
__device__ __forceinline__ uint32_t pow_bits(uint32_t byte)
{
    return (FMT == FATHOM_KV_INT8 ? byte : min(byte + 120u, 255u)) << 7;
}

// x as bf16 parts that sum to it (to 8 bits each).
template <int N>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&part)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        part[i] = bf16x2(x, y);
        x -= __uint_as_float(part[i] << 16);
        y -= __uint_as_float(part[i] & 0xffff0000u);
    }
}

// Tokens that the rows of a tile see at most, and the sequence's facts.
struct KvSpan {
    int64_t first;   // first row of the sequence
    int32_t rows;    // its rows that are computed
    int32_t pos0;    // position of its row 0 (may be negative)
    int32_t keys;    // tokens any of its rows may see
};

__device__ __forceinline__ KvSpan kv_span(const KvAttend& a, int b)
{
    KvSpan s;
    s.first = a.w.cu[b];
    const int64_t end = a.w.cu[b + 1], len = a.w.length[b];
    s.rows = static_cast<int32_t>(max(int64_t{0}, min(min(end, static_cast<int64_t>(a.w.rows)) - s.first, a.max_new)));
    s.pos0 = static_cast<int32_t>(len - end + s.first);
    s.keys = static_cast<int32_t>(max(int64_t{0}, min(len, a.max_len)));
    return s;
}

// Tokens seen by the query rows [r0, r0 + n) of a sequence (rows counted row*G + head).
__device__ __forceinline__ int kv_tile_keys(const KvAttend& a, const KvSpan& s, int r0, int n)
{
    if (!a.causal) return s.keys;
    const int last = min(r0 + n, s.rows * a.G) - 1;
    return max(0, min(s.keys, s.pos0 + last / a.G + 1));
}

template <int D, int FMT, int QT, int NT, bool UNION>
struct RowsShape {
    static constexpr int NQ = QT == FATHOM_KEYS_F32 ? 3 : 1;                   // bf16 parts of a query
    static constexpr int NP = QT == FATHOM_KEYS_F32 ? 3 : (NT == 1 ? 2 : 1);   // and of a weight
    static constexpr int ESZ = kv_elem_bytes<FMT>();
    static constexpr int KPB = FMT == FATHOM_KV_BF16 ? 8 : (D % 64 == 0 ? 16 : 8);                        // channels of a K piece
    static constexpr int VPB = FMT == FATHOM_KV_BF16 ? (D % 64 == 0 ? 8 : 4)
                                                     : (D % 128 == 0 ? 16 : (D % 64 == 0 ? 8 : 4));       // and of a V piece
    static constexpr int KPW = KPB * ESZ / 4, VPW = VPB * ESZ / 4;   // words of a piece
    static constexpr int KP = D / (4 * KPB), VP = D / (8 * VPB);     // pieces of a lane's row
    static constexpr int KS = D / 16;                                // matrix steps
    static constexpr size_t QB = sizeof(uint2) * NQ * KS * NT * 32;   // bytes of Q's operand registers
    static constexpr size_t OB = sizeof(float) * NT * 8 * (D + 8);    // and of the value sums
    static constexpr size_t SUMS = QB > OB ? QB : OB;
    static constexpr size_t SMEM = SUMS + sizeof(float) * 2 * kRowsWarps * NT * 8;
};

template <int D, int FMT, int QT, int NT, bool UNION>
__global__ void __launch_bounds__(kRowsThreads, NT == 1 && D <= 128 ? 4 : 2)
kv_rows_kernel(const KvRowsArgs g)
{
    using S = RowsShape<D, FMT, QT, NT, UNION>;
    constexpr bool CODED = FMT != FATHOM_KV_BF16;
    extern __shared__ __align__(16) unsigned char smem[];
    uint2* qf = reinterpret_cast<uint2*>(smem);              // [NQ][KS][NT][32] operand registers of Q^T
    float* os = reinterpret_cast<float*>(smem);              // [NT*8][D+8] value sums, after the loop
    float* sm_m = reinterpret_cast<float*>(smem + S::SUMS);
    float* sm_l = sm_m + kRowsWarps * NT * 8;

    const KvAttend& a = g.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const int h = blockIdx.y, b = blockIdx.z;
    const int tile = blockIdx.x % g.s.row_tiles, split = blockIdx.x / g.s.row_tiles;
    const int G = a.G;
    const int r0 = tile * NT * 8;   // first query row (row*G + head) of the tile

    KvSpan sp;
    int keys;                       // of the tile's rows
    const int32_t* table = a.w.table;
    if (UNION) {
        sp = KvSpan{0, 1, 0, 0};
        keys = static_cast<int>(min(static_cast<int64_t>(max(a.count[h], 0)), a.M));
    } else {
        sp = kv_span(a, b);
        if (r0 >= sp.rows * G) return;
        keys = kv_tile_keys(a, sp, r0, NT * 8);
        table += b * a.w.table_stride;
    }
    const int begin = split * g.s.chunk;
    const int end = min(keys, begin + g.s.chunk);
    if (begin >= keys && split > 0) return;   // the join knows

    // Q^T operand registers: lane (r, c) of step ks holds channels of row r that match K's.
    for (int e = threadIdx.x; e < S::KS * NT * 32; e += kRowsThreads) {
        const int el = e & 31, nt = (e >> 5) % NT, ks = (e >> 5) / NT;
        const int qr = r0 + nt * 8 + (el >> 2);
        const int d = (ks / (S::KPB / 4)) * 4 * S::KPB + (el & 3) * S::KPB + (ks % (S::KPB / 4)) * 4;
        float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (qr < sp.rows * G) {
            const int64_t at = (sp.first + qr / G) * a.q_tok + (static_cast<int64_t>(h) * G + qr % G) * a.q_head + d;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[j] = QT == FATHOM_KEYS_F32 ? static_cast<const float*>(a.q)[at + j]
                                             : __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[at + j]);
        }
        uint32_t lo[S::NQ], hi[S::NQ];
        split2<S::NQ>(x[0], x[1], lo);
        split2<S::NQ>(x[2], x[3], hi);
#pragma unroll
        for (int p = 0; p < S::NQ; ++p) qf[((p * S::KS + ks) * NT + nt) * 32 + el] = make_uint2(lo[p], hi[p]);
    }

    // Last token that rows 2c, 2c+1 of each tile see (padding rows see all), and the least of any row.
    int seen[NT][2], least = 0x7fffffff;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int qr = r0 + nt * 8 + 2 * c + i;
            seen[nt][i] = !UNION && a.causal && qr < sp.rows * G ? sp.pos0 + qr / G : 0x7fffffff;
        }
    if (!UNION && a.causal) least = sp.pos0 + r0 / G;

    float o[S::KS][NT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
        for (int t = 0; t < S::KS; ++t) o[t][nt][0] = o[t][nt][1] = o[t][nt][2] = o[t][nt][3] = 0.0f;
    }
    const float log2s = a.scale * 1.4426950408889634f;
    __syncthreads();

    uint32_t kw[2][S::KP * S::KPW], vw[4][S::VP * S::VPW];
    uint32_t kb[2][S::KP], vb[4][S::VP];   // exponent bytes of the pieces' blocks
    int kpage, vpage = -1;
    int live_k, live_v = 0, live_at;       // which of the tile's 16 keys there are
    // A lane's keys: K rows r, r + 8; V rows 2c, 2c + 1, 2c + 8, 2c + 9.
    // In a union each key has its own place, kept by lane (key) for the whole warp.
    int upos = -1, upage = -1, vupos = 0, vupage = -1, unext = -1;

    auto find = [&](int at) {   // the places of the tile at `at`
        live_at = at;
        if (UNION) {
            upos = unext;
            upage = upos >= 0 && upos < a.n ? kv_page(a.c, table, a.w.table_pages, upos) : -1;
            live_k = static_cast<int>(__ballot_sync(0xffffffffu, upage >= 0) & 0xffffu);
            const int nx = at + 16 * kRowsWarps + lane;
            unext = lane < 16 && nx < end ? __ldg(a.uni + h * a.M + nx) : -1;
        } else {
            kpage = at < end ? kv_page(a.c, table, a.w.table_pages, at) : -1;
            const int n = end - at;
            live_k = kpage < 0 ? 0 : (n >= 16 ? 0xffff : (1 << n) - 1);
        }
    };
    auto load_k = [&]() {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int key = r + 8 * i;
            int page = kpage, tok = (live_at + key) & (a.c.page_tokens - 1);
            if (UNION) {
                page = __shfl_sync(0xffffffffu, upage, key);
                tok = __shfl_sync(0xffffffffu, upos, key) & (a.c.page_tokens - 1);
            }
            if ((live_k >> key) & 1) {
                const unsigned char* p = a.c.k + kv_off(a.c, page, h, tok) + c * S::KPB * S::ESZ;
#pragma unroll
                for (int q = 0; q < S::KP; ++q) load_words<S::KPW>(p + q * 4 * S::KPB * S::ESZ, &kw[i][q * S::KPW]);
                if (CODED) {
                    const unsigned char* sc = a.c.ks + kv_scale_off(a.c, page, h, tok);
                    if (D == 128) {
                        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(sc));
#pragma unroll
                        for (int q = 0; q < S::KP; ++q) kb[i][q] = (w >> (8 * (2 * q + (c >> 1)))) & 0xff;
                    } else {
#pragma unroll
                        for (int q = 0; q < S::KP; ++q) kb[i][q] = __ldg(sc + ((q * 4 + c) * S::KPB >> 5));
                    }
                }
            } else {
#pragma unroll
                for (int q = 0; q < S::KP * S::KPW; ++q) kw[i][q] = 0;
#pragma unroll
                for (int q = 0; q < S::KP; ++q) kb[i][q] = 0;
            }
        }
    };
    auto load_v = [&](int at) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int key = 2 * c + (i & 1) + 8 * (i >> 1);
            int page = vpage, tok = (at + key) & (a.c.page_tokens - 1);
            if (UNION) {
                page = __shfl_sync(0xffffffffu, vupage, key);
                tok = __shfl_sync(0xffffffffu, vupos, key) & (a.c.page_tokens - 1);
            }
            if ((live_v >> key) & 1) {
                const unsigned char* p = a.c.v + kv_off(a.c, page, h, tok) + r * S::VPB * S::ESZ;
#pragma unroll
                for (int q = 0; q < S::VP; ++q) load_words<S::VPW>(p + q * 8 * S::VPB * S::ESZ, &vw[i][q * S::VPW]);
                if (CODED) {
                    const unsigned char* sc = a.c.vs + kv_scale_off(a.c, page, h, tok);
#pragma unroll
                    for (int q = 0; q < S::VP; ++q) vb[i][q] = __ldg(sc + ((q * 8 + r) * S::VPB >> 5));
                }
            } else {
#pragma unroll
                for (int q = 0; q < S::VP * S::VPW; ++q) vw[i][q] = 0;
#pragma unroll
                for (int q = 0; q < S::VP; ++q) vb[i][q] = 0;
            }
        }
    };

    int at = begin + 16 * warp;
    if (UNION) unext = lane < 16 && at + lane < end ? __ldg(a.uni + h * a.M + at + lane) : -1;
    if (at < end) {
        find(at);
        load_k();
    }
    for (; at < end; at += 16 * kRowsWarps) {
        vpage = kpage;
        vupage = upage;
        vupos = upos;
        live_v = live_k;
        load_v(at);
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < S::KS; ++ks) {
            uint32_t a0, a1, a2, a3;
            if (CODED) {
                const int q = ks / (S::KPB / 4), w = q * S::KPW + ks % (S::KPB / 4);
                const uint32_t f0 = pow_bits<FMT>(kb[0][q]) * 0x10001u, f1 = pow_bits<FMT>(kb[1][q]) * 0x10001u;
                a0 = decode2<FMT, 0, 1>(kw[0][w], kw[0][w], f0);
                a2 = decode2<FMT, 2, 3>(kw[0][w], kw[0][w], f0);
                a1 = decode2<FMT, 0, 1>(kw[1][w], kw[1][w], f1);
                a3 = decode2<FMT, 2, 3>(kw[1][w], kw[1][w], f1);
            } else {
                a0 = kw[0][2 * ks];
                a2 = kw[0][2 * ks + 1];
                a1 = kw[1][2 * ks];
                a3 = kw[1][2 * ks + 1];
            }
#pragma unroll
            for (int p = 0; p < S::NQ; ++p)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint2 q = qf[((p * S::KS + ks) * NT + nt) * 32 + lane];
                    mma16816(s[nt], a0, a1, a2, a3, q.x, q.y);
                }
        }
        // The next tile's keys are on their way while this one's weights are taken.
        if (at + 16 * kRowsWarps < end) {
            find(at + 16 * kRowsWarps);
            load_k();
        }

        const bool whole = live_v == 0xffff && at + 15 <= least;
        uint32_t pb[NT][S::NP][2];
        float f[NT][2];
        bool grew = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[nt][i] *= log2s;
                if (!whole) {
                    const int key = r + 8 * (i >> 1);
                    if (!((live_v >> key) & 1) || at + key > seen[nt][i & 1]) s[nt][i] = -INFINITY;
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float top = fmaxf(s[nt][i], s[nt][i + 2]);
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                const float old = m[nt][i];
                grew |= top > old;
                m[nt][i] = fmaxf(old, top);
                const float base = m[nt][i] == -INFINITY ? 0.0f : m[nt][i];
                f[nt][i] = exp2_fast(old - base);
                s[nt][i] = exp2_fast(s[nt][i] - base);
                s[nt][i + 2] = exp2_fast(s[nt][i + 2] - base);
                l[nt][i] = l[nt][i] * f[nt][i] + (s[nt][i] + s[nt][i + 2]);
            }
            uint32_t lo[S::NP], hi[S::NP];
            split2<S::NP>(s[nt][0], s[nt][1], lo);
            split2<S::NP>(s[nt][2], s[nt][3], hi);
#pragma unroll
            for (int p = 0; p < S::NP; ++p) {
                pb[nt][p][0] = transpose8x8(lo[p]);
                pb[nt][p][1] = transpose8x8(hi[p]);
            }
        }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
            for (int t = 0; t < S::KS; ++t)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    o[t][nt][0] *= f[nt][0];
                    o[t][nt][1] *= f[nt][1];
                    o[t][nt][2] *= f[nt][0];
                    o[t][nt][3] *= f[nt][1];
                }
        }
#pragma unroll
        for (int q = 0; q < S::VP; ++q) {
            uint32_t f01 = 0, f89 = 0;
            if (CODED) {
                f01 = pow_bits<FMT>(vb[0][q]) | pow_bits<FMT>(vb[1][q]) << 16;
                f89 = pow_bits<FMT>(vb[2][q]) | pow_bits<FMT>(vb[3][q]) << 16;
            }
#pragma unroll
            for (int j = 0; j < S::VPB / 2; ++j) {
                uint32_t a0, a1, a2, a3;
                if (CODED) {
                    const int w = q * S::VPW + j / 2;
                    if (j & 1) {
                        a0 = decode2<FMT, 2, 2>(vw[0][w], vw[1][w], f01);
                        a1 = decode2<FMT, 3, 3>(vw[0][w], vw[1][w], f01);
                        a2 = decode2<FMT, 2, 2>(vw[2][w], vw[3][w], f89);
                        a3 = decode2<FMT, 3, 3>(vw[2][w], vw[3][w], f89);
                    } else {
                        a0 = decode2<FMT, 0, 0>(vw[0][w], vw[1][w], f01);
                        a1 = decode2<FMT, 1, 1>(vw[0][w], vw[1][w], f01);
                        a2 = decode2<FMT, 0, 0>(vw[2][w], vw[3][w], f89);
                        a3 = decode2<FMT, 1, 1>(vw[2][w], vw[3][w], f89);
                    }
                } else {
                    const int w = q * S::VPW + j;
                    a0 = __byte_perm(vw[0][w], vw[1][w], 0x5410);
                    a1 = __byte_perm(vw[0][w], vw[1][w], 0x7632);
                    a2 = __byte_perm(vw[2][w], vw[3][w], 0x5410);
                    a3 = __byte_perm(vw[2][w], vw[3][w], 0x7632);
                }
#pragma unroll
                for (int p = 0; p < S::NP; ++p)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma16816(o[q * (S::VPB / 2) + j][nt], a0, a1, a2, a3, pb[nt][p][0], pb[nt][p][1]);
            }
        }
    }

    // Join the warps.
    __syncthreads();   // Q has been read
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float x = l[nt][i];
            x += __shfl_xor_sync(0xffffffffu, x, 4);
            x += __shfl_xor_sync(0xffffffffu, x, 8);
            x += __shfl_xor_sync(0xffffffffu, x, 16);
            if (r == 0) {
                sm_m[warp * NT * 8 + nt * 8 + 2 * c + i] = m[nt][i];
                sm_l[warp * NT * 8 + nt * 8 + 2 * c + i] = x;
            }
        }
    __syncthreads();
    float w8[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kRowsWarps; ++w) top = fmaxf(top, sm_m[w * NT * 8 + nt * 8 + 2 * c + i]);
            w8[nt][i] = exp2_fast(m[nt][i] - (top == -INFINITY ? 0.0f : top));
        }
    for (int w = 0; w < kRowsWarps; ++w) {
        if (warp == w) {
#pragma unroll
            for (int t = 0; t < S::KS; ++t)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float* to = os + (nt * 8 + 2 * c + (i & 1)) * (D + 8) + (2 * t + (i >> 1)) * 8 + r;
                        const float x = o[t][nt][i] * w8[nt][i & 1];
                        *to = w == 0 ? x : *to + x;
                    }
        }
        __syncthreads();
    }
    const bool parts = g.s.splits > 1;
    for (int e = threadIdx.x; e < NT * 8 * D; e += kRowsThreads) {
        const int row = e / D, d = e % D;
        const int qr = r0 + row;
        if (qr >= sp.rows * G) break;
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kRowsWarps; ++w) top = fmaxf(top, sm_m[w * NT * 8 + row]);
        const float low = top == -INFINITY ? 0.0f : top;
#pragma unroll
        for (int w = 0; w < kRowsWarps; ++w) sum += sm_l[w * NT * 8 + row] * exp2_fast(sm_m[w * NT * 8 + row] - low);
        // channel d = 8 VPB q + VPB r + j is kept at (VPB q + j) 8 + r
        const float x = os[row * (D + 8) + ((d / (8 * S::VPB)) * S::VPB + d % S::VPB) * 8 + (d / S::VPB) % 8];
        const int64_t head = ((sp.first + qr / G) * a.c.H + h) * G + qr % G;
        if (parts) {
            const int64_t at_p = split * g.heads + head;
            g.po[at_p * D + d] = x;
            if (d == 0) {
                g.pm[at_p] = top;
                g.pl[at_p] = sum;
            }
        } else {
            const float y = sum == 0.0f ? 0.0f : x / sum;   // no token was seen (NaN scores make the sum NaN)
            if (QT == FATHOM_KEYS_F32) static_cast<float*>(a.out)[head * D + d] = y;
            else static_cast<__nv_bfloat16*>(a.out)[head * D + d] = __float2bfloat16(y);
        }
    }
    pdl_launch_dependents();
}

template <int D, int FMT, int QT, int NT, bool UNION>
int launch_rows_t(const KvRowsArgs& g, cudaStream_t stream)
{
    using S = RowsShape<D, FMT, QT, NT, UNION>;
    const int st = ensure_dynamic_smem(reinterpret_cast<const void*>(kv_rows_kernel<D, FMT, QT, NT, UNION>), S::SMEM);
    if (st) return st;
    const dim3 grid(static_cast<unsigned>(g.s.splits) * g.s.row_tiles, static_cast<unsigned>(g.a.c.H),
                    static_cast<unsigned>(UNION ? 1 : g.a.w.B));
    kv_rows_kernel<D, FMT, QT, NT, UNION><<<grid, kRowsThreads, S::SMEM, stream>>>(g);
    return launch_status();
}

template <int D, int FMT>
int launch_rows_d(const KvRowsArgs& g, int q_dtype, cudaStream_t stream)
{
    constexpr int WIDE = D <= 128 ? 4 : 2;   // accumulators of 4 tiles of 256 channels do not fit a thread's registers
    if (g.a.uni) return launch_rows_t<D, FMT, FATHOM_KEYS_F32, 1, true>(g, stream);
    if (q_dtype == FATHOM_KEYS_F32)
        return g.s.nt == 1 ? launch_rows_t<D, FMT, FATHOM_KEYS_F32, 1, false>(g, stream)
                           : launch_rows_t<D, FMT, FATHOM_KEYS_F32, WIDE, false>(g, stream);
    return g.s.nt == 1 ? launch_rows_t<D, FMT, FATHOM_KEYS_BF16, 1, false>(g, stream)
                       : launch_rows_t<D, FMT, FATHOM_KEYS_BF16, WIDE, false>(g, stream);
}

template <int FMT>
int launch_rows_f(const KvRowsArgs& g, int q_dtype, cudaStream_t stream)
{
    switch (g.a.c.D) {
        case 32: return launch_rows_d<32, FMT>(g, q_dtype, stream);
        case 64: return launch_rows_d<64, FMT>(g, q_dtype, stream);
        case 96: return launch_rows_d<96, FMT>(g, q_dtype, stream);
        case 128: return launch_rows_d<128, FMT>(g, q_dtype, stream);
        case 160: return launch_rows_d<160, FMT>(g, q_dtype, stream);
        case 192: return launch_rows_d<192, FMT>(g, q_dtype, stream);
        case 224: return launch_rows_d<224, FMT>(g, q_dtype, stream);
        default: return launch_rows_d<256, FMT>(g, q_dtype, stream);
    }
}

// One file per format.
int launch_rows_bf16(const KvRowsArgs& g, int q_dtype, cudaStream_t stream);
int launch_rows_int8(const KvRowsArgs& g, int q_dtype, cudaStream_t stream);
int launch_rows_e4m3(const KvRowsArgs& g, int q_dtype, cudaStream_t stream);

}  // namespace fathom
