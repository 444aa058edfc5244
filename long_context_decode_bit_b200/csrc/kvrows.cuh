// Attention of few query rows over rows of the paged cache, on the matrix
// units a warp drives by itself (mma.sync, m16n8k16): single tokens, the
// union of the scan's winners, and what kvchunk.cuh does not take (fp32
// queries, and up to 32 rows of bf16 ones).
//
// The work is bound by reading K and V, so the products are turned round to
// have the cached rows as the 16-row operand and the (few) query rows as the
// 8-column one:
//   S^T [16 keys x 8 rows] = K [16 x D] Q^T,  O^T [D x 8] += V^T [D x 16] P^T.
// P^T comes out of S^T's registers by transposing 8x8 tiles in registers
// (movmatrix).  A CTA takes 8*NT query rows of one sequence and group and one
// stretch of its tokens; its four warps take 16-key tiles in turn.  Each has
// a ring of its own for them, filled by cp.async (zeros for keys that are not
// there), so that no warp waits for another until the end, where maxima and
// sums are joined in shared memory.  Stretches are joined by kv_join_kernel
// in a fixed order, so results do not depend on timing.
//
// 16-bit rows are operands as they are (ldmatrix, V transposed).  8-bit codes
// become bf16 on their way to the operand registers, exactly: INT8 as
// 128 + low bits less 128 or 256, E4M3 by moving its fields, times the block's
// power of two.  (fp16 operands take two instructions less to a pair of INT8
// codes, but then powers have to be kept relative to a running largest and
// weights below 2^-40 are lost; both took the same time.)  A dot product may
// run over the channels in any order, so a lane takes consecutive bytes of a
// row, and Q is laid out to match.  fp32 queries and their weights are three
// bf16 parts each (24 bits), and a tile's three products are summed apart from
// the tiles before, to which they are added with a rounding: the matrix units
// cut sums off, which over a session of a million tokens came to 1e-4 (now
// 7e-7, for 1 to 2% of the time).  The weights of bf16 queries are rounded to bf16,
// up to 2^-8 of each, like the output they go into.  (Two parts of a weight
// would leave the output's own rounding, 1.65e-3 of its size instead of 1.85e-3
// over an int8 session, and take the 128k int8 token from 69.4 to 72.1 us.)
#pragma once

#include "kv.cuh"
#include "ring.cuh"

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
#ifdef FATHOM_TEST_HOOKS
    int32_t withhold;   // test build: tile of K or V (in the order they are brought) whose arrival is withheld, or -1
#endif
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

// Operands of the 4 codes of a word, codes (0, 2) and (1, 3), times the powers f.
template <int FMT>
__device__ __forceinline__ void codes4(uint32_t w, uint32_t f, const CodeMasks& m, uint32_t* a, uint32_t* b)
{
    if (FMT == FATHOM_KV_INT8) {
        *a = decode_low(w, f, m);
        *b = decode_low(w >> 8, f, m);
    } else {
        *a = decode_high(w << 8, f, m);
        *b = decode_high(w, f, m);
    }
}

// x as bf16 parts that sum to it (to 8 bits each).  Several parts are cut off rather than rounded: 8 bits of the 24 each,
// so that nothing is lost, and the first of a value next to the largest is not an infinity.
template <int N>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&part)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        part[i] = N > 1 ? bf16x2_cut(x, y) : bf16x2(x, y);
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
    if (s.first < 0) s.rows = 0;   // no such rows
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

// Stretches of `chunk` that `keys` tokens take.
__device__ __forceinline__ int kv_stretches(int64_t keys, int chunk) { return static_cast<int>((keys + chunk - 1) / chunk); }

// NW words from shared memory.
template <int NW>
__device__ __forceinline__ void lds_words(uint32_t at, uint32_t* w)
{
    if (NW == 4)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
    else if (NW == 2)
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];\n" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
    else
        asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(w[0]) : "r"(at));
}

__device__ __forceinline__ int lds_byte(uint32_t at)
{
    uint32_t r;
    asm volatile("ld.shared.u8 %0, [%1];\n" : "=r"(r) : "r"(at));
    return static_cast<int>(r);
}

// Four 8x8 tiles of 16-bit values, rows at the lanes' addresses.
template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t at, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d)
{
    if (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                     : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(at));
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                     : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(at));
}

// 16-byte copy to shared memory.
__device__ __forceinline__ void cp_async16_to(uint32_t at, const void* gmem)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(at), "l"(gmem) : "memory");
}

// The same, of zeros where `bytes` is 0.
__device__ __forceinline__ void cp_async16_to(uint32_t at, const void* gmem, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(at), "l"(gmem), "r"(bytes) : "memory");
}

template <int D, int FMT, int QT, int NT>
struct RowsShape {
    static constexpr bool CODED = FMT != FATHOM_KV_BF16;
    static constexpr bool WIDEQ = QT == FATHOM_KEYS_F32;
    static constexpr int NQ = WIDEQ ? 3 : 1, NP = NQ;                              // parts of a query and of a weight
    static constexpr int ESZ = kv_elem_bytes<FMT>();
    static constexpr int RB = D * ESZ, PP = RB / 16;                               // bytes of a row, and 16-byte pieces
    static constexpr int KPB = D % 64 == 0 ? 16 : 8;                               // codes that a lane takes of a K row at a time
    static constexpr int VPB = D % 128 == 0 ? 16 : (D % 64 == 0 ? 8 : 4);          // and of a V row
    static constexpr int KPW = KPB / 4, VPW = VPB / 4;
    static constexpr int KP = D / (4 * KPB), VP = D / (8 * VPB);
    static constexpr int KS = D / 16;                                              // matrix steps
    static constexpr int NB = D / kKvBlock, SBW = NB <= 4 ? 4 : 8;                 // exponent bytes of a row, and their place
    static constexpr int LPR = PP % 4 == 0 ? 4 : 2, RPL = LPR / 2;                 // lanes that copy a row, rows of a lane
    static constexpr int STAGE = 32 * RB + (CODED ? 32 * SBW : 0);                 // 16 rows of K and of V
    // Of wide tiles and three parts of Q, two: two CTAs fit an SM (128 channels of bf16, fp32 queries: 78 -> 63 us).
    static constexpr int STAGES = !CODED && WIDEQ && NT > 1 && STAGE >= 8192 ? 2 : 3;
    static constexpr int RING = kRowsWarps * STAGES * STAGE;
    static constexpr int QB = static_cast<int>(sizeof(uint2)) * NQ * KS * NT * 32; // Q's operand registers
    static constexpr int OB = static_cast<int>(sizeof(float)) * NT * 8 * (D + 8);  // value sums, where the ring was
    static constexpr int SUMS = QB + (RING > OB ? RING : OB);
    static constexpr int SMEM = SUMS + static_cast<int>(sizeof(float)) * NT * 8 * (2 * kRowsWarps + 2);
    static constexpr int FIT = 228 * 1024 / (SMEM + 1024);
    static constexpr int CTAS = NT == 1 && D <= 128 ? (FIT < 4 ? FIT : 4) : (FIT < 2 ? FIT : 2);   // to an SM

    // 16-byte piece of a row in its tile: moved so that the lanes that read together find different banks.
    static __device__ __forceinline__ int swizzle(bool v, int row, int piece)
    {
        if (!CODED) return PP % 8 == 0 ? piece ^ (row & 7) : piece ^ ((row >> 1) & 3);
        if (PP % 8 != 0) return piece;
        return v ? piece ^ (((row >> 1) & 3) << 1) : piece ^ ((row & 1) << 2);
    }
    static __device__ __forceinline__ uint32_t at(bool v, int row, int piece)
    {
        return (v ? 16 * RB : 0) + row * RB + swizzle(v, row, piece) * 16;
    }
    // From the address of a row's piece p below N to that of piece p + N*i (N a power of two, tiles on 128 bytes).
    template <int N>
    static __device__ __forceinline__ uint32_t step(uint32_t from, int i)
    {
        const int span = PP % 8 == 0 ? 8 : (CODED ? 1 : 4);   // pieces among which a row's are moved
        return N >= span ? from + 16 * N * i : (from ^ (16 * N * (i % (span / N)))) + 16 * span * (i / (span / N));
    }
};

template <int D, int FMT, int QT, int NT, bool UNION>
__global__ void __launch_bounds__(kRowsThreads, RowsShape<D, FMT, QT, NT>::CTAS)
kv_rows_kernel(const KvRowsArgs g)
{
    using S = RowsShape<D, FMT, QT, NT>;
    constexpr bool CODED = S::CODED;
    extern __shared__ __align__(128) unsigned char smem[];
    uint2* qf = reinterpret_cast<uint2*>(smem);                       // [NQ][KS][NT][32] operand registers of Q^T
    float* os = reinterpret_cast<float*>(smem + S::QB);               // [NT*8][D+8] value sums, after the loop
    float* sm_m = reinterpret_cast<float*>(smem + S::SUMS);
    float* sm_l = sm_m + kRowsWarps * NT * 8;
    float2* sm_t = reinterpret_cast<float2*>(sm_l + kRowsWarps * NT * 8);   // of the joined warps

    const KvAttend& a = g.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const int h = blockIdx.y, b = blockIdx.z;
    const int tile = blockIdx.x % g.s.row_tiles, split = blockIdx.x / g.s.row_tiles;
    const int G = a.G;
    const int r0 = tile * NT * 8;   // first query row (row*G + head) of the tile

    pdl_launch_dependents();   // kv_join_kernel gets ready meanwhile; it waits for all of this before it reads the parts

    // The first tile's place does not wait for the lengths: what it finds beyond them is not used.
    const int32_t* table = a.w.table + (UNION ? 0 : b * a.w.table_stride);
    const int begin = split * g.s.chunk;
    int to_issue = begin + 16 * warp;
    auto union_at = [&](int at) { return lane < 16 && at + lane < a.M ? __ldg(a.uni + h * a.M + at + lane) : -1; };
    auto place = [&](int pos) {
        return pos >= 0 && (!UNION || pos < a.n) ? kv_page(a.c, table, a.w.table_pages, pos) : -1;
    };
    // All the ring's tiles at once, so that their loads do not wait for one another.
    int pos[S::STAGES], page[S::STAGES];   // of tiles to come: their first token, or (union) their keys'
#pragma unroll
    for (int i = 0; i < S::STAGES; ++i) pos[i] = UNION ? union_at(to_issue + 16 * kRowsWarps * i) : to_issue + 16 * kRowsWarps * i;
    int pos2 = UNION ? union_at(to_issue + 16 * kRowsWarps * S::STAGES) : 0;   // and of the one after them
#pragma unroll
    for (int i = 0; i < S::STAGES; ++i) page[i] = place(pos[i]);

    KvSpan sp;
    int keys;                       // of the tile's rows
    if (UNION) {
        sp = KvSpan{0, 1, 0, 0};
        keys = static_cast<int>(min(static_cast<int64_t>(max(a.count[h], 0)), a.M));
    } else {
        sp = kv_span(a, b);
        if (r0 >= sp.rows * G) return;
        keys = kv_tile_keys(a, sp, r0, NT * 8);
    }
    const int end = min(keys, begin + g.s.chunk);
    if (begin >= keys && split > 0) return;   // the join knows

    // ---- bringing tiles.  A lane copies piece lane % LPR, + LPR, ... of the rows lane / LPR (and + 8).
    const uint32_t ring = smem_addr(smem) + S::QB + warp * (S::STAGES * S::STAGE);
    const int lr = lane / S::LPR, lq = lane % S::LPR;
    const unsigned char* k_lane = a.c.k + h * a.c.head_stride + (UNION ? 0 : lr * a.c.token_stride) + lq * 16;
    const unsigned char* v_lane = a.c.v + h * a.c.head_stride + (UNION ? 0 : lr * a.c.token_stride) + lq * 16;
    // and the exponent bytes of row lane % 16 of K (lanes below 16) or V
    const unsigned char* s_lane =
        CODED ? (lane < 16 ? a.c.ks : a.c.vs) + h * a.c.shead_stride + (UNION ? 0 : (lane & 15) * a.c.stoken_stride) : nullptr;
    int live_of[S::STAGES];                    // which keys of a held tile there are (kept in step with the ring)
    uint32_t sc[2] = {0, 0};                   // exponent bytes on their way
    int slot = 0;
    const uint32_t k_to = S::at(false, lr, lq), v_to = S::at(true, lr, lq);

    // The tile at to_issue, whose place is given, into `slot`; the exponents of the one before to theirs.
    auto issue = [&](int pos1, int page1) {
        if (CODED) {
            const uint32_t at = ring + (slot == 0 ? S::STAGES - 1 : slot - 1) * S::STAGE + 32 * S::RB + lane * S::SBW;
            if (S::SBW == 4) asm volatile("st.shared.u32 [%0], %1;\n" ::"r"(at), "r"(sc[0]) : "memory");
            else asm volatile("st.shared.v2.u32 [%0], {%1,%2};\n" ::"r"(at), "r"(sc[0]), "r"(sc[1]) : "memory");
        }
        const int at = to_issue;
        to_issue = min(at, end) + 16 * kRowsWarps;
        int live = 0;
        if (at < end) {
            const uint32_t dst = ring + slot * S::STAGE;
            const unsigned char *kp[S::RPL], *vp[S::RPL], *sp_;
            if (UNION) {
                const int tok = pos1 & (a.c.page_tokens - 1);
                live = static_cast<int>(__ballot_sync(0xffffffffu, page1 >= 0 && at + lane < end) & 0xffffu);
                const int64_t off = page1 >= 0 ? page1 * a.c.page_stride + tok * a.c.token_stride : 0;
                const int64_t soff = CODED && page1 >= 0 ? page1 * a.c.spage_stride + tok * a.c.stoken_stride : 0;
#pragma unroll
                for (int j = 0; j < S::RPL; ++j) {
                    const int64_t o = __shfl_sync(0xffffffffu, off, lr + 8 * j);
                    kp[j] = k_lane + o;
                    vp[j] = v_lane + o;
                }
                sp_ = s_lane + __shfl_sync(0xffffffffu, soff, lane & 15);
            } else {
                const int tok = at & (a.c.page_tokens - 1);
                live = page1 < 0 ? 0 : (end - at >= 16 ? 0xffff : (1 << (end - at)) - 1);
                const int64_t off = page1 >= 0 ? page1 * a.c.page_stride + tok * a.c.token_stride : 0;
#pragma unroll
                for (int j = 0; j < S::RPL; ++j) {
                    kp[j] = k_lane + off + 8 * j * a.c.token_stride;
                    vp[j] = v_lane + off + 8 * j * a.c.token_stride;
                }
                sp_ = s_lane + (page1 >= 0 ? page1 * a.c.spage_stride + tok * a.c.stoken_stride : 0);
            }
            if (live == 0xffff) {
#pragma unroll
                for (int j = 0; j < S::RPL; ++j)
#pragma unroll
                    for (int i = 0; i < S::PP / S::LPR; ++i) {
                        if (!kv_in(a.c, kp[j] - a.c.k + 16 * S::LPR * i, 16) || !kv_in(a.c, vp[j] - a.c.v + 16 * S::LPR * i, 16)) continue;
                        cp_async16_to(S::template step<S::LPR>(dst + k_to, i) + 8 * j * S::RB, kp[j] + 16 * S::LPR * i);
                        cp_async16_to(S::template step<S::LPR>(dst + v_to, i) + 8 * j * S::RB, vp[j] + 16 * S::LPR * i);
                    }
            } else {
#pragma unroll
                for (int j = 0; j < S::RPL; ++j) {
                    const bool on = (live >> (lr + 8 * j)) & 1;
                    const unsigned char* kf = on ? kp[j] : a.c.k;   // dead rows' addresses are not used: their size is 0
                    const unsigned char* vf = on ? vp[j] : a.c.v;
#pragma unroll
                    for (int i = 0; i < S::PP / S::LPR; ++i) {
                        if (on && (!kv_in(a.c, kf - a.c.k + 16 * S::LPR * i, 16) || !kv_in(a.c, vf - a.c.v + 16 * S::LPR * i, 16))) continue;
                        cp_async16_to(S::template step<S::LPR>(dst + k_to, i) + 8 * j * S::RB, kf + 16 * S::LPR * i, on ? 16 : 0);
                        cp_async16_to(S::template step<S::LPR>(dst + v_to, i) + 8 * j * S::RB, vf + 16 * S::LPR * i, on ? 16 : 0);
                    }
                }
            }
            if (CODED) {
                const bool on = ((live >> (lane & 15)) & 1) && kv_scale_in(a.c, sp_ - (lane < 16 ? a.c.ks : a.c.vs), S::NB);
                sc[0] = sc[1] = 0;
                if (on) {
                    if (S::NB == 4) {
                        sc[0] = __ldg(reinterpret_cast<const uint32_t*>(sp_));
                    } else if (S::NB == 8) {
                        sc[0] = __ldg(reinterpret_cast<const uint32_t*>(sp_));
                        sc[1] = __ldg(reinterpret_cast<const uint32_t*>(sp_) + 1);
                    } else {
#pragma unroll
                        for (int i = 0; i < S::NB; ++i) sc[i >> 2] |= static_cast<uint32_t>(__ldg(sp_ + i)) << (8 * (i & 3));
                    }
                }
            }
        }
        asm volatile("cp.async.commit_group;\n" ::: "memory");
#pragma unroll
        for (int i = 0; i + 1 < S::STAGES; ++i) live_of[i] = live_of[i + 1];
        live_of[S::STAGES - 1] = live;
        slot = slot + 1 == S::STAGES ? 0 : slot + 1;
    };
#pragma unroll
    for (int i = 0; i < S::STAGES; ++i) live_of[i] = 0;
#pragma unroll
    for (int i = 0; i + 1 < S::STAGES; ++i) issue(pos[i], page[i]);
    int pos1 = pos[S::STAGES - 1], page1 = page[S::STAGES - 1];   // of the next tile

    // ---- Q^T operand registers: lane (r, c) of step ks holds channels of row r that match K's.
    for (int e = threadIdx.x; e < S::KS * NT * 32; e += kRowsThreads) {
        const int el = e & 31, nt = (e >> 5) % NT, ks = (e >> 5) / NT, qr = r0 + nt * 8 + (el >> 2);
        const int d = CODED ? (ks / S::KPW) * 4 * S::KPB + (el & 3) * S::KPB + (ks % S::KPW) * 4 : 16 * ks + 2 * (el & 3);
        constexpr int D1 = CODED ? 2 : 1, D2 = CODED ? 1 : 8, D3 = CODED ? 3 : 9;
        float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (qr < sp.rows * G) {
            const int tok = UNION ? 0 : qr / G;
            const int64_t at = (sp.first + tok) * a.q_tok + (static_cast<int64_t>(h) * G + (qr - tok * G)) * a.q_head + d;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t from = at + (j == 0 ? 0 : j == 1 ? D1 : j == 2 ? D2 : D3);
                x[j] = QT == FATHOM_KEYS_F32 ? static_cast<const float*>(a.q)[from]
                                             : __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[from]);
            }
        }
        uint32_t lo[S::NQ], hi[S::NQ];
        split2<S::NQ>(x[0], x[1], lo);
        split2<S::NQ>(x[2], x[3], hi);
#pragma unroll
        for (int p = 0; p < S::NQ; ++p) qf[((p * S::KS + ks) * NT + nt) * 32 + el] = make_uint2(lo[p], hi[p]);
    }

    // Last token that rows 2c, 2c+1 of each tile see (padding rows see all), and the least of any row.
    int seen[NT][2], least = 0x7fffffff;
    const float log2s = a.scale * 1.4426950408889634f;
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
    __syncthreads();

    // Where a lane reads: rows r of K and 2c of V (the others lie 1 and 8 rows behind), or the rows ldmatrix asks for.
    const uint32_t k_rd = CODED ? S::at(false, r, c * S::KPB >> 4) + (c * S::KPB & 15) : S::at(false, lane & 15, lane >> 4);
    const uint32_t v_rd = CODED ? S::at(true, 2 * c, r * S::VPB >> 4) + (r * S::VPB & 15)
                                : S::at(true, (lane & 7) + 8 * (lane >> 4), (lane >> 3) & 1);
    const uint32_t ks_rd = 32 * S::RB + r * S::SBW + (c * S::KPB >> 5);
    const uint32_t vs_rd = 32 * S::RB + (16 + 2 * c) * S::SBW + (r * S::VPB >> 5);
    const CodeMasks masks = code_masks<FMT>();
    int cur = 0;
    for (int at = begin + 16 * warp; at < end; at += 16 * kRowsWarps) {
        asm volatile("cp.async.wait_group %0;\n" ::"n"(S::STAGES - 2) : "memory");
        __syncwarp();
        const int live = live_of[1];   // the oldest tile but the one just used up
        const int next = to_issue + 16 * kRowsWarps;
        issue(pos1, page1);
        pos1 = UNION ? pos2 : next;
        page1 = next < end ? place(pos1) : -1;
        if (UNION) pos2 = union_at(next + 16 * kRowsWarps);
        const uint32_t here = ring + cur * S::STAGE;
        cur = cur + 1 == S::STAGES ? 0 : cur + 1;

        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.0f;
        auto scores = [&](int ks, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
            for (int p = 0; p < S::NQ; ++p)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint2 q = qf[((p * S::KS + ks) * NT + nt) * 32 + lane];
                    mma16816(s[nt], a0, a1, a2, a3, q.x, q.y);
                }
        };
        if constexpr (CODED) {
#pragma unroll
            for (int q = 0; q < S::KP; ++q) {
                uint32_t w[2][S::KPW], f[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    lds_words<S::KPW>(S::template step<S::KPB / 4>(here + k_rd, q) + 8 * i * S::RB, w[i]);
                    f[i] = pow_bits2<FMT>(lds_byte(here + ks_rd + 8 * i * S::SBW + (q * 4 * S::KPB >> 5)));
                }
#pragma unroll
                for (int j = 0; j < S::KPW; ++j) {
                    uint32_t a0, a1, a2, a3;
                    codes4<FMT>(w[0][j], f[0], masks, &a0, &a2);
                    codes4<FMT>(w[1][j], f[1], masks, &a1, &a3);
                    scores(q * S::KPW + j, a0, a1, a2, a3);
                }
            }
        } else {
#pragma unroll
            for (int ks = 0; ks < S::KS; ++ks) {
                uint32_t a0, a1, a2, a3;
                ldmatrix4<false>(S::template step<2>(here + k_rd, ks), a0, a1, a2, a3);
                scores(ks, a0, a1, a2, a3);
            }
        }

        const bool whole = live == 0xffff && at + 15 <= least;
        bool grew = false;
        uint32_t pb[NT][S::NP][2];
        float f[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[nt][i] = __fmul_rn(s[nt][i], log2s);   // never fused with what follows: a step of the maximum may be large
                if (!whole) {
                    const int key = r + 8 * (i >> 1);
                    if (!((live >> key) & 1) || at + key > seen[nt][i & 1]) s[nt][i] = -INFINITY;
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
                const float low = m[nt][i] == -INFINITY ? 0.0f : m[nt][i];
                f[nt][i] = exp2_fast(old - low);
                s[nt][i] = exp2_fast(s[nt][i] - low);
                s[nt][i + 2] = exp2_fast(s[nt][i + 2] - low);
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
        auto values = [&](int t, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int p = 0; p < S::NP; ++p) mma16816(S::WIDEQ ? sum : o[t][nt], a0, a1, a2, a3, pb[nt][p][0], pb[nt][p][1]);
                if (S::WIDEQ) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[t][nt][i] += sum[i];
                }
            }
        };
        if constexpr (CODED) {
#pragma unroll
            for (int q = 0; q < S::VP; ++q) {
                uint32_t w[4][S::VPW], p2[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int on = (i & 1) + 8 * (i >> 1);
                    lds_words<S::VPW>(here + v_rd + on * S::RB + q * 8 * S::VPB, w[i]);
                    p2[i] = pow_bits<FMT>(lds_byte(here + vs_rd + on * S::SBW + (q * 8 * S::VPB >> 5)));
                }
                const uint32_t f01 = p2[0] | p2[1] << 16, f89 = p2[2] | p2[3] << 16;
#pragma unroll
                for (int j = 0; j < S::VPW; ++j) {
                    const int t = (q * S::VPB) / 2 + 2 * j;
                    values(t, decode2<FMT, 0, 0>(w[0][j], w[1][j], f01, masks), decode2<FMT, 1, 1>(w[0][j], w[1][j], f01, masks),
                           decode2<FMT, 0, 0>(w[2][j], w[3][j], f89, masks), decode2<FMT, 1, 1>(w[2][j], w[3][j], f89, masks));
                    values(t + 1, decode2<FMT, 2, 2>(w[0][j], w[1][j], f01, masks), decode2<FMT, 3, 3>(w[0][j], w[1][j], f01, masks),
                           decode2<FMT, 2, 2>(w[2][j], w[3][j], f89, masks), decode2<FMT, 3, 3>(w[2][j], w[3][j], f89, masks));
                }
            }
        } else {
#pragma unroll
            for (int t = 0; t < S::KS; ++t) {
                uint32_t a0, a1, a2, a3;
                ldmatrix4<true>(S::template step<2>(here + v_rd, t), a0, a1, a2, a3);
                values(t, a0, a1, a2, a3);
            }
        }
    }

    // Join the warps.
    cp_async_wait_all();
    __syncthreads();   // the rings have been read
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
            const int row = nt * 8 + 2 * c + i;
            float top = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kRowsWarps; ++w) top = fmaxf(top, sm_m[w * NT * 8 + row]);
            const float low = top == -INFINITY ? 0.0f : top;
            w8[nt][i] = exp2_fast(m[nt][i] - low);
            if (warp == 0 && r == 0) {
#pragma unroll
                for (int w = 0; w < kRowsWarps; ++w) sum += sm_l[w * NT * 8 + row] * exp2_fast(sm_m[w * NT * 8 + row] - low);
                sm_t[row] = make_float2(top, sum);
            }
        }
    // The warps' sums side by side where the ring has room for them, else one after another in one place.
    constexpr int SIDES = S::RING >= kRowsWarps * S::OB ? kRowsWarps : 1;
    constexpr int SIDE = S::OB / sizeof(float);
    for (int w = 0; w < kRowsWarps; w += SIDES) {
        if (SIDES > 1 || warp == w) {
            float* mine = os + (SIDES > 1 ? warp * SIDE : 0);
#pragma unroll
            for (int t = 0; t < S::KS; ++t)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float* to = mine + (nt * 8 + 2 * c + (i & 1)) * (D + 8) + (2 * t + (i >> 1)) * 8 + r;
                        const float x = o[t][nt][i] * w8[nt][i & 1];
                        *to = w == 0 ? x : *to + x;
                    }
        }
        __syncthreads();
    }
    const bool parts = g.s.splits > 1;
    for (int row = warp; row < NT * 8; row += kRowsWarps) {
        const int qr = r0 + row;
        if (qr >= sp.rows * G) break;
        const float2 t = sm_t[row];   // maximum and weight sum
        const int tok = UNION ? 0 : qr / G;
        const int64_t head = ((sp.first + tok) * a.c.H + h) * G + (qr - tok * G), at_p = split * g.heads + head;
        if (!kv_place_in(a.c, head, g.heads) || !kv_place_in(a.c, at_p, g.s.splits * g.heads)) continue;
        if (parts && lane == 0) {
            g.pm[at_p] = t.x;
            g.pl[at_p] = t.y;
        }
#pragma unroll
        for (int d = lane; d < D; d += 32) {
            // with codes, channel d = 8 VPB q + VPB r + j is kept at (VPB q + j) 8 + r
            const int at = row * (D + 8) + (CODED ? ((d / (8 * S::VPB)) * S::VPB + d % S::VPB) * 8 + (d / S::VPB) % 8 : d);
            float x = os[at];
#pragma unroll
            for (int w = 1; w < SIDES; ++w) x += os[w * SIDE + at];
            if (parts) {
                g.po[at_p * D + d] = x;
            } else {
                const float y = t.y == 0.0f ? 0.0f : x / t.y;   // no token was seen (NaN scores make the sum NaN)
                if (QT == FATHOM_KEYS_F32) static_cast<float*>(a.out)[head * D + d] = y;
                else static_cast<__nv_bfloat16*>(a.out)[head * D + d] = __float2bfloat16(y);
            }
        }
    }
}

template <int D, int FMT, int QT, int NT, bool UNION>
int launch_rows_t(const KvRowsArgs& g, cudaStream_t stream)
{
    using S = RowsShape<D, FMT, QT, NT>;
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
