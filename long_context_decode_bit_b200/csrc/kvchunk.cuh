// Attention of prompt chunks over the paged cache on the tensor memory's
// matrix units (tcgen05): bf16 queries, 64, 128 or 256 channels and, with
// zeros behind, the widths between.
//
// A CTA takes 256 query rows (a row is one head of one token; the G heads of
// a group lie next to each other, so they share every cached byte) as two
// tiles of 128, and the tokens of one stretch in tiles of 128; beyond 128
// channels, whose O leaves no room for a second, one tile of rows and tiles
// of 64 tokens, which take the same shared memory.  Per tile of tokens and of rows
//   S [128 x 128] = Q K^T  (both in shared memory, accumulators in tensor memory),
//   P = 2^(S scale log2 e - m), l += row sums,
//   O [128 x D] += P V     (P in tensor memory over S, V in shared memory).
// Roles: warps 0-3 and 4-7 are the softmax of the two row tiles, a thread to
// a row; warps 8-11 bring K and V; one thread of warp 12 issues the products.
// The row tiles take turns: while one's softmax runs, the other's products do.
//
// Both operands are kept with 64 channels (128 bytes) to a row and the
// 128-byte swizzle, K read along the channels and V along the tokens from the
// same layout.  16-bit pages are copied there by cp.async, 16 bytes a thread,
// zeros for tokens that are not there; 8-bit pages are copied beside them, by
// the threads that then decode them to bf16 (once for 256 query rows).
//
// The running maximum m of a row is raised only when it grew by more than
// 2^8 (P and l then stay below 2^8 times what the true maximum gives, far
// inside bf16's and fp32's range), so O is rarely touched between products.
// P enters the product in bf16 (off by up to 2^-8 of a weight); l sums the
// unrounded weights in fp32.  (A second part would be half as many products
// again, on a kernel whose products are active two thirds of the time.)
//
// Every wait on a barrier has an iteration limit; a role whose wait runs out
// sets the fault word and leaves its loop, and the CTA frees its tensor memory.
#pragma once

#include <atomic>
#include <type_traits>

#include "kvrows.cuh"
#include "ring.cuh"

namespace fathom {

constexpr int kChunkThreads = 512;
// Query rows of a CTA and tokens of a tile, by the width of a row.
constexpr int chunk_rows(int D) { return D <= 128 ? 256 : 128; }
constexpr int chunk_keys(int D) { return D <= 128 ? 128 : 64; }
// S scale log2 e - m is one fused operation, and m a rounded product: they differ by half a step of m, which is part of the
// weight's exponent.  From here on (where a step is 2) the product is rounded too.
constexpr float kFarScore = 16777216.0f;
// Registers a thread of each role keeps; their sum is the launch's 4 x 128.
constexpr int kRegsSoftmax = 192, kRegsLoad = 80, kRegsIssue = 48;
static_assert(2 * kRegsSoftmax + kRegsLoad + kRegsIssue <= 512, "more registers than the block has");

template <int D, int FMT>
struct ChunkShape {
    static constexpr bool CODED = FMT != FATHOM_KV_BF16;
    static constexpr bool PAIR = D <= 128;                        // two row tiles in turn, or two tiles of tokens of one
    static constexpr int ROWS = chunk_rows(D), KEYS = chunk_keys(D);
    static constexpr int DB = D / 64;                             // 64-channel blocks of a row
    static constexpr int QTILE = 128 * 128 * DB;                  // bytes of 128 rows of Q
    static constexpr int TILE = KEYS * 128 * DB;                  // and of a tile of K or V
    static constexpr int STAGES = D == 64 ? (CODED ? 6 : 8) : (CODED ? 3 : 5);   // tiles of K or V held as operands
    static constexpr int RAWS = CODED ? (D == 64 ? 4 : 3) : 0;    // and as they come
    static constexpr int RAW = KEYS * D + 2048;                   // codes, and exponents in 16 bytes a thread
    static constexpr int QB = (ROWS / 128) * QTILE;
    static constexpr size_t BARS = QB + static_cast<size_t>(STAGES) * TILE + static_cast<size_t>(RAWS) * RAW;
    static constexpr size_t SMEM = BARS + 256 + 1024;             // the base is moved up to a multiple of 1024
    static_assert(SMEM <= 227 * 1024, "fits an SM, and only once");
    static_assert(SMEM > 114 * 1024, "a CTA has the SM's tensor memory to itself");
};

// ---- tensor memory and its products (cta_group::1)

__device__ __forceinline__ void tmem_alloc(uint32_t smem_at, uint32_t cols)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_at), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
}

__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t cols)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(at), "r"(cols));
}

__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }

// `bar` gets one arrival when every product issued so far by this thread is done.
__device__ __forceinline__ void tc_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar) : "memory");
}

// 32 or 16 columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t at, float* x)
{
    uint32_t* r = reinterpret_cast<uint32_t*>(x);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at)
        : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t at, float* x)
{
    uint32_t* r = reinterpret_cast<uint32_t*>(x);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t* r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Shared-memory operand in 128-byte rows with the 128-byte swizzle: groups of
// 8 rows are 1024 bytes apart; `lbo` is the distance of 64-channel blocks
// where the product runs along the rows (V).
__device__ __forceinline__ uint64_t tc_operand(uint32_t smem_at, uint32_t lbo)
{
    constexpr uint32_t hi = (2u << 29) | (1u << 14) | (1024 >> 4);
    return static_cast<uint64_t>(hi) << 32 | (((lbo >> 4) << 16) + (smem_at >> 4));
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}

// bf16 x bf16 -> fp32, 128 rows, N columns; `along_rows`: B is stored [k][n].
__host__ __device__ constexpr uint32_t tc_shape(int N, bool along_rows)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (along_rows ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(128 >> 4) << 24);
}

__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t shape, bool add)
{
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
                 "l"(a), "l"(b), "r"(shape), "r"(static_cast<uint32_t>(add))
                 : "memory");
}

__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t shape, bool add)
{
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
                 "r"(a), "l"(b), "r"(shape), "r"(static_cast<uint32_t>(add))
                 : "memory");
}

template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N)); }

// ---- pairs of fp32

__device__ __forceinline__ uint64_t pack2(float x, float y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(x), "f"(y));
    return r;
}

__device__ __forceinline__ void unpack2(uint64_t v, float& x, float& y)
{
    asm("mov.b64 {%0, %1}, %2;\n" : "=f"(x), "=f"(y) : "l"(v));
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// ---- bringing K and V

// 16-byte piece `piece` (of D/8) of row `row` of a tile of ROWS rows.
template <int ROWS>
__device__ __forceinline__ uint32_t tile_at(int row, int piece)
{
    return (piece >> 3) * (ROWS * 128) + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
}

__device__ __forceinline__ void st_shared16(uint32_t at, uint4 x)
{
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(at), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
}

// Page of the 16 tokens from `at` + 16*lane (lanes 0..7), -1 for none of this stretch's.
__device__ __forceinline__ int chunk_page(const KvCache& c, const int32_t* table, int table_pages, int at, int end, int lane)
{
    const int pos = at + 16 * lane;
    return lane < 8 && pos < end ? kv_page(c, table, table_pages, pos) : -1;
}

// Where those tokens are, from the start of K or V (-1: nowhere).
__device__ __forceinline__ int64_t chunk_off(const KvCache& c, int page, int at, int h, int lane)
{
    return page < 0 ? -1 : kv_off(c, page, h, (at + 16 * lane) & (c.page_tokens - 1));
}

// The whole tiles of K and V from `begin` on, in the order K0 V0 K1 V1 ..., into the ring.
// D is the width of the operands, c.D (less where not FULL) that of the rows.
template <int D, int FMT, bool FULL>
__device__ __forceinline__ bool chunk_load(const KvRowsArgs& g, const int32_t* table, int h, int begin, int end, uint32_t ring,
                                           uint32_t full, uint32_t empty)
{
    const KvCache& c = g.a.c;
    const int table_pages = g.a.w.table_pages;
    using S = ChunkShape<D, FMT>;
    constexpr int KEYS = S::KEYS;
    constexpr uint32_t ALL = (1u << (KEYS / 16)) - 1;
    const int t = threadIdx.x & 127, lane = threadIdx.x & 31;
    const int tiles = (end - begin + KEYS - 1) / KEYS;
    // This thread's part of tile k is in its place.
    auto filled = [&](int k) {
#ifdef FATHOM_TEST_HOOKS
        // Test build only: one thread of the first CTA of group 0 withholds its arrival for one tile, so that the waits on
        // it run out, and those on what would follow.
        if (k == g.withhold && t == 0 && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) return;
#endif
        mbar_arrive(full + 8 * (k % S::STAGES));
    };
    bool ok = true;
    int page = chunk_page(c, table, table_pages, begin, end, lane);
    if constexpr (FMT == FATHOM_KV_BF16) {
        constexpr int PIECES = D / 8, ROWS = 128 / PIECES;   // rows of a pass
        constexpr int AHEAD = S::STAGES - 2;                 // stages that may be on their way
        const int piece = t % PIECES, r0 = t / PIECES;
        const bool there = FULL || piece * 8 < c.D;
        const uint32_t to0 = ring + tile_at<KEYS>(r0, piece);
        const int64_t row_off = r0 * c.token_stride + piece * 16;
        int i = 0;
        for (int j = 0; j < tiles && ok; ++j) {
            const int at = begin + j * KEYS;
            const int64_t off = chunk_off(c, page, at, h, lane);
            const bool whole = FULL && end - at >= KEYS && (__ballot_sync(0xffffffffu, page >= 0) & ALL) == ALL;
            page = chunk_page(c, table, table_pages, at + KEYS, end, lane);
            for (int s = 0; s < 2; ++s, ++i) {
                const int st = i % S::STAGES;
                ok = __all_sync(0xffffffffu, mbar_wait(empty + 8 * st, ((i / S::STAGES) & 1) ^ 1));
                if (!ok) break;
                const unsigned char* data = s ? c.v : c.k;
#pragma unroll
                for (int p = 0; p < KEYS / ROWS; ++p) {
                    const int64_t o = __shfl_sync(0xffffffffu, off, p * ROWS >> 4);
                    const unsigned char* from = data + o + row_off + (p * ROWS & 15) * c.token_stride;
                    // p*ROWS rows behind; where ROWS is 4, every other time 4 chunks on in the swizzle
                    const uint32_t to = ((to0 + st * S::TILE) ^ ((p * ROWS & 7) << 4)) + p * ROWS * 128;
                    if (whole) {
                        if (kv_in(c, from - data, 16)) cp_async16_to(to, from);
                    } else {
                        const bool live = there && o >= 0 && at + r0 + p * ROWS < end && kv_in(c, from - data, 16);
                        cp_async16_to(to, live ? from : data, live ? 16 : 0);
                    }
                }
                asm volatile("cp.async.commit_group;\n" ::: "memory");
                if (i == 1) {   // the first scores need not wait for what follows
                    asm volatile("cp.async.wait_group 1;\n" ::: "memory");
                    fence_async_smem();
                    filled(0);
                } else if (i > AHEAD) {
                    asm volatile("cp.async.wait_group %0;\n" ::"n"(AHEAD) : "memory");
                    fence_async_smem();
                    filled(i - AHEAD);
                }
            }
        }
        cp_async_wait_all();
        fence_async_smem();
        if (ok)
            for (int k = max(1, i - AHEAD); k < i; ++k) filled(k);
    } else {
        // A thread copies 16-code pieces lq, lq + 4, ... of the rows lr, lr + 32, ... to a place of its own some tiles ahead, and decodes those same pieces from there.
        constexpr int KP = D / 64, RP = KEYS / 32, SW = 4 / RP, AHEAD = S::RAWS - 1;   // SW words of exponents to a row
        const int lr = t >> 2, lq = t & 3, group = lr >> 4;
        const CodeMasks masks = code_masks<FMT>();
        const uint32_t mine = ring + S::STAGES * S::TILE + t * 16;
        const int64_t row_off = (lr & 15) * c.token_stride + lq * 16;
        const int64_t row_soff = (lr & 15) * c.stoken_stride + (FULL && D == 64 ? lq >> 1 : 0);
        const int stages = 2 * tiles;
        int is = 0, at = begin;
        int64_t off = -1, soff = 0;
        uint32_t sc[4] = {0, 0, 0, 0};   // exponent bytes on their way
        auto issue = [&]() {
            const uint32_t slot = mine + (is % S::RAWS) * S::RAW;
            if (is > 0)
                st_shared16(mine + ((is - 1) % S::RAWS) * S::RAW + RP * KP * 2048, make_uint4(sc[0], sc[1], sc[2], sc[3]));
            if (is < stages) {
                if ((is & 1) == 0) {
                    at = begin + (is >> 1) * KEYS;
                    off = chunk_off(c, page, at, h, lane);
                    soff = page < 0 ? 0 : kv_scale_off(c, page, h, (at + 16 * lane) & (c.page_tokens - 1));
                    page = chunk_page(c, table, table_pages, at + KEYS, end, lane);
                }
                const unsigned char* data = (is & 1) ? c.v : c.k;
                const unsigned char* scale = (is & 1) ? c.vs : c.ks;
#pragma unroll
                for (int i = 0; i < RP; ++i) {
                    const int64_t o = __shfl_sync(0xffffffffu, off, group + 2 * i), so = __shfl_sync(0xffffffffu, soff, group + 2 * i);
                    const bool live = o >= 0 && at + lr + 32 * i < end;
                    const unsigned char* from = live ? data + o + row_off : data;
#pragma unroll
                    for (int k = 0; k < KP; ++k) {
                        const bool there = live && (FULL || (lq + 4 * k) * 16 < c.D) && kv_in(c, from + 64 * k - data, 16);
                        cp_async16_to(slot + (i * KP + k) * 2048, there ? from + 64 * k : data, there ? 16 : 0);
                    }
#pragma unroll
                    for (int n = 0; n < SW; ++n) sc[SW * i + n] = 0;
                    if (live && kv_scale_in(c, so + row_soff, 1)) {
                        const unsigned char* sp = scale + so + row_soff;
                        if (FULL && D >= 128) {
#pragma unroll
                            for (int n = 0; n < SW; ++n) sc[SW * i + n] = __ldg(reinterpret_cast<const uint32_t*>(sp) + n);
                        } else if (D == 64) {
                            sc[i] = __ldg(sp);
                        } else {
#pragma unroll
                            for (int n = 0; n < D / kKvBlock; ++n)
                                if (n * kKvBlock < c.D) sc[SW * i + (n >> 2)] |= static_cast<uint32_t>(__ldg(sp + n)) << (8 * (n & 3));
                        }
                    }
                }
            }
            asm volatile("cp.async.commit_group;\n" ::: "memory");
            ++is;
        };
        for (int i = 0; i < AHEAD; ++i) issue();
        int i = 0;
        for (; i < stages && ok; ++i) {
            asm volatile("cp.async.wait_group %0;\n" ::"n"(AHEAD - 1) : "memory");
            issue();
            const int st = i % S::STAGES;
            ok = __all_sync(0xffffffffu, mbar_wait(empty + 8 * st, ((i / S::STAGES) & 1) ^ 1));
            if (!ok) break;
            const uint32_t from = mine + (i % S::RAWS) * S::RAW, to = ring + st * S::TILE + tile_at<KEYS>(lr, 2 * lq);
            uint32_t ps[4];
            lds_words<4>(from + RP * KP * 2048, ps);
#pragma unroll
            for (int r = 0; r < RP; ++r)
#pragma unroll
                for (int k = 0; k < KP; ++k) {
                    uint32_t w[4];
                    lds_words<4>(from + (r * KP + k) * 2048, w);
                    const uint32_t byte = D == 64 ? ps[r] : (ps[SW * r + (k >> 1)] >> (16 * (k & 1) + 8 * (lq >> 1))) & 0xff;
                    const uint32_t f = pow_bits2<FMT>(byte);
                    // the row's two 16-byte pieces, the second one chunk on in the swizzle
                    const uint32_t there = to + r * 32 * 128 + k * (KEYS * 128);
                    st_shared16(there, make_uint4(decode2<FMT, 0, 1>(w[0], w[0], f, masks), decode2<FMT, 2, 3>(w[0], w[0], f, masks),
                                                  decode2<FMT, 0, 1>(w[1], w[1], f, masks), decode2<FMT, 2, 3>(w[1], w[1], f, masks)));
                    st_shared16(there ^ 16, make_uint4(decode2<FMT, 0, 1>(w[2], w[2], f, masks), decode2<FMT, 2, 3>(w[2], w[2], f, masks),
                                                       decode2<FMT, 0, 1>(w[3], w[3], f, masks), decode2<FMT, 2, 3>(w[3], w[3], f, masks)));
                }
            fence_async_smem();
            filled(i);
        }
        cp_async_wait_all();
    }
    return ok;
}

template <int D, int FMT, bool FULL>
__global__ void __launch_bounds__(kChunkThreads, 1)
kv_chunk_kernel(const KvRowsArgs g, int32_t* __restrict__ fault)
{
    using S = ChunkShape<D, FMT>;
    constexpr int ST = S::STAGES, KEYS = S::KEYS;
    constexpr uint32_t ALL = (1u << (KEYS / 16)) - 1;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* base = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const uint32_t q_s = smem_addr(base), ring = q_s + S::QB, bars = q_s + static_cast<uint32_t>(S::BARS);
    const uint32_t full = bars, empty = bars + 8 * ST, s_full = bars + 16 * ST, p_full = s_full + 16, o_full = p_full + 32,
                   q_full = o_full + 16, drain = q_full + 8, tmem_slot = drain + 8;
    static_assert(16 * ST + 16 * 4 + 8 * 2 + 4 <= 256, "barriers fit their space");

    pdl_launch_dependents();   // kv_join_kernel gets ready meanwhile
    const KvAttend& a = g.a;
    // the same in all lanes, as the compiler can tell
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int h = blockIdx.y, b = blockIdx.z, G = a.G;
    // Later rows see more tokens: they start first.
    const int tile = g.s.row_tiles - 1 - static_cast<int>(blockIdx.x % g.s.row_tiles), split = blockIdx.x / g.s.row_tiles;
    const int r0 = tile * S::ROWS;
    const KvSpan sp = kv_span(a, b);
    const int nrows = sp.rows * G;
    if (r0 >= nrows) return;
    const int keys = kv_tile_keys(a, sp, r0, S::ROWS);
    const int begin = split * g.s.chunk, end = min(keys, begin + g.s.chunk);
    if (begin >= keys && split > 0) return;   // the join knows
    const int tiles = (max(end - begin, 0) + KEYS - 1) / KEYS;
    const bool two = S::PAIR && r0 + 128 < nrows;   // the second row tile has rows
    const int32_t* table = a.w.table + b * a.w.table_stride;

    if (warp == 12) {
        tmem_alloc(tmem_slot, 512);
        if (lane == 0) {
            for (int i = 0; i < ST; ++i) {
                mbar_init(full + 8 * i, 128);
                mbar_init(empty + 8 * i, 1);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(s_full + 8 * i, 1);
                mbar_init(p_full + 8 * i, 128);        // the first half of the weights
                mbar_init(p_full + 16 + 8 * i, 128);   // and the second
                mbar_init(o_full + 8 * i, 1);
            }
            mbar_init(q_full, 256);
            mbar_init(drain, 1);
            asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
        }
        tc_before();
    }
    __syncthreads();
    tc_after();
    uint32_t tmem;
    asm volatile("ld.shared.b32 %0, [%1];\n" : "=r"(tmem) : "r"(tmem_slot));

    if (warp >= 12) {
        regs_down<kRegsIssue>();
        if (warp == 12 && tiles > 0) {
            // The whole warp goes along, so that operands are in uniform registers; one lane issues.  (A lane on its own
            // took 90 cycles to a product, more than the product.)
            constexpr uint32_t shape_s = tc_shape(KEYS, false), shape_o = tc_shape(D, true);
            auto scores = [&](int t, int st) {
                const uint64_t q = tc_operand(q_s + (S::PAIR ? t * S::QTILE : 0), 0), k = tc_operand(ring + st * S::TILE, 0);
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t off = (ks & 3) * 32 >> 4;
                        tc_mma_ss(tmem + 128 * t, q + ((ks >> 2) * (128 * 128) >> 4) + off, k + ((ks >> 2) * (KEYS * 128) >> 4) + off,
                                  shape_s, ks > 0);
                    }
                    tc_commit(s_full + 8 * t);
                }
                __syncwarp();
            };
            auto values = [&](int t, int st, int half, bool add) {
                const uint64_t v = tc_operand(ring + st * S::TILE + half * (KEYS / 2) * 128, KEYS * 128);
                const uint32_t p = tmem + 128 * t + half * (KEYS / 4);
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < KEYS / 32; ++ks)
                        tc_mma_ts(tmem + 256 + (S::PAIR ? 128 * t : 0), p + 8 * ks, v + ks * (2048 >> 4), shape_o, add || ks > 0);
                }
                __syncwarp();
            };
            auto done = [&](uint32_t bar) {
                if (elect_one()) tc_commit(bar);
                __syncwarp();
            };
            auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity)); };
            const int nt = two ? 2 : 1;
            bool ok = wait(q_full, 0) && wait(full, 0);
            if (ok) {
                tc_after();
                for (int t = 0; t < nt; ++t) scores(t, 0);
                done(empty);
            }
            if constexpr (S::PAIR) {
                for (int j = 0; j < tiles && ok; ++j) {
                    const int iv = 2 * j + 1, ik = iv + 1;
                    const bool more = j + 1 < tiles;
                    ok = wait(full + 8 * (iv % ST), (iv / ST) & 1);
                    for (int t = 0; t < nt && ok; ++t) {
                        for (int half = 0; half < 2 && ok; ++half) {
                            ok = wait(p_full + 16 * half + 8 * t, j & 1);
                            if (!ok) break;
                            tc_after();
                            values(t, iv % ST, half, j > 0 || half > 0);
                        }
                        if (!ok) break;
                        if (!more) done(o_full + 8 * t);
                        if (t == nt - 1) done(empty + 8 * (iv % ST));
                        if (more) {
                            if (t == 0) ok = wait(full + 8 * (ik % ST), (ik / ST) & 1);
                            if (!ok) break;
                            scores(t, ik % ST);
                        }
                    }
                    if (ok && more) done(empty + 8 * (ik % ST));
                }
            } else {
                // The next tile's scores are taken while this one's softmax runs.
                for (int j = 0; j < tiles && ok; ++j) {
                    const int iv = 2 * j + 1, ik = iv + 1, t = j & 1;
                    if (j + 1 < tiles) {
                        ok = wait(full + 8 * (ik % ST), (ik / ST) & 1);
                        if (!ok) break;
                        tc_after();
                        scores(1 - t, ik % ST);
                        done(empty + 8 * (ik % ST));
                    }
                    ok = wait(full + 8 * (iv % ST), (iv / ST) & 1);
                    for (int half = 0; half < 2 && ok; ++half) {
                        ok = wait(p_full + 16 * half + 8 * t, (j >> 1) & 1);
                        if (!ok) break;
                        tc_after();
                        values(t, iv % ST, half, j > 0 || half > 0);
                    }
                    if (!ok) break;
                    done(empty + 8 * (iv % ST));
                    done(o_full + 8 * t);
                }
            }
            // Nothing is on its way in tensor memory when it is freed.
            done(drain);
            if (!wait(drain, 0)) ok = false;
            if (!ok && lane == 0) atomicOr(fault, kFaultTimeout);
        }
        __syncwarp();
    } else if (warp >= 8) {
        regs_down<kRegsLoad>();
        if (!chunk_load<D, FMT, FULL>(g, table, h, begin, end, ring, full, empty)) atomicOr(fault, kFaultTimeout);
    } else {
        regs_up<kRegsSoftmax>();
        {   // Q, by all these warps
            constexpr int PIECES = D / 8, ROWS = 256 / PIECES;
            const int piece = threadIdx.x % PIECES, at_row = threadIdx.x / PIECES;
            const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + static_cast<int64_t>(h) * G * a.q_head + piece * 8;
            const bool wide = FULL || piece * 8 < a.c.D;
            const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;   // the softmax uses |scale|
            const bool vec = flip == 0 && ((reinterpret_cast<uintptr_t>(q) & 15) | (a.q_tok & 7) | (a.q_head & 7)) == 0;
#pragma unroll 4
            for (int row = at_row; row < S::ROWS; row += ROWS) {
                const unsigned qr = min(r0 + row, nrows - 1), tok = qr / static_cast<unsigned>(G), g1 = qr - tok * G;
                const bool there = wide && r0 + row < nrows;
                const uint32_t to = q_s + (row >> 7) * S::QTILE + tile_at<128>(row & 127, piece);
                const __nv_bfloat16* from = q + (sp.first + tok) * a.q_tok + g1 * a.q_head;
                if (vec) {
                    cp_async16_to(to, there ? from : static_cast<const __nv_bfloat16*>(a.q), there ? 16 : 0);
                } else {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = there ? (__bfloat16_as_ushort(from[2 * i]) |
                                        static_cast<uint32_t>(__bfloat16_as_ushort(from[2 * i + 1])) << 16) ^ flip
                                     : 0u;
                    st_shared16(to, make_uint4(w[0], w[1], w[2], w[3]));
                }
            }
            cp_async_wait_all();
            fence_async_smem();
            mbar_arrive(q_full);
        }
        const int t = warp >> 2;
        const int qr = r0 + threadIdx.x;
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t o_at = tmem + lanes + 256 + 128 * t;
        // Tokens before `mine` are seen by this thread's row (a row that is not there: all).
        const int mine = a.causal && qr < nrows ? min(end, sp.pos0 + qr / G + 1) : end;
        // No smaller than the least normal number: -inf times it stays -inf, and 2^(x 1e-38) is 1.
        const float log2s = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1.17549435e-38f);
        const uint64_t log2s2 = pack2(log2s, log2s);
        float m = -INFINITY, l = 0.0f;
        bool ok = true, far = false;   // far: a row of the warp has a maximum that fp32 holds to no better than 1
        if (t == 0 || two) {
            int page = chunk_page(a.c, table, a.w.table_pages, begin, end, lane);
            for (int j = 0; j < tiles; ++j) {
                const int at = begin + j * KEYS;
                const uint32_t live = __ballot_sync(0xffffffffu, page >= 0) & ALL;
                const int buf = S::PAIR ? t : j & 1, phase = S::PAIR ? j & 1 : (j >> 1) & 1;
                const uint32_t s_at = tmem + lanes + 128 * buf;
                page = chunk_page(a.c, table, a.w.table_pages, at + KEYS, end, lane);
                ok = __all_sync(0xffffffffu, mbar_wait(s_full + 8 * buf, phase));
                // Of one row tile: product j reports to barrier j & 1.  Waiting for product j - 2 here keeps the phases
                // apart: the next one of that barrier, product j, cannot be before this iteration's weights.
                if (!S::PAIR && j >= 2) ok = __all_sync(0xffffffffu, ok && mbar_wait(o_full + 8 * (j & 1), ((j - 2) >> 1) & 1));
                if (!ok) break;
                tc_after();
                float s[KEYS];
#pragma unroll
                for (int i = 0; i < KEYS / 32; ++i) tmem_ld32(s_at + 32 * i, s + 32 * i);
                tmem_ld_wait();
                const int lim = mine - at;
                if (!__all_sync(0xffffffffu, lim >= KEYS) || live != ALL) {
#pragma unroll
                    for (int i = 0; i < KEYS; ++i)
                        if (i >= lim || !((live >> (i >> 4)) & 1)) s[i] = -INFINITY;
                }
                float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int i = 4; i < KEYS; i += 8)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        top[k] = i + 4 + k < KEYS ? fmaxf(fmaxf(top[k], s[i + k]), s[i + 4 + k]) : fmaxf(top[k], s[i + k]);
                const float peak = fmaxf(m, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * log2s);
                if (__any_sync(0xffffffffu, peak > m + 8.0f)) {
                    const float f = exp2_fast(m - (peak == -INFINITY ? 0.0f : peak));
                    l *= f;
                    m = peak;
                    far = __any_sync(0xffffffffu, fabsf(m) >= kFarScore && m > -INFINITY);
                    if (j > 0) {
                        if (!S::PAIR) {   // of a pair, the product before is done: this tile's scores came after it
                            ok = __all_sync(0xffffffffu, mbar_wait(o_full + 8 * ((j - 1) & 1), ((j - 1) >> 1) & 1));
                            if (!ok) break;
                            tc_after();
                        }
#pragma unroll
                        for (int i = 0; i < D; i += 16) {
                            float o[16];
                            tmem_ld16(o_at + i, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] *= f;
                            tmem_st16(o_at + i, reinterpret_cast<const uint32_t*>(o));
                        }
                    }
                }
                const float low = m == -INFINITY ? 0.0f : -m;
                const uint64_t low2 = pack2(low, low);
                uint64_t sum[2] = {pack2(l, 0.0f), pack2(0.0f, 0.0f)};
                auto weights = [&](auto rounded) {
#pragma unroll
                    for (int part = 0; part < KEYS / 32; ++part) {
                        uint32_t p[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float x = s[32 * part + 2 * i], y = s[32 * part + 2 * i + 1];
                            if constexpr (decltype(rounded)::value) {   // as the maximum was, so that no weight is above 2^8
                                x = __fadd_rn(__fmul_rn(x, log2s), low);
                                y = __fadd_rn(__fmul_rn(y, log2s), low);
                            } else {
                                unpack2(fma2(pack2(x, y), log2s2, low2), x, y);
                            }
                            x = exp2_fast(x);
                            y = exp2_fast(y);
                            sum[i & 1] = add2(sum[i & 1], pack2(x, y));
                            p[i] = bf16x2(x, y);
                        }
                        tmem_st16(s_at + 16 * part, p);
                        if (KEYS == 64 || (part & 1)) {   // half of the tile
                            tmem_st_wait();
                            tc_before();
                            mbar_arrive(p_full + 16 * (KEYS == 64 ? part : part >> 1) + 8 * buf);
                        }
                    }
                };
                if (far) weights(std::true_type{});
                else weights(std::false_type{});
                float l0, l1;
                unpack2(add2(sum[0], sum[1]), l0, l1);
                l = l0 + l1;
            }
            if (ok && tiles > 0) {
                const int last = tiles - 1;
                ok = __all_sync(0xffffffffu, S::PAIR ? mbar_wait(o_full + 8 * t, 0) : mbar_wait(o_full + 8 * (last & 1), (last >> 1) & 1));
                tc_after();
            }
            if (!ok) {
                if (lane == 0) atomicOr(fault, kFaultTimeout);
            } else {
                const int64_t head = ((sp.first + qr / G) * a.c.H + h) * G + qr % G;
                const int64_t width = FULL ? D : a.c.D;
                const bool parts = g.s.splits > 1;
                const float f = parts ? 1.0f : (l > 0.0f ? 1.0f / l : 0.0f);
                const int64_t at_p = split * g.heads + head;
                const bool nothing = l == 0.0f;   // no token was seen (NaN scores make l NaN)
#pragma unroll
                for (int i = 0; i < D; i += 32) {
                    if (!FULL && i >= a.c.D) break;
                    float o[32];
                    if (tiles > 0) {
                        tmem_ld32(o_at + i, o);
                        tmem_ld_wait();
                    }
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = nothing ? 0.0f : o[k] * f;
                    if (qr < nrows && kv_place_in(a.c, head, g.heads) && kv_place_in(a.c, at_p, g.s.splits * g.heads)) {
                        if (parts) {
                            float* to = g.po + at_p * width + i;
#pragma unroll
                            for (int k = 0; k < 32; k += 8) st_global32(to + k, reinterpret_cast<const uint32_t*>(o + k));
                        } else {
                            __nv_bfloat16* to = static_cast<__nv_bfloat16*>(a.out) + head * width + i;
                            if ((reinterpret_cast<uintptr_t>(a.out) & 31) == 0) {
                                uint32_t w[16];
#pragma unroll
                                for (int k = 0; k < 16; ++k) w[k] = bf16x2(o[2 * k], o[2 * k + 1]);
                                st_global32(to, w);
                                st_global32(to + 16, w + 8);
                            } else {
#pragma unroll
                                for (int k = 0; k < 32; ++k) to[k] = __float2bfloat16(o[k]);
                            }
                        }
                    }
                }
                if (parts && qr < nrows) {
                    g.pm[at_p] = m;
                    g.pl[at_p] = l;
                }
            }
        }
        tc_before();
    }
    __syncthreads();
    if (warp == 12) {
        tc_after();
        tmem_free(tmem, 512);
    }
}

template <int D, int FMT, bool FULL>
int launch_chunk_t(const KvRowsArgs& g, cudaStream_t stream)
{
    using S = ChunkShape<D, FMT>;
    const void* f = reinterpret_cast<const void*>(kv_chunk_kernel<D, FMT, FULL>);
    // The roles' registers must add up to no more than the block is launched with, or the softmax waits for ever.
    static std::atomic<int> launch_regs{0};   // the same on every device
    if (launch_regs.load(std::memory_order_relaxed) == 0) {
        cudaFuncAttributes attr;
        const cudaError_t e = cudaFuncGetAttributes(&attr, f);
        if (e != cudaSuccess) return cuda_status(e);
        launch_regs.store(attr.numRegs, std::memory_order_relaxed);
    }
    if (4 * launch_regs.load(std::memory_order_relaxed) < 2 * kRegsSoftmax + kRegsLoad + kRegsIssue) return FATHOM_ERR_UNSUPPORTED;
    int32_t* fault = nullptr;
    int st = device_fault_word(&fault);
    if (st) return st;
    st = ensure_dynamic_smem(f, S::SMEM);
    if (st) return st;
    const dim3 grid(static_cast<unsigned>(g.s.splits) * g.s.row_tiles, static_cast<unsigned>(g.a.c.H),
                    static_cast<unsigned>(g.a.w.B));
    kv_chunk_kernel<D, FMT, FULL><<<grid, kChunkThreads, S::SMEM, stream>>>(g, fault);
    return launch_status();
}

// kvchunk.cu: chunks of bf16 queries over caches of 32 to 256 channels (widths between 64, 128 and 256 with zeros behind).
int launch_chunk(const KvRowsArgs& g, int format, cudaStream_t stream);

}  // namespace fathom
