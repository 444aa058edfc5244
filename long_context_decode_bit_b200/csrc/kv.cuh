// The paged KV cache on the device: addressing, the rows of a call, and the
// decoding of cached elements (include/fathom.h has the formats).
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace fathom {

constexpr int kKvBlock = 32;     // channels that share a power of two
constexpr int kKvLowest = -100;  // smallest exponent kept
constexpr int kKvThreads = 256;  // of a CTA that writes or reads rows

struct KvCache {
    const unsigned char* k;
    const unsigned char* v;
    const unsigned char* ks;
    const unsigned char* vs;
    int64_t page_stride, head_stride, token_stride;      // bytes
    int64_t spage_stride, shead_stride, stoken_stride;   // bytes
    int32_t pages, H, D, page_tokens, page_shift;
#ifdef FATHOM_DEBUG_BOUNDS
    int64_t bytes, scale_bytes;   // from the first to behind the last byte of K or V, and of their exponents
    int32_t* fault;
#endif
};

struct KvRows {
    const int32_t* table;
    const int32_t* cu;
    const int32_t* length;
    int64_t table_stride;
    int32_t rows, table_pages, B;
};

// One call of either attention.
struct KvAttend {
    KvCache c;
    KvRows w;               // table, cu, length (paged attention); table alone (union)
    const void* q;
    void* out;
    int64_t q_tok, q_head;  // elements
    int64_t n;              // union: tokens an index may name
    int64_t M;
    const int32_t* uni;     // union: [H][M]
    const int32_t* count;
    int64_t max_new, max_len;
    float scale;
    int G, causal;
};

// CTAs of a write: a thread takes 16 channels of a row.
inline int64_t kv_write_ctas(int64_t rows, int H, int D) { return ceil_div(rows * H * (D / 16), kKvThreads); }

// Bytes of a cached element.
template <int FMT>
__host__ __device__ constexpr int kv_elem_bytes() { return FMT == FATHOM_KV_BF16 ? 2 : 1; }

// Page of position `pos` of table row `t`, or -1 where it names no token.
__device__ __forceinline__ int kv_page(const KvCache& c, const int32_t* t, int table_pages, int64_t pos)
{
    const int64_t i = pos >> c.page_shift;
    if (pos < 0 || i >= table_pages) return -1;
    const int p = __ldg(t + i);
    return p >= 0 && p < c.pages ? p : -1;
}

__device__ __forceinline__ int64_t kv_off(const KvCache& c, int page, int h, int token)
{
    return page * c.page_stride + h * c.head_stride + token * c.token_stride;
}

__device__ __forceinline__ int64_t kv_scale_off(const KvCache& c, int page, int h, int token)
{
    return page * c.spage_stride + h * c.shead_stride + token * c.stoken_stride;
}

// Debug build: `n` bytes `off` from the start of K or V, or of their exponents, are the cache's (bounds_ok).
__device__ __forceinline__ bool kv_in(const KvCache& c, int64_t off, int n)
{
#ifdef FATHOM_DEBUG_BOUNDS
    return bounds_ok(off >= 0 && off + n <= c.bytes, c.fault);
#else
    return true;
#endif
}

__device__ __forceinline__ bool kv_scale_in(const KvCache& c, int64_t off, int n)
{
#ifdef FATHOM_DEBUG_BOUNDS
    return bounds_ok(off >= 0 && off + n <= c.scale_bytes, c.fault);
#else
    return true;
#endif
}

// The same of place `at` of the `n` that an output or a call's scratch has.
__device__ __forceinline__ bool kv_place_in(const KvCache& c, int64_t at, int64_t n)
{
#ifdef FATHOM_DEBUG_BOUNDS
    return bounds_ok(at >= 0 && at < n, c.fault);
#else
    return true;
#endif
}

// Sequence of row r (cu[b] <= r < cu[b+1]), or -1: the last b whose cu[b] <= r.
__device__ __forceinline__ int kv_sequence(const KvRows& w, int r)
{
    int lo = 0, hi = w.B;   // the answer lies in [lo, hi)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(w.cu + mid) <= r) lo = mid;
        else hi = mid;
    }
    return r >= __ldg(w.cu + lo) && r < __ldg(w.cu + lo + 1) ? lo : -1;
}

// fp32 value of 2^e from its byte (e + 127); 255 is an infinity, which turns
// the zero codes kept with it into NaN.
__device__ __forceinline__ float kv_pow2(uint32_t byte) { return __uint_as_float(byte << 23); }

// ---- 8-bit codes to bf16, two at a time

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

// (x & y) | z
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t y, uint32_t z)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;\n" : "=r"(r) : "r"(x), "r"(y), "r"(z));
    return r;
}

// Masks of the decoders, kept in registers: an instruction takes one constant only.
struct CodeMasks {
    uint32_t a, b, c;
};

template <int FMT>
__device__ __forceinline__ CodeMasks code_masks()
{
    CodeMasks m;
    asm volatile("mov.b32 %0, %3;\n mov.b32 %1, %4;\n mov.b32 %2, %5;\n"
                 : "=r"(m.a), "=r"(m.b), "=r"(m.c)
                 : "n"(FMT == FATHOM_KV_INT8 ? 0x007f007f : 0x07f007f0), "n"(FMT == FATHOM_KV_INT8 ? 0x00800080 : 0x80008000),
                   "n"(0x43004300));
    return m;
}

// INT8 codes in the low bytes of each 16 bits as bf16 values, times the powers f:
// 128 + low 7 bits, less 128, or 256 for a negative code.
__device__ __forceinline__ uint32_t decode_low(uint32_t t, uint32_t f, const CodeMasks& m)
{
    return bmul2(bsub2(and_or(t, m.a, m.c), and_or(t, m.b, m.c)), f);
}

// E4M3 codes in the high bytes: sign in place, exponent and mantissa 4 below; 2^120 of the power makes up for the bias.
__device__ __forceinline__ uint32_t decode_high(uint32_t t, uint32_t f, const CodeMasks& m)
{
    return bmul2(and_or(t, m.b, (t >> 4) & m.a), f);
}

// Bytes BLO of x and BHI of y.
template <int FMT, int BLO, int BHI>
__device__ __forceinline__ uint32_t decode2(uint32_t x, uint32_t y, uint32_t f, const CodeMasks& m)
{
    if (FMT == FATHOM_KV_INT8) return decode_low(__byte_perm(x, y, BLO | ((4 + BHI) << 8)), f, m);
    return decode_high(__byte_perm(x, y, (BLO << 4) | ((4 + BHI) << 12)), f, m);
}

// The 16 bits that decode2 multiplies with, from the exponent byte.
template <int FMT>
__device__ __forceinline__ uint32_t pow_bits(uint32_t byte)
{
    return (FMT == FATHOM_KV_INT8 ? byte : min(byte + 120u, 255u)) << 7;
}

// The same twice over.
template <int FMT>
__device__ __forceinline__ uint32_t pow_bits2(uint32_t byte)
{
    return FMT == FATHOM_KV_INT8 ? byte * 0x00800080u : pow_bits<FMT>(byte) * 0x10001u;
}

// 32 bytes at once: half as many lines to a warp's stores as with 16, where each thread has its own.
__device__ __forceinline__ void st_global32(void* p, const uint32_t* w)
{
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Two bf16 from two fp32, the first in the low half.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The same, rounded towards zero.
__device__ __forceinline__ uint32_t bf16x2_cut(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rz.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace fathom
