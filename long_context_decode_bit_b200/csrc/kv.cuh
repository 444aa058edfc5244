// The paged KV cache on the device: addressing, the rows of a call, and the
// decoding of cached elements (include/fathom.h has the formats).
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace fathom {

constexpr int kKvBlock = 32;     // channels that share a power of two
constexpr int kKvLowest = -100;  // smallest exponent kept

struct KvCache {
    const unsigned char* k;
    const unsigned char* v;
    const unsigned char* ks;
    const unsigned char* vs;
    int64_t page_stride, head_stride, token_stride;      // bytes
    int64_t spage_stride, shead_stride, stoken_stride;   // bytes
    int32_t pages, H, D, page_tokens, page_shift;
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

// Two bf16 from two fp32, the first in the low half.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace fathom
