// fathom_kv_write and fathom_kv_read: rows into the paged cache and back.
//
// A thread takes 16 channels of one row of K and of V; the two threads of a
// 32-channel block find its largest magnitude with a shuffle.  Magnitudes are
// compared as bit patterns, which orders NaN above infinity above every
// number, so one compare finds the blocks that cannot be kept.  The exponent
// comes from the pattern too (exponent field, and one compare of the fraction
// with the value that would round over the largest code), so no division or
// logarithm is rounded anywhere and x 2^-e is exact before the one rounding to
// the code.
//
// Both kernels stream: bound by HBM, or by the launch when a decode step
// writes one token.  A row's place is three loads that wait for one another
// (its sequence, its length, its page); many small threads hide the chain
// better than several rows to a thread (a 128k int8 session of 8 groups read
// back in bf16: 131 us, 6.2 TB/s, against 137 us with four; 32k tokens written and
// read back 70 us against 80, bf16 and e4m3 caches 90 and 70; a token 4.4 us
// against 6.6).
#include "kv.cuh"

namespace fathom {

namespace {

__device__ __forceinline__ void ld_global32(const void* p, uint4* u)
{
    asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                 : "=r"(u[0].x), "=r"(u[0].y), "=r"(u[0].z), "=r"(u[0].w), "=r"(u[1].x), "=r"(u[1].y), "=r"(u[1].z), "=r"(u[1].w)
                 : "l"(p));
}

// 16 elements as they lie: two 16-byte pieces of bf16, four of fp32.
template <int DT>
struct Raw16 {
    uint4 u[DT == FATHOM_KEYS_BF16 ? 2 : 4];
};

// VEC: bytes that all pieces are aligned to (32, 16, or 0 for less).  Whole sectors with one instruction where that is 32.
template <int DT, int VEC>
__device__ __forceinline__ void kv_load16(const void* p, int64_t at, Raw16<DT>* raw)
{
    constexpr int N = DT == FATHOM_KEYS_BF16 ? 2 : 4;
    if (VEC) {
        const uint4* s = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(p) + at * (DT == FATHOM_KEYS_BF16 ? 2 : 4));
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            if (VEC == 32) {
                ld_global32(s + i, &raw->u[i]);
            } else {
                raw->u[i] = __ldg(s + i);
                raw->u[i + 1] = __ldg(s + i + 1);
            }
        }
    } else if (DT == FATHOM_KEYS_BF16) {
        const unsigned short* s = static_cast<const unsigned short*>(p) + at;
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = s[2 * i] | static_cast<uint32_t>(s[2 * i + 1]) << 16;
#pragma unroll
        for (int i = 0; i < N; ++i) raw->u[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else {
        const uint32_t* s = static_cast<const uint32_t*>(p) + at;
#pragma unroll
        for (int i = 0; i < N; ++i) raw->u[i] = make_uint4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
    }
}

template <int DT>
__device__ __forceinline__ void kv_values(const Raw16<DT>& raw, float (&x)[16])
{
#pragma unroll
    for (int i = 0; i < (DT == FATHOM_KEYS_BF16 ? 2 : 4); ++i) {
        const uint32_t w[4] = {raw.u[i].x, raw.u[i].y, raw.u[i].z, raw.u[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (DT == FATHOM_KEYS_BF16) {
                x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
                x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            } else {
                x[4 * i + j] = __uint_as_float(w[j]);
            }
        }
    }
}

// Bit pattern (fp32) of the largest magnitude of a 32-channel block, of which this thread and its neighbour have half each.
template <int DT>
__device__ __forceinline__ uint32_t kv_largest(const Raw16<DT>& raw)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < (DT == FATHOM_KEYS_BF16 ? 2 : 4); ++i) {
        const uint32_t w[4] = {raw.u[i].x, raw.u[i].y, raw.u[i].z, raw.u[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) m = DT == FATHOM_KEYS_BF16 ? __vmaxu2(m, w[j] & 0x7fff7fffu) : max(m, w[j] & 0x7fffffffu);
    }
    if (DT == FATHOM_KEYS_BF16) m = max(m << 16, m & 0xffff0000u);
    return max(m, __shfl_xor_sync(0xffffffffu, m, 1));
}

// Codes of 16 channels and their block's exponent byte, m from kv_largest.
template <int FMT>
__device__ __forceinline__ uint4 kv_encode16(float (&x)[16], uint32_t m, uint32_t* byte)
{
    if (m >= 0x7f800000u) {
        *byte = 255;
        return make_uint4(0, 0, 0, 0);
    }
    const int ex = static_cast<int>(m >> 23) - 127;
    const uint32_t frac = m & 0x7fffffu;
    // INT8: 64 f in [64, 128) rounds to 128 from 127.5 on.  E4M3: 256 f rounds to 448 up to 464 (a tie, to even).
    int e = FMT == FATHOM_KV_INT8 ? ex - 6 + (frac >= 0x7f0000u) : ex - 8 + (frac > 0x680000u);
    e = min(max(e, kKvLowest), FMT == FATHOM_KV_INT8 ? 121 : 7);
    *byte = static_cast<uint32_t>(e + 127);
    const float f = kv_pow2(static_cast<uint32_t>(127 - e));
    uint32_t w[4];
    if (FMT == FATHOM_KV_INT8 && e == 121) {   // only there a code could become 128
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = fminf(fmaxf(x[i], -0x7fp121f), 0x7fp121f);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (FMT == FATHOM_KV_INT8) {
            // x f + 1.5 2^23: the product is exact, the sum is rounded to a whole number, kept in its low bits
            uint32_t r[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                r[j] = __float_as_uint(fmaf(x[4 * i + j], f, 12582912.0f));
            w[i] = __byte_perm(__byte_perm(r[0], r[1], 0x0040), __byte_perm(r[2], r[3], 0x0040), 0x5410);
        } else {
            const float2 lo = make_float2(x[4 * i] * f, x[4 * i + 1] * f), hi = make_float2(x[4 * i + 2] * f, x[4 * i + 3] * f);
            w[i] = static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(lo, __NV_SATFINITE, __NV_E4M3)) |
                   static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(hi, __NV_SATFINITE, __NV_E4M3)) << 16;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Values of 16 codes as bf16 pairs (exact: at most 7 bits times a power of two).
template <int FMT>
__device__ __forceinline__ void kv_decode16(uint4 c, uint32_t byte, uint32_t (&x)[8])
{
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    if constexpr (FMT == FATHOM_KV_INT8) {
        const CodeMasks m = code_masks<FMT>();
        const uint32_t f = pow_bits2<FMT>(byte);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = decode2<FMT, 0, 1>(w[i], w[i], f, m);
            x[2 * i + 1] = decode2<FMT, 2, 3>(w[i], w[i], f, m);
        }
    } else {
        const float f = kv_pow2(byte);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
            const float2 v = __half22float2(__half2(r));
            x[i] = bf16x2(v.x * f, v.y * f);
        }
    }
}

// Where row r of the call is kept: page and token, or page -1.
__device__ __forceinline__ int kv_place(const KvCache& c, const KvRows& w, int r, int* token)
{
    const int b = kv_sequence(w, r);
    if (b < 0) return -2;
    const int64_t pos = static_cast<int64_t>(__ldg(w.length + b)) - __ldg(w.cu + b + 1) + r;
    *token = static_cast<int>(pos & (c.page_tokens - 1));
    return kv_page(c, w.table + b * w.table_stride, w.table_pages, pos);
}

template <int FMT, int DT, int VEC>
__global__ void __launch_bounds__(kKvThreads)
kv_write_kernel(const KvCache c, const KvRows w, const void* __restrict__ k, const void* __restrict__ v,
                int64_t stride_tok, int64_t stride_h)
{
    const int per = c.D >> 4, units = c.H * per;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kKvThreads + threadIdx.x, row = t / units;
    const int unit = static_cast<int>(t - row * units), h = unit / per, j = (unit - h * per) << 4;
    int token = 0;
    const int page = row < w.rows ? kv_place(c, w, static_cast<int>(row), &token) : -2;
    const bool live = page >= 0;   // the same for both threads of a block
    Raw16<DT> x[2] = {};
    if (live) {
        const int64_t at = row * stride_tok + h * stride_h + j;
        kv_load16<DT, VEC>(k, at, &x[0]);
        kv_load16<DT, VEC>(v, at, &x[1]);
    }
    const int64_t to = live ? kv_off(c, page, h, token) : 0;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        unsigned char* data = const_cast<unsigned char*>(s ? c.v : c.k);
        float y[16];
        kv_values<DT>(x[s], y);
        if (FMT == FATHOM_KV_BF16) {
            if (live && kv_in(c, to + 2 * j, 32)) {
                uint4* o = reinterpret_cast<uint4*>(data + to + 2 * j);
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    o[q] = make_uint4(bf16x2(y[8 * q], y[8 * q + 1]), bf16x2(y[8 * q + 2], y[8 * q + 3]),
                                      bf16x2(y[8 * q + 4], y[8 * q + 5]), bf16x2(y[8 * q + 6], y[8 * q + 7]));
            }
        } else {
            uint32_t byte;
            const uint4 codes = kv_encode16<FMT>(y, kv_largest<DT>(x[s]), &byte);
            if (live && kv_in(c, to + j, 16)) {
                *reinterpret_cast<uint4*>(data + to + j) = codes;
                unsigned char* sc = const_cast<unsigned char*>(s ? c.vs : c.ks);
                const int64_t at = kv_scale_off(c, page, h, token) + (j >> 5);
                if ((j & 31) == 0 && kv_scale_in(c, at, 1)) sc[at] = static_cast<unsigned char>(byte);
            }
        }
    }
}

// 16 values, given as bf16 pairs.
template <int DT, int VEC>
__device__ __forceinline__ void kv_store16(void* out, int64_t to, const uint32_t (&x)[8])
{
    if (DT == FATHOM_KEYS_BF16) {
        unsigned short* o = static_cast<unsigned short*>(out) + to;
        if (VEC == 32) {
            st_global32(o, x);
        } else if (VEC) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
                reinterpret_cast<uint4*>(o)[q] = make_uint4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = static_cast<unsigned short>(x[i >> 1] >> (16 * (i & 1)));
        }
    } else {
        uint32_t* o = static_cast<uint32_t*>(out) + to;
        if (VEC == 32) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = (i & 1) ? x[4 * q + (i >> 1)] & 0xffff0000u : x[4 * q + (i >> 1)] << 16;
                st_global32(o + 8 * q, y);
            }
        } else if (VEC) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                reinterpret_cast<uint4*>(o)[q] = make_uint4(x[2 * q] << 16, x[2 * q] & 0xffff0000u, x[2 * q + 1] << 16,
                                                            x[2 * q + 1] & 0xffff0000u);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = (i & 1) ? x[i >> 1] & 0xffff0000u : x[i >> 1] << 16;
        }
    }
}

template <int FMT, int DT, int VEC>
__global__ void __launch_bounds__(kKvThreads)
kv_read_kernel(const KvCache c, const KvRows w, void* out_k, void* out_v, int64_t stride_h, int64_t stride_tok)
{
    constexpr int PIECES = FMT == FATHOM_KV_BF16 ? 2 : 1;
    const int per = c.D >> 4;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kKvThreads + threadIdx.x, row = t / per;
    const int j = static_cast<int>(t - row * per) << 4, h = blockIdx.y;
    if (row >= w.rows) return;
    int token = 0;
    const int page = kv_place(c, w, static_cast<int>(row), &token);
    if (page == -2) return;   // not a row of any sequence
    uint4 raw[2][PIECES] = {};
    uint32_t byte[2] = {0, 0};
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        if (page >= 0 && (s ? out_v : out_k)) {
            const int64_t at = kv_off(c, page, h, token) + j * kv_elem_bytes<FMT>();
            const uint4* from = reinterpret_cast<const uint4*>((s ? c.v : c.k) + at);
            if (kv_in(c, at, 16 * PIECES)) {
#pragma unroll
                for (int q = 0; q < PIECES; ++q) raw[s][q] = __ldg(from + q);
            }
            if (FMT != FATHOM_KV_BF16) {
                const int64_t sat = kv_scale_off(c, page, h, token) + (j >> 5);
                if (kv_scale_in(c, sat, 1)) byte[s] = __ldg((s ? c.vs : c.ks) + sat);
            }
        }
    }
    const int64_t to = h * stride_h + row * stride_tok + j;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        void* out = s ? out_v : out_k;
        if (!out) continue;
        uint32_t x[8];
        if constexpr (FMT == FATHOM_KV_BF16) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                x[4 * q] = raw[s][q].x;
                x[4 * q + 1] = raw[s][q].y;
                x[4 * q + 2] = raw[s][q].z;
                x[4 * q + 3] = raw[s][q].w;
            }
        } else {
            kv_decode16<FMT>(raw[s][0], byte[s], x);
        }
        kv_store16<DT, VEC>(out, to, x);
    }
}

template <int FMT, int DT, int VEC>
int launch_kv_write_v(const KvCache& c, const KvRows& w, const void* k, const void* v, int64_t stride_tok, int64_t stride_h,
                      cudaStream_t stream)
{
    const unsigned grid = static_cast<unsigned>(kv_write_ctas(w.rows, c.H, c.D));
    kv_write_kernel<FMT, DT, VEC><<<grid, kKvThreads, 0, stream>>>(c, w, k, v, stride_tok, stride_h);
    return launch_status();
}

template <int FMT, int DT, int VEC>
int launch_kv_read_v(const KvCache& c, const KvRows& w, void* out_k, void* out_v, int64_t stride_h, int64_t stride_tok,
                     cudaStream_t stream)
{
    const dim3 grid(static_cast<unsigned>(ceil_div(static_cast<int64_t>(w.rows) * (c.D / 16), kKvThreads)),
                    static_cast<unsigned>(c.H));
    kv_read_kernel<FMT, DT, VEC><<<grid, kKvThreads, 0, stream>>>(c, w, out_k, out_v, stride_h, stride_tok);
    return launch_status();
}

template <int FMT>
int launch_kv_write_f(const KvCache& c, const KvRows& w, const void* k, const void* v, int dtype, int vec, int64_t st, int64_t sh,
                      cudaStream_t stream)
{
    if (dtype == FATHOM_KEYS_BF16)
        return vec == 32 ? launch_kv_write_v<FMT, FATHOM_KEYS_BF16, 32>(c, w, k, v, st, sh, stream)
               : vec     ? launch_kv_write_v<FMT, FATHOM_KEYS_BF16, 16>(c, w, k, v, st, sh, stream)
                         : launch_kv_write_v<FMT, FATHOM_KEYS_BF16, 0>(c, w, k, v, st, sh, stream);
    return vec == 32 ? launch_kv_write_v<FMT, FATHOM_KEYS_F32, 32>(c, w, k, v, st, sh, stream)
           : vec     ? launch_kv_write_v<FMT, FATHOM_KEYS_F32, 16>(c, w, k, v, st, sh, stream)
                     : launch_kv_write_v<FMT, FATHOM_KEYS_F32, 0>(c, w, k, v, st, sh, stream);
}

template <int FMT>
int launch_kv_read_f(const KvCache& c, const KvRows& w, void* k, void* v, int dtype, int vec, int64_t sh, int64_t st,
                     cudaStream_t stream)
{
    if (dtype == FATHOM_KEYS_BF16)
        return vec == 32 ? launch_kv_read_v<FMT, FATHOM_KEYS_BF16, 32>(c, w, k, v, sh, st, stream)
               : vec     ? launch_kv_read_v<FMT, FATHOM_KEYS_BF16, 16>(c, w, k, v, sh, st, stream)
                         : launch_kv_read_v<FMT, FATHOM_KEYS_BF16, 0>(c, w, k, v, sh, st, stream);
    return vec == 32 ? launch_kv_read_v<FMT, FATHOM_KEYS_F32, 32>(c, w, k, v, sh, st, stream)
           : vec     ? launch_kv_read_v<FMT, FATHOM_KEYS_F32, 16>(c, w, k, v, sh, st, stream)
                     : launch_kv_read_v<FMT, FATHOM_KEYS_F32, 0>(c, w, k, v, sh, st, stream);
}

// Bytes that every 16 elements of `dtype` are aligned to: 32, 16, or 0 for less.
int kv_vec(const void* a, const void* b, int dtype, int64_t s0, int64_t s1)
{
    const int64_t esz = dtype == FATHOM_KEYS_F32 ? 4 : 2;
    const uintptr_t all = reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) |   // NULL adds no bits
                          static_cast<uintptr_t>(s0 * esz) | static_cast<uintptr_t>(s1 * esz);
    return (all & 31) == 0 ? 32 : (all & 15) == 0 ? 16 : 0;
}

}  // namespace

int launch_kv_write(const KvCache& c, int format, const KvRows& w, const void* k, const void* v, int dtype,
                    int64_t stride_tok, int64_t stride_h, cudaStream_t stream)
{
    const int vec = kv_vec(k, v, dtype, stride_tok, stride_h);
    switch (format) {
        case FATHOM_KV_BF16: return launch_kv_write_f<FATHOM_KV_BF16>(c, w, k, v, dtype, vec, stride_tok, stride_h, stream);
        case FATHOM_KV_INT8: return launch_kv_write_f<FATHOM_KV_INT8>(c, w, k, v, dtype, vec, stride_tok, stride_h, stream);
        default: return launch_kv_write_f<FATHOM_KV_E4M3>(c, w, k, v, dtype, vec, stride_tok, stride_h, stream);
    }
}

int launch_kv_read(const KvCache& c, int format, const KvRows& w, void* out_k, void* out_v, int dtype,
                   int64_t stride_h, int64_t stride_tok, cudaStream_t stream)
{
    const int vec = kv_vec(out_k, out_v, dtype, stride_h, stride_tok);
    switch (format) {
        case FATHOM_KV_BF16: return launch_kv_read_f<FATHOM_KV_BF16>(c, w, out_k, out_v, dtype, vec, stride_h, stride_tok, stream);
        case FATHOM_KV_INT8: return launch_kv_read_f<FATHOM_KV_INT8>(c, w, out_k, out_v, dtype, vec, stride_h, stride_tok, stream);
        default: return launch_kv_read_f<FATHOM_KV_E4M3>(c, w, out_k, out_v, dtype, vec, stride_h, stride_tok, stream);
    }
}

}  // namespace fathom
