// fathom_kv_write and fathom_kv_read: rows into the paged cache and back.
//
// One thread takes 8 channels of one row of K and of V; the four threads of a
// 32-channel block find its largest magnitude with two shuffles.  Magnitudes
// are compared as bit patterns, which orders NaN above infinity above every
// number, so one compare finds the blocks that cannot be kept.  The exponent
// comes from the pattern too (exponent field, and one compare of the fraction
// with the value that would round over the largest code), so no division or
// logarithm is rounded anywhere and x 2^-e is exact before the one rounding
// to the code.  Both kernels stream: bound by HBM, or by the launch when a
// decode step writes one token.
#include "kv.cuh"

namespace fathom {

namespace {

constexpr int kKvThreads = 256;

// 8 consecutive elements as fp32.
template <int DT, bool VEC>
__device__ __forceinline__ void kv_load8(const void* p, int64_t at, float (&x)[8])
{
    if (DT == FATHOM_KEYS_BF16) {
        const __nv_bfloat16* s = static_cast<const __nv_bfloat16*>(p) + at;
        if (VEC) {
            const uint4 u = __ldg(reinterpret_cast<const uint4*>(s));
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __bfloat162float(s[i]);
        }
    } else {
        const float* s = static_cast<const float*>(p) + at;
        if (VEC) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(s)), b = __ldg(reinterpret_cast<const float4*>(s) + 1);
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
            x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = s[i];
        }
    }
}

// Codes of 8 channels and their block's exponent byte.  All four threads of
// the block take part.
template <int FMT>
__device__ __forceinline__ uint2 kv_encode8(const float (&x)[8], uint32_t* byte)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    if (m >= 0x7f800000u) {
        *byte = 255;
        return make_uint2(0, 0);
    }
    const int ex = static_cast<int>(m >> 23) - 127;
    const uint32_t frac = m & 0x7fffffu;
    // INT8: 64 f in [64, 128) rounds to 128 from 127.5 on.  E4M3: 256 f rounds to 448 up to 464 (a tie, to even).
    int e = FMT == FATHOM_KV_INT8 ? ex - 6 + (frac >= 0x7f0000u) : ex - 8 + (frac > 0x680000u);
    e = min(max(e, kKvLowest), FMT == FATHOM_KV_INT8 ? 121 : 7);
    *byte = static_cast<uint32_t>(e + 127);
    const float f = kv_pow2(static_cast<uint32_t>(127 - e));
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (FMT == FATHOM_KV_INT8) {
            w[i] = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = min(127, max(-127, __float2int_rn(x[4 * i + j] * f)));
                w[i] |= static_cast<uint32_t>(c & 0xff) << (8 * j);
            }
        } else {
            const float2 lo = make_float2(x[4 * i] * f, x[4 * i + 1] * f), hi = make_float2(x[4 * i + 2] * f, x[4 * i + 3] * f);
            w[i] = static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(lo, __NV_SATFINITE, __NV_E4M3)) |
                   static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(hi, __NV_SATFINITE, __NV_E4M3)) << 16;
        }
    }
    return make_uint2(w[0], w[1]);
}

// Values of 8 codes (exact: at most 7 bits times a power of two).
template <int FMT>
__device__ __forceinline__ void kv_decode8(uint2 c, uint32_t byte, float (&x)[8])
{
    const float f = kv_pow2(byte);
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t b = (w[i >> 2] >> (8 * (i & 3))) & 0xff;
        if (FMT == FATHOM_KV_INT8) {
            x[i] = static_cast<float>(static_cast<int8_t>(b)) * f;
        } else {
            const __half_raw r = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(b), __NV_E4M3);
            x[i] = __half2float(__half(r)) * f;
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

template <int FMT, int DT, bool VEC>
__global__ void __launch_bounds__(kKvThreads)
kv_write_kernel(const KvCache c, const KvRows w, const void* __restrict__ k, const void* __restrict__ v,
                int64_t stride_tok, int64_t stride_h)
{
    const int per = c.D >> 3;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kKvThreads + threadIdx.x;
    const int64_t unit = t / per;
    const int j = static_cast<int>(t - unit * per) << 3;
    const int64_t row = unit / c.H;
    const int h = static_cast<int>(unit - row * c.H);
    int page = -2, token = 0;
    if (row < w.rows) page = kv_place(c, w, static_cast<int>(row), &token);
    const bool live = page >= 0;   // the same for the four threads of a block
    float x[2][8];
    const int64_t at = live ? row * stride_tok + h * stride_h + j : 0;
    if (live) {
        kv_load8<DT, VEC>(k, at, x[0]);
        kv_load8<DT, VEC>(v, at, x[1]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[0][i] = x[1][i] = 0.0f;
    }
    const int64_t to = live ? kv_off(c, page, h, token) : 0;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        unsigned char* data = const_cast<unsigned char*>(s ? c.v : c.k);
        if (FMT == FATHOM_KV_BF16) {
            if (live)
                *reinterpret_cast<uint4*>(data + to + 2 * j) =
                    make_uint4(bf16x2(x[s][0], x[s][1]), bf16x2(x[s][2], x[s][3]), bf16x2(x[s][4], x[s][5]),
                               bf16x2(x[s][6], x[s][7]));
        } else {
            uint32_t byte;
            const uint2 codes = kv_encode8<FMT>(x[s], &byte);
            if (live) {
                *reinterpret_cast<uint2*>(data + to + j) = codes;
                unsigned char* sc = const_cast<unsigned char*>(s ? c.vs : c.ks);
                if ((j & 31) == 0) sc[kv_scale_off(c, page, h, token) + (j >> 5)] = static_cast<unsigned char>(byte);
            }
        }
    }
}

template <int FMT, int DT, bool VEC>
__global__ void __launch_bounds__(kKvThreads)
kv_read_kernel(const KvCache c, const KvRows w, void* out_k, void* out_v, int64_t stride_h, int64_t stride_tok)
{
    const int per = c.D >> 3;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kKvThreads + threadIdx.x;
    const int64_t row = t / per;
    const int j = static_cast<int>(t - row * per) << 3;
    const int h = blockIdx.y;
    if (row >= w.rows) return;
    int token = 0;
    const int page = kv_place(c, w, static_cast<int>(row), &token);
    if (page == -2) return;   // not a row of any sequence
    const int64_t from = page >= 0 ? kv_off(c, page, h, token) : 0;
    const int64_t to = h * stride_h + row * stride_tok + j;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        void* out = s ? out_v : out_k;
        if (!out) continue;
        const unsigned char* data = s ? c.v : c.k;
        float x[8] = {};
        if (page >= 0) {
            if (FMT == FATHOM_KV_BF16) {
                kv_load8<FATHOM_KEYS_BF16, true>(data + from, j, x);
            } else {
                const uint2 codes = __ldg(reinterpret_cast<const uint2*>(data + from + j));
                const uint32_t byte = __ldg((s ? c.vs : c.ks) + kv_scale_off(c, page, h, token) + (j >> 5));
                kv_decode8<FMT>(codes, byte, x);
            }
        }
        if (DT == FATHOM_KEYS_BF16) {
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out) + to;
            const uint4 u = make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
            if (VEC) {
                *reinterpret_cast<uint4*>(o) = u;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = __float2bfloat16(x[i]);
            }
        } else {
            float* o = static_cast<float*>(out) + to;
            if (VEC) {
                reinterpret_cast<float4*>(o)[0] = make_float4(x[0], x[1], x[2], x[3]);
                reinterpret_cast<float4*>(o)[1] = make_float4(x[4], x[5], x[6], x[7]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = x[i];
            }
        }
    }
}

template <int FMT>
int launch_kv_write_f(const KvCache& c, const KvRows& w, const void* k, const void* v, int dtype, bool vec,
                      int64_t stride_tok, int64_t stride_h, cudaStream_t stream)
{
    const int64_t threads = static_cast<int64_t>(w.rows) * c.H * (c.D / 8);
    const unsigned grid = static_cast<unsigned>(ceil_div(threads, kKvThreads));
    if (dtype == FATHOM_KEYS_BF16) {
        if (vec) kv_write_kernel<FMT, FATHOM_KEYS_BF16, true><<<grid, kKvThreads, 0, stream>>>(c, w, k, v, stride_tok, stride_h);
        else kv_write_kernel<FMT, FATHOM_KEYS_BF16, false><<<grid, kKvThreads, 0, stream>>>(c, w, k, v, stride_tok, stride_h);
    } else {
        if (vec) kv_write_kernel<FMT, FATHOM_KEYS_F32, true><<<grid, kKvThreads, 0, stream>>>(c, w, k, v, stride_tok, stride_h);
        else kv_write_kernel<FMT, FATHOM_KEYS_F32, false><<<grid, kKvThreads, 0, stream>>>(c, w, k, v, stride_tok, stride_h);
    }
    return launch_status();
}

template <int FMT>
int launch_kv_read_f(const KvCache& c, const KvRows& w, void* out_k, void* out_v, int dtype, bool vec,
                     int64_t stride_h, int64_t stride_tok, cudaStream_t stream)
{
    const int64_t threads = static_cast<int64_t>(w.rows) * (c.D / 8);
    const dim3 grid(static_cast<unsigned>(ceil_div(threads, kKvThreads)), static_cast<unsigned>(c.H));
    if (dtype == FATHOM_KEYS_BF16) {
        if (vec) kv_read_kernel<FMT, FATHOM_KEYS_BF16, true><<<grid, kKvThreads, 0, stream>>>(c, w, out_k, out_v, stride_h, stride_tok);
        else kv_read_kernel<FMT, FATHOM_KEYS_BF16, false><<<grid, kKvThreads, 0, stream>>>(c, w, out_k, out_v, stride_h, stride_tok);
    } else {
        if (vec) kv_read_kernel<FMT, FATHOM_KEYS_F32, true><<<grid, kKvThreads, 0, stream>>>(c, w, out_k, out_v, stride_h, stride_tok);
        else kv_read_kernel<FMT, FATHOM_KEYS_F32, false><<<grid, kKvThreads, 0, stream>>>(c, w, out_k, out_v, stride_h, stride_tok);
    }
    return launch_status();
}

// 16-byte pieces: 8 elements of `dtype` start on a multiple of 16 bytes everywhere.
bool kv_vec(const void* a, const void* b, int dtype, int64_t s0, int64_t s1)
{
    const int64_t esz = dtype == FATHOM_KEYS_F32 ? 4 : 2;
    const uintptr_t p = reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b);   // NULL adds no bits
    return (p & 15) == 0 && (s0 * esz) % 16 == 0 && (s1 * esz) % 16 == 0;
}

}  // namespace

int launch_kv_write(const KvCache& c, int format, const KvRows& w, const void* k, const void* v, int dtype,
                    int64_t stride_tok, int64_t stride_h, cudaStream_t stream)
{
    const bool vec = kv_vec(k, v, dtype, stride_tok, stride_h);
    switch (format) {
        case FATHOM_KV_BF16: return launch_kv_write_f<FATHOM_KV_BF16>(c, w, k, v, dtype, vec, stride_tok, stride_h, stream);
        case FATHOM_KV_INT8: return launch_kv_write_f<FATHOM_KV_INT8>(c, w, k, v, dtype, vec, stride_tok, stride_h, stream);
        default: return launch_kv_write_f<FATHOM_KV_E4M3>(c, w, k, v, dtype, vec, stride_tok, stride_h, stream);
    }
}

int launch_kv_read(const KvCache& c, int format, const KvRows& w, void* out_k, void* out_v, int dtype,
                   int64_t stride_h, int64_t stride_tok, cudaStream_t stream)
{
    const bool vec = kv_vec(out_k, out_v, dtype, stride_h, stride_tok);
    switch (format) {
        case FATHOM_KV_BF16: return launch_kv_read_f<FATHOM_KV_BF16>(c, w, out_k, out_v, dtype, vec, stride_h, stride_tok, stream);
        case FATHOM_KV_INT8: return launch_kv_read_f<FATHOM_KV_INT8>(c, w, out_k, out_v, dtype, vec, stride_h, stride_tok, stream);
        default: return launch_kv_read_f<FATHOM_KV_E4M3>(c, w, out_k, out_v, dtype, vec, stride_h, stride_tok, stream);
    }
}

}  // namespace fathom
