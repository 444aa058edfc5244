// fathom_paged_attention and fathom_paged_union_attention: softmax attention
// of a group's query heads over rows of the paged cache.
//
// One CTA per (row of queries, group): warp w scores the keys w, w + 8, ...
// with its lanes across the channels and keeps a running maximum, weight sum
// and value sum per head; the eight warps' results are joined at the end.
#include "kv.cuh"

namespace fathom {

namespace {

constexpr int kSimpleWarps = 8;

template <int FMT>
__device__ __forceinline__ float kv_value(const unsigned char* data, int j, uint32_t byte)
{
    if (FMT == FATHOM_KV_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(data)[j]);
    if (FMT == FATHOM_KV_INT8) return static_cast<float>(reinterpret_cast<const int8_t*>(data)[j]) * kv_pow2(byte);
    const __half_raw r = __nv_cvt_fp8_to_halfraw(data[j], __NV_E4M3);
    return __half2float(__half(r)) * kv_pow2(byte);
}

template <int FMT, int QT, bool UNION>
__global__ void __launch_bounds__(32 * kSimpleWarps)
kv_attend_kernel(const KvAttend a)
{
    extern __shared__ float sm[];   // [warps][G][D] value sums, [warps][G] maxima, [warps][G] weight sums
    const int G = a.G, D = a.c.D;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.y;
    const int row = blockIdx.x;
    const int32_t* table = a.w.table;
    int64_t keys;
    if (UNION) {
        keys = min(static_cast<int64_t>(max(a.count[h], 0)), a.M);
    } else {
        const int b = kv_sequence(a.w, row);
        if (b < 0) return;
        const int64_t first = a.w.cu[b], end = a.w.cu[b + 1], len = a.w.length[b];
        if (row - first >= a.max_new) return;
        const int64_t pos = len - end + row;
        keys = max(int64_t{0}, min(min(a.causal ? pos + 1 : len, len), a.max_len));
        table += b * a.w.table_stride;
    }
    float qv[kMaxG][kMaxD / 32], o[kMaxG][kMaxD / 32], m[kMaxG], l[kMaxG];
#pragma unroll
    for (int g = 0; g < kMaxG; ++g) {
        m[g] = -INFINITY;
        l[g] = 0.0f;
#pragma unroll
        for (int i = 0; i < kMaxD / 32; ++i) {
            o[g][i] = qv[g][i] = 0.0f;
            if (g < G && i < D / 32) {
                const int64_t at = row * a.q_tok + (static_cast<int64_t>(h) * G + g) * a.q_head + lane + 32 * i;
                qv[g][i] = QT == FATHOM_KEYS_F32 ? static_cast<const float*>(a.q)[at]
                                                 : __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[at]);
            }
        }
    }
    for (int64_t i0 = warp; i0 < keys; i0 += kSimpleWarps) {
        int64_t pos = i0;
        if (UNION) {
            pos = a.uni[h * a.M + i0];
            if (pos < 0 || pos >= a.n) continue;
        }
        const int page = kv_page(a.c, table, a.w.table_pages, pos);
        if (page < 0) continue;
        const int token = static_cast<int>(pos & (a.c.page_tokens - 1));
        const int64_t at = kv_off(a.c, page, h, token);
        const int64_t sat = FMT == FATHOM_KV_BF16 ? 0 : kv_scale_off(a.c, page, h, token);
        float kx[kMaxD / 32], vx[kMaxD / 32];
#pragma unroll
        for (int i = 0; i < kMaxD / 32; ++i) {
            kx[i] = vx[i] = 0.0f;
            if (i < D / 32) {
                kx[i] = kv_value<FMT>(a.c.k + at, lane + 32 * i, FMT == FATHOM_KV_BF16 ? 0 : a.c.ks[sat + i]);
                vx[i] = kv_value<FMT>(a.c.v + at, lane + 32 * i, FMT == FATHOM_KV_BF16 ? 0 : a.c.vs[sat + i]);
            }
        }
#pragma unroll
        for (int g = 0; g < kMaxG; ++g) {
            if (g >= G) break;
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < kMaxD / 32; ++i) s = fmaf(qv[g][i], kx[i], s);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            s *= a.scale;
            const float top = fmaxf(m[g], s);
            const float f = m[g] == -INFINITY ? 0.0f : expf(m[g] - top), p = expf(s - top);
            m[g] = top;
            l[g] = l[g] * f + p;
#pragma unroll
            for (int i = 0; i < kMaxD / 32; ++i) o[g][i] = o[g][i] * f + p * vx[i];
        }
    }
    float* sm_m = sm + kSimpleWarps * G * D;
    float* sm_l = sm_m + kSimpleWarps * G;
#pragma unroll
    for (int g = 0; g < kMaxG; ++g) {
        if (g >= G) break;
#pragma unroll
        for (int i = 0; i < kMaxD / 32; ++i)
            if (i < D / 32) sm[(warp * G + g) * D + lane + 32 * i] = o[g][i];
        if (lane == 0) {
            sm_m[warp * G + g] = m[g];
            sm_l[warp * G + g] = l[g];
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < G * D; e += blockDim.x) {
        const int g = e / D;
        float top = -INFINITY, sum = 0.0f, val = 0.0f;
        for (int w = 0; w < kSimpleWarps; ++w) top = fmaxf(top, sm_m[w * G + g]);
        if (top != -INFINITY)
            for (int w = 0; w < kSimpleWarps; ++w) {
                const float f = sm_m[w * G + g] == -INFINITY ? 0.0f : expf(sm_m[w * G + g] - top);
                sum += sm_l[w * G + g] * f;
                val += sm[(w * G + g) * D + e % D] * f;
            }
        const float r = top == -INFINITY ? 0.0f : val / sum;
        const int64_t to = (static_cast<int64_t>(row) * a.c.H + h) * G * D + e;
        if (QT == FATHOM_KEYS_F32) static_cast<float*>(a.out)[to] = r;
        else static_cast<__nv_bfloat16*>(a.out)[to] = __float2bfloat16(r);
    }
}

template <int FMT, int QT, bool UNION>
int launch_simple(const KvAttend& a, int rows, cudaStream_t stream)
{
    const size_t smem = sizeof(float) * kSimpleWarps * a.G * (a.c.D + 2);
    const int st = ensure_dynamic_smem(reinterpret_cast<const void*>(kv_attend_kernel<FMT, QT, UNION>), smem);
    if (st) return st;
    kv_attend_kernel<FMT, QT, UNION><<<dim3(rows, a.c.H), 32 * kSimpleWarps, smem, stream>>>(a);
    return launch_status();
}

template <int FMT>
int launch_attend_f(const KvAttend& a, int q_dtype, bool uni, cudaStream_t stream)
{
    if (uni) return launch_simple<FMT, FATHOM_KEYS_F32, true>(a, 1, stream);
    if (q_dtype == FATHOM_KEYS_F32) return launch_simple<FMT, FATHOM_KEYS_F32, false>(a, a.w.rows, stream);
    return launch_simple<FMT, FATHOM_KEYS_BF16, false>(a, a.w.rows, stream);
}

}  // namespace

size_t paged_attention_workspace_bytes(int, int, int, int64_t, int, int64_t, int64_t, int) { return 0; }
size_t paged_union_attention_workspace_bytes(int64_t, int, int, int64_t) { return 0; }

int launch_paged_attention(const KvAttend& a, int format, int q_dtype, void*, cudaStream_t stream)
{
    const bool uni = a.uni != nullptr;
    switch (format) {
        case FATHOM_KV_BF16: return launch_attend_f<FATHOM_KV_BF16>(a, q_dtype, uni, stream);
        case FATHOM_KV_INT8: return launch_attend_f<FATHOM_KV_INT8>(a, q_dtype, uni, stream);
        default: return launch_attend_f<FATHOM_KV_E4M3>(a, q_dtype, uni, stream);
    }
}

}  // namespace fathom
