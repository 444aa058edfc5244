// extern "C" entry points of the paged KV cache (declared in
// include/fathom.h): argument checks on the host, then the launches.
#include <cuda.h>
#include <stdlib.h>

#include <algorithm>

#include "args.cuh"
#include "kv.cuh"

namespace fathom {

int launch_kv_write(const KvCache& c, int format, const KvRows& w, const void* k, const void* v, int dtype,
                    int64_t stride_tok, int64_t stride_h, cudaStream_t stream);
int launch_kv_read(const KvCache& c, int format, const KvRows& w, void* out_k, void* out_v, int dtype,
                   int64_t stride_h, int64_t stride_tok, cudaStream_t stream);
size_t paged_attention_workspace_bytes(int H, int G, int D, int64_t rows, int B, int64_t max_new, int64_t max_len,
                                       int q_dtype);
size_t paged_union_attention_workspace_bytes(int64_t H, int G, int D, int64_t M);
int launch_paged_attention(const KvAttend& a, int format, int q_dtype, void* ws, cudaStream_t stream);

namespace {

constexpr int64_t kMaxTokens = 1LL << 30;                 // of a sequence: token + stretch stays an int
constexpr int64_t kMaxQueryRows = (1LL << 31) - 1;        // of a sequence: rows times heads of a group
constexpr int64_t kMaxRows = (1LL << 31) - 1, kMaxSequences = 65535;

#define FATHOM_TRY(expr)                 \
    do {                                 \
        const int _st = (expr);          \
        if (_st != FATHOM_OK) return _st; \
    } while (0)

// Of two faults in a call the sizes' is reported first, then alignment, then the pointers'.
int check_sizes(const fathom_kv_cache* c)
{
    if (!c) return FATHOM_ERR_INVALID_ARG;
    if (c->format < FATHOM_KV_BF16 || c->format > FATHOM_KV_E4M3) return FATHOM_ERR_INVALID_ARG;
    if (c->H < 0 || c->pages < 0 || c->pages >= (1LL << 31)) return FATHOM_ERR_INVALID_ARG;
    if (!dims_ok(c->D, 1) || c->H > 65535) return FATHOM_ERR_UNSUPPORTED;
    const int p = c->page_tokens;
    if (p < 16 || p > 256 || (p & (p - 1))) return FATHOM_ERR_UNSUPPORTED;
    if (c->token_stride < c->D || c->page_stride < 0 || c->head_stride < 0) return FATHOM_ERR_INVALID_ARG;
    if (c->format != FATHOM_KV_BF16 &&
        (c->scale_token_stride < c->D / kKvBlock || c->scale_page_stride < 0 || c->scale_head_stride < 0))
        return FATHOM_ERR_INVALID_ARG;
    return FATHOM_OK;
}

int check_rows(const fathom_kv_rows* w)
{
    if (!w || w->B < 0 || w->B > kMaxSequences || w->rows < 0 || w->rows > kMaxRows) return FATHOM_ERR_INVALID_ARG;
    if (w->table_pages < 0 || w->table_stride < 0) return FATHOM_ERR_INVALID_ARG;
    return FATHOM_OK;
}

// Device memory of the current device, by two attributes of the driver rather
// than the runtime's query of all of them: a write of nine pointers takes the
// host 4.6 us instead of 5.7, its launch included.
using PointerAttributes = CUresult (*)(unsigned int, CUpointer_attribute*, void**, CUdeviceptr);

PointerAttributes pointer_attributes()
{
    static const PointerAttributes fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuPointerGetAttributes", &f, 12000, cudaEnableDefault, &found);
        if (e != cudaSuccess) (void)cudaGetLastError();
        return e == cudaSuccess && found == cudaDriverEntryPointSuccess ? reinterpret_cast<PointerAttributes>(f) : nullptr;
    }();
    return fn;
}

// As check_device_ptr, and device memory has to be the current device's.
int check_here(const void* p, int dev)
{
    if (const PointerAttributes query = p ? pointer_attributes() : nullptr) {
        unsigned int type = 0;
        int ordinal = -1;
        CUpointer_attribute what[2] = {CU_POINTER_ATTRIBUTE_MEMORY_TYPE, CU_POINTER_ATTRIBUTE_DEVICE_ORDINAL};
        void* to[2] = {&type, &ordinal};
        if (query(2, what, to, reinterpret_cast<CUdeviceptr>(p)) == CUDA_SUCCESS && type == CU_MEMORYTYPE_DEVICE &&
            ordinal == dev)
            return FATHOM_OK;
    }
    FATHOM_TRY(check_device_ptr(p));
    cudaPointerAttributes attr;
    const cudaError_t e = cudaPointerGetAttributes(&attr, p);
    if (e != cudaSuccess) return cuda_status(e);
    return attr.type != cudaMemoryTypeDevice || attr.device == dev ? FATHOM_OK : FATHOM_ERR_INVALID_ARG;
}

// Every pointer of a call.
template <typename... P>
int check_all_here(const P*... p)
{
    int dev = -1;
    // Without a device every pointer is refused below.
    if (cudaGetDevice(&dev) != cudaSuccess) (void)cudaGetLastError();
    int st = FATHOM_OK;
    (void)((st = check_here(p, dev), st == FATHOM_OK) && ...);
    return st;
}

int check_cache(const fathom_kv_cache* c, KvCache* out)
{
    const int64_t esz = c->format == FATHOM_KV_BF16 ? 2 : 1;
    const bool coded = c->format != FATHOM_KV_BF16;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || (c->page_stride * esz) % 16 || (c->head_stride * esz) % 16 ||
        (c->token_stride * esz) % 16)
        return FATHOM_ERR_UNSUPPORTED;
    if (coded && c->D % 128 == 0 &&
        (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) || c->scale_page_stride % 4 || c->scale_head_stride % 4 ||
         c->scale_token_stride % 4))
        return FATHOM_ERR_UNSUPPORTED;
    FATHOM_TRY(check_all_here(c->k, c->v));
    if (coded) FATHOM_TRY(check_all_here(c->k_scale, c->v_scale));
    out->k = static_cast<const unsigned char*>(c->k);
    out->v = static_cast<const unsigned char*>(c->v);
    out->ks = c->k_scale;
    out->vs = c->v_scale;
    out->page_stride = c->page_stride * esz;
    out->head_stride = c->head_stride * esz;
    out->token_stride = c->token_stride * esz;
    out->spage_stride = c->scale_page_stride;
    out->shead_stride = c->scale_head_stride;
    out->stoken_stride = c->scale_token_stride;
    out->pages = static_cast<int32_t>(c->pages);
    out->H = c->H;
    out->D = c->D;
    out->page_tokens = c->page_tokens;
    out->page_shift = 0;
    while ((1 << out->page_shift) < c->page_tokens) ++out->page_shift;
#ifdef FATHOM_DEBUG_BOUNDS
    FATHOM_TRY(device_fault_word(&out->fault));
    auto bytes = [&](int64_t page, int64_t head, int64_t token, int64_t row) {
        return c->pages ? (c->pages - 1) * page + (c->H - 1) * head + (c->page_tokens - 1) * token + row : 0;
    };
    out->bytes = bytes(out->page_stride, out->head_stride, out->token_stride, c->D * esz);
    out->scale_bytes = coded ? bytes(out->spage_stride, out->shead_stride, out->stoken_stride, c->D / kKvBlock) : 0;
    // Test build only: let the checks allow half of the cache, so that a test sees a failed one reach the host.
    const char* e = getenv("FATHOM_TEST_SHRINK_CAP");
    if (e != nullptr && e[0] == '1') {
        out->bytes /= 2;
        out->scale_bytes /= 2;
    }
#endif
    return FATHOM_OK;
}

int check_row_ptrs(const fathom_kv_rows* w, KvRows* out)
{
    if (!aligned(w->table, 4) || !aligned(w->cu, 4) || !aligned(w->length, 4)) return FATHOM_ERR_UNSUPPORTED;
    if (w->table_pages > 0) FATHOM_TRY(check_all_here(w->table));
    FATHOM_TRY(check_all_here(w->cu, w->length));
    *out = KvRows{w->table, w->cu, w->length, w->table_stride, static_cast<int32_t>(w->rows), w->table_pages, w->B};
    return FATHOM_OK;
}

bool dtype_ok(int t) { return t == FATHOM_KEYS_F32 || t == FATHOM_KEYS_BF16; }
size_t dtype_bytes(int t) { return t == FATHOM_KEYS_F32 ? 4 : 2; }
bool scale_ok(float s) { return s <= 1.0e38f && s >= -1.0e38f; }   // times log2 e it is finite too; false for NaN

}  // namespace
}  // namespace fathom

using namespace fathom;

extern "C" {

int fathom_kv_write(const fathom_kv_cache* cache, const fathom_kv_rows* rows, const void* k, const void* v,
                    int dtype, int64_t stride_tok, int64_t stride_h, fathom_stream_t stream)
{
    NvtxRange range("fathom_kv_write");
    FATHOM_TRY(check_sizes(cache));
    FATHOM_TRY(check_rows(rows));
    if (!dtype_ok(dtype) || stride_tok < 0 || stride_h < 0) return FATHOM_ERR_INVALID_ARG;
    if (cache->H == 0 || rows->B == 0 || rows->rows == 0) return FATHOM_OK;
    if (kv_write_ctas(rows->rows, cache->H, cache->D) > 0x7FFFFFFF) return FATHOM_ERR_UNSUPPORTED;
    if (!aligned(k, dtype_bytes(dtype)) || !aligned(v, dtype_bytes(dtype))) return FATHOM_ERR_UNSUPPORTED;
    KvCache c;
    KvRows w;
    FATHOM_TRY(check_cache(cache, &c));
    FATHOM_TRY(check_row_ptrs(rows, &w));
    FATHOM_TRY(check_all_here(k, v));
    return launch_kv_write(c, cache->format, w, k, v, dtype, stride_tok, stride_h,
                           reinterpret_cast<cudaStream_t>(stream));
}

int fathom_kv_read(const fathom_kv_cache* cache, const fathom_kv_rows* rows, void* out_k, void* out_v, int dtype,
                   int64_t stride_h, int64_t stride_tok, fathom_stream_t stream)
{
    NvtxRange range("fathom_kv_read");
    FATHOM_TRY(check_sizes(cache));
    FATHOM_TRY(check_rows(rows));
    if (!dtype_ok(dtype)) return FATHOM_ERR_INVALID_ARG;
    if (cache->H == 0 || rows->B == 0 || rows->rows == 0) return FATHOM_OK;
    // Rows of the output must not overlap: tokens within groups, or groups within tokens.
    const int64_t D = cache->D;
    const bool by_group = stride_tok >= D && (cache->H == 1 || stride_h >= (rows->rows - 1) * stride_tok + D);
    const bool by_token = stride_h >= D && (rows->rows == 1 || stride_tok >= (cache->H - 1) * stride_h + D);
    if (!by_group && !by_token) return FATHOM_ERR_INVALID_ARG;
    if (!out_k && !out_v) return FATHOM_ERR_INVALID_ARG;
    if (!aligned(out_k, dtype_bytes(dtype)) || !aligned(out_v, dtype_bytes(dtype))) return FATHOM_ERR_UNSUPPORTED;
    KvCache c;
    KvRows w;
    FATHOM_TRY(check_cache(cache, &c));
    FATHOM_TRY(check_row_ptrs(rows, &w));
    FATHOM_TRY(check_all_here(out_k ? out_k : out_v, out_v ? out_v : out_k));
    if (out_k == out_v) return FATHOM_ERR_INVALID_ARG;
    return launch_kv_read(c, cache->format, w, out_k, out_v, dtype, stride_h, stride_tok,
                          reinterpret_cast<cudaStream_t>(stream));
}

size_t fathom_paged_attention_workspace_bytes(int H, int G, int D, int64_t rows, int B, int64_t max_new,
                                              int64_t max_len, int q_dtype)
{
    if (H <= 0 || H > 65535 || !dims_ok(D, G) || rows <= 0 || rows > kMaxRows || B <= 0 || B > kMaxSequences || max_new <= 0 ||
        max_len <= 0 || max_len > kMaxTokens || std::min(max_new, rows) * G > kMaxQueryRows || !dtype_ok(q_dtype))
        return 0;   // sizes that the call refuses too: the cut counts tokens and query rows in ints
    return paged_attention_workspace_bytes(H, G, D, rows, B, max_new, max_len, q_dtype);
}

int fathom_paged_attention(const fathom_kv_cache* cache, const fathom_kv_rows* rows, const void* q, int q_dtype,
                           int64_t q_stride_tok, int64_t q_stride_h, int G, int64_t max_new, int64_t max_len,
                           int causal, float scale, void* out, void* workspace, size_t ws_bytes,
                           fathom_stream_t stream)
{
    NvtxRange range("fathom_paged_attention");
    FATHOM_TRY(check_sizes(cache));
    FATHOM_TRY(check_rows(rows));
    if (!dtype_ok(q_dtype) || q_stride_tok < 0 || q_stride_h < 0 || !scale_ok(scale)) return FATHOM_ERR_INVALID_ARG;
    if (max_new < 0 || max_len < 0) return FATHOM_ERR_INVALID_ARG;
    if (G < 1 || G > kMaxG || max_len > kMaxTokens) return FATHOM_ERR_UNSUPPORTED;
    if (cache->H == 0 || rows->B == 0 || rows->rows == 0 || max_new == 0) return FATHOM_OK;
    if (max_new > rows->rows) max_new = rows->rows;
    if (max_new * G > kMaxQueryRows) return FATHOM_ERR_UNSUPPORTED;
    const size_t need = fathom_paged_attention_workspace_bytes(cache->H, G, cache->D, rows->rows, rows->B, max_new,
                                                               max_len, q_dtype);
    if (ws_bytes < need) return FATHOM_ERR_WORKSPACE;
    if (!aligned(q, dtype_bytes(q_dtype)) || !aligned(out, dtype_bytes(q_dtype)) || (need && !aligned(workspace, 256)))
        return FATHOM_ERR_UNSUPPORTED;
    KvAttend a{};
    FATHOM_TRY(check_cache(cache, &a.c));
    FATHOM_TRY(check_row_ptrs(rows, &a.w));
    FATHOM_TRY(check_all_here(q, static_cast<const void*>(out)));
    if (need) FATHOM_TRY(check_all_here(workspace));
    a.q = q;
    a.out = out;
    a.q_tok = q_stride_tok;
    a.q_head = q_stride_h;
    a.max_new = max_new;
    a.max_len = max_len;
    a.scale = scale;
    a.G = G;
    a.causal = causal != 0;
    return launch_paged_attention(a, cache->format, q_dtype, workspace, reinterpret_cast<cudaStream_t>(stream));
}

size_t fathom_paged_union_attention_workspace_bytes(int64_t H, int G, int D, int64_t M)
{
    if (H <= 0 || H > 65535 || M < 1 || M > 65536 || !dims_ok(D, G)) return 0;
    return paged_union_attention_workspace_bytes(H, G, D, M);
}

int fathom_paged_union_attention(const fathom_kv_cache* cache, const int32_t* table, int32_t table_pages, int64_t n,
                                 const float* q, int G, const int32_t* union_idx, const int32_t* union_count,
                                 int64_t M, float scale, float* out, void* workspace, size_t ws_bytes,
                                 fathom_stream_t stream)
{
    NvtxRange range("fathom_paged_union_attention");
    FATHOM_TRY(check_sizes(cache));
    if (table_pages < 0 || n < 0 || n >= (1LL << 31) || M < 1 || M > 65536 || !scale_ok(scale))
        return FATHOM_ERR_INVALID_ARG;
    if (G < 1 || G > kMaxG) return FATHOM_ERR_UNSUPPORTED;
    if (cache->H == 0) return FATHOM_OK;
    const size_t need = fathom_paged_union_attention_workspace_bytes(cache->H, G, cache->D, M);
    if (ws_bytes < need) return FATHOM_ERR_WORKSPACE;
    if (!aligned(table, 4) || !aligned(q, 4) || !aligned(union_idx, 4) || !aligned(union_count, 4) || !aligned(out, 4) ||
        (need && !aligned(workspace, 256)))
        return FATHOM_ERR_UNSUPPORTED;
    KvAttend a{};
    FATHOM_TRY(check_cache(cache, &a.c));
    if (table_pages > 0) FATHOM_TRY(check_all_here(table));
    FATHOM_TRY(check_all_here(q, union_idx, union_count, out));
    if (need) FATHOM_TRY(check_all_here(workspace));
    a.w.table = table;
    a.w.table_pages = table_pages;
    a.w.rows = 1;
    a.w.B = 1;
    a.q = q;
    a.q_head = cache->D;
    a.out = out;
    a.n = n;
    a.M = M;
    a.uni = union_idx;
    a.count = union_count;
    a.scale = scale;
    a.G = G;
    return launch_paged_attention(a, cache->format, FATHOM_KEYS_F32, workspace, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
