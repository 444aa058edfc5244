// fathom_paged_attention and fathom_paged_union_attention: how a call is cut
// up, and the joining of its stretches.
#include <stdlib.h>

#include <algorithm>

#include "kvchunk.cuh"

namespace fathom {

namespace {

constexpr int kSms = 148;        // the machine this library is written for; only the cut depends on it

int64_t round_up(int64_t x, int64_t to) { return ceil_div(x, to) * to; }

// The cut of `tiles` tiles of tokens into stretches that ends soonest: waves of
// CTAs (`at_once` to the machine) times a stretch's tiles (`us` each, and the
// time of `start` of them to begin and end a CTA), and writing and joining the
// stretches' sums.  A batch's longest sequence is `longest` of the `items`;
// the others are taken to be half as long, since only the device knows.
// From eight waves of CTAs on there is nothing to gain, and with longer bounds
// than the sequences have the parts would only take memory.
// Returns the tiles of a stretch.
int64_t cut(int64_t tiles, int64_t items, int64_t longest, int64_t heads, int D, int64_t at_once, double us, int64_t start)
{
    double best = 0.0;
    int64_t each = tiles;
    const int64_t most = std::min({int64_t{32}, tiles, ceil_div(8 * at_once, items)});
    for (int64_t n = 1; n <= most; ++n) {
        const int64_t len = ceil_div(tiles, n);
        const int64_t waves = ceil_div(longest * n + (items - longest) * ceil_div(n, 2), at_once);
        const double cost = waves * (len + start) * us + (n > 1 ? 4.0 + static_cast<double>(n) * heads * D * 8 / 5e6 : 0.0);
        if (n == 1 || cost < best) {
            best = cost;
            each = len;
        }
    }
    return each;
}

// How rows of queries and tokens are cut into CTAs.
KvSplit rows_split(int H, int G, int D, int64_t rows, int B, int64_t max_new, int64_t max_len, int q_dtype)
{
    KvSplit s{};
    const int64_t qrows = max_new * G, len = std::max<int64_t>(max_len, 1);
    // kvchunk.cuh takes bf16 queries from 33 rows (heads of tokens) on.  One session of 8 groups, 32k int8 tokens, 128
    // channels: 16 rows 45 us there and 44 here, 32 rows 46 and 46, 64 rows 50 and 73, 128 rows 57 and 116; eight
    // sessions of up to 8k bf16 tokens: 16 rows 66 and 73, 32 rows 66 and 77, 64 rows 70 and 122.
    const bool chunk = q_dtype == FATHOM_KEYS_BF16 && qrows > 32;
    s.nt = chunk ? 0 : (qrows <= 8 ? 1 : (D <= 128 ? 4 : 2));
    s.tile_rows = chunk ? chunk_rows(D) : 8 * s.nt;
    s.row_tiles = static_cast<int32_t>(ceil_div(qrows, s.tile_rows));
    if (s.nt == 1) {
        // Single tokens.  Four CTAs fit an SM.  One session: its stretches are equal, one wave of CTAs.  Several of
        // uneven lengths: shorter stretches, so that the longest session does not end alone.
        const int64_t items = static_cast<int64_t>(B) * H, want = B == 1 ? 4 * kSms : 16 * kSms;
        const int64_t splits = std::max<int64_t>(1, want / items);
        s.chunk = static_cast<int32_t>(std::max<int64_t>(round_up(ceil_div(len, splits), 64), 256));
    } else {
        // A batch has no more row tiles than all its rows fill, and one begun by each sequence.
        const int64_t items = H * std::min(static_cast<int64_t>(B) * s.row_tiles, ceil_div(rows * G, s.tile_rows) + B - 1);
        const int64_t longest = std::min(items, static_cast<int64_t>(H) * s.row_tiles), heads = rows * H * G;
        // A CTA to an SM and 128 tokens in 1.7 us (64 in 1.0 beyond 128 channels), or two and 64 tokens in 1.5.
        const int64_t tile = chunk ? chunk_keys(D) : 16 * kRowsWarps;
        s.chunk = static_cast<int32_t>(tile * cut(ceil_div(len, tile), items, longest, heads, D, chunk ? kSms : 2 * kSms,
                                                  !chunk ? 1.5 : D <= 128 ? 1.7 : 1.0, !chunk ? 4 : D <= 128 ? 5 : 9));
    }
    s.splits = static_cast<int32_t>(ceil_div(len, s.chunk));
    return s;
}

// A union has between 1/G of M rows and all of them, only the device knows:
// 5/8 is taken (the mean at G = 4; 288 groups of 25%, 62% and 99% of 2048 rows
// take 33, 48 and 73 us), and one wave of CTAs, four to an SM, for that (a group's last
// stretch is half one on average).
KvSplit union_split(int64_t H, int64_t M)
{
    KvSplit s{1, 8, 1, 1, 0};
    const double per_group = 4.0 * kSms / static_cast<double>(H) - 0.5;
    const int64_t chunk = per_group > 0.625 ? static_cast<int64_t>(0.625 * static_cast<double>(M) / per_group) : M;
    // To the nearest 64: 36 groups of up to 2048 rows take 17 us by 64 and 21 by 128.
    s.chunk = static_cast<int32_t>(std::max<int64_t>((std::min(chunk, M) + 32) / 64 * 64, 64));
    s.splits = static_cast<int32_t>(ceil_div(M, s.chunk));
    return s;
}

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

size_t parts_bytes(int64_t heads, int64_t splits, int D)
{
    return splits > 1 ? up256(sizeof(float) * splits * heads * D) + 2 * up256(sizeof(float) * splits * heads) : 0;
}

// The stretches' value sums, each times 2^(its maximum - the largest), over
// the weight sums treated alike: WARPS warps to a query head of a row.  A
// decode step's many stretches of few heads have 16, so that all loads are on
// their way at once; a chunk's few stretches of many heads one, and 8 heads to
// a CTA (a CTA each took 110 us for 65536 heads of 4 stretches; a token each
// of 9 sessions, 576 heads of up to 27 stretches, takes 49 us with 16 warps to
// the join's heads and 61 with one, attention included).
template <int QT, int WARPS>
__global__ void __launch_bounds__(WARPS == 1 ? 256 : 32 * WARPS)
kv_join_kernel(const KvRowsArgs g)
{
    constexpr int HEADS = WARPS == 1 ? 8 : 1;   // of a CTA
    const KvAttend& a = g.a;
    const int D = a.c.D, lane = threadIdx.x & 31, heads_row = a.c.H * a.G;
    const int warp = WARPS == 1 ? 0 : threadIdx.x >> 5;
    const int64_t head = static_cast<int64_t>(blockIdx.x) * HEADS + (WARPS == 1 ? threadIdx.x >> 5 : 0);
    int n = 0;   // stretches that were computed; -1: the row is not
    if (head >= g.heads) {
        n = -1;
    } else if (a.uni) {
        n = kv_stretches(min(static_cast<int64_t>(max(a.count[head / a.G], 0)), a.M), g.s.chunk);
    } else {
        const int row = static_cast<int>(head / heads_row), b = kv_sequence(a.w, row);
        const KvSpan sp = kv_span(a, max(b, 0));
        if (b < 0 || row - sp.first >= sp.rows) {
            n = -1;
        } else {
            const int qr = static_cast<int>(row - sp.first) * a.G + static_cast<int>(head % heads_row) % a.G;
            n = kv_stretches(kv_tile_keys(a, sp, qr / g.s.tile_rows * g.s.tile_rows, g.s.tile_rows), g.s.chunk);
        }
    }
    // The lengths are the caller's; the parts are written by the kernel before.  Every CTA waits: the stream's next
    // kernel starts when this one has ended, and counts on both.
    pdl_wait();
    if (n < 0) return;
    float top = -INFINITY;
    for (int s = lane; s < n; s += 32) top = fmaxf(top, g.pm[s * g.heads + head]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float acc[kMaxD / 32], l = 0.0f;
#pragma unroll
    for (int i = 0; i < kMaxD / 32; ++i) acc[i] = 0.0f;
    const float low = top == -INFINITY ? 0.0f : top;
#pragma unroll 4
    for (int s = warp; s < n; s += WARPS) {
        const int64_t at = s * g.heads + head;
        if (!kv_place_in(a.c, at, g.s.splits * g.heads)) continue;
        const float f = exp2_fast(g.pm[at] - low);
        l += g.pl[at] * f;
#pragma unroll
        for (int i = 0; i < kMaxD / 32; ++i)
            if (i < D / 32) acc[i] = fmaf(g.po[at * D + lane + 32 * i], f, acc[i]);
    }
    auto store = [&](int d, float x, float sum) {
        const float y = sum == 0.0f ? 0.0f : x / sum;   // no token was seen (NaN scores make the sum NaN)
        if (QT == FATHOM_KEYS_F32) static_cast<float*>(a.out)[head * D + d] = y;
        else static_cast<__nv_bfloat16*>(a.out)[head * D + d] = __float2bfloat16(y);
    };
    if constexpr (WARPS == 1) {
#pragma unroll
        for (int i = 0; i < kMaxD / 32; ++i)
            if (i < D / 32) store(lane + 32 * i, acc[i], l);
    } else {
        __shared__ float part[WARPS][kMaxD];
        __shared__ float part_l[WARPS];
#pragma unroll
        for (int i = 0; i < kMaxD / 32; ++i)
            if (i < D / 32) part[warp][lane + 32 * i] = acc[i];
        if (lane == 0) part_l[warp] = l;
        __syncthreads();
        for (int d = threadIdx.x; d < D; d += 32 * WARPS) {
            float x = 0.0f, sum = 0.0f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                x += part[w][d];
                sum += part_l[w];
            }
            store(d, x, sum);
        }
    }
}

template <int QT>
int launch_join_t(const KvRowsArgs& g, cudaStream_t stream)
{
    if (g.s.splits > 16 && g.heads <= 4096) return launch_pdl(kv_join_kernel<QT, 16>, static_cast<unsigned>(g.heads), 512, 0, stream, g);
    return launch_pdl(kv_join_kernel<QT, 1>, static_cast<unsigned>(ceil_div(g.heads, 8)), 256, 0, stream, g);
}

int launch_join(const KvRowsArgs& g, int q_dtype, cudaStream_t stream)
{
    return q_dtype == FATHOM_KEYS_F32 ? launch_join_t<FATHOM_KEYS_F32>(g, stream) : launch_join_t<FATHOM_KEYS_BF16>(g, stream);
}

}  // namespace

size_t paged_attention_workspace_bytes(int H, int G, int D, int64_t rows, int B, int64_t max_new, int64_t max_len,
                                       int q_dtype)
{
    const KvSplit s = rows_split(H, G, D, rows, B, std::min(max_new, rows), max_len, q_dtype);
    return parts_bytes(rows * H * G, s.splits, D);
}

size_t paged_union_attention_workspace_bytes(int64_t H, int G, int D, int64_t M)
{
    return parts_bytes(H * G, union_split(H, M).splits, D);
}

int launch_paged_attention(const KvAttend& a, int format, int q_dtype, void* ws, cudaStream_t stream)
{
    KvRowsArgs g{};
    g.a = a;
    g.s = a.uni ? union_split(a.c.H, a.M) : rows_split(a.c.H, a.G, a.c.D, a.w.rows, a.w.B, a.max_new, a.max_len, q_dtype);
    g.heads = static_cast<int64_t>(a.w.rows) * a.c.H * a.G;
#ifdef FATHOM_TEST_HOOKS
    {
        const char* e = getenv("FATHOM_TEST_WITHHOLD_TILE");
        g.withhold = e != nullptr ? atoi(e) : -1;
    }
#endif
    unsigned char* base = static_cast<unsigned char*>(ws);
    if (g.s.splits > 1) {
        g.po = reinterpret_cast<float*>(base);
        g.pm = reinterpret_cast<float*>(base + up256(sizeof(float) * g.s.splits * g.heads * a.c.D));
        g.pl = reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(g.pm) + up256(sizeof(float) * g.s.splits * g.heads));
    }
    const int st = g.s.nt == 0                 ? launch_chunk(g, format, stream)
                   : format == FATHOM_KV_BF16 ? launch_rows_bf16(g, q_dtype, stream)
                   : format == FATHOM_KV_INT8 ? launch_rows_int8(g, q_dtype, stream)
                                              : launch_rows_e4m3(g, q_dtype, stream);
    if (st || g.s.splits <= 1) return st;
    // heads < 2^31: there are stretches only where CTAs along rows and heads are few
    return launch_join(g, q_dtype, stream);
}

}  // namespace fathom
