// The kernels of kvchunk.cuh.
#include "kvchunk.cuh"

namespace fathom {

namespace {

template <int D, bool FULL>
int launch_chunk_d(const KvRowsArgs& g, int format, cudaStream_t stream)
{
    switch (format) {
        case FATHOM_KV_BF16: return launch_chunk_t<D, FATHOM_KV_BF16, FULL>(g, stream);
        case FATHOM_KV_INT8: return launch_chunk_t<D, FATHOM_KV_INT8, FULL>(g, stream);
        default: return launch_chunk_t<D, FATHOM_KV_E4M3, FULL>(g, stream);
    }
}

}  // namespace

int launch_chunk(const KvRowsArgs& g, int format, cudaStream_t stream)
{
    switch (g.a.c.D) {
        case 32: return launch_chunk_d<64, false>(g, format, stream);
        case 64: return launch_chunk_d<64, true>(g, format, stream);
        case 96: return launch_chunk_d<128, false>(g, format, stream);
        case 128: return launch_chunk_d<128, true>(g, format, stream);
        case 256: return launch_chunk_d<256, true>(g, format, stream);
        default: return launch_chunk_d<256, false>(g, format, stream);   // 160, 192, 224
    }
}

}  // namespace fathom
