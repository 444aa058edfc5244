// The kernels of kvchunk.cuh.
#include "kvchunk.cuh"

namespace fathom {

namespace {

template <int D>
int launch_chunk_d(const KvRowsArgs& g, int format, cudaStream_t stream)
{
    switch (format) {
        case FATHOM_KV_BF16: return launch_chunk_t<D, FATHOM_KV_BF16>(g, stream);
        case FATHOM_KV_INT8: return launch_chunk_t<D, FATHOM_KV_INT8>(g, stream);
        default: return launch_chunk_t<D, FATHOM_KV_E4M3>(g, stream);
    }
}

}  // namespace

int launch_chunk(const KvRowsArgs& g, int format, cudaStream_t stream)
{
    return g.a.c.D == 128 ? launch_chunk_d<128>(g, format, stream) : launch_chunk_d<64>(g, format, stream);
}

}  // namespace fathom
