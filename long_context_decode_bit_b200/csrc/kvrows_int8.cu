// The kernels of kvrows.cuh for caches in FATHOM_KV_INT8.
#include "kvrows.cuh"

namespace fathom {

int launch_rows_int8(const KvRowsArgs& g, int q_dtype, cudaStream_t stream)
{
    return launch_rows_f<FATHOM_KV_INT8>(g, q_dtype, stream);
}

}  // namespace fathom
