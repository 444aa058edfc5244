// The kernels of kvrows.cuh for caches in FATHOM_KV_E4M3.
#include "kvrows.cuh"

namespace fathom {

int launch_rows_e4m3(const KvRowsArgs& g, int q_dtype, cudaStream_t stream)
{
    return launch_rows_f<FATHOM_KV_E4M3>(g, q_dtype, stream);
}

}  // namespace fathom
