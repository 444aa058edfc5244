// The kernels of kvrows.cuh for caches in FATHOM_KV_BF16.
#include "kvrows.cuh"

namespace fathom {

int launch_rows_bf16(const KvRowsArgs& g, int q_dtype, cudaStream_t stream)
{
    return launch_rows_f<FATHOM_KV_BF16>(g, q_dtype, stream);
}

}  // namespace fathom
