// Attention over the paged KV cache: the tcgen05 kernel for many query rows.
#include "hadq_kernels.h"
#include "hadq_paged_tc.cuh"

namespace hadq {

const void* paged_chunk_kernel_ptr(int ng, int bits) {
  if (bits == 8)
    return ng == 4 ? (const void*)paged_chunk_kernel<4, 8> : ng == 2 ? (const void*)paged_chunk_kernel<2, 8> : (const void*)paged_chunk_kernel<1, 8>;
  return ng == 4 ? (const void*)paged_chunk_kernel<4, 4> : ng == 2 ? (const void*)paged_chunk_kernel<2, 4> : (const void*)paged_chunk_kernel<1, 4>;
}
size_t paged_chunk_smem() { return pt_smem_bytes(); }

}  // namespace hadq
