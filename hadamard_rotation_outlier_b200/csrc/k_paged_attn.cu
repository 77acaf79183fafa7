// Attention over the paged KV cache: the kernel for few query rows.
#include "hadq_kernels.h"
#include "hadq_paged_attn.cuh"

namespace hadq {

template <int RG, int NG, int BITS>
static const void* pd_get(size_t* smem) {
  *smem = sizeof(PdSmem<RG, NG, BITS>);
  return reinterpret_cast<const void*>(&paged_decode_kernel<RG, NG, BITS>);
}
template <int NG, int BITS>
static const void* pd_rows(int rg, size_t* smem) {
  return rg == 2 ? pd_get<2, NG, BITS>(smem) : pd_get<1, NG, BITS>(smem);
}
const void* paged_decode_kernel_ptr(int rg, int ng, int bits, size_t* smem) {
  if (bits == 8) return ng == 4 ? pd_rows<4, 8>(rg, smem) : ng == 2 ? pd_rows<2, 8>(rg, smem) : pd_rows<1, 8>(rg, smem);
  return ng == 4 ? pd_rows<4, 4>(rg, smem) : ng == 2 ? pd_rows<2, 4>(rg, smem) : pd_rows<1, 4>(rg, smem);
}

}  // namespace hadq
