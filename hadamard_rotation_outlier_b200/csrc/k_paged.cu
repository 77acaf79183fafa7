// The paged KV cache: slots, append, gather.
#include "hadq_kernels.h"
#include "hadq_paged.cuh"

namespace hadq {

const void* paged_slots_kernel_ptr() { return reinterpret_cast<const void*>(&paged_slots_kernel<kSlotsThreads>); }

template <int BITS, int NG>
static const void* append_ptr(bool signs) {
  return signs ? reinterpret_cast<const void*>(&paged_append_kernel<BITS, NG, true>)
               : reinterpret_cast<const void*>(&paged_append_kernel<BITS, NG, false>);
}
const void* paged_append_kernel_ptr(int bits, int ng, bool signs) {
  if (bits == 8) return ng == 4 ? append_ptr<8, 4>(signs) : ng == 2 ? append_ptr<8, 2>(signs) : append_ptr<8, 1>(signs);
  return ng == 4 ? append_ptr<4, 4>(signs) : ng == 2 ? append_ptr<4, 2>(signs) : append_ptr<4, 1>(signs);
}

template <int BITS, int NG>
static const void* gather_ptr(bool f32) {
  return f32 ? reinterpret_cast<const void*>(&paged_gather_kernel<BITS, NG, true>)
             : reinterpret_cast<const void*>(&paged_gather_kernel<BITS, NG, false>);
}
const void* paged_gather_kernel_ptr(int bits, int ng, bool f32) {
  if (bits == 8) return ng == 4 ? gather_ptr<8, 4>(f32) : ng == 2 ? gather_ptr<8, 2>(f32) : gather_ptr<8, 1>(f32);
  return ng == 4 ? gather_ptr<4, 4>(f32) : ng == 2 ? gather_ptr<4, 2>(f32) : gather_ptr<4, 1>(f32);
}

}  // namespace hadq
