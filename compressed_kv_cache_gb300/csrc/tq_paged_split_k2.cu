// The split of tq_decode_paged for 2-bit keys (one unit per key width, to build in parallel).
#define TQ_SPLIT_KERNEL
#include "tq_paged_split.cuh"

namespace tq {

cudaError_t launch_split_k2(const SplitArgs& a, int vbits, int variant, int ctas, cudaStream_t st) {
  return launch_split<2>(a, vbits, variant, ctas, st);
}

cudaError_t take_faults_split_k2(unsigned int* bits) { return take_unit_faults(bits); }

}  // namespace tq
