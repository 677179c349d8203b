// The split of tq_attend_int8 for bf16 queries and heads of 128 dimensions (a unit of its own: compiled in parallel).
#define TQ_INT8_SPLIT
#include "tq_int8_split.cuh"

namespace tq {

cudaError_t launch_attend_split_bf16_128(const AttendArgs& a, int nt, int ctas, cudaStream_t st) {
  return launch_split_of<__nv_bfloat16, 128>(a, nt, ctas, st);
}

cudaError_t take_faults_attend_bf16_128(unsigned int* bits) { return take_unit_faults(bits); }

}  // namespace tq
