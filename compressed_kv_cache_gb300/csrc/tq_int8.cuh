// Shared pieces of the kernels of the 8-bit paged cache (tq_int8_rows.cu, tq_int8_attend.cu) and of
// tq_norm_rope.cu, and what tq_api.cu calls of them.
#pragma once

#include "tq_internal.cuh"
#include "tq_paged.cuh"

namespace tq {

// Tokens of a step as the kernels see them: `starts` [B + 1], `lengths` [B], n in all.
struct Step {
  const int* starts;
  const int* lengths;
  int n, B;
};

struct NormRope {
  const void* q;
  const void* k;
  int64_t q_token, q_head, k_token, k_head;   // strides in elements
  const void* q_weight;
  const void* k_weight;
  const int* positions;
  const uint64_t* turns;
  const uint8_t* axis;
  void* q_out;
  void* k_out;
  int n, Hq, Hk, D, axes, pairs;
  bool paired, weights_bf16;
  float eps;
};

cudaError_t launch_norm_rope(const NormRope& a, tq_qtype type, cudaStream_t st);
cudaError_t launch_append_int8(const tq_int8_cache& c, const void* K, int64_t k_stride, const void* V,
                               int64_t v_stride, tq_qtype type, const Step& step, const int* table, int max_pages,
                               cudaStream_t st);
cudaError_t launch_read_int8(const tq_int8_cache& c, void* K, void* V, tq_qtype type, const Step& step,
                             const int* table, int max_pages, cudaStream_t st);
size_t attend_int8_bytes(int n, int B, int H, int G, int D);
cudaError_t launch_attend_int8(const tq_int8_cache& c, const void* Q, tq_qtype type, const Step& step, int G,
                               const int* table, int max_pages, int window, int sinks, float scale, void* out,
                               void* ws, cudaStream_t st);
cudaError_t take_faults_int8_rows(unsigned int* bits);
cudaError_t take_faults_int8_attend(unsigned int* bits);

namespace {

constexpr int kBlockSlots = 16;   // slots of a head that share an exponent
// Exponents: code u stands for (u - 127.5) * 2^e.  At 121 the codes reach the largest finite float,
// at -120 and above 2^e and 2^-e are normal numbers.
constexpr int kExpLow = -120, kExpHigh = 121;

// The cache as the kernels see it.  page_size is a power of two.
struct Int8View {
  uint8_t* kc;
  uint8_t* vc;
  int8_t* ex;       // [n_pages, H, page_size / 16, 2]: key's, value's
  const int* table;
  int n_pages, H, shift, max_pages;   // page_size = 1 << shift

  // Page of slot s of sequence b, or -1 (absent: a number out of range, recorded).
  __device__ __forceinline__ int page(int b, int s) const {
    const int i = s >> shift;
    int id = -1;
    if (i < max_pages) id = table[static_cast<size_t>(b) * max_pages + i];
    if (static_cast<unsigned>(id) < static_cast<unsigned>(n_pages)) return id;
    atomicOr(&g_wait_fault, static_cast<unsigned int>(kFaultPaged));
    return -1;
  }
  // Row number of slot s on a page, in the planes of head h; 16 rows on from a block's first row is the
  // next block of exponents.
  __device__ __forceinline__ size_t row(int pg, int h, int s) const {
    return ((static_cast<size_t>(pg) * H + h) << shift) + (s & ((1 << shift) - 1));
  }
};

inline Int8View int8_view(const tq_int8_cache& c, const int* table, int max_pages) {
  int shift = 0;
  while ((1 << shift) < c.page_size) ++shift;
  return {c.k_codes, c.v_codes, c.exponents, table, c.n_pages, c.H, shift, max_pages};
}

// Tokens [first, first + count) of sequence b, at slots [len, len + count).  Numbers that do not fit
// together (starts that descend or leave [0, n], a negative length) give no tokens and are recorded.
struct Run {
  int first, count, len;
};
__device__ __forceinline__ bool fits(const Step& s, int a, int z, int len) {
  return a >= 0 && a <= z && z <= s.n && len >= 0 && len <= INT32_MAX - 4096 - (z - a);
}
__device__ __forceinline__ Run run_of(const Step& s, int b) {
  const int a = s.starts[b], z = s.starts[b + 1], len = s.lengths[b];
  if (fits(s, a, z, len)) return {a, z - a, len};
  atomicOr(&g_wait_fault, static_cast<unsigned int>(kFaultPaged));
  return {0, 0, 0};
}

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127

}  // namespace
}  // namespace tq
