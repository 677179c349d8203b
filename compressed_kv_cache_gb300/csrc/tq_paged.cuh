// Shared pieces of the paged-cache kernels (tq_append.cu, tq_paged_*.cu, tq_evict.cu), and what
// tq_api.cu calls of them.
#pragma once

#include "tq_internal.cuh"

namespace tq {

// Launches (D == 128): quantise and write new rows, decode, evict.
cudaError_t launch_append_paged(const tq_paged_cache& c, const void* K, const void* V, tq_qtype type,
                                const int* rows, int n, const int* table, int B, int max_pages, float* mass,
                                int* positions, int S, cudaStream_t st);
size_t decode_paged_bytes(int B, int H, int G, int S, bool with_mass);
cudaError_t launch_decode_paged(const tq_paged_cache& c, const void* Q, tq_qtype qtype, const int* table,
                                const int* lengths, int B, int G, int max_pages, float scale, float* mass,
                                int S, void* out, void* ws, cudaStream_t st);
size_t evict_paged_bytes(int B, int H, int S, int budget);
cudaError_t launch_evict_paged(const tq_paged_cache& c, const int* table, const int* lengths, const int* seen,
                               int B, int max_pages, const float* mass, const int* positions, int S, int budget,
                               int recent, float* mass_out, int* positions_out, void* ws, cudaStream_t st);

// Fault bits: a number out of range, a wait of the append that ran out.
enum : unsigned int { kFaultPaged = 32u, kFaultPagedWait = 64u };
cudaError_t take_faults_append(unsigned int* bits);
cudaError_t take_faults_paged(unsigned int* bits);
cudaError_t take_faults_evict(unsigned int* bits);

namespace {

constexpr int kPD = 128;   // head dimension

// The cache as the kernels see it.  page_size is a power of two.
struct Paged {
  uint8_t* kp;
  uint8_t* vp;
  uint16_t* kn;
  uint16_t* vn;
  const int* table;
  int n_pages, H, shift, max_pages;   // page_size = 1 << shift

  // Page of slot s of sequence b, or -1 (absent: a number out of range, recorded).
  __device__ __forceinline__ int page(int b, int s) const {
    const int id = table[static_cast<size_t>(b) * max_pages + (s >> shift)];
    if (static_cast<unsigned>(id) < static_cast<unsigned>(n_pages)) return id;
    atomicOr(&g_wait_fault, static_cast<unsigned int>(kFaultPaged));
    return -1;
  }
  // Row number of slot s on a page, in the planes of head h.
  __device__ __forceinline__ size_t row(int pg, int h, int s) const {
    return ((static_cast<size_t>(pg) * H + h) << shift) + (s & ((1 << shift) - 1));
  }
};

inline Paged paged_view(const tq_paged_cache& c, const int* table, int max_pages) {
  int shift = 0;
  while ((1 << shift) < c.page_size) ++shift;
  return {c.k_plane, c.v_plane, c.k_norm, c.v_norm, table, c.n_pages, c.H, shift, max_pages};
}

inline size_t paged_round(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace
}  // namespace tq
