// The write side of the paged cache (tq_append_paged): rotate, search the midpoints, pack
// the codes and write the row to its slot.
#include "tq_paged.cuh"

namespace tq {
namespace {

__device__ __forceinline__ float load_x(const float* x, size_t i) { return x[i]; }
__device__ __forceinline__ float load_x(const __nv_bfloat16* x, size_t i) { return __bfloat162float(x[i]); }

__device__ __forceinline__ float block_max(float v, float* red) {
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
}
__device__ __forceinline__ double block_sum(double v, double* red) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return red[0] + red[1] + red[2] + red[3];
}

// One block per (row, head), one thread per coordinate, everything in 64 bits.
template <typename T>
__global__ void __launch_bounds__(kPD)
append_kernel(Paged pg, const T* __restrict__ K, const T* __restrict__ V, const int* __restrict__ rows,
              int B, const float* __restrict__ Pik, const float* __restrict__ Piv,
              const float* __restrict__ kcb, const float* __restrict__ vcb, int kbits, int vbits, int rot,
              float* __restrict__ mass, int* __restrict__ positions, int S, int cap) {
  __shared__ float x[kPD];
  __shared__ float red[4];
  __shared__ double dred[4];
  __shared__ unsigned char code[kPD];
  const int i = blockIdx.x, h = blockIdx.y, d = threadIdx.x;
  const int seq = rows[3 * i], slot = rows[3 * i + 1], pos = rows[3 * i + 2];
  if (seq < 0 || slot < 0) return;
  if (seq >= B || slot >= cap) {
    if (d == 0) atomicOr(&g_wait_fault, static_cast<unsigned int>(kFaultPaged));
    return;
  }
  const int page = pg.page(seq, slot);
  if (page < 0) return;
  const size_t row = pg.row(page, h, slot);
  for (int part = 0; part < 2; ++part) {
    const float v = load_x(part ? V : K, (static_cast<size_t>(i) * pg.H + h) * kPD + d);
    const float* Pi = (part ? Piv : Pik) + static_cast<size_t>(h % rot) * kPD * kPD;
    const float* cb = part ? vcb : kcb;
    const int bits = part ? vbits : kbits;
    const float top = block_max(isfinite(v) ? fabsf(v) : INFINITY, red);
    x[d] = v;
    const double n = sqrt(block_sum(static_cast<double>(v) * v, dred));
    int c = 0;
    if (top < INFINITY) {
      double y = 0.0;
      for (int j = 0; j < kPD; ++j) y += static_cast<double>(Pi[d * kPD + j]) * x[j];
      for (int k = 0; k + 1 < (1 << bits); ++k) {
        const double mid = 0.5 * (static_cast<double>(cb[k]) + cb[k + 1]);
        c += n > 0.0 ? y > mid * n : 0.0 > mid;
      }
    }
    code[d] = static_cast<unsigned char>(c);
    __syncthreads();
    uint32_t* dst = reinterpret_cast<uint32_t*>((part ? pg.vp : pg.kp) + row * (16 * bits));
    if (d < 4 * bits) {
      uint32_t w = 0;
      for (int t = 0; t < 32; ++t) {
        const int bit = 32 * d + t;
        w |= static_cast<uint32_t>((code[bit / bits] >> (bit % bits)) & 1) << t;
      }
      dst[d] = w;
    }
    if (d == 0) (part ? pg.vn : pg.kn)[row] = __half_as_ushort(__double2half(n));
    __syncthreads();
  }
  if (d == 0) {
    const size_t at = (static_cast<size_t>(seq) * pg.H + h) * S + slot;
    if (mass != nullptr) mass[at] = 0.f;
    if (positions != nullptr) positions[at] = pos;
  }
}

template <typename T>
cudaError_t launch(const tq_paged_cache& c, const T* K, const T* V, const int* rows, int n, const int* table,
                   int B, int max_pages, float* mass, int* positions, int S, cudaStream_t st) {
  int cap = max_pages * c.page_size;
  if ((mass != nullptr || positions != nullptr) && S < cap) cap = S;
  append_kernel<T><<<dim3(n, c.H), kPD, 0, st>>>(paged_view(c, table, max_pages), K, V, rows, B, c.Pi_k, c.Pi_v,
                                                 c.k_codebook, c.v_codebook, c.k_bits, c.v_bits, c.rot_heads,
                                                 mass, positions, S, cap);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append_paged(const tq_paged_cache& c, const void* K, const void* V, tq_qtype type,
                                const int* rows, int n, const int* table, int B, int max_pages, float* mass,
                                int* positions, int S, cudaStream_t st) {
  if (type == TQ_Q_F32)
    return launch(c, static_cast<const float*>(K), static_cast<const float*>(V), rows, n, table, B, max_pages,
                  mass, positions, S, st);
  return launch(c, static_cast<const __nv_bfloat16*>(K), static_cast<const __nv_bfloat16*>(V), rows, n, table, B,
                max_pages, mass, positions, S, st);
}

cudaError_t take_faults_append(unsigned int* bits) { return take_unit_faults(bits); }

}  // namespace tq
