// Attention of one new token over the paged cache (tq_decode_paged).
#include "tq_paged.cuh"

namespace tq {
namespace {

__device__ __forceinline__ float load_q(const float* q, size_t i) { return q[i]; }
__device__ __forceinline__ float load_q(const __nv_bfloat16* q, size_t i) { return __bfloat162float(q[i]); }
__device__ __forceinline__ void store_o(float* o, size_t i, float v) { o[i] = v; }
__device__ __forceinline__ void store_o(__nv_bfloat16* o, size_t i, float v) { o[i] = __float2bfloat16_rn(v); }

__device__ __forceinline__ unsigned code_at(const uint8_t* row, int bits, int d) {
  const int at = bits * d;
  unsigned w = row[at >> 3];
  if ((at & 7) + bits > 8) w |= static_cast<unsigned>(row[(at >> 3) + 1]) << 8;
  return (w >> (at & 7)) & ((1u << bits) - 1);
}

// One block per (sequence, head): its queries in turn, the keys in tiles of 128, the softmax
// with a running maximum and sum, fp32 throughout.  z keeps the logits where mass is asked for.
template <typename T>
__global__ void __launch_bounds__(kPD)
decode_simple_kernel(Paged pg, const T* __restrict__ Q, const int* __restrict__ lengths, int G,
                     const float* __restrict__ Pik, const float* __restrict__ Piv,
                     const float* __restrict__ kcb, const float* __restrict__ vcb, int kbits, int vbits,
                     int rot, float scale, float* __restrict__ mass, int S, int cap, T* __restrict__ out,
                     float* __restrict__ z) {
  __shared__ float q[kPD], a[kPD], w[kPD], red[4], ck[16], cv[16];
  __shared__ size_t rows[kPD];
  const int b = blockIdx.x, h = blockIdx.y, d = threadIdx.x;
  const int n = pg.length(lengths, b, cap);
  if (d < 1 << kbits) ck[d] = kcb[d];
  if (d < 1 << vbits) cv[d] = vcb[d];
  const float* Pk = Pik + static_cast<size_t>(h % rot) * kPD * kPD;
  const float* Pv = Piv + static_cast<size_t>(h % rot) * kPD * kPD;
  for (int g = 0; g < G; ++g) {
    const size_t qo = (static_cast<size_t>(b) * pg.H + h) * G + g;
    float* zq = z == nullptr ? nullptr : z + qo * S;
    __syncthreads();
    q[d] = load_q(Q, qo * kPD + d);
    __syncthreads();
    float y = 0.f;
    for (int j = 0; j < kPD; ++j) y = fmaf(Pk[d * kPD + j], q[j], y);
    a[d] = y;
    float M = -INFINITY, L = 0.f, acc = 0.f;
    for (int s0 = 0; s0 < n; s0 += kPD) {
      const int s = s0 + d;
      __syncthreads();
      float v = -INFINITY, nv = 0.f;
      rows[d] = 0;
      if (s < n) {
        const int page = pg.page(b, s);
        if (page >= 0) {
          const size_t r = pg.row(page, h, s);
          rows[d] = r;
          const uint8_t* kr = pg.kp + r * 16 * kbits;
          float t = 0.f;
          for (int j = 0; j < kPD; ++j) t = fmaf(a[j], ck[code_at(kr, kbits, j)], t);
          v = t * __half2float(__ushort_as_half(pg.kn[r])) * scale;
          nv = __half2float(__ushort_as_half(pg.vn[r]));
        }
        if (zq != nullptr) zq[s] = v;
      }
      float m = v;
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if ((d & 31) == 0) red[d >> 5] = m;
      __syncthreads();
      m = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), M);
      const float r = M > -INFINITY ? expf(M - m) : 0.f;
      const float p = v > -INFINITY ? expf(v - m) : 0.f;
      M = m;
      w[d] = p > 0.f ? p * nv : 0.f;
      float l = p;
      for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      __syncthreads();
      if ((d & 31) == 0) red[d >> 5] = l;
      __syncthreads();
      L = L * r + (red[0] + red[1] + red[2] + red[3]);
      acc *= r;
      const int cnt = min(kPD, n - s0);
      for (int j = 0; j < cnt; ++j)
        if (w[j] != 0.f) acc = fmaf(w[j], cv[code_at(pg.vp + rows[j] * 16 * vbits, vbits, d)], acc);
    }
    __syncthreads();
    q[d] = L > 0.f ? acc / L : 0.f;
    __syncthreads();
    y = 0.f;
    for (int j = 0; j < kPD; ++j) y = fmaf(Pv[j * kPD + d], q[j], y);
    store_o(out, qo * kPD + d, y);
    if (mass != nullptr && L > 0.f)
      for (int s = d; s < n; s += kPD)
        mass[(static_cast<size_t>(b) * pg.H + h) * S + s] += expf(zq[s] - M) / L;
  }
}

template <typename T>
cudaError_t launch(const tq_paged_cache& c, const T* Q, const int* table, const int* lengths, int B, int G,
                   int max_pages, float scale, float* mass, int S, T* out, void* ws, cudaStream_t st) {
  int cap = max_pages * c.page_size;
  if (mass != nullptr && S < cap) cap = S;
  decode_simple_kernel<T><<<dim3(B, c.H), kPD, 0, st>>>(
      paged_view(c, table, max_pages), Q, lengths, G, c.Pi_k, c.Pi_v, c.k_codebook, c.v_codebook, c.k_bits,
      c.v_bits, c.rot_heads, scale, mass, S, cap, out, mass != nullptr ? static_cast<float*>(ws) : nullptr);
  return cudaGetLastError();
}

}  // namespace

size_t decode_paged_bytes(int B, int H, int G, int S, bool with_mass) {
  return paged_round(with_mass ? static_cast<size_t>(B) * H * G * S * 4 : 256);
}

cudaError_t launch_decode_paged(const tq_paged_cache& c, const void* Q, tq_qtype qtype, const int* table,
                                const int* lengths, int B, int G, int max_pages, float scale, float* mass,
                                int S, void* out, void* ws, cudaStream_t st) {
  if (qtype == TQ_Q_F32)
    return launch(c, static_cast<const float*>(Q), table, lengths, B, G, max_pages, scale, mass, S,
                  static_cast<float*>(out), ws, st);
  return launch(c, static_cast<const __nv_bfloat16*>(Q), table, lengths, B, G, max_pages, scale, mass, S,
                static_cast<__nv_bfloat16*>(out), ws, st);
}

cudaError_t take_faults_paged(unsigned int* bits) { return take_unit_faults(bits); }

}  // namespace tq
