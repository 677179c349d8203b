// Attention of a step's tokens over the 8-bit paged cache (tq_attend_int8), the plain way: a block of threads takes one
// token and query head, a thread a slot for the logits and a dimension for the sum of values.
#include "tq_int8.cuh"

namespace tq {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <typename T>
__global__ void __launch_bounds__(kThreads)
attend_kernel(const Int8View c, const T* __restrict__ Q, const Step step, int G, int D, int window, int sinks, float scale2, T* __restrict__ out) {
  __shared__ float q[128], p[kThreads], red[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int token = blockIdx.x, head = blockIdx.y, h = head / G;
  int lo = 0, hi = step.B;      // the last sequence that starts at or before the token
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (step.starts[mid] <= token) lo = mid;
    else hi = mid;
  }
  const Run r = run_of(step, lo);
  if (token < r.first || token >= r.first + r.count) return;
  const int at = r.len + token - r.first;
  const size_t qi = (static_cast<size_t>(token) * c.H * G + head) * D;
  if (tid < D) q[tid] = load1(Q + qi + tid) * scale2;
  float top = -INFINITY, sum = 0.0f, acc = 0.0f;
  for (int64_t s0 = 0; s0 <= at; s0 += kThreads) {
    __syncthreads();
    const int s = static_cast<int>(s0) + tid;
    float z = -INFINITY;
    const bool seen = s <= at && (window <= 0 || s > at - window || s < sinks);
    const int pg = seen ? c.page(lo, s) : -1;
    if (pg >= 0) {
      const size_t row = c.row(pg, h, s);
      const uint8_t* k = c.kc + row * D;
      float dot = 0.0f;
      for (int d = 0; d < D; ++d) dot = fmaf(q[d], k[d] - 127.5f, dot);
      z = dot * pow2(c.ex[row / kBlockSlots * 2]);
    }
    float m = z;
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) red[warp] = m;
    __syncthreads();
    m = top;
    for (int i = 0; i < kThreads / 32; ++i) m = fmaxf(m, red[i]);
    const float rescale = m == -INFINITY ? 1.0f : exp2f(top - m);
    top = m;
    p[tid] = pg >= 0 ? exp2f(z - top) : 0.0f;
    __syncthreads();
    sum *= rescale;
    acc *= rescale;
    for (int i = 0; i < kThreads; ++i) {
      if (p[i] == 0.0f) continue;
      sum += p[i];
      const size_t row = c.row(c.page(lo, static_cast<int>(s0) + i), h, static_cast<int>(s0) + i);
      if (tid < D) acc = fmaf(p[i] * pow2(c.ex[row / kBlockSlots * 2 + 1]), c.vc[row * D + tid] - 127.5f, acc);
    }
  }
  if (tid < D) store1(out + qi + tid, sum == 0.0f ? 0.0f : acc / sum);
}

}  // namespace

size_t attend_int8_bytes(int n, int B, int H, int G, int D) { return 256; }

cudaError_t launch_attend_int8(const tq_int8_cache& c, const void* Q, tq_qtype type, const Step& step, int G,
                               const int* table, int max_pages, int window, int sinks, float scale, void* out,
                               void* ws, cudaStream_t st) {
  const Int8View v = int8_view(c, table, max_pages);
  const float scale2 = scale * 1.4426950408889634f;
  const dim3 grid(step.n, c.H * G);
  if (type == TQ_Q_F32)
    attend_kernel<<<grid, kThreads, 0, st>>>(v, static_cast<const float*>(Q), step, G, c.D, window, sinks, scale2, static_cast<float*>(out));
  else
    attend_kernel<<<grid, kThreads, 0, st>>>(v, static_cast<const __nv_bfloat16*>(Q), step, G, c.D, window, sinks, scale2,
                                             static_cast<__nv_bfloat16*>(out));
  return cudaGetLastError();
}

cudaError_t take_faults_int8_attend(unsigned int* bits) { return take_unit_faults(bits); }

}  // namespace tq
