// Attention of a step's tokens over the 8-bit paged cache (tq_attend_int8): two launches, the second a programmatic
// dependent of the first.
//   split   tq_int8_split.cuh: every unit's sums, written out where one block of threads had all of it
//   join    the parts of a unit that lies across blocks
#include "tq_int8_split.cuh"

namespace tq {
namespace {

constexpr int kJoinWarps = 8;
constexpr float kLifted = 7.0f;      // weights were taken 2^7 above their range


// Block (i, k) takes columns 8 k .. 8 k + 7 of the unit that block i of the split starts in the middle of, if that is the
// first start inside it: parts (i - 1, 1), (i, 0), (i + 1, 0) and on.  A warp takes a column, a lane its D / 32
// dimensions; the factors of 32 parts are made by 32 lanes.
template <typename T, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) attend_join_kernel(const AttendArgs a, int NC) {
  constexpr int kDims = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const AttendRecord r = a.rec[blockIdx.x];
  if (r.off == 0 || r.off > r.chunk) return;
  const int lane = threadIdx.x & 31, col = blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
  const int64_t cc = static_cast<int64_t>(r.cb) * NC + col;
  if (cc >= static_cast<int64_t>(r.count) * a.G) return;
  const int pieces = 1 + static_cast<int>((r.quads - r.off + r.chunk - 1) / r.chunk);
  auto place = [&](int p) {
    return (static_cast<size_t>(p == 0 ? blockIdx.x - 1 : blockIdx.x + p - 1) * 2 + (p == 0 ? 1 : 0)) * NC + col;
  };
  float mt = -3.4e38f, Mt = -3.4e38f;
  for (int p = lane; p < pieces; p += 32) {
    const float4 v = a.top[place(p)];
    mt = fmaxf(mt, v.x);
    Mt = fmaxf(Mt, v.y);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
    Mt = fmaxf(Mt, __shfl_xor_sync(0xffffffffu, Mt, o));
  }
  float l = 0.0f, acc[kDims];
#pragma unroll
  for (int d = 0; d < kDims; ++d) acc[d] = 0.0f;
  for (int p0 = 0; p0 < pieces; p0 += 32) {
    float f = 0.0f;
    if (p0 + lane < pieces) {
      const float4 v = a.top[place(p0 + lane)];
      l = fmaf(v.z, exp2f(v.x - mt), l);
      f = exp2f(v.y - Mt);
    }
    const int n = min(32, pieces - p0);
#pragma unroll 8
    for (int p = 0; p < n; ++p) {
      const float g = __shfl_sync(0xffffffffu, f, p);
      const float* from = a.part + place(p0 + p) * D + lane * kDims;
      if constexpr (kDims == 4) {
        const float4 v = *reinterpret_cast<const float4*>(from);
        acc[0] = fmaf(v.x, g, acc[0]); acc[1] = fmaf(v.y, g, acc[1]); acc[2] = fmaf(v.z, g, acc[2]); acc[3] = fmaf(v.w, g, acc[3]);
      } else {
        const float2 v = *reinterpret_cast<const float2*>(from);
        acc[0] = fmaf(v.x, g, acc[0]); acc[1] = fmaf(v.y, g, acc[1]);
      }
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const float f = 1.0f / l, up = exp2f(Mt - mt - kLifted);
  const int token = static_cast<int>(cc / a.G), head = static_cast<int>(cc - static_cast<int64_t>(token) * a.G);
  T* to = static_cast<T*>(a.out) + ((static_cast<size_t>(r.first) + token) * a.c.H * a.G + static_cast<size_t>(r.h) * a.G + head) * D + lane * kDims;
#pragma unroll
  for (int d = 0; d < kDims; ++d) {
    const float v = l == 0.0f ? 0.0f : acc[d] * f * up;
    if constexpr (sizeof(T) == 4) to[d] = v;
    else to[d] = __float2bfloat16_rn(v);
  }
}

// Columns of 8 that a unit holds: as many as an average sequence fills, 4 at most (registers).  The
// cache is read once for all columns of a unit, and a second time, from L2, for the next ones.
int column_tiles(int n, int B, int G) {
  const int64_t columns = (static_cast<int64_t>(n) * G + B - 1) / B;
  return columns <= 8 ? 1 : columns <= 16 ? 2 : 4;
}

struct Space {
  size_t top, part, all;
  Space(int nt, int D) {
    size_t at = paged_round(kAttendCtas * sizeof(AttendRecord));
    top = at;
    at += paged_round(static_cast<size_t>(kAttendCtas) * 2 * 8 * nt * sizeof(float4));
    part = at;
    all = at + static_cast<size_t>(kAttendCtas) * 2 * 8 * nt * D * sizeof(float);
  }
};

}  // namespace

size_t attend_int8_bytes(int n, int B, int H, int G, int D) { return Space(column_tiles(n, B, G), D).all; }

cudaError_t launch_attend_int8(const tq_int8_cache& c, const void* Q, tq_qtype type, const Step& step, int G,
                               const int* table, int max_pages, int window, int sinks, float scale, void* out,
                               void* ws, cudaStream_t st) {
  static std::atomic<int> sms_cache[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int sms = sms_cache[dev & 63].load(std::memory_order_relaxed);
  if (sms == 0) {
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    sms_cache[dev & 63].store(sms, std::memory_order_relaxed);
  }
  const int ctas = 2 * sms < kAttendCtas ? 2 * sms : kAttendCtas;
  const int nt = column_tiles(step.n, step.B, G);
  const Space sp(nt, c.D);
  char* w = static_cast<char*>(ws);
  const AttendArgs a = {int8_view(c, table, max_pages), step, Q, out, G, window, sinks, scale * 1.4426950408889634f,
                        reinterpret_cast<AttendRecord*>(w), reinterpret_cast<float4*>(w + sp.top), reinterpret_cast<float*>(w + sp.part)};
  const bool f32 = type == TQ_Q_F32;
  if (c.D == 64) e = f32 ? launch_attend_split_f32_64(a, nt, ctas, st) : launch_attend_split_bf16_64(a, nt, ctas, st);
  else e = f32 ? launch_attend_split_f32_128(a, nt, ctas, st) : launch_attend_split_bf16_128(a, nt, ctas, st);
  if (e != cudaSuccess) return e;

  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(ctas, nt);
  cfg.blockDim = dim3(kJoinWarps * 32);
  if (c.D == 64)
    return f32 ? cudaLaunchKernelEx(&cfg, attend_join_kernel<float, 64>, a, 8 * nt)
               : cudaLaunchKernelEx(&cfg, attend_join_kernel<__nv_bfloat16, 64>, a, 8 * nt);
  return f32 ? cudaLaunchKernelEx(&cfg, attend_join_kernel<float, 128>, a, 8 * nt)
             : cudaLaunchKernelEx(&cfg, attend_join_kernel<__nv_bfloat16, 128>, a, 8 * nt);
}

cudaError_t take_faults_int8_attend(unsigned int* bits) {
  cudaError_t e = take_faults_attend_bf16_64(bits);
  if (e == cudaSuccess) e = take_faults_attend_bf16_128(bits);
  if (e == cudaSuccess) e = take_faults_attend_f32_64(bits);
  if (e == cudaSuccess) e = take_faults_attend_f32_128(bits);
  return e;
}

}  // namespace tq
