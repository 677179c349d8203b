// Attention of a step's tokens over the 8-bit paged cache (tq_attend_int8): two launches, the second a programmatic
// dependent of the first.
//   split   tq_int8_split.cuh, or tq_int8_prompt.cu for pieces of prompts: every unit's sums, written out where one
//           block of threads had all of it
//   join    the parts of a unit that lies across blocks
#include "tq_int8_split.cuh"

namespace tq {
namespace {

constexpr int kJoinWarps = 8;
constexpr float kLifted = 7.0f;      // weights were taken 2^7 above their range

// Block i of the split that starts in the middle of a unit, as the first to do so, names a unit to be joined: its parts are
// (i - 1, 1), (i, 0), (i + 1, 0) and on.  Every block of the join lists these units and takes its share of their
// columns.  Many columns: a warp each.  Few (one long sequence): a block each, its warps taking every eighth part, so
// that all parts are on their way at once.  A lane holds D / 32 dimensions.
template <typename T, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) attend_join_kernel(const AttendArgs a, int nc_log2, int ctas) {
  constexpr int kDims = D / 32;
  const int NC = 1 << nc_log2;
  __shared__ AttendRecord records[kAttendCtas];
  __shared__ int warp_count[kJoinWarps];
  __shared__ float4 warp_top[kJoinWarps];
  __shared__ float warp_acc[kJoinWarps][D];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // all records are on their way at once: two a thread
  static_assert(kAttendCtas <= 2 * kJoinWarps * 32, "records a thread");
  AttendRecord mine[2];
  bool first[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = 2 * tid + k;
    first[k] = false;
    if (i < ctas) {
      mine[k] = a.rec[i];
      first[k] = mine[k].off > 0 && mine[k].off <= mine[k].chunk;
    }
  }
  int at = (first[0] ? 1 : 0) + (first[1] ? 1 : 0);
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, at, o);
    if (lane >= o) at += y;
  }
  if (lane == 31) warp_count[warp] = at;
  __syncthreads();
  int units = 0;
  for (int w = 0; w < kJoinWarps; ++w) {
    if (w < warp) at += warp_count[w];
    units += warp_count[w];
  }
#pragma unroll
  for (int k = 1; k >= 0; --k)
    if (first[k]) records[--at] = mine[k];
  __syncthreads();
  const int items = units * NC;
  const bool shared = items < static_cast<int>(gridDim.x) * 2;      // a block an item
  const int step = shared ? kJoinWarps : 1, w0 = shared ? warp : 0;
  for (int item = shared ? blockIdx.x : blockIdx.x * kJoinWarps + warp; item < items; item += gridDim.x * (shared ? 1 : kJoinWarps)) {
    const AttendRecord& r = records[item >> nc_log2];
    const int i = r.block, col = item & (NC - 1), cc = r.cb * NC + col;      // all columns of a step are below 2^31
    if (cc >= r.count * a.G) continue;
    const int pieces = 1 + (r.quads - r.off + r.chunk - 1) / r.chunk;
    float mt = -3.4e38f, Mt = -3.4e38f, l = 0.0f, acc[kDims];
#pragma unroll
    for (int d = 0; d < kDims; ++d) acc[d] = 0.0f;
    constexpr int kAhead = 4;
    for (int p0 = w0; p0 < pieces; p0 += kAhead * step) {
      float4 top[kAhead], v[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int p = p0 + k * step;
        top[k] = make_float4(-3.4e38f, -3.4e38f, 0.0f, 0.0f);
        v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (p < pieces) {
          const size_t place = (static_cast<size_t>(p == 0 ? i - 1 : i + p - 1) * 2 + (p == 0 ? 1 : 0)) * NC + col;
          top[k] = a.top[place];
          const float* from = a.part + place * D + lane * kDims;
          if constexpr (kDims == 4) v[k] = *reinterpret_cast<const float4*>(from);
          else {
            const float2 u = *reinterpret_cast<const float2*>(from);
            v[k].x = u.x;
            v[k].y = u.y;
          }
        }
      }
      float m1 = mt, M1 = Mt;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        m1 = fmaxf(m1, top[k].x);
        M1 = fmaxf(M1, top[k].y);
      }
      l *= exp2f(mt - m1);
      const float back = exp2f(Mt - M1);
#pragma unroll
      for (int d = 0; d < kDims; ++d) acc[d] *= back;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        l = fmaf(top[k].z, exp2f(top[k].x - m1), l);
        const float f = exp2f(top[k].y - M1);
        acc[0] = fmaf(v[k].x, f, acc[0]);
        acc[1] = fmaf(v[k].y, f, acc[1]);
        if constexpr (kDims == 4) {
          acc[2] = fmaf(v[k].z, f, acc[2]);
          acc[3] = fmaf(v[k].w, f, acc[3]);
        }
      }
      mt = m1;
      Mt = M1;
    }
    if (shared) {
      __syncthreads();      // the last item's sums have been read
      if (lane == 0) warp_top[warp] = make_float4(mt, Mt, l, 0.0f);
#pragma unroll
      for (int d = 0; d < kDims; ++d) warp_acc[warp][lane * kDims + d] = acc[d];
      __syncthreads();
      if (warp != 0) continue;
      mt = Mt = -3.4e38f;
      for (int w = 0; w < kJoinWarps; ++w) {
        mt = fmaxf(mt, warp_top[w].x);
        Mt = fmaxf(Mt, warp_top[w].y);
      }
      l = 0.0f;
#pragma unroll
      for (int d = 0; d < kDims; ++d) acc[d] = 0.0f;
      for (int w = 0; w < kJoinWarps; ++w) {
        l = fmaf(warp_top[w].z, exp2f(warp_top[w].x - mt), l);
        const float f = exp2f(warp_top[w].y - Mt);
#pragma unroll
        for (int d = 0; d < kDims; ++d) acc[d] = fmaf(warp_acc[w][lane * kDims + d], f, acc[d]);
      }
    }
    const float f = 1.0f / l, up = exp2f(Mt - mt - kLifted);
    const int token = static_cast<unsigned>(cc) / static_cast<unsigned>(a.G), head = cc - token * a.G;
    T* to = static_cast<T*>(a.out) + ((static_cast<size_t>(r.first) + token) * a.c.H * a.G + static_cast<size_t>(r.h) * a.G + head) * D + lane * kDims;
#pragma unroll
    for (int d = 0; d < kDims; ++d) {
      const float v = l == 0.0f ? 0.0f : acc[d] * f * up;
      if constexpr (sizeof(T) == 4) to[d] = v;
      else to[d] = __float2bfloat16_rn(v);
    }
  }
}

// Columns of a unit: 8, 16 or 32 in the warp-wide form, as many as an average sequence fills (the cache is read
// once for all columns of a unit, and again, from L2, for the next ones); 256 in the prompts' form, for bf16 queries with more than 32.
// The average of the step decides for all of its sequences, known to the host without a look at `starts`.  Steps of both kinds pay
// for it: 255 single tokens and a piece of 512, behind 2048 slots each, 32 heads on 8, take 340 us (172 and 64 apart), 32 and a piece of
// 2048 take 281 (33 and 201).
int columns_of(int n, int B, int G, bool f32) {
  const int64_t columns = (static_cast<int64_t>(n) * G + B - 1) / B;
  return columns <= 8 ? 8 : columns <= 16 ? 16 : columns <= 32 || f32 ? 32 : 256;
}

struct Space {
  size_t top, part, all;
  Space(int NC, int D) {
    const size_t parts = static_cast<size_t>(NC == 256 ? kPromptCtas : kAttendCtas) * 2 * NC;
    top = paged_round(kAttendCtas * sizeof(AttendRecord));
    part = top + paged_round(parts * sizeof(float4));
    all = part + parts * D * sizeof(float);
  }
};

}  // namespace

size_t attend_int8_bytes(int n, int B, int H, int G, int D) {
  const size_t one = Space(columns_of(n, B, G, false), D).all, two = Space(columns_of(n, B, G, true), D).all;
  return one > two ? one : two;
}

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
  const bool f32 = type == TQ_Q_F32;
  const int NC = columns_of(step.n, step.B, G, f32), nt = NC / 8, room = NC == 256 ? kPromptCtas : kAttendCtas;
  const int blocks = NC == 256 ? 1 : attend_blocks(f32, c.D, nt), ctas = blocks * sms < room ? blocks * sms : room;
  const Space sp(NC, c.D);
  char* w = static_cast<char*>(ws);
  const AttendArgs a = {int8_view(c, table, max_pages), step, Q, out, G, window, sinks, scale * 1.4426950408889634f,
                        reinterpret_cast<AttendRecord*>(w), reinterpret_cast<float4*>(w + sp.top), reinterpret_cast<float*>(w + sp.part)};
  if (NC == 256) e = launch_attend_prompt(a, c.D, ctas, st);
  else if (c.D == 64) e = f32 ? launch_attend_split_f32_64(a, nt, ctas, st) : launch_attend_split_bf16_64(a, nt, ctas, st);
  else e = f32 ? launch_attend_split_f32_128(a, nt, ctas, st) : launch_attend_split_bf16_128(a, nt, ctas, st);
  if (e != cudaSuccess) return e;

  int nc_log2 = 3;
  while (1 << nc_log2 < NC) ++nc_log2;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // the prompts' 256 columns a unit are many short joins, each a trip to memory: all warps that fit
  cfg.gridDim = dim3((NC == 256 ? 4 : 2) * sms);
  cfg.blockDim = dim3(kJoinWarps * 32);
  if (c.D == 64)
    return f32 ? cudaLaunchKernelEx(&cfg, attend_join_kernel<float, 64>, a, nc_log2, ctas)
               : cudaLaunchKernelEx(&cfg, attend_join_kernel<__nv_bfloat16, 64>, a, nc_log2, ctas);
  return f32 ? cudaLaunchKernelEx(&cfg, attend_join_kernel<float, 128>, a, nc_log2, ctas)
             : cudaLaunchKernelEx(&cfg, attend_join_kernel<__nv_bfloat16, 128>, a, nc_log2, ctas);
}

cudaError_t take_faults_int8_attend(unsigned int* bits) {
  cudaError_t e = take_faults_attend_bf16_64(bits);
  if (e == cudaSuccess) e = take_faults_attend_bf16_128(bits);
  if (e == cudaSuccess) e = take_faults_attend_f32_64(bits);
  if (e == cudaSuccess) e = take_faults_attend_f32_128(bits);
  if (e == cudaSuccess) e = take_faults_attend_prompt(bits);
  return e;
}

}  // namespace tq
