// Norms of queries and keys by head, and the rotation by their positions, in one pass (tq_norm_rope):
//
//   y = x / sqrt(mean(x^2) + eps) * w,   (a, b) -> (a cos t - b sin t, b cos t + a sin t),
//   t = positions[axis of the pair] * frequency of the pair
//
// A row (one head of one token) lies across 2 to 32 lanes; a lane holds both members of four pairs, so that
// the rotation needs no exchange between lanes and a lane's four sines and cosines serve every head of its
// token.  Sums are held in 32 bits, the result is rounded once.
//
// The angle: turns[i] = frequency / (2 pi) as a 64-bit fraction of a turn.  position * turns[i] modulo 2^64
// drops the whole turns exactly, whatever the position, and its top 32 bits are the angle to 2^-32 of a turn;
// one 64-bit product replaces the double-precision range reduction that an fp32 angle of a far position
// (131072 radians have a step of 0.0078) would need.
#include "tq_int8.cuh"

namespace tq {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;         // rows a lane has in flight

template <typename T>
struct Four;
template <>
struct Four<float> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void get(float* f) const { f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w; }
  __device__ static __forceinline__ void put(float* p, const float* f) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <>
struct Four<__nv_bfloat16> {
  uint2 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = __uint_as_float(v.x << 16); f[1] = __uint_as_float(v.x & 0xffff0000u);
    f[2] = __uint_as_float(v.y << 16); f[3] = __uint_as_float(v.y & 0xffff0000u);
  }
  __device__ static __forceinline__ void put(__nv_bfloat16* p, const float* f) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
};

// A warp takes `per` heads of one token, queries' or keys' (parts: slices of queries, then of keys).
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRope a, int lanes_log2, int per, int q_parts, int parts) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t token = unit / parts;
  if (token >= a.n) return;
  int part = static_cast<int>(unit - token * parts);
  const bool keys = part >= q_parts;
  if (keys) part -= q_parts;
  const int heads = keys ? a.Hk : a.Hq;
  const int stop = min(heads, (part + 1) * per);
  const T* x = static_cast<const T*>(keys ? a.k : a.q) + token * (keys ? a.k_token : a.q_token);
  const int64_t head_stride = keys ? a.k_head : a.q_head;
  T* out = static_cast<T*>(keys ? a.k_out : a.q_out) + token * heads * a.D;
  const void* weight = keys ? a.k_weight : a.q_weight;

  // where this lane's two groups of four lie: members of four pairs, or eight that are not rotated
  const int j = lane & ((1 << lanes_log2) - 1), sub = lane >> lanes_log2, rows = 32 >> lanes_log2;
  const int rot = 2 * a.pairs;
  const bool turned = 8 * j < rot, there = 8 * j < a.D;
  const int at_a = turned && !a.paired ? 4 * j : 8 * j;
  const int at_b = turned && !a.paired ? rot / 2 + 4 * j : 8 * j + 4;

  Four<T> xa[kRows], xb[kRows];
  auto fetch = [&](int h0) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int h = h0 + r * rows + sub;
      if (there && h < stop) {
        xa[r].load(x + h * head_stride + at_a);
        xb[r].load(x + h * head_stride + at_b);
      }
    }
  };
  int h0 = part * per;
  fetch(h0);

  float w[8], c[4], s[4];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 1.0f;
  if (weight != nullptr && there) {
    if (a.weights_bf16) {
      Four<__nv_bfloat16> u, v;
      u.load(static_cast<const __nv_bfloat16*>(weight) + at_a);
      v.load(static_cast<const __nv_bfloat16*>(weight) + at_b);
      u.get(w); v.get(w + 4);
    } else {
      Four<float> u, v;
      u.load(static_cast<const float*>(weight) + at_a);
      v.load(static_cast<const float*>(weight) + at_b);
      u.get(w); v.get(w + 4);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = 1.0f;
    s[i] = 0.0f;
    if (turned) {
      const int axis = min(static_cast<int>(__ldg(a.axis + 4 * j + i)), a.axes - 1);
      const int64_t pos = __ldg(a.positions + token * a.axes + axis);
      const uint64_t turn = __ldg(reinterpret_cast<const unsigned long long*>(a.turns) + 4 * j + i) * static_cast<uint64_t>(pos);
      sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &s[i], &c[i]);
    }
  }

  for (; h0 < stop; h0 += kRows * rows) {
    if (h0 != part * per) fetch(h0);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int h = h0 + r * rows + sub;
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = 0.0f;
      if (there && h < stop) {
        xa[r].get(f);
        xb[r].get(f + 4);
      }
      if (weight != nullptr) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
        for (int o = 1; o < 1 << lanes_log2; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = rsqrtf(ss / static_cast<float>(a.D) + a.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = f[i] * inv * w[i];
      }
      float g[8];
      if (!turned) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = f[i];
      } else if (a.paired) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          g[2 * i] = f[2 * i] * c[i] - f[2 * i + 1] * s[i];
          g[2 * i + 1] = f[2 * i + 1] * c[i] + f[2 * i] * s[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          g[i] = f[i] * c[i] - f[4 + i] * s[i];
          g[4 + i] = f[4 + i] * c[i] + f[i] * s[i];
        }
      }
      if (there && h < stop) {
        Four<T>::put(out + static_cast<int64_t>(h) * a.D + at_a, g);
        Four<T>::put(out + static_cast<int64_t>(h) * a.D + at_b, g + 4);
      }
    }
  }
}

}  // namespace

cudaError_t launch_norm_rope(const NormRope& a, tq_qtype type, cudaStream_t st) {
  int lanes_log2 = 0;
  while ((8 << lanes_log2) < a.D) ++lanes_log2;
  const int rows = 32 >> lanes_log2;
  // As many heads a warp as leave 16 warps for each of 152 SMs: a token's sines are then made once for
  // its queries and once for its keys, and a single token is spread over warps of one row a lane.
  const int heads = a.Hq > a.Hk ? a.Hq : a.Hk;
  int per = static_cast<int>(static_cast<int64_t>(a.n) * (a.Hq + a.Hk) / (152 * 16));
  per = (per < 1 ? 1 : per > heads ? heads : per);
  per = (per + rows - 1) / rows * rows;
  const int q_parts = (a.Hq + per - 1) / per, parts = q_parts + (a.Hk + per - 1) / per;
  const int64_t blocks = (static_cast<int64_t>(a.n) * parts + kThreads / 32 - 1) / (kThreads / 32);
  if (type == TQ_Q_F32)
    norm_rope_kernel<float><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(a, lanes_log2, per, q_parts, parts);
  else
    norm_rope_kernel<__nv_bfloat16><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(a, lanes_log2, per, q_parts, parts);
  return cudaGetLastError();
}

}  // namespace tq
