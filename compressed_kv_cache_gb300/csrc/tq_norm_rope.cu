// Norms of queries and keys by head, and the rotation by their positions, in one pass (tq_norm_rope):
//
//   y = x / sqrt(mean(x^2) + eps) * w,   (a, b) -> (a cos t - b sin t, b cos t + a sin t),
//   t = positions[axis of the pair] * frequency of the pair
//
// A row (one head of one token) lies across 8 to 32 lanes; a lane holds both members of four pairs, so that
// the rotation needs no exchange between lanes and a lane's four sines and cosines serve every head of its
// token.  Sums are held in 32 bits, the result is rounded once.
//
// The angle: turns[i] = frequency / (2 pi) as a 64-bit fraction of a turn.  position * turns[i] modulo 2^64
// drops the whole turns exactly, whatever the position, and its top 32 bits are the angle to 2^-32 of a turn.  As an fp32
// number of half turns it is off by up to 2^-26 of a turn, 1e-7 radians, of the order of the sine's own fp32 step.
// One 64-bit product replaces the double-precision range reduction that an fp32 angle of a far position
// (131072 radians have a step of 0.0078) would need.
//
// Bound by memory with the issue close behind (8191 tokens, 32 + 8 heads of 128 in bf16: 168 MB in 33 us, 75 % of the copy
// rate, 68 % of the issue slots; in fp32 335 MB in 57 us, 86 %); lanes of 16 bytes in two halves, whole lines a warp, four rows in flight.
#include "tq_int8.cuh"

namespace tq {
namespace {

constexpr int kThreads = 256;
template <typename T>
constexpr int kRowsOf = sizeof(T) == 4 ? 2 : 4;      // rows a lane has in flight, 16 registers either way

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

// A warp takes `per` heads of one token, of the queries' heads and the keys' behind them.  kLanes lanes a row.
template <typename T, int kLanes, bool kPaired>
__global__ void __launch_bounds__(kThreads, 4) norm_rope_kernel(const NormRope a, int per, int parts, float inv_d) {
  constexpr int kAt = 32 / kLanes, kRows = kRowsOf<T>;         // rows at a time, loads of them in flight
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t token = unit / parts;
  if (token >= a.n) return;
  const int part = static_cast<int>(unit - token * parts);

  // where this lane's two groups of four lie: members of four pairs, or eight that are not rotated
  const int j = lane % kLanes, sub = lane / kLanes, rot = 2 * a.pairs;
  const bool turned = 8 * j < rot, there = 8 * j < a.D;
  const int at_a = turned && !kPaired ? 4 * j : 8 * j;
  const int at_b = turned && !kPaired ? a.pairs + 4 * j : 8 * j + 4;

  float c[4], s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = 1.0f;
    s[i] = 0.0f;
  }
  bool made = false;
  auto heads = [&](const T* x, int64_t stride, T* out, const void* weight, int h0, int h1) {
    if (h0 >= h1) return;
    const T* from = x + (h0 + sub) * stride;
    T* to = out + static_cast<int64_t>(h0 + sub) * a.D;
    Four<T> xa[kRows], xb[kRows];
    auto fetch = [&](int left) {
#pragma unroll
      for (int r = 0; r < kRows; ++r)
        if (there && r * kAt + sub < left) {
          xa[r].load(from + r * kAt * stride + at_a);
          xb[r].load(from + r * kAt * stride + at_b);
        }
    };
    fetch(h1 - h0);
    if (!made && turned) {      // under way while the rows come
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int axis = min(static_cast<int>(__ldg(a.axis + 4 * j + i)), a.axes - 1);
        const int64_t pos = __ldg(a.positions + token * a.axes + axis);
        const uint64_t turn = __ldg(reinterpret_cast<const unsigned long long*>(a.turns) + 4 * j + i) * static_cast<uint64_t>(pos);
        sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &s[i], &c[i]);
      }
    }
    made = true;
    float w[8];
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
    for (int left = h1 - h0;;) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (r * kAt >= left) break;      // the whole warp's
        const bool mine = there && r * kAt + sub < left;
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 0.0f;
        if (mine) {
          xa[r].get(f);
          xb[r].get(f + 4);
        }
        if (weight != nullptr) {
          float ss = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
#pragma unroll
          for (int o = 1; o < kLanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float inv = rsqrtf(fmaf(ss, inv_d, a.eps));
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] *= inv * w[i];
        }
        if (turned) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int u = kPaired ? 2 * i : i, v = kPaired ? 2 * i + 1 : 4 + i;
            const float y = f[u];
            f[u] = y * c[i] - f[v] * s[i];
            f[v] = f[v] * c[i] + y * s[i];
          }
        }
        if (mine) {
          Four<T>::put(to + r * kAt * a.D + at_a, f);
          Four<T>::put(to + r * kAt * a.D + at_b, f + 4);
        }
      }
      left -= kRows * kAt;
      if (left <= 0) break;
      from += kRows * kAt * stride;
      to += kRows * kAt * a.D;
      fetch(left);
    }
  };
  const int h0 = part * per, h1 = min(a.Hq + a.Hk, h0 + per);
  heads(static_cast<const T*>(a.q) + token * a.q_token, a.q_head, static_cast<T*>(a.q_out) + token * a.Hq * a.D, a.q_weight, min(h0, a.Hq),
        min(h1, a.Hq));
  heads(static_cast<const T*>(a.k) + token * a.k_token, a.k_head, static_cast<T*>(a.k_out) + token * a.Hk * a.D, a.k_weight, max(h0 - a.Hq, 0),
        max(h1 - a.Hq, 0));
}

template <typename T, int kLanes>
void launch(const NormRope& a, int per, int parts, cudaStream_t st) {
  const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(a.n) * parts + kThreads / 32 - 1) / (kThreads / 32));
  const float inv_d = 1.0f / static_cast<float>(a.D);
  if (a.paired) norm_rope_kernel<T, kLanes, true><<<blocks, kThreads, 0, st>>>(a, per, parts, inv_d);
  else norm_rope_kernel<T, kLanes, false><<<blocks, kThreads, 0, st>>>(a, per, parts, inv_d);
}

template <typename T>
cudaError_t launch_of(const NormRope& a, cudaStream_t st) {
  const int lanes = a.D <= 64 ? 8 : a.D <= 128 ? 16 : 32, rows = 32 / lanes;
  // As many heads a warp as leave 16 warps for each of 152 SMs: a token's sines are then made once, and a
  // single token is spread over warps of one row a lane.
  const int heads = a.Hq + a.Hk;
  const int64_t share = static_cast<int64_t>(a.n) * heads / (152 * 16);
  int per = share < 1 ? 1 : share > heads ? heads : static_cast<int>(share);
  per = (per + rows - 1) / rows * rows;
  const int parts = (heads + per - 1) / per;
  if (lanes == 8) launch<T, 8>(a, per, parts, st);
  else if (lanes == 16) launch<T, 16>(a, per, parts, st);
  else launch<T, 32>(a, per, parts, st);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRope& a, tq_qtype type, cudaStream_t st) {
  return type == TQ_Q_F32 ? launch_of<float>(a, st) : launch_of<__nv_bfloat16>(a, st);
}

}  // namespace tq
