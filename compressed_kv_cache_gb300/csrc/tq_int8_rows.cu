// Rows of the 8-bit paged cache: written (tq_append_int8) and read back (tq_read_int8).
//
// A code u of a block of 16 slots stands for (u - 127.5) * 2^e, e one exponent for the block and head.  Written:
//   e = the least with |x| < 2^(e + 7) for every row of the block that is live, old or new,
//   u = floor(x * 2^-e) + 128.
// floor(floor(x) / 2^s) = floor(x / 2^s), so a block whose exponent grows by s has its old codes shifted and
// holds exactly what it would hold had all its rows come at once: no row is rounded twice, and an error is at
// most half of the block's present step however the tokens arrived.  (With the nearest code of a scale that
// follows the largest value, each growth would round the old rows again.)  The power of two costs at most one of
// the 8 bits; the half step in the middle of a cell is exact in bf16 (an odd number below 256 over two).
//
// A warp takes one block of one head's keys or values: its 16 rows lie one instruction's load apart, all in
// flight at once, so that a unit is one trip to memory for its numbers, one for page and rows, one out.
// Both directions are bound by memory, 2 D (size + 1) bytes a token and head: 8192 tokens of 8 heads in bf16 written in 9.5 us
// (78 % of the copy rate; in fp32 15.8, 78 %; 64 single tokens 3.3 us, four trips to memory one after the other), 15003 slots read as fp32
// in 28.8 (79 %).  With 8 values a lane in fp32 too, half a sector an access, the read took 36.
#include "tq_int8.cuh"

namespace tq {
namespace {

constexpr int kWarps = 4;

// Unit u of a step: a block of 16 slots of one sequence.  Sequence b has at most starts[b + 1] / 16 - starts[b] / 16
// + 2 blocks, so the units from starts[b] / 16 + 2 b on are its own and no prefix sum is needed: n / 16 + 2 B in all.
__host__ __device__ __forceinline__ int64_t units_of(const Step& s) { return s.n / kBlockSlots + 2 * static_cast<int64_t>(s.B); }

struct Unit {
  int b, slot, rows0, rows1, token;   // block from `slot` on; its rows [rows0, rows1) are the step's tokens from `token` on
  bool old;                           // rows before rows0 are live
};

__device__ __forceinline__ int64_t first_unit(int start, int b) { return (start >> 4) + 2 * static_cast<int64_t>(b); }

// The sequence is looked for by 32 lanes at a time: 2 loads in a row for 1024 sequences.  Where starts do not ascend the search may end
// anywhere.  It is right where it ends at a sequence whose numbers fit and whose unit this is, or before the first
// or behind the last (tokens of none); else every sequence is asked whether it has rows in this unit, so that what is wrong of
// one costs no other its rows.  (Of two that have tokens in common, and this unit both, one is served.)
__device__ __forceinline__ bool unit_of(const Step& s, int u, int lane, Unit& t) {
  int lo = 0, hi = s.B;
  while (hi - lo > 1) {
    const int stride = (hi - lo + 31) / 32;
    const int i = lo + lane * stride;
    const bool below = i < hi && first_unit(s.starts[i], i) <= u;
    const int n = __popc(__ballot_sync(0xffffffffu, below));
    lo += (n > 0 ? n - 1 : 0) * stride;
    hi = min(hi, lo + stride);
  }
  int a = s.starts[lo], z = s.starts[lo + 1], len = s.lengths[lo];
  const bool good = fits(s, a, z, len), before = u < first_unit(a, lo), behind = u >= first_unit(z, lo + 1);
  if (!good || before || behind) {
    if (good && (before ? lo == 0 : lo == s.B - 1)) return false;
    atomicOr(&g_wait_fault, static_cast<unsigned int>(kFaultPaged));
    uint32_t owners = 0;
    int b0 = -32;
    while (owners == 0 && b0 + 32 < s.B) {
      b0 += 32;
      const int b = b0 + lane;
      bool own = false;
      if (b < s.B) {
        a = s.starts[b];
        z = s.starts[b + 1];
        len = s.lengths[b];
        const int64_t k = u - first_unit(a, b);
        own = a < z && fits(s, a, z, len) && k >= 0 && ((len >> 4) + k) << 4 < static_cast<int64_t>(len) + z - a;
      }
      owners = __ballot_sync(0xffffffffu, own);
    }
    if (owners == 0) return false;
    lo = b0 + __ffs(owners) - 1;
    a = s.starts[lo];
    z = s.starts[lo + 1];
    len = s.lengths[lo];
  }
  const Run r = {a, z - a, len};
  const int64_t k = u - first_unit(a, lo);
  const int64_t slot = ((r.len >> 4) + k) << 4;
  const int64_t first = slot > r.len ? slot : r.len, stop = min(slot + kBlockSlots, static_cast<int64_t>(r.len) + r.count);
  if (first >= stop) return false;
  t = {lo, static_cast<int>(slot), static_cast<int>(first - slot), static_cast<int>(stop - slot), r.first + static_cast<int>(first - r.len),
       slot < r.len};
  return true;
}

// Sixteen bytes of a row: 8 values of bf16 or 4 of fp32, so that a warp's accesses are whole lines of either.
template <typename T>
struct Piece;
template <>
struct Piece<float> {
  static constexpr int kN = 4;
  uint4 a;
  // the largest |x| as bits of fp32; above 0x7f800000 or at it where one is not finite
  __device__ __forceinline__ uint32_t most() const {
    const uint32_t m = 0x7fffffffu;
    return max(max(a.x & m, a.y & m), max(a.z & m, a.w & m));
  }
  __device__ __forceinline__ void bits(uint32_t* w) const { w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w; }
  __device__ __forceinline__ void set(const uint32_t* w) { a = make_uint4(w[0], w[1], w[2], w[3]); }
};
template <>
struct Piece<__nv_bfloat16> {
  static constexpr int kN = 8;
  uint4 a;
  __device__ __forceinline__ uint32_t most() const {
    const uint32_t m = 0x7fff7fffu;
    const uint32_t v = __vmaxu2(__vmaxu2(a.x & m, a.y & m), __vmaxu2(a.z & m, a.w & m));
    return max(v << 16, v & 0xffff0000u);
  }
  __device__ __forceinline__ void bits(uint32_t* w) const {
    const uint32_t v[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) { w[2 * i] = v[i] << 16; w[2 * i + 1] = v[i] & 0xffff0000u; }
  }
  __device__ __forceinline__ void set(const uint32_t* w) {
    a = make_uint4(__byte_perm(w[0], w[1], 0x7632), __byte_perm(w[2], w[3], 0x7632), __byte_perm(w[4], w[5], 0x7632), __byte_perm(w[6], w[7], 0x7632));
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32, sizeof(T) == 4 ? 4 : 6)
append_kernel(const Int8View c, const T* __restrict__ K, int64_t k_stride, const T* __restrict__ V, int64_t v_stride, const Step step) {
  constexpr int kN = Piece<T>::kN, kLanes = D / kN, kAt = 32 / kLanes, kIt = kBlockSlots / kAt;   // lanes a row, rows at a time, times
  constexpr int kOld = kBlockSlots * D / 512;                                 // 16-byte pieces of the old codes a lane holds
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int of = static_cast<int>(w & 1), h = static_cast<int>((w >> 1) % c.H);
  const int64_t u = (w >> 1) / c.H;
  if (u >= units_of(step)) return;
  Unit t;
  if (!unit_of(step, static_cast<int>(u), lane, t)) return;

  const int col = lane % kLanes * kN, sub = lane / kLanes;
  const int64_t stride = of ? v_stride : k_stride;
  const T* x = (of ? V : K) + t.token * stride + static_cast<int64_t>(h) * D + col;
  Piece<T> in[kIt];
#pragma unroll
  for (int i = 0; i < kIt; ++i) {
    const int r = i * kAt + sub;
    in[i].a = r >= t.rows0 && r < t.rows1 ? __ldg(reinterpret_cast<const uint4*>(x + (r - t.rows0) * stride)) : make_uint4(0u, 0u, 0u, 0u);
  }
  const int pg = c.page(t.b, t.slot);
  if (pg < 0) return;
  const size_t row = c.row(pg, h, t.slot);
  uint8_t* to = (of ? c.vc : c.kc) + row * D;
  int8_t* ex = c.ex + row / kBlockSlots * 2 + of;
  uint4 was[kOld];
  int e_old = kExpLow;
  if (t.old) {
    e_old = min(static_cast<int>(*ex), kExpHigh);
#pragma unroll
    for (int i = 0; i < kOld; ++i)
      if ((i * 512 + lane * 16) / D < t.rows0) was[i] = *reinterpret_cast<const uint4*>(to + i * 512 + lane * 16);
  }

  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < kIt; ++i) most = max(most, in[i].most());
  most = __reduce_max_sync(0xffffffffu, most);
  const bool odd = most >= 0x7f800000u;      // an infinity or NaN: the exponent goes by the finite values
  if (odd) {
    most = 0;
#pragma unroll
    for (int i = 0; i < kIt; ++i) {
      uint32_t b[kN];
      in[i].bits(b);
#pragma unroll
      for (int k = 0; k < kN; ++k)
        if ((b[k] & 0x7fffffffu) < 0x7f800000u) most = max(most, b[k] & 0x7fffffffu);
    }
    most = __reduce_max_sync(0xffffffffu, most);
  }
  int e = min(max(static_cast<int>(most >> 23) - 133, kExpLow), kExpHigh);   // 2^(e + 6) <= most < 2^(e + 7)
  if (t.old) e = max(e, e_old);
  if (odd) {
    // infinity takes the highest code, minus infinity and NaN the lowest (both whole numbers times 2^e, exact in bf16)
#pragma unroll
    for (int i = 0; i < kIt; ++i) {
      uint32_t b[kN];
      in[i].bits(b);
#pragma unroll
      for (int k = 0; k < kN; ++k)
        if ((b[k] & 0x7fffffffu) >= 0x7f800000u) b[k] = __float_as_uint((b[k] == 0x7f800000u ? 127.0f : -128.0f) * pow2(e));
      in[i].set(b);
    }
  }

  if (t.old && e > e_old) {
    // bytes: ((u - 128) >> s) + 128 = (u >> s) + 128 - (128 >> s); beyond 7 every code is next to the middle, as at 7
    const int s = min(e - e_old, 7);
    const uint32_t mask = (0xffu >> s) * 0x01010101u, add = (128u - (128u >> s)) * 0x01010101u;
#pragma unroll
    for (int i = 0; i < kOld; ++i)
      if ((i * 512 + lane * 16) / D < t.rows0) {
        const uint4 v = was[i];
        *reinterpret_cast<uint4*>(to + i * 512 + lane * 16) = make_uint4((v.x >> s & mask) + add, (v.y >> s & mask) + add,
                                                                         (v.z >> s & mask) + add, (v.w >> s & mask) + add);
      }
  }

  // x * 2^-e, rounded down to a whole number by an addition at 1.5 * 2^23: its low byte is the code
  const float scale = pow2(-e);
#pragma unroll
  for (int i = 0; i < kIt; ++i) {
    const int r = i * kAt + sub;
    uint32_t b[kN];
    in[i].bits(b);
#pragma unroll
    for (int k = 0; k < kN; ++k) b[k] = __float_as_uint(__fmaf_rd(__uint_as_float(b[k]), scale, 12582912.0f + 128.0f));
    uint32_t o[kN / 4];
#pragma unroll
    for (int k = 0; k < kN / 4; ++k)
      o[k] = __byte_perm(__byte_perm(b[4 * k], b[4 * k + 1], 0x0040), __byte_perm(b[4 * k + 2], b[4 * k + 3], 0x0040), 0x5410);
    if (r >= t.rows0 && r < t.rows1) {
      if constexpr (kN == 8) *reinterpret_cast<uint2*>(to + r * D + col) = make_uint2(o[0], o[1]);
      else *reinterpret_cast<uint32_t*>(to + r * D + col) = o[0];
    }
  }
  if (lane == 0) *ex = static_cast<int8_t>(e);
}

__device__ __forceinline__ void put(float* p, const float* f) { *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]); }
__device__ __forceinline__ void put(__nv_bfloat16* p, const float* f) {      // exact: the upper halves
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __byte_perm(__float_as_uint(f[2 * i]), __float_as_uint(f[2 * i + 1]), 0x7632);
  *reinterpret_cast<uint4*>(p) = make_uint4(v[0], v[1], v[2], v[3]);
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32)
read_kernel(const Int8View c, T* __restrict__ K, T* __restrict__ V, const Step step) {
  constexpr int kN = Piece<T>::kN, kLanes = D / kN, kAt = 32 / kLanes, kIt = kBlockSlots / kAt;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int of = static_cast<int>(w & 1), h = static_cast<int>((w >> 1) % c.H);
  const int64_t u = (w >> 1) / c.H;
  if (u >= units_of(step)) return;
  Unit t;
  if (!unit_of(step, static_cast<int>(u), lane, t)) return;

  const int col = lane % kLanes * kN, sub = lane / kLanes;
  const int pg = c.page(t.b, t.slot);
  uint32_t in[kIt][kN / 4];
  int e = 0;
  if (pg >= 0) {
    const size_t row = c.row(pg, h, t.slot);
    const uint8_t* from = (of ? c.vc : c.kc) + row * D + col;
    e = c.ex[row / kBlockSlots * 2 + of];
#pragma unroll
    for (int i = 0; i < kIt; ++i) {
      const int r = i * kAt + sub;
      if (r >= t.rows0 && r < t.rows1) {
        if constexpr (kN == 8) {
          const uint2 v = *reinterpret_cast<const uint2*>(from + r * D);
          in[i][0] = v.x;
          in[i][1] = v.y;
        } else {
          in[i][0] = *reinterpret_cast<const uint32_t*>(from + r * D);
        }
      }
    }
  }
  // an exponent outside the range that is written has no power of two in fp32's normal numbers: cut to it
  const float scale = pg >= 0 ? pow2(min(max(e, kExpLow), kExpHigh)) : 0.0f;
  T* out = (of ? V : K) + (static_cast<int64_t>(t.token) * c.H + h) * D + col;
  const int64_t stride = static_cast<int64_t>(c.H) * D;
#pragma unroll
  for (int i = 0; i < kIt; ++i) {
    const int r = i * kAt + sub;
    if (r >= t.rows0 && r < t.rows1) {
      float f[kN];
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        // the byte below 2^23 is a whole number; u * 2^e - 127.5 * 2^e has one rounding, and none is needed
        const float whole = __uint_as_float(__byte_perm(in[i][k / 4], 0x4b000000u, 0x7550 + (k & 3))) - 8388608.0f;
        f[k] = pg >= 0 ? fmaf(whole, scale, -127.5f * scale) : 0.0f;
      }
      put(out + (r - t.rows0) * stride, f);
    }
  }
}

template <typename T>
cudaError_t append(const Int8View& v, int D, const void* K, int64_t ks, const void* V, int64_t vs, const Step& s, cudaStream_t st) {
  const unsigned blocks = static_cast<unsigned>((units_of(s) * v.H * 2 + kWarps - 1) / kWarps);
  const T* k = static_cast<const T*>(K);
  const T* x = static_cast<const T*>(V);
  if (D == 64) append_kernel<T, 64><<<blocks, kWarps * 32, 0, st>>>(v, k, ks, x, vs, s);
  else append_kernel<T, 128><<<blocks, kWarps * 32, 0, st>>>(v, k, ks, x, vs, s);
  return cudaGetLastError();
}

template <typename T>
cudaError_t read(const Int8View& v, int D, void* K, void* V, const Step& s, cudaStream_t st) {
  const unsigned blocks = static_cast<unsigned>((units_of(s) * v.H * 2 + kWarps - 1) / kWarps);
  if (D == 64) read_kernel<T, 64><<<blocks, kWarps * 32, 0, st>>>(v, static_cast<T*>(K), static_cast<T*>(V), s);
  else read_kernel<T, 128><<<blocks, kWarps * 32, 0, st>>>(v, static_cast<T*>(K), static_cast<T*>(V), s);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append_int8(const tq_int8_cache& c, const void* K, int64_t k_stride, const void* V,
                               int64_t v_stride, tq_qtype type, const Step& step, const int* table, int max_pages,
                               cudaStream_t st) {
  const Int8View v = int8_view(c, table, max_pages);
  return type == TQ_Q_F32 ? append<float>(v, c.D, K, k_stride, V, v_stride, step, st)
                          : append<__nv_bfloat16>(v, c.D, K, k_stride, V, v_stride, step, st);
}

cudaError_t launch_read_int8(const tq_int8_cache& c, void* K, void* V, tq_qtype type, const Step& step,
                             const int* table, int max_pages, cudaStream_t st) {
  const Int8View v = int8_view(c, table, max_pages);
  return type == TQ_Q_F32 ? read<float>(v, c.D, K, V, step, st) : read<__nv_bfloat16>(v, c.D, K, V, step, st);
}

cudaError_t take_faults_int8_rows(unsigned int* bits) { return take_unit_faults(bits); }

}  // namespace tq
