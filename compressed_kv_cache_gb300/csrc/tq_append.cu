// The write side of the paged cache (tq_append_paged): rotate, search the midpoints, pack
// the codes and write the row to its slot.
//
// A tile is 128 rows of one KV head's keys or values against N rows of its rotation: a
// 128 x N x 128 product on the tensor cores (tcgen05, fp32 sums in tensor memory).  Both sides
// are fp16 pairs hi + lo (22 bits; a bf16 row, scaled by a power of two, needs no lo), and
// hi hi + hi lo + lo hi are summed.  Tensor memory hands each thread one row, so it
// searches and packs its coordinates in registers.
//
// The codes are those of a 64-bit product: a coordinate within kNear of a midpoint (in units of
// the row's length) is summed again in 64 bits from the inputs.  kNear = 5e-6 covers, in that
// unit: the operands' 2^-21; the up to 24 fp32 sums of 16 products, each of which is at most the
// row's length and is off by at most 2^-23 of it even where bits are cut off instead of rounded
// (2.9e-6 together); the fp32 length (8e-7, a coordinate being at most 1) and the scaling by it:
// 4.4e-6.  Where the tensor core cuts is not documented, so it was measured: without the second
// sums the farthest coordinate from a midpoint with another code than in 64 bits was 7e-7 away
// (rows that are one, two or five rows of the rotation, whose products all point one way; 1.3e-7
// for random rows).  The window meets about 1 coordinate in 4000 (3 bits).
//
// N is 128 (the rotation of a head stays in shared memory from tile to tile) or, where that
// leaves SMs without a tile, 32: a decode step of 64 tokens then runs on four times the SMs.
//
// Bound: latency and issue, not yet memory.  8192 tokens x 8 heads, bf16, 3-bit codes: 44 us, of
// which 5 are set-up (tensor memory, the rotation's fp16 form) and about 5 a tile (7 tiles an SM):
// rows to fp16 0.8, the search of the cells 2 to 3, waits on the slowest warp and on the product
// the rest; 0.94 TB/s of the rows' and codes' bytes.  15003 fp32 rows x 8 heads, 4-bit codes: 95
// us, 1.48 TB/s.  Measured on the way there (8192 tokens): everything in 64 bits 13.5 ms; near
// coordinates listed and summed again in 64 bits 75 us (a 64-bit instruction takes a warp 16
// cycles); in pairs of fp32 50 us; binary search of the midpoints instead of the cells 52 us;
// rows prefetched in registers 53 us (they spill); two CTAs of 8 warps an SM 52 us; a barrier
// a tile instead of the product's own warp 49 us; four copies of a cell instead of sixteen 47 us,
// of which the second sums took 9 and the search 7.
#include "tq_paged.cuh"

namespace tq {
namespace {

constexpr int kRows = 128;             // rows of a tile
constexpr int kCells = 128;            // cells of the search table
constexpr int kCopies = 16;            // of each, one for every lane that a load serves at a time
constexpr float kNear = 5e-6f;
constexpr float kLength = 8e-7f;       // an fp32 length is off by less: 19 roundings of its square (half of 19 x 2^-24), two of its own

__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));   // the table stays as it is while its readers run
  return v;
}
__device__ __forceinline__ uint32_t smem_u32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

// Shared-memory matrix descriptor, K-major, no swizzle: core matrices of 8 rows x 16 bytes,
// `lbo` bytes between neighbours along K, 128 between neighbours along the rows.
__device__ __forceinline__ uint64_t operand(uint32_t saddr, uint32_t lbo) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>(128 >> 4) << 32) | (1ull << 46);
}
// fp16 operands, fp32 sums
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t N, bool add) {
  const uint32_t idesc = (1u << 4) | ((N >> 3) << 17) | ((kRows >> 4) << 24);
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
      "r"(static_cast<uint32_t>(add))
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float half_round(float x) { return __half2float(__float2half_rn(x)); }

// Eight values, and the 16-byte chunk of their hi (or lo) parts.
__device__ __forceinline__ uint4 hi_chunk(const float (&x)[8]) {
  return make_uint4(pack_h2(x[0], x[1]), pack_h2(x[2], x[3]), pack_h2(x[4], x[5]), pack_h2(x[6], x[7]));
}
__device__ __forceinline__ uint4 lo_chunk(const float (&x)[8]) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = x[i] - half_round(x[i]);
  return hi_chunk(y);
}
__device__ __forceinline__ void widen(const uint4 (&v)[1], float (&x)[8]) {   // 8 bf16
  const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void widen(const uint4 (&v)[2], float (&x)[8]) {   // 8 fp32
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[4 * i] = __uint_as_float(v[i].x);
    x[4 * i + 1] = __uint_as_float(v[i].y);
    x[4 * i + 2] = __uint_as_float(v[i].z);
    x[4 * i + 3] = __uint_as_float(v[i].w);
  }
}

struct AppendArgs {
  Paged pg;
  const void* X[2];          // keys, values [n, H, 128]
  const float* Pi[2];
  const float* cb[2];
  const int* rows;
  float* mass;
  int* positions;
  int n, B, rot, S, cap, N, tiles, bits[2];
  uint32_t step;             // bytes from cell to cell
  int items;                 // (head, keys or values, part of the rotation, tile)
};

// Search table: the midpoints' range in cells, each with the midpoint k nearest to it; the code
// of a v in the cell is k + (v > midpoint k).  The cells are a 62nd of the range or less
// apart from every other midpoint (or the table is not used: count16), so that no v has
// another midpoint nearer by.  A v at the edge of a cell may be as near as half a cell to the
// next midpoint unseen: a cell is 2 kNear or wider.  The cell of v is a saturating FMA and a
// rounding.
struct Cell {
  float mid;
  int above;       // k + 1
};
struct Grid {
  float scale, shift;                                      // v * scale + shift in [0, 1] over the cells
  int ok;
};

__device__ __forceinline__ float cell_u(float y, float scale, float shift) {   // 2^23 + cell
  return fmaf(__saturatef(fmaf(y, scale, shift)), static_cast<float>(kCells - 1), 8388608.f);
}

// One warp: the grid of n ascending midpoints.
__device__ __forceinline__ Grid make_grid(const float* mids, int n, int lane) {
  const float lo = mids[0], hi = mids[n - 1], w = (hi - lo) / static_cast<float>(kCells - 4);
  const bool close = lane + 1 < n && !(mids[min(lane + 1, n - 1)] - mids[min(lane, n - 1)] >= 2.f * w);
  Grid g;
  g.ok = !__any_sync(0xffffffffu, close) && w >= 2.f * kNear && w < 1e30f;
  g.scale = 1.f / (w * static_cast<float>(kCells - 1));
  g.shift = (1.5f * w - lo) * g.scale;
  return g;
}
// Entry i, by the cell's centre.
__device__ __forceinline__ Cell make_cell(const float* mids, int n, const Grid& g, int i) {
  const float c = (static_cast<float>(i) / static_cast<float>(kCells - 1) - g.shift) / g.scale;
  int k = 0;
  for (int j = 1; j < n; ++j)
    if (fabsf(mids[j] - c) < fabsf(mids[k] - c)) k = j;
  return {mids[k], k + 1};
}

// 16 coordinates from J of 32 where the grid does not serve: every midpoint in turn.
template <int BITS, int J>
__device__ __forceinline__ void count16(const float (&y)[16], float inv, const float* mids, uint32_t (&w)[BITS], uint32_t& mask) {
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float v = y[j] * inv;
    uint32_t code = 0;
    float least = 1.f;
#pragma unroll 1
    for (int i = 0; i + 1 < (1 << BITS); ++i) {
      const float d = v - mids[i];
      code += d > 0.f ? 1u : 0u;
      least = fminf(least, fabsf(d));
    }
    if (least < kNear) mask |= 1u << (J + j);
    const int bit = BITS * (J + j);
    w[bit / 32] += code << (bit % 32);
    if (bit % 32 + BITS > 32) w[bit / 32 + 1] += code >> (32 - bit % 32);
  }
}

// Coordinates J .. J + 15 of 32 (J 0 or 16): packed codes to w, near ones to the mask.  at:
// what takes the bits of cell_u to the address of the lane's copy.
template <int BITS, int J>
__device__ __forceinline__ void look_up16(const float (&y)[16], float inv, float scale, float shift, uint32_t at, uint32_t step,
                                          uint32_t (&w)[BITS], uint32_t& mask) {
  float least = 1.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const uint2 e = lds64(__float_as_uint(cell_u(y[j], scale, shift)) * step + at);
    const float d = fmaf(y[j], inv, -__uint_as_float(e.x));
    const uint32_t code = e.y + static_cast<uint32_t>(static_cast<int>(__float_as_uint(d)) >> 31);
    least = fminf(least, fabsf(d));
    const int bit = BITS * (J + j);
    w[bit / 32] += code << (bit % 32);
    if (bit % 32 + BITS > 32) w[bit / 32 + 1] += code >> (32 - bit % 32);
  }
  if (least < kNear) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const uint2 e = lds64(__float_as_uint(cell_u(y[j], scale, shift)) * step + at);
      if (fabsf(fmaf(y[j], inv, -__uint_as_float(e.x))) < kNear) mask |= 1u << (J + j);
    }
  }
}

// s + x rounded to s; returns the rounding error, exactly.
__device__ __forceinline__ float add_exact(float& s, float x) {
  const float t = s + x, b = t - s;
  const float e = (s - (t - b)) + (x - b);
  s = t;
  return e;
}

// What the threads of a tile know of its rows.
struct RowInfo {
  float inv;         // 1 / (length * scales): turns a sum into a unit coordinate; 0 where there is none
  float scale;       // the power of two that takes the row to 2^7 (in two factors for tiny rows)
  int kind;          // 0: no row, 1: an ordinary one, 2: zero, 3: NaN or infinity within
  float norm;        // length, to kLength
  int tiny;          // the other factor is 2^64
  int code;          // kinds 2 and 3: the code of every coordinate
  long long at;      // row on the cache's planes
};

// The code of coordinate c of a row, as 64 bits decide it.  Eight lanes (j = 0 .. 7) with 16
// coordinates each: sums of products as pairs of fp32 (each product and each addition with its
// rounding error, 2^-45 of the row's length); where they cannot tell (an exact tie, say), the
// sums in 64 bits.  P, x: the rows, widened on the way.
template <typename T, int BITS>
__device__ __forceinline__ uint32_t exact_cell(const float* P, const T* x, const RowInfo& ri, const float* cb, const float* mids, bool live, int j) {
  const float s0 = ri.tiny ? 18446744073709551616.f : 1.f, s1 = ri.scale;
  float s = 0.f, se = 0.f, q = 0.f, qe = 0.f;
  if (live) {
    const float4* P4 = reinterpret_cast<const float4*>(P + 16 * j);
    const uint4* x4 = reinterpret_cast<const uint4*>(x + 16 * j);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint4 raw[sizeof(T) / 2];
#pragma unroll
      for (int v = 0; v < static_cast<int>(sizeof(T) / 2); ++v) raw[v] = __ldg(x4 + k * (sizeof(T) / 2) + v);
      float xv[8];
      widen(raw, xv);
      const float4 u = __ldg(P4 + 2 * k), v = __ldg(P4 + 2 * k + 1);
      const float pv[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xs = xv[i] * s0 * s1;
        const float d = __fmul_rn(xs, pv[i]), d2 = __fmul_rn(xs, xs);   // never fused with the additions
        se += fmaf(xs, pv[i], -d) + add_exact(s, d);
        qe += fmaf(xs, xs, -d2) + add_exact(q, d2);
      }
    }
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    const float so = __shfl_xor_sync(0xffffffffu, s, o), qo = __shfl_xor_sync(0xffffffffu, q, o);
    const float seo = __shfl_xor_sync(0xffffffffu, se, o), qeo = __shfl_xor_sync(0xffffffffu, qe, o);
    se += seo + add_exact(s, so);
    qe += qeo + add_exact(q, qo);
  }
  uint32_t code = 0;
  if (live && j == 0) {
    const float len = sqrtf(q);                            // len + le: the length to 2^-45
    const float le = (fmaf(-len, len, q) + qe) / (2.f * len);
    const float y = s / len;
    for (int i = 0; i + 1 < (1 << BITS); ++i) {
      bool above = y > mids[i];
      if (fabsf(y - mids[i]) < 4.f * kNear) {
        float mid = 0.5f * cb[i];                          // mid + me, exactly
        const float me = add_exact(mid, 0.5f * cb[i + 1]);
        const float at = __fmul_rn(mid, len);
        const float ae = fmaf(mid, len, -at) + fmaf(mid, le, me * len);
        const float diff = (s - at) + (se - ae);           // s - at is exact so near the midpoint
        if (fabsf(diff) > 1e-11f * len) {
          above = diff > 0.f;
        } else {
          const double sc = static_cast<double>(s1) * static_cast<double>(s0);
          double q64 = 0.0, s64 = 0.0;
          for (int k = 0; k < kPD; ++k) {
            const double xv = static_cast<double>(static_cast<float>(x[k])) * sc;
            s64 += xv * static_cast<double>(P[k]);
            q64 += xv * xv;
          }
          above = s64 > 0.5 * (static_cast<double>(cb[i]) + static_cast<double>(cb[i + 1])) * sqrt(q64);
        }
      }
      code += above ? 1u : 0u;
    }
  }
  return code;
}

// The code of a near coordinate, eight lanes for it: its sum to 2^-24 of the row's length
// against the fp32 length (within 2^-20), which settles all but a quarter of them, and
// exact_cell for those.  All 32 lanes come here.
template <typename T, int BITS>
__device__ __forceinline__ uint32_t near_cell(const float* P, const T* x, const RowInfo& ri, const float* cb, const float* mids, bool live, int j) {
  constexpr float kSure = 1.f / 524288.f;
  const float s0 = ri.tiny ? 18446744073709551616.f : 1.f, s1 = ri.scale;
  float s = 0.f, se = 0.f;
  if (live) {
    const float4* P4 = reinterpret_cast<const float4*>(P + 16 * j);
    const uint4* x4 = reinterpret_cast<const uint4*>(x + 16 * j);
    uint4 raw[2][sizeof(T) / 2];
    float4 u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) u[k] = __ldg(P4 + k);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int v = 0; v < static_cast<int>(sizeof(T) / 2); ++v) raw[k][v] = __ldg(x4 + k * (sizeof(T) / 2) + v);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float xv[8];
      widen(raw[k], xv);
      const float pv[8] = {u[2 * k].x, u[2 * k].y, u[2 * k].z, u[2 * k].w, u[2 * k + 1].x, u[2 * k + 1].y, u[2 * k + 1].z, u[2 * k + 1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xs = xv[i] * s0 * s1;
        const float d = __fmul_rn(xs, pv[i]);
        se += fmaf(xs, pv[i], -d) + add_exact(s, d);
      }
    }
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    const float so = __shfl_xor_sync(0xffffffffu, s, o), seo = __shfl_xor_sync(0xffffffffu, se, o);
    se += seo + add_exact(s, so);
  }
  const float y = (s + se) * (128.f * ri.inv);
  uint32_t code = 0;
  float least = 1.f;
#pragma unroll
  for (int i = 0; i + 1 < (1 << BITS); ++i) {
    const float d = y - mids[i];
    code += d > 0.f ? 1u : 0u;
    least = fminf(least, fabsf(d));
  }
  // one answer for the eight: their sums may differ in the last bit (all lanes shuffle)
  const float lead = __shfl_sync(0xffffffffu, least, threadIdx.x & 24);
  const bool open = live && lead < kSure;
  if (__any_sync(0xffffffffu, open)) {
    const uint32_t exact = exact_cell<T, BITS>(P, x, ri, cb, mids, open, j);
    if (open) code = exact;                                // lane 0 of the eight has it
  }
  return code;
}

// The length of a row, as fp16, of which `below` or the next number is the nearest: the sum of
// squares as a pair of fp32 against the square of the middle (12 bits, so the square is exact; the
// even one on it).  The whole warp, four coordinates a lane.  A row in 300 to 600 comes here; inlined
// it cost prompts 1 to 2 us, in the warps that make operands 1.5 (bf16) and 14 (fp32).
template <typename T>
__device__ __noinline__ uint32_t nearest_length(const T* x, float scale, uint32_t below, int lane) {
  float v[4], q = 0.f, e = 0.f;
  if constexpr (sizeof(T) == 4) {
    const float4 u = __ldg(reinterpret_cast<const float4*>(x) + lane);
    v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
  } else {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(x) + lane);
    v[0] = __uint_as_float(u.x << 16); v[1] = __uint_as_float(u.x & 0xffff0000u);
    v[2] = __uint_as_float(u.y << 16); v[3] = __uint_as_float(u.y & 0xffff0000u);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float z = v[i] * scale, z2 = __fmul_rn(z, z);
    e += fmaf(z, z, -z2) + add_exact(q, z2);
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float qo = __shfl_xor_sync(0xffffffffu, q, o), eo = __shfl_xor_sync(0xffffffffu, e, o);
    e += eo + add_exact(q, qo);
  }
  // behind the largest number comes 65536
  const float next = below == 0x7bffu ? 65536.f : __half2float(__ushort_as_half(static_cast<uint16_t>(below + 1)));
  const float mid = 0.5f * (__half2float(__ushort_as_half(static_cast<uint16_t>(below))) + next) * scale;
  const float diff = (q - __fmul_rn(mid, mid)) + e;
  return diff > 0.f || (diff == 0.f && (below & 1)) ? below + 1 : below;
}

// A warp's share of a tile: 32 rows, 32 coordinates each (where N is 32, on the first four
// warps), from tensor memory to the planes.
template <typename T, int BITS>
__device__ __forceinline__ void search_tile(const AppendArgs& a, int kv, int h, int part, int tile, uint32_t tmem,
                                            const RowInfo* info, const float* mids, const Grid* grid, uint32_t cells) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool whole = a.N == kPD;
  if (!whole && warp >= 4) return;
  const Grid g = *grid;
  const uint32_t step = a.step, at = cells + (lane & (kCopies - 1)) * 8 - 0x4b000000u * step;
  const int r0 = 32 * (warp & 3), r = r0 + lane;
  RowInfo ri = info[r];
  if (ri.at < 0) ri.kind = 0;
  const T* X = static_cast<const T*>(a.X[kv]);
  const float* P = a.Pi[kv] + (static_cast<size_t>(h % a.rot) * kPD + part * a.N) * kPD;
  uint32_t* dst = reinterpret_cast<uint32_t*>((kv ? a.pg.vp : a.pg.kp) + ri.at * (16 * BITS)) + part * (whole ? 0 : BITS);
  const int c0 = whole ? warp >> 2 : 0;
  uint32_t w[BITS], mask = 0;
#pragma unroll
  for (int i = 0; i < BITS; ++i) w[i] = 0;
  {
    const uint32_t from = tmem + (static_cast<uint32_t>(r0) << 16) + 32 * c0;
    float y[16];
    if (g.ok) {
      const float scale = ri.inv * g.scale;
      tmem_ld16(from, y);
      look_up16<BITS, 0>(y, ri.inv, scale, g.shift, at, step, w, mask);
      tmem_ld16(from + 16, y);
      look_up16<BITS, 16>(y, ri.inv, scale, g.shift, at, step, w, mask);
    } else {
      tmem_ld16(from, y);
      count16<BITS, 0>(y, ri.inv, mids, w, mask);
      tmem_ld16(from + 16, y);
      count16<BITS, 16>(y, ri.inv, mids, w, mask);
    }
  }
  if (ri.kind != 1) {
    mask = 0;
#pragma unroll
    for (int i = 0; i < BITS; ++i) {                       // one code throughout
      uint32_t x = 0;
      for (int j = 0; j < 32; ++j) x |= ((static_cast<uint32_t>(ri.code) >> ((32 * i + j) % BITS)) & 1u) << j;
      w[i] = x;
    }
  }
  // near coordinates, four lanes' at a time
  for (uint32_t waiting = __ballot_sync(0xffffffffu, mask != 0); waiting != 0; waiting = __ballot_sync(0xffffffffu, mask != 0)) {
    uint32_t left = waiting;
    for (int k = 0; k < (lane >> 3); ++k) left &= left - 1;
    const bool live = left != 0;
    const int owner = live ? __ffs(left) - 1 : 0;
    const int mine = __ffs(mask) - 1;
    const int at = __shfl_sync(0xffffffffu, mine, owner);
    const uint32_t code = near_cell<T, BITS>(P + (32 * c0 + (live ? at : 0)) * kPD,
                                              X + (static_cast<size_t>(tile * kRows + r0 + owner) * a.pg.H + h) * kPD,
                                              info[r0 + owner], a.cb[kv], mids, live, lane & 7);
    const int rank = __popc(waiting & ((1u << lane) - 1));
    const uint32_t exact = __shfl_sync(0xffffffffu, code, 8 * (rank & 3));
    if (mask != 0 && rank < 4) {
      mask &= mask - 1;
      constexpr uint32_t ones = (1u << BITS) - 1;
#pragma unroll
      for (int i = 0; i < BITS; ++i) {
        const int sh = BITS * mine - 32 * i;               // where the code begins in this word
        if (sh > -BITS && sh < 32) {
          const uint32_t on = sh >= 0 ? ones << sh : ones >> -sh, v = sh >= 0 ? exact << sh : exact >> -sh;
          w[i] = (w[i] & ~on) | v;
        }
      }
    }
  }
  if (ri.kind != 0) {
    uint32_t* o = dst + BITS * c0;
    if constexpr (BITS == 4) {
      *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
    } else if constexpr (BITS == 2) {
      *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < BITS; ++i) o[i] = w[i];
    }
  }
  {                                                        // lengths: each warp (or part) those of 8 of the rows
    const bool mine = ri.kind != 0 && (lane >> 3) == (whole ? c0 : part);
    const uint32_t below = __half_as_ushort(__float2half_rn(ri.norm * (1.f - kLength)));
    uint32_t norm = __half_as_ushort(__float2half_rn(ri.norm * (1.f + kLength)));   // another number: the next
    for (uint32_t left = __ballot_sync(0xffffffffu, mine && ri.kind == 1 && below != norm); left != 0; left &= left - 1) {
      const int owner = __ffs(left) - 1;
      const uint32_t near = nearest_length(X + (static_cast<size_t>(tile * kRows + r0 + owner) * a.pg.H + h) * kPD, info[r0 + owner].scale,
                                           __shfl_sync(0xffffffffu, below, owner), lane);
      if (lane == owner) norm = near;
    }
    if (mine) (kv ? a.pg.vn : a.pg.kn)[ri.at] = static_cast<uint16_t>(norm);
  }
}

constexpr int kWorkers = 512;          // 16 warps that make operands and search, and one more:
constexpr int kThreads = 544;          // it issues the products

template <typename T>
constexpr int append_smem(int N) {
  return kRows * 256 * (sizeof(T) == 4 ? 2 : 1) + kRows * kPD * static_cast<int>(sizeof(T)) + N * 256 * 2 + 3 * kRows * static_cast<int>(sizeof(RowInfo)) +
         kCells * kCopies * 8 + 64 + 64;
}

// Where a CTA is among the items: tile by tile, then the next part of a rotation.
struct Place {
  int item, tile, hkp;
  __device__ __forceinline__ void next(int tiles) {
    ++item;
    if (++tile == tiles) {
      tile = 0;
      ++hkp;
    }
  }
};

// One CTA of 16 + 1 warps an SM.  While a tile is searched, the product of the next one runs and
// the rows of the one behind it are on their way to shared memory (each thread's own places:
// registers would not hold them through the search; one bulk copy a row measured slower).  The
// warps meet only where the last warp waits for an operand to be whole, so one that has
// near coordinates to settle holds the others up a tile later, if at all.
template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr bool XLO = sizeof(T) == 4;                     // rows need a lo part
  constexpr int V = sizeof(T) / 2;                         // 16-byte loads of 8 values
  constexpr int kA = kRows * 256 * (XLO ? 2 : 1);          // operand of a tile: hi, then lo
  extern __shared__ __align__(128) char smem[];
  const int N = a.N;
  char* sA = smem;
  char* sB = sA + kA;                                      // hi, then lo of the rotation
  char* sRaw = sB + N * 512;                               // rows as they come
  RowInfo* infos = reinterpret_cast<RowInfo*>(sRaw + kRows * kPD * sizeof(T));   // of three tiles: a warp may still search the one before
  Cell* cells = reinterpret_cast<Cell*>(infos + 3 * kRows);
  float* mids = reinterpret_cast<float*>(cells + kCells * kCopies);
  uint64_t* bars = reinterpret_cast<uint64_t*>(mids + 16);
  uint32_t* slot = reinterpret_cast<uint32_t*>(bars + 3);
  Grid* grid = reinterpret_cast<Grid*>(slot + 1);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  const bool whole = N == kPD;
  const int per = a.items / gridDim.x, more = a.items - per * gridDim.x;
  const int cta = blockIdx.x;
  const int first = cta * per + min(cta, more), last = first + per + (cta < more ? 1 : 0);
  auto part_of = [&](int hkp) { return whole ? 0 : hkp & 3; };
  auto hk_of = [&](int hkp) { return whole ? hkp : hkp >> 2; };

  const uint32_t done = smem_u32(bars), whole_op = smem_u32(bars + 2);
  const bool worker = warp < kWorkers / 32;
  int seq = -1, slt = -1, pos = 0, page = -1;
  // A worker's share of a tile's rows, to places of its own.  Lane 8g + j of warp w takes chunks
  // g, g + 4, g + 8, g + 12 (eight values) of row 8w + j.
  const uint32_t mine = smem_u32(sRaw) + tid * 16;
  auto request = [&](const Place& p) {
    const int hk = hk_of(p.hkp), i = p.tile * kRows + 8 * warp + (lane & 7);
    const int bytes = i < a.n ? 16 : 0;                    // zeros behind the last row
    const T* src = static_cast<const T*>(a.X[hk & 1]);
    if (i < a.n) src += (static_cast<size_t>(i) * a.pg.H + (hk >> 1)) * kPD + 8 * (lane >> 3);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(mine + (k * V + v) * (kWorkers * 16)),
                     "l"(reinterpret_cast<const uint4*>(src + 32 * k) + v), "r"(bytes)
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // Where a tile's rows go, asked for a tile ahead.
  auto places = [&](const Place& p) {
    const int j = p.tile * kRows + tid;
    seq = -1;
    if (tid < kRows && j < a.n) {
      const int* r = a.rows + 3 * static_cast<size_t>(j);
      seq = r[0];
      slt = r[1];
      pos = r[2];
    }
  };
  auto find_page = [&]() {
    const bool in = seq >= 0 && slt >= 0 && seq < a.B && slt < a.cap;
    page = in ? a.pg.table[static_cast<size_t>(seq) * a.pg.max_pages + (slt >> a.pg.shift)] : -1;
  };

  Place ahead = {first, first % a.tiles, first / a.tiles};   // the tile whose loads are under way
  if (tid == 0) {
    const int counts[3] = {1, 1, kWorkers / 32};
#pragma unroll
    for (int i = 0; i < 3; ++i)
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bars + i)), "r"(counts[i]) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (first < last && worker) {
    request(ahead);
    places(ahead);
    find_page();
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(2 * N) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *slot;

  // A warp whose wait ran out makes no operand and announces none, issues no product and writes
  // nothing more.  The others' waits for what it leaves out then run out as well, so that no warp
  // searches a product whose operand may not have been whole.
  bool lost = false;
  auto wait = [&](uint32_t bar, int n) {                   // for the bar's n-th use, from 0
    if (!lost) lost = __any_sync(0xffffffffu, !wait_parity_bounded(bar, n & 1, kFaultPagedWait));
  };

  // Rows part * N .. of a head's rotation, times 2^7, and its codebook's midpoints.  Every warp is
  // past the products and the search of the tiles before.
  auto load_rotation = [&](int hkp) {
    if (!worker) {
      __syncthreads();
      return;
    }
    const int hk = hk_of(hkp), kv = hk & 1, h = hk >> 1;
    const float* P = a.Pi[kv] + (static_cast<size_t>(h % a.rot) * kPD + part_of(hkp) * N) * kPD;
#pragma unroll 4
    for (int e = tid; e < N * 16; e += kWorkers) {
      const int d = (e >> 5) / 4 * 8 + (e & 7), c = (e >> 5) % 4 * 4 + ((e >> 3) & 3);   // as the rows: 8 rows x 4 chunks a warp
      const float4 u = __ldg(reinterpret_cast<const float4*>(P + d * kPD + 8 * c));
      const float4 v = __ldg(reinterpret_cast<const float4*>(P + d * kPD + 8 * c + 4));
      const float x[8] = {128.f * u.x, 128.f * u.y, 128.f * u.z, 128.f * u.w, 128.f * v.x, 128.f * v.y, 128.f * v.z, 128.f * v.w};
      const int at = c * (N * 16) + (d >> 3) * 128 + (d & 7) * 16;
      *reinterpret_cast<uint4*>(sB + at) = hi_chunk(x);
      *reinterpret_cast<uint4*>(sB + N * 256 + at) = lo_chunk(x);
    }
    const int n = (1 << a.bits[kv]) - 1;
    if (tid < n) mids[tid] = 0.5f * (a.cb[kv][tid] + a.cb[kv][tid + 1]);   // within 2^-24: kNear has room
    __syncthreads();
    const Grid g = make_grid(mids, n, lane);
    if (tid == 0) *grid = g;
    constexpr int kShare = kCells * kCopies / kWorkers;    // copies of one cell a thread writes
    if (g.ok) {
      const Cell c = make_cell(mids, n, g, tid * kShare / kCopies);
#pragma unroll
      for (int k = 0; k < kShare; ++k) cells[tid * kShare + k] = c;
    }
  };

  // The last warp: a tile's product, once its operand is whole.
  auto issue_tile = [&]() {
    const int i = ahead.item - first;
    wait(whole_op, i);
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (lane == 0 && !lost) {
      const uint32_t Aa = smem_u32(sA), Bm = smem_u32(sB), d = tmem + (i & 1) * N;
      const uint32_t la = kRows * 16, lb = N * 16;
#pragma unroll
      for (int k = 0; k < 8; ++k) mma_f16(d, operand(Aa + k * 2 * la, la), operand(Bm + k * 2 * lb, lb), N, k != 0);
#pragma unroll
      for (int k = 0; k < 8; ++k) mma_f16(d, operand(Aa + k * 2 * la, la), operand(Bm + N * 256 + k * 2 * lb, lb), N, true);
      if constexpr (XLO) {
#pragma unroll
        for (int k = 0; k < 8; ++k) mma_f16(d, operand(Aa + kRows * 256 + k * 2 * la, la), operand(Bm + k * 2 * lb, lb), N, true);
      }
      asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(done + 8 * (i & 1)) : "memory");
    }
    __syncwarp();
    ahead.next(a.tiles);
  };

  // A worker's rows of the tile that has come, as fp16, where they go, and the next tile's loads.
  auto make_operand = [&]() {
    if (lost) {
      ahead.next(a.tiles);
      return;
    }
    const int hk = hk_of(ahead.hkp), kv = hk & 1, h = hk >> 1;
    RowInfo* info = infos + (ahead.item % 3) * kRows;
    char* A = sA;
    if (tid < kRows) {                                     // where each row goes
      long long at = -1;
      if (seq >= 0 && slt >= 0) {
        if (static_cast<unsigned>(page) < static_cast<unsigned>(a.pg.n_pages)) {
          at = static_cast<long long>(a.pg.row(page, h, slt));
          if (kv == 0 && part_of(ahead.hkp) == 0) {
            const size_t m = (static_cast<size_t>(seq) * a.pg.H + h) * a.S + slt;
            if (a.mass != nullptr) a.mass[m] = 0.f;
            if (a.positions != nullptr) a.positions[m] = pos;
          }
        } else {                                           // a sequence, slot or page out of range
          atomicOr(&g_wait_fault, static_cast<unsigned int>(kFaultPaged));
        }
      }
      info[tid].at = at;
    }
    ahead.next(a.tiles);
    if (ahead.item < last) places(ahead);
    // rows scaled to 2^7
    const int r = 8 * warp + (lane & 7);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    uint32_t top = 0;
    float x[4][8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint4 raw[V];
#pragma unroll
      for (int v = 0; v < V; ++v) raw[v] = *reinterpret_cast<const uint4*>(sRaw + (k * V + v) * (kWorkers * 16) + tid * 16);
      widen(raw, x[k]);
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[k][i]) & 0x7fffffffu);
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 8));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 16));
    const bool finite = top < 0x7f800000u;
    // powers of two: up to 2^64 first for rows that are tiny throughout, then to 2^7
    const float s0 = top < 0x21800000u ? 18446744073709551616.f : 1.f;            // below 2^-60
    const int e = static_cast<int>(__float_as_uint(__uint_as_float(top) * s0) >> 23);   // 1 .. 254 for a row that is neither zero nor infinite
    int k2 = 134 - e;                                                             // -120 .. 126
    k2 = k2 > 126 ? 126 : k2;
    const float s1 = finite && top != 0 ? __uint_as_float(static_cast<uint32_t>(127 + k2) << 23) : 0.f;
    if (s0 != 1.f) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[k][i] *= s0;
    }
    float sums[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float& sum2 = sums[k & 1];                           // two chains: 19 roundings instead of 34
#pragma unroll
      for (int i = 0; i < 8; ++i) {                        // NaN and infinity stay within their row, which takes no codes from it
        x[k][i] *= s1;
        sum2 = fmaf(x[k][i], x[k][i], sum2);
      }
      const int at = ((lane >> 3) + 4 * k) * (kRows * 16) + (r >> 3) * 128 + (r & 7) * 16;
      *reinterpret_cast<uint4*>(A + at) = hi_chunk(x[k]);
      if constexpr (XLO) *reinterpret_cast<uint4*>(A + kRows * 256 + at) = lo_chunk(x[k]);
    }
    float sum = sums[0] + sums[1];
    sum += __shfl_xor_sync(0xffffffffu, sum, 8);
    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
    if (lane < 8) {
      RowInfo& ri = info[r];
      const float len = sqrtf(sum);
      const int kind = !finite ? 3 : top == 0 ? 2 : 1;
      ri.kind = kind;
      ri.scale = s1;
      ri.tiny = s0 != 1.f;
      ri.inv = kind == 1 ? 1.f / (128.f * len) : 0.f;
      // the length, the powers of two taken back
      const float back = __uint_as_float(static_cast<uint32_t>(127 - k2) << 23) * (s0 != 1.f ? 5.42101086e-20f : 1.f);
      const float n = kind == 1 ? len * back : kind == 2 ? 0.f : __uint_as_float(top > 0x7f800000u ? 0x7fc00000u : 0x7f800000u);
      ri.norm = n;
      int zero = 0;
      if (kind == 2)
        for (int i = 0; i + 1 < (1 << a.bits[kv]); ++i) zero += a.cb[kv][i] + a.cb[kv][i + 1] < 0.f ? 1 : 0;   // the sign is exact
      ri.code = zero;
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");   // and this warp's reads of the tile before last
    __syncwarp();
    if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(whole_op) : "memory");
    if (ahead.item < last) {
      request(ahead);
      find_page();
    }
  };

  Place now = ahead;
  int loaded = -1;
  while (now.item < last) {
    if (ahead.item == now.item) {                          // nothing is under way
      if (loaded != now.hkp) {
        __syncthreads();
        load_rotation(now.hkp);
        loaded = now.hkp;
      }
      if (worker) make_operand();
      else issue_tile();
    }
    const int i = now.item - first;
    if (!worker) {
      if (ahead.item < last && ahead.hkp == loaded) issue_tile();
      now.next(a.tiles);
      continue;
    }
    wait(done + 8 * (i & 1), i >> 1);
    // the operand is free again
    if (ahead.item < last && ahead.hkp == loaded) make_operand();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (!lost) {
      const int hk = hk_of(now.hkp), kv = hk & 1, h = hk >> 1, part = part_of(now.hkp);
      const RowInfo* info = infos + (now.item % 3) * kRows;
      const uint32_t d = tmem + (i & 1) * N;
      switch (a.bits[kv]) {
        case 2: search_tile<T, 2>(a, kv, h, part, now.tile, d, info, mids, grid, smem_u32(cells)); break;
        case 3: search_tile<T, 3>(a, kv, h, part, now.tile, d, info, mids, grid, smem_u32(cells)); break;
        default: search_tile<T, 4>(a, kv, h, part, now.tile, d, info, mids, grid, smem_u32(cells)); break;
      }
    }
    now.next(a.tiles);
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * N) : "memory");
}

template <typename T>
cudaError_t launch(const tq_paged_cache& c, const T* K, const T* V, const int* rows, int n, const int* table,
                   int B, int max_pages, float* mass, int* positions, int S, cudaStream_t st) {
  static std::atomic<int> sms_cache[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int sms = sms_cache[dev & 63].load(std::memory_order_acquire);
  if (sms == 0) {
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(append_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, append_smem<T>(kPD));
    if (e != cudaSuccess) return e;
    sms_cache[dev & 63].store(sms, std::memory_order_release);
  }
  AppendArgs a;
  a.pg = paged_view(c, table, max_pages);
  a.X[0] = K;
  a.X[1] = V;
  a.Pi[0] = c.Pi_k;
  a.Pi[1] = c.Pi_v;
  a.cb[0] = c.k_codebook;
  a.cb[1] = c.v_codebook;
  a.rows = rows;
  a.mass = mass;
  a.positions = positions;
  a.n = n;
  a.step = kCopies * 8;
  a.B = B;
  a.rot = c.rot_heads;
  a.S = S;
  a.cap = max_pages * c.page_size;
  if ((mass != nullptr || positions != nullptr) && S < a.cap) a.cap = S;
  a.bits[0] = c.k_bits;
  a.bits[1] = c.v_bits;
  a.tiles = ceil_div(n, kRows);
  const int64_t whole = static_cast<int64_t>(a.tiles) * c.H * 2;
  a.N = whole * 4 <= sms ? 32 : kPD;
  const int64_t items = whole * (kPD / a.N);
  if (items > INT32_MAX) return cudaErrorInvalidValue;
  a.items = static_cast<int>(items);
  const int64_t most = sms;
  append_kernel<T><<<static_cast<int>(items < most ? items : most), kThreads, append_smem<T>(a.N), st>>>(a);
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
