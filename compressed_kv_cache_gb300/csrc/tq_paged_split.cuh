// The split of tq_decode_paged over the cache's length: logits, softmax and value sum of
// one token per sequence, read straight from the packed codes of the pages.
//
// Work: the cache of every unit (sequence, KV head, query tile) in tiles of 32 slots, all
// units end to end; every warp of the grid (one CTA of 12 warps per SM) takes an equal run of
// that line (the tiles are counted on the device: lengths are not known to the host) and
// leaves one partial (maximum, sum, weighted value sum) for each unit it touched.  No two
// warps ever wait for each other.
//
// Products: mma.m16n8k16 (fp16 operands, fp32 sums) with the keys or values as the 16-row
// operand and up to 8 queries as its 8 columns, so grouped heads cost what one head costs.
// The 16-row operand is made in registers: neighbouring codes select fp16 pairs of centroids
// from tables in shared memory, where every lane that a load serves has a copy in its own banks,
// so that a look-up never conflicts.  tcgen05 would need that operand written to shared memory
// and read back (512 bytes a slot instead of none), where the kernel is already bound; at up
// to 8 queries the tensor pipe is busy for 23 % of the time as it is.
//
// Bound: shared memory.  The look-ups read 512 bytes a slot whatever the codes' width, 4
// wavefronts; codes, lengths and the copies into the ring add 2.8.  131072 slots x 8 heads, 3-bit
// codes: 245 cycles a tile of 32 slots in the loop, 217 of them wavefronts; over the whole kernel
// shared memory is 65 %, issue 58 % and the ALU pipe 46 % busy.  It takes 37 us (2.9 TB/s of codes)
// of a call of 42: 26.5 in the loop, 4 for tables, set-up, first tiles and partials, the rest at the
// grid's start and end.  32 x 32768 x 8 heads, 4-bit keys: a call of 275 us, 3.6 TB/s.  With
// the look-ups' addresses in the place of what they read, the two calls take 38 and 197 us.
// hi + lo look-ups (KX) are 8 bytes each: 335 cycles a tile.
// Measured on the way there (131072 slots x 8 heads, whole call): two-code tables in 64 entries
// with shifts and masks on the ALU pipe 63 us; shifts to the left on the FMA pipe and
// aligned tables 49 us; 256 entries picked by a byte permute 46 us; 8, 12 or 16 warps within
// 5 % of each other.
//
// The order of the sum over coordinates and over slots is free, and is chosen for the loads:
// lane (g, t) of a warp (g = lane / 4, t = lane % 4) takes coordinates 32t .. 32t+31 of two
// keys (whole words of their rows), and coordinates 16g .. 16g+15 of four values.
//
// Precision: a factor x is an fp16 pair hi + lo (22 bits) where KX / VX ask for it; then
// hi hi + hi lo + lo hi are summed.  bf16 queries get a bf16 output, so fp16 operands (2^-11) are
// finer than what comes in and goes out: rotated queries, key and value centroids and weights are
// single fp16 numbers (131072 slots: 2.2e-3 of the output's norm from 64 bits, products of fp32
// operands 1.8e-3, mostly the output's rounding).  With mass the keys' factors are pairs, as the
// weights are summed over many steps (and up to 4 queries a unit the weights).  fp32 queries: pairs
// everywhere.  COL: four queries, whose hi and lo parts are columns
// 0..3 and 4..7 of one product.  Centroids, queries, and values' lengths are scaled by
// powers of two to 2^7 before they become fp16, so that lo stays out of the subnormals.
//
// The tensor core's additions cut bits off, so that the errors of a long sum of like terms add up
// (fp32 queries, flat weights, 1150 tiles a run: 6.8e-5).  With VX the value products of 16 slots
// begin at zero and are added to the sums with rounded additions, two a tile.  A warp takes a unit in
// pieces of at most kPiece tiles, and adds each piece to its partial; with VX it keeps the rounding
// errors of that too.  What is left is the error of one piece, whatever the cache's length: fp32 256
// additions of 2^-24 of a sum that grows evenly, 7.6e-6 at worst and 7e-7 measured (flat
// weights, one value row).  32 x 32768 x 64 heads on 8, fp32: 731 us, and 691 without either; one
// chain of the tensor core in pieces of 64 tiles 721 (5.5e-6 off), of 32 tiles 758 (2.6e-6).
// Additions to the partial from within the loop (721) take registers that the other variants miss.
#pragma once

#include "tq_paged.cuh"

namespace tq {

constexpr int kSplitWarps = 12;
constexpr int kTile = 32;            // slots a warp takes at a time
constexpr int kPartF = 132;          // partial of a query: 128 sums, maximum, sum, 2 unused
constexpr int kMaxCtas = 192;        // partials are laid out for at most this many CTAs
constexpr int kPieceX = 128, kPiece = 256;   // tiles of a piece

// A unit's share of the tiles is cut where the warps' runs are cut: run w covers
// [w q + min(w, r), ...) of T = q W + r tiles.
__host__ __device__ __forceinline__ int run_start(int w, int q, int r) { return w * q + (w < r ? w : r); }
__device__ __forceinline__ int run_of(int tile, int q, int r) {
  const int big = r * (q + 1);
  return tile < big ? tile / (q + 1) : r + (tile - big) / q;
}

struct SplitArgs {
  const uint8_t* kp;
  const uint8_t* vp;
  const uint16_t* kn;
  const uint16_t* vn;
  const int* table;
  int n_pages, H, shift, max_pages;
  const float* A;        // [B, H*G, 128] rotated queries
  const int* tiles;      // [B + 1] tiles before each sequence
  const int* lengths;    // [B] as cut by the plan
  const float* kcb;
  const float* vcb;
  float* part;           // [runs + units][QT][kPartF]; VX: and [runs][QT][kPartF] rounding errors
  float* z;              // [units][Sz][QT] logits times log2(e), or null
  int B, G, nqt, Sz;
  float scale2;          // scale * log2(e)
  uint32_t pow2[8];      // 1, 2, 4 ... 128
};

cudaError_t launch_split_k2(const SplitArgs& a, int vbits, int variant, int ctas, cudaStream_t st);
cudaError_t launch_split_k3(const SplitArgs& a, int vbits, int variant, int ctas, cudaStream_t st);
cudaError_t launch_split_k4(const SplitArgs& a, int vbits, int variant, int ctas, cudaStream_t st);

// Variants: bf16 queries; bf16 with mass, up to 4 and up to 8 queries a unit; fp32.
enum { kVarFast = 0, kVarMass4 = 1, kVarMass8 = 2, kVarF32 = 3 };

#ifdef TQ_SPLIT_KERNEL
namespace {

// Tables of centroids, 256 entries of 128 bytes each: an entry is picked by a byte of the code
// stream, so that its address (table | byte << 8 | lane's copy) is one byte permute.  The
// entry holds copies of what the byte's codes stand for, one for each lane that a load serves
// at a time, each in banks of its own.
//   4 bits: the byte's two codes.        2 bits: its four codes.
//   3 bits: two codes in its low six bits (LOW) or in its high six bits (HIGH); the other two
//           bits are whatever lies there in the stream.
// Two tables interleave in a block of 64 KB (the halves of 256-byte rows); blocks lie at shared
// addresses that are multiples of 64 KB.
constexpr int kBlock = 65536;
constexpr int kSmem = 232448;          // all a CTA can have
constexpr int kFirst = 4096;           // it begins here at the latest: behind what the driver keeps (1 KB)

template <int BITS>
constexpr int tables_of() { return BITS == 3 ? 2 : 1; }

template <int KB, int VB>
struct Lay {
  static constexpr int blocks = (tables_of<KB>() + tables_of<VB>() + 1) / 2;
  static constexpr int kBytes = kTile * 16 * KB, vBytes = kTile * 16 * VB;
  static constexpr int norms = kBytes + vBytes;          // 32 fp16 of keys, 32 of values
  static constexpr int mask = norms + 4 * kTile;         // which slots of the tile are there
  static constexpr int stage = mask + 16;
  // The warps' rings of stages lie before and behind the blocks; the dynamic shared memory
  // begins somewhere in the first 4 KB (kFirst).
  static constexpr int room0 = kBlock - kFirst, room1 = kSmem - (1 + blocks) * kBlock;
  static constexpr int rings(int stages) { return room0 / (stage * stages) + room1 / (stage * stages); }
  static constexpr int stages = rings(4) >= kSplitWarps ? 4 : rings(3) >= kSplitWarps ? 3 : 2;   // a warp's tiles in flight or in use
  static constexpr int ring = stage * stages;
  static constexpr int before = room0 / ring;            // rings before the blocks
  static_assert(rings(stages) >= kSplitWarps, "two stages have to fit");
};

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
// Table entries: the tables never change, so these may move freely.
__device__ __forceinline__ uint32_t lds32t(uint32_t a) {
  uint32_t v;
  asm("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64t(uint32_t a) {
  uint2 v;
  asm("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128t(uint32_t a) {
  uint4 v;
  asm("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ float lds_half(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return __half2float(__ushort_as_half(v));
}
// Copies of 16 and 4 bytes; nothing is read where ok is false (zeros are written).
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with sums that begin at zero.
__device__ __forceinline__ void mma0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float half_round(float x) { return __half2float(__float2half_rn(x)); }

// Power of two that takes |x| = m to [2^7, 2^8) (1 for zero, infinity, NaN), and its inverse.
__device__ __forceinline__ float scale_to_2p7(float m, float* inv) {
  const int e = static_cast<int>((__float_as_uint(m) >> 23) & 255u);
  if (e == 0 || e == 255) { *inv = 1.f; return 1.f; }
  int k = 134 - e;                              // 2^(k) m lies in [2^7, 2^8)
  k = k > 126 ? 126 : (k < -126 ? -126 : k);
  *inv = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
  return __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
}

// Fills table `id` (half id % 2 of block id / 2) from the scaled centroids, one a lane.  X: the
// fp16 pairs of hi parts are followed by those of lo parts.  SHIFT: where the byte's codes
// begin.  A thread writes an entry's eight 16-byte pieces, beginning at its own.
template <int BITS, bool X, int SHIFT>
__device__ __forceinline__ void build_table(char* blocks, int id, float cb) {
  constexpr int m = (1 << BITS) - 1;
  char* tab = blocks + (id >> 1) * kBlock + (id & 1) * 128;
  for (int e0 = 0; e0 < 256; e0 += kSplitWarps * 32) {     // whole warps: the centroids come from lanes
    const int e = e0 + static_cast<int>(threadIdx.x);
    const int i = (e & 255) >> SHIFT;
    const float a = __shfl_sync(0xffffffffu, cb, i & m), b = __shfl_sync(0xffffffffu, cb, (i >> BITS) & m);
    const uint32_t hi = pack2(a, b);
    const uint32_t lo = X ? pack2(a - half_round(a), b - half_round(b)) : hi;
    uint4 v = make_uint4(hi, lo, hi, lo);
    if constexpr (BITS == 2) {
      const float c = __shfl_sync(0xffffffffu, cb, (i >> 4) & m), d = __shfl_sync(0xffffffffu, cb, (i >> 6) & m);
      const uint32_t hi2 = pack2(c, d);
      const uint32_t lo2 = X ? pack2(c - half_round(c), d - half_round(d)) : hi2;
      v = X ? make_uint4(hi, hi2, lo, lo2) : make_uint4(hi, hi2, hi, hi2);
    }
    if (e < 256) {
#pragma unroll
      for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4*>(tab + e * 256 + ((k + e) & 7) * 16) = v;
    }
  }
}
template <int BITS, bool X>
__device__ __forceinline__ void build_tables(char* blocks, int id, float cb) {
  build_table<BITS, X, 0>(blocks, id, cb);
  if constexpr (BITS == 3) build_table<BITS, X, 2>(blocks, id + 1, cb);
}

// A lane's copy within an entry: 4 bytes of a pair, 8 of a pair in two parts or of two
// pairs, 16 of two pairs in two parts.
template <int BITS, bool X>
__device__ __forceinline__ uint32_t copy_of(int lane) {
  constexpr int n = 4 * (X ? 2 : 1) * (BITS == 2 ? 2 : 1);
  return (lane * n) & 127;
}

// Address of the entry that byte I of w names; tab: the table's address and the lane's copy.
template <int I>
__device__ __forceinline__ uint32_t entry(uint32_t w, uint32_t tab) {
  return __byte_perm(w, tab, 0x7604 | I << 4);
}

// The fp16 pairs (X: and their lo parts) of the four pairs of neighbouring codes of one word
// of the stream: 8 codes of 3 or 4 bits.  For 3 bits u is the word moved up by four bits, so that
// its second and third pair lie in one byte each.  2-bit words hold eight pairs.
template <int BITS, bool X>
struct Pairs {
  static constexpr int n = BITS == 2 ? 8 : 4;
  uint32_t hi[n], lo[X ? n : 1];
  template <int K>
  __device__ __forceinline__ void one(uint32_t at) {
    if constexpr (X) {
      const uint2 v = lds64t(at);
      hi[K] = v.x;
      lo[K] = v.y;
    } else {
      hi[K] = lds32t(at);
    }
  }
  template <int K>
  __device__ __forceinline__ void two(uint32_t at) {
    if constexpr (X) {
      const uint4 v = lds128t(at);
      hi[2 * K] = v.x;
      hi[2 * K + 1] = v.y;
      lo[2 * K] = v.z;
      lo[2 * K + 1] = v.w;
    } else {
      const uint2 v = lds64t(at);
      hi[2 * K] = v.x;
      hi[2 * K + 1] = v.y;
    }
  }
  // B0, B1: the bytes of the first pair in w0 and of the last one in w1
  template <int B0, int B1>
  __device__ __forceinline__ void look_up3(uint32_t w0, uint32_t w1, uint32_t u, uint32_t low, uint32_t high) {
    one<0>(entry<B0>(w0, low));
    one<1>(entry<1>(u, high));
    one<2>(entry<2>(u, low));
    one<3>(entry<B1>(w1, high));
  }
  __device__ __forceinline__ void look_up(uint32_t w, uint32_t tab) {
    if constexpr (BITS == 2) {
      two<0>(entry<0>(w, tab));
      two<1>(entry<1>(w, tab));
      two<2>(entry<2>(w, tab));
      two<3>(entry<3>(w, tab));
    } else {
      one<0>(entry<0>(w, tab));
      one<1>(entry<1>(w, tab));
      one<2>(entry<2>(w, tab));
      one<3>(entry<3>(w, tab));
    }
  }
};

// Word I of the 32 codes of a key row that a lane takes.
template <int KB, bool X, int I>
__device__ __forceinline__ void key_pairs(Pairs<KB, X>& r, const uint32_t (&w)[KB], uint32_t low, uint32_t high,
                                          const SplitArgs& p) {
  if constexpr (KB != 3) r.look_up(w[I], low);
  else if constexpr (I == 0) r.template look_up3<0, 2>(w[0], w[0], w[0] * p.pow2[4], low, high);
  else if constexpr (I == 1) r.template look_up3<3, 1>(w[0], w[1], __funnelshift_r(w[0], w[1], 20), low, high);
  else if constexpr (I == 2) r.template look_up3<2, 0>(w[1], w[2], __funnelshift_r(w[1], w[2], 12), low, high);
  else r.template look_up3<1, 3>(w[2], w[2], w[2] >> 4, low, high);
}

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], uint32_t a) {
  if constexpr (N == 2) {
    const uint2 v = lds64(a);
    w[0] = v.x; w[1] = v.y;
  } else if constexpr (N == 4) {
    const uint4 v = lds128(a);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = lds32(a + 4 * i);
  }
}

// The 16 codes 16g .. 16g+15 of a value row as words (3-bit rows: six bytes, picked from the
// two aligned words around them by the lane's selectors).
template <int VB>
__device__ __forceinline__ void load_value(uint32_t (&w)[2], uint32_t row, int g, uint32_t sel0, uint32_t sel1) {
  if constexpr (VB == 2) {
    w[0] = lds32(row + 4 * g);
    w[1] = 0;
  } else if constexpr (VB == 4) {
    const uint2 v = lds64(row + 8 * g);
    w[0] = v.x; w[1] = v.y;
  } else {
    const uint32_t a = row + ((6 * g) & ~3);
    const uint32_t x = lds32(a), y = lds32(a + 4);
    w[0] = __byte_perm(x, y, sel0);
    w[1] = __byte_perm(x, y, sel1);
  }
}

// Products of two keys (rows g and g + 8) with the queries, word I of their codes and on.  With KX
// the coordinates are summed in four parts: the tensor core's additions cut bits off, and two
// of them in a row cost half the error of eight (fp32 queries, 8 x 32 heads of up to 2049
// slots: 9.6e-7 of the output's norm in one part).
template <bool KX>
constexpr int parts_of() { return KX ? 4 : 1; }
template <int KB, bool KX, int NB, int I>
__device__ __forceinline__ void key_products(float (&c)[parts_of<KX>()][4], float (&cl)[4], const uint32_t (&w0)[KB], const uint32_t (&w1)[KB],
                                             uint32_t low, uint32_t high, const SplitArgs& p, const uint32_t (&q)[16],
                                             const uint32_t (&ql)[NB]) {
  using Pr = Pairs<KB, KX>;
  constexpr int n = Pr::n / 2;                             // products of 16 coordinates in a word
  Pr a, b;
  key_pairs<KB, KX, I>(a, w0, low, high, p);
  key_pairs<KB, KX, I>(b, w1, low, high, p);
#pragma unroll
  for (int k = 0; k < n; ++k) {
    const int m = I * n + k;
    float (&cm)[4] = c[m % parts_of<KX>()];
    if (m < parts_of<KX>()) mma0(cm, a.hi[2 * k], b.hi[2 * k], a.hi[2 * k + 1], b.hi[2 * k + 1], q[2 * m], q[2 * m + 1]);
    else mma(cm, a.hi[2 * k], b.hi[2 * k], a.hi[2 * k + 1], b.hi[2 * k + 1], q[2 * m], q[2 * m + 1]);
    if constexpr (KX) {
      if (m == 0) mma0(cl, a.lo[0], b.lo[0], a.lo[1], b.lo[1], q[0], q[1]);
      else mma(cl, a.lo[2 * k], b.lo[2 * k], a.lo[2 * k + 1], b.lo[2 * k + 1], q[2 * m], q[2 * m + 1]);
    }
    if constexpr (NB == 16) mma(cl, a.hi[2 * k], b.hi[2 * k], a.hi[2 * k + 1], b.hi[2 * k + 1], ql[2 * m], ql[2 * m + 1]);
  }
  if constexpr ((I + 1) * n < 8) key_products<KB, KX, NB, I + 1>(c, cl, w0, w1, low, high, p, q, ql);
}

// Two keys' codes of one coordinate side by side: even coordinates of the word to `e`, odd
// ones to `o` (shifts to the left are products: they run on the FMA pipe, the ALU pipe being
// the busier one).
template <int VB>
__device__ __forceinline__ void interleave(uint32_t a, uint32_t b, const SplitArgs& p, uint32_t& e, uint32_t& o) {
  constexpr uint32_t m = VB == 2 ? 0x33333333u : VB == 3 ? 0x1c71c7u : 0x0f0f0f0fu;
  e = (a & m) | ((b * p.pow2[VB]) & ~m);
  o = ((a >> VB) & m) | (b & ~m);
}

template <int VB, bool VX>
__device__ __forceinline__ void value_pairs(Pairs<VB, VX>& r, uint32_t w, uint32_t low, uint32_t high, const SplitArgs& p) {
  if constexpr (VB == 3) r.template look_up3<0, 2>(w, w, w * p.pow2[4], low, high);
  else r.look_up(w, low);
}

// Weighted sum of four keys' values (slots 2t, 2t+1, 2t+8, 2t+9 of the product), word I and on.
// VX: the product is added with a rounding of its own.
template <int VB, bool VX, int I>
__device__ __forceinline__ void value_products(float (&acc)[8][4], const uint32_t (&wa)[2], const uint32_t (&wb)[2],
                                               const uint32_t (&wc)[2], const uint32_t (&wd)[2], uint32_t low,
                                               uint32_t high, const SplitArgs& p, uint32_t b0, uint32_t b1) {
  using Pr = Pairs<VB, VX>;
  uint32_t e0, o0, e1, o1;
  interleave<VB>(wa[I], wb[I], p, e0, o0);
  interleave<VB>(wc[I], wd[I], p, e1, o1);
  Pr f0, f1, f2, f3;
  value_pairs<VB, VX>(f0, e0, low, high, p);
  value_pairs<VB, VX>(f1, o0, low, high, p);
  value_pairs<VB, VX>(f2, e1, low, high, p);
  value_pairs<VB, VX>(f3, o1, low, high, p);
#pragma unroll
  for (int k = 0; k < Pr::n; ++k) {
    const int m = I * Pr::n + k;
    if constexpr (VX) {
      float c[4];
      mma0(c, f0.hi[k], f1.hi[k], f2.hi[k], f3.hi[k], b0, b1);
      mma(c, f0.lo[k], f1.lo[k], f2.lo[k], f3.lo[k], b0, b1);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][i] += c[i];
    } else {
      mma(acc[m], f0.hi[k], f1.hi[k], f2.hi[k], f3.hi[k], b0, b1);
    }
  }
  if constexpr ((I + 1) * Pr::n < 8)
    value_products<VB, VX, I + 1>(acc, wa, wb, wc, wd, low, high, p, b0, b1);
}

// Largest b with tiles[b] * per <= t, by 32-way steps of the whole warp.
__device__ __forceinline__ int find_sequence(const int* tiles, int B, int per, int t, int lane) {
  int lo = 0, n = B;                                      // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lane * step;
    const bool le = i < n && tiles[lo + i] * per <= t;    // lane 0 always
    const int k = 31 - __clz(__ballot_sync(0xffffffffu, le));
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// a * f + b rounded, and its rounding error.
__device__ __forceinline__ float add_err(float a, float f, float b, float* err) {
  const float p = __fmul_rn(a, f), s = p + b, x = s - p;
  *err = ((p - (s - x)) + (b - x)) + fmaf(a, f, -p);
  return s;
}
// Four sums of a partial: what it has, times f, and v.  X: `rest` has (`more`) and gets their
// rounding errors, which go to the sums at the end.
template <bool X>
__device__ __forceinline__ float4 join_sum(const float4& a, const float4& v, float f, float4* rest, bool more, bool last) {
  if constexpr (!X) {
    return make_float4(fmaf(a.x, f, v.x), fmaf(a.y, f, v.y), fmaf(a.z, f, v.z), fmaf(a.w, f, v.w));
  } else {
    float4 e, s;
    s.x = add_err(a.x, f, v.x, &e.x);
    s.y = add_err(a.y, f, v.y, &e.y);
    s.z = add_err(a.z, f, v.z, &e.z);
    s.w = add_err(a.w, f, v.w, &e.w);
    if (more) {
      const float4 r = *rest;
      e = make_float4(fmaf(r.x, f, e.x), fmaf(r.y, f, e.y), fmaf(r.z, f, e.z), fmaf(r.w, f, e.w));
    }
    if (last) return make_float4(s.x + e.x, s.y + e.y, s.z + e.z, s.w + e.w);
    *rest = e;
    return s;
  }
}

template <int KB, int VB, bool KX, bool VX, bool COL>
__global__ void __launch_bounds__(kSplitWarps * 32, 1)
paged_split_kernel(const __grid_constant__ SplitArgs p) {
  using L = Lay<KB, VB>;
  constexpr int QT = COL ? 4 : 8;
  constexpr int NL = (KX && !COL) ? 16 : 1;
  extern __shared__ __align__(128) char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;

  const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(smem));   // kFirst or less: checked by the host
  const uint32_t ring = warp < L::before ? base + warp * L::ring
                                         : (1 + L::blocks) * kBlock + (warp - L::before) * L::ring;

  // tables: inputs of the call, so they may be read before the plan is there
  constexpr int vid = tables_of<KB>();                     // numbers of the values' tables
  float kinv, vinv;
  {
    const float kc = lane < 1 << KB ? p.kcb[lane] : 0.f, vc = lane < 1 << VB ? p.vcb[lane] : 0.f;
    float mk = fabsf(kc), mv = fabsf(vc);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, o));
      mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, o));
    }
    const float ks = scale_to_2p7(mk, &kinv), vs = scale_to_2p7(mv, &vinv);
    build_tables<KB, KX>(smem + (kBlock - base), 0, kc * ks);
    build_tables<VB, VX>(smem + (kBlock - base), vid, vc * vs);
  }
  __syncthreads();
  const uint32_t klow = kBlock + copy_of<KB, KX>(lane), khigh = klow + 128;
  const uint32_t vlow = (1 + vid / 2) * kBlock + (vid & 1) * 128 + copy_of<VB, VX>(lane);
  const uint32_t vhigh = (1 + (vid + 1) / 2) * kBlock + ((vid + 1) & 1) * 128 + copy_of<VB, VX>(lane);
  const uint32_t sel0 = g & 1 ? 0x5432u : 0x3210u, sel1 = g & 1 ? 0x7765u : 0x6543u;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int per = p.H * p.nqt;
  const bool few = p.B <= 32;                              // then lane b knows sequence b
  const int mine = few ? p.tiles[min(lane, p.B)] : 0, mylen = few ? p.lengths[min(lane, p.B - 1)] : 0;
  const int T = p.tiles[p.B] * per;
  const int W = gridDim.x * kSplitWarps;
  const int run = warp * gridDim.x + blockIdx.x;           // short lines reach every SM
  const int rq = T / W, rr = T % W;
  const int end = run_start(run + 1, rq, rr);
  for (int at = run_start(run, rq, rr); at < end;) {
    int b, first, nt, n;
    if (few) {
      b = 31 - __clz(__ballot_sync(0xffffffffu, lane < p.B && mine * per <= at));
      first = __shfl_sync(0xffffffffu, mine, b);
      nt = (b + 1 < 32 ? __shfl_sync(0xffffffffu, mine, (b + 1) & 31) : T / per) - first;
      n = __shfl_sync(0xffffffffu, mylen, b);
    } else {
      b = find_sequence(p.tiles, p.B, per, at, lane);
      first = p.tiles[b];
      nt = p.tiles[b + 1] - first;
      n = p.lengths[b];
    }
    const int in = at - first * per;
    const int u = in / nt;                                 // (head, query tile) of the sequence
    const int tile0 = in - u * nt;
    constexpr int piece = VX ? kPieceX : kPiece;
    const int tile1 = min(min(nt, tile0 + (end - at)), tile0 + piece);
    const int before = min(tile0, at - run_start(run, rq, rr));   // tiles of the unit that this warp has had
    at += tile1 - tile0;
    const int h = u / p.nqt, j = u - h * p.nqt;
    const int unit = b * per + u;
    const int* table = p.table + static_cast<size_t>(b) * p.max_pages;

    // a tile is two runs of 16 rows, each on one page (both on one where a page holds 32)
    int pg0 = -1, pg1 = -1;
    auto look_up = [&](int tile) {
      const int s = min(tile, tile1 - 1) * kTile;
      pg0 = table[s >> p.shift];
      if (p.shift == 4) pg1 = s + 16 < n ? table[(s >> 4) + 1] : -1;
    };
    auto issue = [&](int tile, uint32_t st) {
      const int s = tile * kTile, left = n - s;
      const bool live = tile < tile1;                      // behind the last tile nothing is read
      const bool ok0 = live && static_cast<unsigned>(pg0) < static_cast<unsigned>(p.n_pages);
      const uint32_t ph0 = (ok0 ? pg0 : 0) * p.H + h;
      uint32_t there = left >= 32 ? 0xffffffffu : (1u << (left & 31)) - 1;
      uint32_t gone = ok0 ? 0u : 0xffffu;
      if (p.shift >= 5) {
        const size_t r = (static_cast<size_t>(ph0) << p.shift) + (s & ((1 << p.shift) - 1));
        const uint8_t* ks = p.kp + r * (16 * KB) + lane * 16;
        const uint8_t* vs = p.vp + r * (16 * VB) + lane * 16;
#pragma unroll
        for (int i = 0; i < KB; ++i) cp16(st + lane * 16 + i * 512, ks + i * 512, ok0);
#pragma unroll
        for (int i = 0; i < VB; ++i) cp16(st + lane * 16 + L::kBytes + i * 512, vs + i * 512, ok0);
        cp4(st + L::norms + lane * 4, (lane < 16 ? p.kn : p.vn - 32) + r + 2 * lane, ok0);
        gone = ok0 ? 0u : 0xffffffffu;
      } else {
        const bool ok1 = live && static_cast<unsigned>(pg1) < static_cast<unsigned>(p.n_pages);
        const uint32_t ph1 = (ok1 ? pg1 : 0) * p.H + h;
        const size_t r0 = static_cast<size_t>(ph0) << 4, r1 = static_cast<size_t>(ph1) << 4;
#pragma unroll
        for (int i = 0; i < KB; ++i) {
          const int c = i * 32 + lane;
          const bool second = c >= 16 * KB;
          cp16(st + c * 16, p.kp + (second ? r1 : r0) * (16 * KB) + (second ? c - 16 * KB : c) * 16, second ? ok1 : ok0);
        }
#pragma unroll
        for (int i = 0; i < VB; ++i) {
          const int c = i * 32 + lane;
          const bool second = c >= 16 * VB;
          cp16(st + L::kBytes + c * 16, p.vp + (second ? r1 : r0) * (16 * VB) + (second ? c - 16 * VB : c) * 16,
               second ? ok1 : ok0);
        }
        const bool second = (lane & 15) >= 8;
        cp4(st + L::norms + lane * 4, (lane < 16 ? p.kn : p.vn) + (second ? r1 : r0) + 2 * (lane & 7), second ? ok1 : ok0);
        if (!ok1) gone |= 0xffff0000u;
      }
      if (live && (there & gone) != 0 && lane == 0) atomicOr(&g_wait_fault, static_cast<unsigned int>(kFaultPaged));
      there &= ~gone;
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(st + L::mask), "r"(there) : "memory");
      look_up(tile + 1);
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    look_up(tile0);
    // queries: column g is query g (COL: g % 4; its hi part for g < 4, its lo part above); they
    // are asked for with the first pages, and made ready while the first tiles come
    const int qi = j * QT + (COL ? (g & 3) : g);
    float4 qraw[8];
    {
      const float4* src = reinterpret_cast<const float4*>(
          p.A + (static_cast<size_t>(b * p.H + h) * p.G + min(qi, p.G - 1)) * kPD + 32 * t);
#pragma unroll
      for (int i = 0; i < 8; ++i) qraw[i] = src[i];
    }
    // The ring is free once its readers are done and the unit before has no copies left under way:
    // those behind its last tile read nothing, but write zeros.
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
#pragma unroll
    for (int i = 0; i < L::stages - 1; ++i) issue(tile0 + i, ring + i * L::stage);
    uint32_t q[16], ql[NL];
    float qinv;
    {
      float x[32], m = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 v = qraw[i];
        x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) m = fmaxf(m, fabsf(x[i]));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      float s = scale_to_2p7(m, &qinv);
      if (qi >= p.G) s = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float a = x[2 * i] * s, c = x[2 * i + 1] * s;
        const float al = a - half_round(a), cl = c - half_round(c);
        if constexpr (COL) q[i] = g < 4 ? pack2(a, c) : pack2(al, cl);
        else q[i] = pack2(a, c);
        if constexpr (NL == 16) ql[i] = pack2(al, cl);
      }
      if (qi >= p.G) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          q[i] = 0;
          if constexpr (NL == 16) ql[i] = 0;
        }
      }
    }
    // logit factors of columns 2t and 2t + 1 (COL: of their queries)
    const int c0 = COL ? 2 * (t & 1) : 2 * t;
    const float f0 = __shfl_sync(0xffffffffu, qinv, 4 * c0) * kinv * p.scale2;
    const float f1 = __shfl_sync(0xffffffffu, qinv, 4 * (c0 + 1)) * kinv * p.scale2;

    float acc[8][4];
#pragma unroll
    for (int m = 0; m < 8; ++m) acc[m][0] = acc[m][1] = acc[m][2] = acc[m][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float vs = 0.f, vsinv = 0.f, vtop = 0.f;               // values' lengths: scale, inverse, largest so far
    float* zrow = p.z == nullptr ? nullptr : p.z + (static_cast<size_t>(unit) * p.Sz) * QT;

    int rs = 0, ws = L::stages - 1;
    for (int tile = tile0; tile < tile1; ++tile) {
      asm volatile("cp.async.wait_group %0;" ::"n"(L::stages - 2) : "memory");
      __syncwarp();
      issue(tile + L::stages - 1, ring + ws * L::stage);
      ws = ws + 1 == L::stages ? 0 : ws + 1;
      const uint32_t st = ring + rs * L::stage;
      rs = rs + 1 == L::stages ? 0 : rs + 1;

      const uint32_t there = lds32(st + L::mask);
      const int r0 = (g >> 1) + (g & 1) * 4;               // row g of the product is this key of its 8
      float z[2][4], f[2][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        uint32_t w0[KB], w1[KB];
        load_words(w0, st + (16 * mt + r0) * (16 * KB) + t * 4 * KB);
        load_words(w1, st + (16 * mt + 8 + r0) * (16 * KB) + t * 4 * KB);
        float c[parts_of<KX>()][4], cl[4];
        key_products<KB, KX, NL, 0>(c, cl, w0, w1, klow, khigh, p, q, ql);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (KX) z[mt][i] = ((c[0][i] + c[1][i]) + (c[2][i] + c[3][i])) + cl[i];
          else z[mt][i] = c[0][i];
        }
        if constexpr (COL) {
#pragma unroll
          for (int i = 0; i < 4; ++i) z[mt][i] += __shfl_xor_sync(0xffffffffu, z[mt][i], 2);
        }
        const int ka = 16 * mt + r0, kb = ka + 8;
        const float na = lds_half(st + L::norms + 2 * ka), nb = lds_half(st + L::norms + 2 * kb);
        f[mt][0] = na * f0;
        f[mt][1] = na * f1;
        f[mt][2] = nb * f0;
        f[mt][3] = nb * f1;
        if (zrow != nullptr && (!COL || t < 2)) {
          float* zt = zrow + static_cast<size_t>(tile * kTile) * QT + c0;
          const bool ha = (there >> ka) & 1, hb = (there >> kb) & 1;
          if (tile * kTile + ka < n)
            *reinterpret_cast<float2*>(zt + ka * QT) = ha ? make_float2(z[mt][0] * f[mt][0], z[mt][1] * f[mt][1])
                                                          : make_float2(-INFINITY, -INFINITY);
          if (tile * kTile + kb < n)
            *reinterpret_cast<float2*>(zt + kb * QT) = hb ? make_float2(z[mt][2] * f[mt][2], z[mt][3] * f[mt][3])
                                                          : make_float2(-INFINITY, -INFINITY);
        }
      }
      float nv = lds_half(st + L::norms + 64 + 2 * lane);
      const bool part_tile = there != 0xffffffffu;
      if (part_tile) {                                     // absent slots: a factor that leaves no weight whatever z is
        if (!((there >> lane) & 1)) nv = 0.f;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          if (!((there >> (16 * mt + r0)) & 1)) z[mt][0] = z[mt][1] = -INFINITY, f[mt][0] = f[mt][1] = 1.f;
          if (!((there >> (16 * mt + r0 + 8)) & 1)) z[mt][2] = z[mt][3] = -INFINITY, f[mt][2] = f[mt][3] = 1.f;
        }
      }
      // Logits relative to the running maximum.  It moves only when one passes it by 2^8 (so
      // weights stay below 2^8 and their fp16 form below 2^16), which is rare after the first
      // tile; before there is one, everything passes it.
      float x[2][4], top = -INFINITY;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        x[mt][0] = fmaf(z[mt][0], f[mt][0], -m0);
        x[mt][1] = fmaf(z[mt][1], f[mt][1], -m1);
        x[mt][2] = fmaf(z[mt][2], f[mt][2], -m0);
        x[mt][3] = fmaf(z[mt][3], f[mt][3], -m1);
        top = fmaxf(top, fmaxf(fmaxf(x[mt][0], x[mt][1]), fmaxf(x[mt][2], x[mt][3])));
      }
      if (__any_sync(0xffffffffu, top > 8.f || m0 == -INFINITY || m1 == -INFINITY || nv > vtop)) {
        float a = -INFINITY, c = -INFINITY, v = nv;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          a = fmaxf(a, fmaxf(z[mt][0] * f[mt][0], z[mt][2] * f[mt][2]));
          c = fmaxf(c, fmaxf(z[mt][1] * f[mt][1], z[mt][3] * f[mt][3]));
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
          c = fmaxf(c, __shfl_xor_sync(0xffffffffu, c, o));
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
        a = fmaxf(a, m0);
        c = fmaxf(c, m1);
        const float e0 = m0 > -INFINITY ? ex2(m0 - a) : 0.f, e1 = m1 > -INFINITY ? ex2(m1 - c) : 0.f;
        m0 = a;
        m1 = c;
        l0 *= e0;
        l1 *= e1;
        float r = 1.f;
        if (v > vtop) {                                    // to the next power of two, and no further this way
          float inv;
          const float s = scale_to_2p7(v, &inv) * 0.5f;    // lengths up to 2^7 after it
          r = vs > 0.f ? s * vsinv : 0.f;
          vs = s;
          vsinv = 2.f * inv;
          vtop = __uint_as_float(__float_as_uint(v) | 0x7fffffu);
        }
        const float x0 = e0 * r, x1 = e1 * r;
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          acc[m][0] *= x0;
          acc[m][1] *= x1;
          acc[m][2] *= x0;
          acc[m][3] *= x1;
        }
        // no slot yet: every logit here is -inf, and stays so
        const float s0 = m0 > -INFINITY ? m0 : 0.f, s1 = m1 > -INFINITY ? m1 : 0.f;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          x[mt][0] = fmaf(z[mt][0], f[mt][0], -s0);
          x[mt][1] = fmaf(z[mt][1], f[mt][1], -s1);
          x[mt][2] = fmaf(z[mt][2], f[mt][2], -s0);
          x[mt][3] = fmaf(z[mt][3], f[mt][3], -s1);
        }
      }
      nv *= vs;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const int ka = 16 * mt + r0, kb = ka + 8;
        const float va = __shfl_sync(0xffffffffu, nv, ka), vb = __shfl_sync(0xffffffffu, nv, kb);
        const float p0 = ex2(x[mt][0]), p1 = ex2(x[mt][1]), p2 = ex2(x[mt][2]), p3 = ex2(x[mt][3]);
        l0 += p0 + p2;
        l1 += p1 + p3;
        float w0 = p0 * va, w1 = p1 * va, w2 = p2 * vb, w3 = p3 * vb;
        if constexpr (COL) {
          if (t >= 2) {
            w0 -= half_round(w0);
            w1 -= half_round(w1);
            w2 -= half_round(w2);
            w3 -= half_round(w3);
          }
        }
        const uint32_t b0 = transpose8x8(pack2(w0, w1)), b1 = transpose8x8(pack2(w2, w3));
        // slots 2t and 2t + 1 of the product are keys t and t + 4 of their 8
        const uint32_t row = st + L::kBytes + (16 * mt + t) * (16 * VB);
        uint32_t wa[2], wb[2], wc[2], wd[2];
        load_value<VB>(wa, row, g, sel0, sel1);
        load_value<VB>(wb, row + 4 * 16 * VB, g, sel0, sel1);
        load_value<VB>(wc, row + 8 * 16 * VB, g, sel0, sel1);
        load_value<VB>(wd, row + 12 * 16 * VB, g, sel0, sel1);
        value_products<VB, VX, 0>(acc, wa, wb, wc, wd, vlow, vhigh, p, b0, b1);
      }
    }

    // this warp's partial of the unit, or what is added to it
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, o);
      l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }
    if constexpr (COL) {
#pragma unroll
      for (int m = 0; m < 8; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][i] += __shfl_xor_sync(0xffffffffu, acc[m][i], 2);
    }
    const float fin = vs > 0.f ? vsinv * vinv : 0.f;
    float* part = p.part + static_cast<size_t>(run + unit) * (QT * kPartF);
    float* rest = p.part + (static_cast<size_t>(W) + p.B * per + run) * (QT * kPartF);
    const int live = min(QT, p.G - j * QT);
    const bool last = tile1 == nt || at == end;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool writes = (!COL || t < 2) && c0 + i < live;
      float* o = part + (c0 + i) * kPartF;
      float4* r4 = reinterpret_cast<float4*>(rest + (c0 + i) * kPartF);
      float mx = i ? m1 : m0, f = fin, had = 0.f;
      float4 l = make_float4(i ? l1 : l0, 0.f, 0.f, 0.f);
      float2 ml = make_float2(0.f, 0.f);
      if (before > 0) {
        if (writes) ml = *reinterpret_cast<const float2*>(o + kPD);
        __syncwarp();                                      // every lane has read it
        // as in the loop, the maximum moves only by 2^8 and more: what is there is hardly ever rounded again
        const float top = mx > ml.x + 8.f || ml.x == -INFINITY ? mx : ml.x;
        had = ml.x > -INFINITY ? ex2(ml.x - top) : 0.f;
        const float now = mx > -INFINITY ? ex2(mx - top) : 0.f;
        mx = top;
        f *= now;
        l.x *= now;
      }
      if (writes) {
        float4* o4 = reinterpret_cast<float4*>(o + 16 * g);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          float4 v = make_float4(acc[2 * m][i] * f, acc[2 * m][2 + i] * f, acc[2 * m + 1][i] * f, acc[2 * m + 1][2 + i] * f);
          if (before > 0) v = join_sum<VX>(o4[m], v, had, r4 + 4 * g + m, before > piece, last);
          o4[m] = v;
        }
        if (g == 0) {
          if (before > 0) l = join_sum<VX>(make_float4(ml.y, 0.f, 0.f, 0.f), l, had, r4 + kPD / 4, before > piece, last);
          *reinterpret_cast<float2*>(o + kPD) = make_float2(mx, l.x);
        }
      }
    }
  }
}

template <int KB, int VB, bool KX, bool VX, bool COL>
cudaError_t launch_one(const SplitArgs& a, int ctas, cudaStream_t st) {
  auto kernel = paged_split_kernel<KB, VB, KX, VX, COL>;
  static std::atomic<uint64_t> configured{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(configured.load(std::memory_order_acquire) & bit)) {
    int kept = 0;                                          // shared memory before the kernel's own, all of which is dynamic
    e = cudaDeviceGetAttribute(&kept, cudaDevAttrReservedSharedMemoryPerBlock, dev);
    if (e == cudaSuccess && kept > kFirst) e = cudaErrorInvalidConfiguration;
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_acq_rel);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kSplitWarps * 32);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int KB, int VB>
cudaError_t launch_variant(const SplitArgs& a, int variant, int ctas, cudaStream_t st) {
  switch (variant) {
    case kVarFast: return launch_one<KB, VB, false, false, false>(a, ctas, st);
    case kVarMass4: return launch_one<KB, VB, true, false, true>(a, ctas, st);
    case kVarMass8: return launch_one<KB, VB, true, false, false>(a, ctas, st);
    default: return launch_one<KB, VB, true, true, true>(a, ctas, st);
  }
}

template <int KB>
cudaError_t launch_split(const SplitArgs& a, int vbits, int variant, int ctas, cudaStream_t st) {
  switch (vbits) {
    case 2: return launch_variant<KB, 2>(a, variant, ctas, st);
    case 3: return launch_variant<KB, 3>(a, variant, ctas, st);
    default: return launch_variant<KB, 4>(a, variant, ctas, st);
  }
}

}  // namespace
#endif  // TQ_SPLIT_KERNEL

}  // namespace tq
