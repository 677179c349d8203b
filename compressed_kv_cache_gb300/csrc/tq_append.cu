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
// the row's length) is summed again in 64 bits from the inputs.  kNear = 2^-16 covers the
// operands' 2^-21 and, at 2^-23 of the row's length each, the roundings of the up to 24 fp32
// sums of 16 products with room for a tensor core that cuts off instead of rounding; it meets
// about 1 coordinate in 1300 (3 bits).
//
// N is 128 (the rotation of a head stays in shared memory from tile to tile) or, where that
// leaves SMs without a tile, 32: a decode step of 64 tokens then runs on four times the SMs.
#include "tq_paged.cuh"

namespace tq {
namespace {

constexpr int kRows = 128;             // rows of a tile
constexpr int kThreads = 256;
constexpr float kNear = 1.f / 65536.f;
constexpr int kListed = 1024;          // near coordinates a tile can list; with more, all are summed again

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
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
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
  int items;                 // (head, keys or values, part of the rotation, tile)
};

// The cell of v among the midpoints m (ascending): binary search, and whether one of the
// midpoints it met (both neighbours of v are among them) is near.
template <int BITS>
__device__ __forceinline__ uint32_t cell(float v, const float (&m)[15], bool& near) {
  float t = m[(1 << (BITS - 1)) - 1];
  bool p = v > t;
  near = fabsf(v - t) < kNear;
  uint32_t c = p ? 1u << (BITS - 1) : 0u;
  if constexpr (BITS == 2) {
    t = p ? m[2] : m[0];
    c |= v > t ? 1u : 0u;
    near |= fabsf(v - t) < kNear;
  } else if constexpr (BITS == 3) {
    t = p ? m[5] : m[1];
    const float x = p ? m[4] : m[0], y = p ? m[6] : m[2];
    p = v > t;
    near |= fabsf(v - t) < kNear;
    c |= p ? 2u : 0u;
    t = p ? y : x;
    c |= v > t ? 1u : 0u;
    near |= fabsf(v - t) < kNear;
  } else {
    t = p ? m[11] : m[3];
    float x[4];
    float u0 = p ? m[9] : m[1], u1 = p ? m[13] : m[5];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = p ? m[8 + 2 * i] : m[2 * i];
    p = v > t;
    near |= fabsf(v - t) < kNear;
    c |= p ? 4u : 0u;
    t = p ? u1 : u0;
    const float y0 = p ? x[2] : x[0], y1 = p ? x[3] : x[1];
    p = v > t;
    near |= fabsf(v - t) < kNear;
    c |= p ? 2u : 0u;
    t = p ? y1 : y0;
    c |= v > t ? 1u : 0u;
    near |= fabsf(v - t) < kNear;
  }
  return c;
}

// 32 coordinates of a row: packed codes to w, near ones to the returned mask.
template <int BITS>
__device__ __forceinline__ uint32_t search32(const float (&y)[32], float inv, const float (&m)[15], uint32_t (&w)[BITS]) {
  uint32_t mask = 0;
#pragma unroll
  for (int i = 0; i < BITS; ++i) w[i] = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    bool near;
    const uint32_t c = cell<BITS>(y[j] * inv, m, near);
    const int at = BITS * j;
    w[at / 32] |= c << (at % 32);
    if (at % 32 + BITS > 32) w[at / 32 + 1] |= c >> (32 - at % 32);
    if (near) mask |= 1u << j;
  }
  return mask;
}

// What the threads of a tile know of its rows.
struct RowInfo {
  float inv;         // 1 / (length * scales): turns a sum into a unit coordinate; 0 where there is none
  int kind;          // 0: no row, 1: an ordinary one, 2: zero, 3: NaN or infinity within
  uint32_t norm;     // fp16 length
  int code;          // kinds 2 and 3: the code of every coordinate
  long long at;      // row on the cache's planes
};

template <typename T, int BITS>
__device__ __forceinline__ void search_tile(const AppendArgs& a, int kv, int h, int part, int tile, uint32_t tmem,
                                            RowInfo* info, uint32_t* codes, uint16_t* list, int* listed) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunks = a.N / 32, words = chunks * BITS;      // words of a row in this tile
  float m[15];
#pragma unroll
  for (int i = 0; i + 1 < (1 << BITS); ++i)
    m[i] = static_cast<float>(0.5 * (static_cast<double>(a.cb[kv][i]) + static_cast<double>(a.cb[kv][i + 1])));
  {
    const int r = 32 * (warp & 3) + lane;
    const RowInfo ri = info[r];
    const int c0 = chunks == 4 ? 2 * (warp >> 2) : (warp >> 2), c1 = chunks == 4 ? c0 + 2 : (warp < 4 ? 1 : c0);
    for (int c = c0; c < c1; ++c) {
      float y[32];
      tmem_ld32(tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + 32 * c, y);
      uint32_t w[BITS], mask = search32<BITS>(y, ri.inv, m, w);
      if (ri.kind != 1) {
        mask = 0;
#pragma unroll
        for (int i = 0; i < BITS; ++i) {                   // one code throughout
          uint32_t x = 0;
          for (int j = 0; j < 32; ++j) x |= ((static_cast<uint32_t>(ri.code) >> ((32 * i + j) % BITS)) & 1u) << j;
          w[i] = x;
        }
      }
#pragma unroll
      for (int i = 0; i < BITS; ++i) codes[r * words + c * BITS + i] = w[i];
      while (mask != 0) {
        const int j = __ffs(mask) - 1;
        mask &= mask - 1;
        const int at = atomicAdd(listed, 1);
        if (at < kListed) list[at] = static_cast<uint16_t>(r << 7 | (32 * c + j));
      }
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  // near coordinates again, in 64 bits: eight lanes each
  const int total = *listed;
  const bool all = total > kListed;
  const int count = all ? kRows * a.N : total;
  const T* X = static_cast<const T*>(a.X[kv]);
  for (int e0 = warp * 4; e0 < count; e0 += (kThreads / 32) * 4) {
    const int e = e0 + (lane >> 3), j = lane & 7;
    int r = 0, c = 0;
    bool live = e < count;
    if (live) {
      const int v = all ? e : list[e];
      r = all ? e / a.N : v >> 7;
      c = all ? e - r * a.N : v & 127;
      live = info[r].kind == 1;
    }
    double s = 0.0, q = 0.0;
    if (live) {
      const T* x = X + (static_cast<size_t>(tile * kRows + r) * a.pg.H + h) * kPD + j;
      const float* P = a.Pi[kv] + (static_cast<size_t>(h % a.rot) * kPD + part * a.N + c) * kPD + j;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const double xv = static_cast<double>(static_cast<float>(x[8 * i]));
        s += static_cast<double>(P[8 * i]) * xv;
        q += xv * xv;
      }
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      q += __shfl_xor_sync(0xffffffffu, q, o);
    }
    if (live && j == 0) {
      const double len = sqrt(q);
      uint32_t code = 0;
      for (int i = 0; i + 1 < (1 << BITS); ++i)
        code += s > 0.5 * (static_cast<double>(a.cb[kv][i]) + static_cast<double>(a.cb[kv][i + 1])) * len ? 1u : 0u;
      uint32_t* w = codes + r * words + (BITS * c) / 32;
      const int sh = (BITS * c) % 32;
      const bool over = sh + BITS > 32;
      // other lanes and warps may change neighbouring codes of the same words
      uint32_t old = w[0] >> sh;
      if (over) old |= w[1] << (32 - sh);
      const uint32_t flip = (old ^ code) & ((1u << BITS) - 1);
      if (flip != 0) {
        atomicXor(w, flip << sh);
        if (over) atomicXor(w + 1, flip >> (32 - sh));
      }
    }
  }
  __syncthreads();
  // to the planes
  const uint32_t bytes = 16 * BITS, off = part * words;
  uint8_t* plane = kv ? a.pg.vp : a.pg.kp;
  if (chunks == 4) {
    for (int e = tid; e < kRows * BITS; e += kThreads) {
      const int r = e / BITS, i = e - r * BITS;
      if (info[r].kind != 0)
        *reinterpret_cast<uint4*>(plane + info[r].at * bytes + 16 * i) = *reinterpret_cast<const uint4*>(codes + r * words + 4 * i);
    }
  } else {
    for (int e = tid; e < kRows * words; e += kThreads) {
      const int r = e / words, i = e - r * words;
      if (info[r].kind != 0) *reinterpret_cast<uint32_t*>(plane + info[r].at * bytes + 4 * (off + i)) = codes[e];
    }
  }
  if (part == 0 && tid < kRows && info[tid].kind != 0)
    (kv ? a.pg.vn : a.pg.kn)[info[tid].at] = static_cast<uint16_t>(info[tid].norm);
}

template <typename T>
constexpr int append_smem(int N) {
  return kRows * 256 * (sizeof(T) == 4 ? 2 : 1) + N * 256 * 2 + kRows * 64 + kRows * static_cast<int>(sizeof(RowInfo)) +
         kListed * 2 + 64;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 1 : 2)
append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr bool XLO = sizeof(T) == 4;                     // rows need a lo part
  constexpr int V = sizeof(T) / 2;                         // 16-byte loads of 8 values
  extern __shared__ __align__(128) char smem[];
  const int N = a.N;
  char* sA = smem;                                         // hi, then lo of the rows
  char* sB = sA + kRows * 256 * (XLO ? 2 : 1);             // hi, then lo of the rotation
  uint32_t* codes = reinterpret_cast<uint32_t*>(sB + N * 512);
  RowInfo* info = reinterpret_cast<RowInfo*>(codes + kRows * 16);
  uint16_t* list = reinterpret_cast<uint16_t*>(info + kRows);
  uint64_t* bar = reinterpret_cast<uint64_t*>(list + kListed);
  uint32_t* slot = reinterpret_cast<uint32_t*>(bar + 1);
  int* listed = reinterpret_cast<int*>(slot + 1);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(bar)) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(N) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *slot;

  const int parts = kPD / N;
  const int per = a.items / gridDim.x, more = a.items - per * gridDim.x;
  const int cta = blockIdx.x;
  const int first = cta * per + min(cta, more), last = first + per + (cta < more ? 1 : 0);

  // Loads of an item, in registers while the tile before is searched.  Lane 8g + j of warp w
  // holds chunks g, g + 4, g + 8, g + 12 (eight values) of rows 8w + j and 64 + 8w + j.
  uint4 raw[2][4][V];
  int seq = -1, slt = -1, pos = 0;
  auto request = [&](int item) {
    const int tile = item % a.tiles, hk = item / a.tiles / parts;
    const T* X = static_cast<const T*>(a.X[hk & 1]) + static_cast<size_t>(hk >> 1) * kPD;
#pragma unroll
    for (int rg = 0; rg < 2; ++rg) {
      const int i = tile * kRows + 64 * rg + 8 * warp + (lane & 7);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint4* src = reinterpret_cast<const uint4*>(X + static_cast<size_t>(i) * a.pg.H * kPD + 8 * ((lane >> 3) + 4 * k));
#pragma unroll
        for (int v = 0; v < V; ++v) raw[rg][k][v] = i < a.n ? __ldg(src + v) : make_uint4(0, 0, 0, 0);
      }
    }
    seq = -1;
    if (tid < kRows && tile * kRows + tid < a.n) {
      const int* r = a.rows + 3 * static_cast<size_t>(tile * kRows + tid);
      seq = r[0];
      slt = r[1];
      pos = r[2];
    }
  };
  if (first < last) request(first);

  int loaded = -1;
  uint32_t phase = 0;
  bool ok = true;
  for (int item = first; item < last && ok; ++item) {
    const int tile = item % a.tiles, hkp = item / a.tiles, part = hkp % parts, hk = hkp / parts, kv = hk & 1, h = hk >> 1;
    if (hkp != loaded) {                                   // rows part * N .. of the head's rotation, times 2^7
      loaded = hkp;
      const float* P = a.Pi[kv] + (static_cast<size_t>(h % a.rot) * kPD + part * N) * kPD;
      for (int e = tid; e < N * 16; e += kThreads) {
        const int d = (e >> 5) / 4 * 8 + (e & 7), c = (e >> 5) % 4 * 4 + ((e >> 3) & 3);   // as the rows: 8 rows x 4 chunks a warp
        const float4 u = __ldg(reinterpret_cast<const float4*>(P + d * kPD + 8 * c));
        const float4 v = __ldg(reinterpret_cast<const float4*>(P + d * kPD + 8 * c + 4));
        const float x[8] = {128.f * u.x, 128.f * u.y, 128.f * u.z, 128.f * u.w, 128.f * v.x, 128.f * v.y, 128.f * v.z, 128.f * v.w};
        const int at = c * (N * 16) + (d >> 3) * 128 + (d & 7) * 16;
        *reinterpret_cast<uint4*>(sB + at) = hi_chunk(x);
        *reinterpret_cast<uint4*>(sB + N * 256 + at) = lo_chunk(x);
      }
    }
    // where each row goes
    if (tid < kRows) {
      long long at = -1;
      if (seq >= 0 && slt >= 0) {
        if (seq < a.B && slt < a.cap) {
          const int page = a.pg.page(seq, slt);
          if (page >= 0) at = static_cast<long long>(a.pg.row(page, h, slt));
        } else {
          atomicOr(&g_wait_fault, static_cast<unsigned int>(kFaultPaged));
        }
        if (at >= 0 && kv == 0 && part == 0) {
          const size_t m = (static_cast<size_t>(seq) * a.pg.H + h) * a.S + slt;
          if (a.mass != nullptr) a.mass[m] = 0.f;
          if (a.positions != nullptr) a.positions[m] = pos;
        }
      }
      info[tid].at = at;
    }
    if (tid == 0) *listed = 0;
    // rows to fp16, scaled to 2^7
#pragma unroll
    for (int rg = 0; rg < 2; ++rg) {
      uint32_t top = 0;
      float x[4][8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        widen(raw[rg][k], x[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[k][i]) & 0x7fffffffu);
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 8));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 16));
      const bool finite = top < 0x7f800000u;
      // powers of two: up to 2^64 first for rows that are tiny throughout, then to 2^7
      const float s0 = top < 0x21800000u ? 18446744073709551616.f : 1.f;          // below 2^-60
      const float t = __uint_as_float(top) * s0;
      const int e = static_cast<int>(__float_as_uint(t) >> 23);                   // 1 .. 254 for a row that is neither zero nor infinite
      const int k2 = 134 - e;                                                     // -120 .. 126
      const float s1 = finite && top != 0 ? __uint_as_float(static_cast<uint32_t>(127 + (k2 > 126 ? 126 : k2)) << 23) : 0.f;
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[k][i] = finite ? x[k][i] * s0 * s1 : 0.f;
          sum = fmaf(x[k][i], x[k][i], sum);
        }
        const int r = 64 * rg + 8 * warp + (lane & 7), c = (lane >> 3) + 4 * k;
        const int at = c * (kRows * 16) + (r >> 3) * 128 + (r & 7) * 16;
        *reinterpret_cast<uint4*>(sA + at) = hi_chunk(x[k]);
        if constexpr (XLO) *reinterpret_cast<uint4*>(sA + kRows * 256 + at) = lo_chunk(x[k]);
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      if (lane < 8) {
        RowInfo& ri = info[64 * rg + 8 * warp + lane];
        const float len = sqrtf(sum);
        const int kind = !finite ? 3 : top == 0 ? 2 : 1;
        ri.kind = kind;
        ri.inv = kind == 1 ? 1.f / (128.f * len) : 0.f;
        // the length: powers of two taken back, one rounding in fp32 and one to fp16
        const float n = kind == 1 ? len / s1 / s0 : kind == 2 ? 0.f : __uint_as_float(top > 0x7f800000u ? 0x7fc00000u : 0x7f800000u);
        ri.norm = __half_as_ushort(__float2half_rn(n));
        int zero = 0;
        if (kind == 2)
          for (int i = 0; i + 1 < (1 << a.bits[kv]); ++i)
            zero += static_cast<double>(a.cb[kv][i]) + static_cast<double>(a.cb[kv][i + 1]) < 0.0 ? 1 : 0;
        ri.code = zero;
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (tid < kRows && info[tid].at < 0) info[tid].kind = 0;
    if (tid == 0) {
      const uint32_t A = smem_u32(sA), Bm = smem_u32(sB);
      const uint32_t la = kRows * 16, lb = N * 16;
#pragma unroll
      for (int k = 0; k < 8; ++k) mma_f16(tmem, operand(A + k * 2 * la, la), operand(Bm + k * 2 * lb, lb), N, k != 0);
#pragma unroll
      for (int k = 0; k < 8; ++k) mma_f16(tmem, operand(A + k * 2 * la, la), operand(Bm + N * 256 + k * 2 * lb, lb), N, true);
      if constexpr (XLO) {
#pragma unroll
        for (int k = 0; k < 8; ++k) mma_f16(tmem, operand(A + kRows * 256 + k * 2 * la, la), operand(Bm + k * 2 * lb, lb), N, true);
      }
      asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
    }
    if (item + 1 < last) request(item + 1);
    ok = wait_parity_bounded(smem_u32(bar), phase, kFaultPaged) && ok;
    phase ^= 1;
    ok = __syncthreads_and(ok) != 0;
    if (!ok) break;                                        // the product never came: nothing is written
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    switch (a.bits[kv]) {
      case 2: search_tile<T, 2>(a, kv, h, part, tile, tmem, info, codes, list, listed); break;
      case 3: search_tile<T, 3>(a, kv, h, part, tile, tmem, info, codes, list, listed); break;
      default: search_tile<T, 4>(a, kv, h, part, tile, tmem, info, codes, list, listed); break;
    }
    __syncthreads();
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(N) : "memory");
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
  a.B = B;
  a.rot = c.rot_heads;
  a.S = S;
  a.cap = max_pages * c.page_size;
  if ((mass != nullptr || positions != nullptr) && S < a.cap) a.cap = S;
  a.bits[0] = c.k_bits;
  a.bits[1] = c.v_bits;
  a.tiles = ceil_div(n, kRows);
  const int64_t whole = static_cast<int64_t>(a.tiles) * c.H * 2;
  a.N = whole * 4 <= 2 * sms ? 32 : kPD;
  const int64_t items = whole * (kPD / a.N);
  if (items > INT32_MAX) return cudaErrorInvalidValue;
  a.items = static_cast<int>(items);
  const int64_t most = static_cast<int64_t>(sms) * (sizeof(T) == 4 ? 1 : 2);
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
