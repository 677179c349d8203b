// The split of tq_attend_int8: a step's queries over the 8-bit paged cache, its quads of tiles cut evenly over the device.
//
// Mathematics.  A key is (c + 0.5) * 2^e with whole numbers c = u - 128 that fp16 holds exactly, so
//   logit = 2^e * f * (sum_d c_d q_d + 0.5 sum_d q_d),      f = scale * log2(e) * 2^-x,
// with the query times 2^x in fp16 (bf16 queries exactly, fp32 ones as two parts, 22 bits): products are exact and the
// tensor core sums them in fp32.  Values likewise: sum_i p_i 2^(e_i) (c_i + 0.5) takes w_i = p_i 2^(e_i) in fp16 (two
// parts for fp32) against the whole numbers, and half the sum of w.  w has a maximum M of its own, max(z + e): a block of small
// values with all the weight keeps its bits beside one of large values with none.  Both maxima follow only when a logit
// passes them by 2^8 (w is taken 2^7 above its range, so it stays below 2^15), which saves the exchange between lanes in
// nearly every tile.
//
// Roundings.  The products take fp16 operands, so w is rounded: to 2^-11 in one part for bf16 outputs, an eighth of their own half
// step of 2^-8, and differently for every slot, so that it averages out (outputs are as far from 64 bits as those of weights in
// fp32: 0.001698 and 0.001697 of their norm for 1021 slots, 0.001116 and 0.001115 for drafts in a window).  Two parts would
// double the second product.  fp32 queries and weights have two parts, 22 bits, and exp2 two steps of fp32, 2^-22: outputs
// are 2e-7 to 7e-7 of their norm off where plain fp32 is 2e-7 to 5e-7; a third part would add half to the products for the
// last two bits.  The sum of weights that divides needs no operand and stays in fp32, unrounded.
//
// Work.  A unit is (sequence, head, NC = 8 NT columns), a column a (token, query head of the group); its visible slots
// are tiles of 32, first those of the sinks, then those of the window.  Four tiles are a quad, quads of all units are counted
// through and each block of threads takes an even share, whatever the sequences' lengths (two blocks an SM, one wave).  A unit
// counts as many quads as its sequence's last, which is what it has for one token, a few, or a piece of a prompt behind a
// long cache.  Of a prompt from an empty cache the first units have few: there the shares' work is uneven.  Each of
// its four warps takes one tile of every quad; the warps' sums are joined in shared memory at the end of a unit.  A unit
// that lies within one block's share is written out; of the others each block leaves a part in the workspace
// (tq_int8_attend.cu joins them).
//
// A tile: rows go by 16-byte asynchronous copies into the warp's own ring of kStages tiles (no block-wide
// barrier in the loop), 16-byte pieces exchanged by row so that both products read without bank conflicts.  Keys are the
// 16 rows of the matrix instruction and columns its 8: one query a head fills the tensor core no worse than eight.
// Values are its rows too (dimensions), so the weights need one 8x8 transposition per 16 slots and no conversion of layout
// elsewhere.  Bytes become fp16 by placing them below 1024 (0x64) and subtracting 1152: 4 instructions for 4 codes
// of keys, 10 for 8 of values (two rows are interleaved).
//
// Bound by the cache's bytes where there are enough of them: 32 x 32768 slots of 8 heads, 2.15 GB, in 327 us with the
// join, 97 % of the copy rate; 131072 slots of one sequence 55 us, of which 35 are the bytes and the rest start, the
// blocks' uneven ends and the join.  Two blocks an SM with three stages; three with two: 337 us (heads of 64: three).
#pragma once

#include "tq_int8.cuh"

namespace tq {

constexpr int kAttendCtas = 480;      // room for the parts of this many blocks
constexpr int kPromptCtas = 160;      // of the prompts' form
constexpr int kAttendWarps = 4;
constexpr int kTileSlots = 32, kQuadTiles = kAttendWarps;

// Blocks an SM: what registers allow.  Heads of 64 with 8 columns: three (8 ragged sequences of 2049 slots in fp32 19.9 us, two
// 22.3); heads of 128 with 8 columns would fit three only with two stages (32 x 32768 slots 337 us, two blocks with three 327).
constexpr int attend_blocks(bool f32, int D, int nt) { return D == 64 && nt == 1 ? 3 : 2; }

// What a block leaves for the join: the unit that it starts in the middle of.
struct alignas(16) AttendRecord {
  int chunk;                 // quads of a block (cut to 2^30: no unit has more)
  int off, quads;            // of the unit: quads before this block's start, all
  int first, count, h, cb;
  int block;                 // the block's own number
};

struct AttendArgs {
  Int8View c;
  Step step;
  const void* Q;
  void* out;
  int G, window, sinks;
  float scale2;              // scale * log2(e)
  AttendRecord* rec;         // [ctas]
  float4* top;               // [ctas][2][NC]: m, M, sum
  float* part;               // [ctas][2][NC][D]
};

cudaError_t launch_attend_split_bf16_64(const AttendArgs& a, int nt, int ctas, cudaStream_t st);
cudaError_t launch_attend_split_bf16_128(const AttendArgs& a, int nt, int ctas, cudaStream_t st);
cudaError_t launch_attend_split_f32_64(const AttendArgs& a, int nt, int ctas, cudaStream_t st);
cudaError_t launch_attend_split_f32_128(const AttendArgs& a, int nt, int ctas, cudaStream_t st);
cudaError_t launch_attend_prompt(const AttendArgs& a, int D, int ctas, cudaStream_t st);
cudaError_t take_faults_attend_prompt(unsigned int* bits);
cudaError_t take_faults_attend_bf16_64(unsigned int* bits);
cudaError_t take_faults_attend_bf16_128(unsigned int* bits);
cudaError_t take_faults_attend_f32_64(unsigned int* bits);
cudaError_t take_faults_attend_f32_128(unsigned int* bits);

#ifdef TQ_INT8_SPLIT      // the kernels, for the units that hold them
namespace {

constexpr float kNone = -3.4e38f;     // a maximum before the first logit
constexpr float kSlack = 8.0f, kLift = 7.0f;

// The visible slots of a sequence's columns.
struct Plan {
  Run r;
  int ncb;                   // units of a head
  int64_t quads;             // of a unit, at most
};

template <int NC>
__device__ __forceinline__ Plan plan_of(const AttendArgs& a, int b) {
  Plan p;
  p.r = run_of(a.step, b);
  if (p.r.count == 0) return {p.r, 0, 0};
  p.ncb = static_cast<int>((static_cast<int64_t>(p.r.count) * a.G + NC - 1) / NC);
  const int64_t cap = static_cast<int64_t>(a.c.max_pages) << a.c.shift;
  int64_t end = static_cast<int64_t>(p.r.len) + p.r.count;
  if (end > cap) {
    atomicOr(&g_wait_fault, static_cast<unsigned int>(kFaultPaged));
    end = cap;
  }
  int64_t tiles = (end + kTileSlots - 1) / kTileSlots;
  if (a.window > 0) {
    // a column block's tokens see a stretch of window + tokens - 1 slots
    const int64_t tokens = min((NC - 1) / a.G + 2, p.r.count);
    const int64_t most = (a.sinks + static_cast<int64_t>(kTileSlots) - 1) / kTileSlots + (a.window + tokens - 2) / kTileSlots + 2;
    tiles = min(tiles, most);
  }
  p.quads = max((tiles + kQuadTiles - 1) / kQuadTiles, static_cast<int64_t>(1));
  return p;
}

// The tiles of one unit: `sunk` of the sinks, then from slot tile `from` on.
struct Span {
  int t0, t1;                // tokens of the run
  int lo, hi;                // slots seen by any column: [lo, hi], and those below sinks
  int sunk, from, tiles;
};

template <int NC>
__device__ __forceinline__ Span span_of(const AttendArgs& a, const Run& r, int cb) {
  Span s;
  s.t0 = static_cast<int>(static_cast<int64_t>(cb) * NC / a.G);
  s.t1 = static_cast<int>(min((static_cast<int64_t>(cb) * NC + NC - 1) / a.G, static_cast<int64_t>(r.count - 1)));
  const int64_t cap = static_cast<int64_t>(a.c.max_pages) << a.c.shift;
  s.hi = static_cast<int>(min(static_cast<int64_t>(r.len) + s.t1, cap - 1));
  s.lo = a.window > 0 ? max(0, r.len + s.t0 - a.window + 1) : 0;
  s.from = min(s.lo, s.hi + 1) / kTileSlots;
  s.sunk = min((min(a.sinks, s.hi + 1) + kTileSlots - 1) / kTileSlots, s.from);
  if (a.window <= 0) s.sunk = 0;
  // where the window lies beyond the table (lo > hi) the last tile may still hold first slots
  s.tiles = s.sunk + max(0, s.hi / kTileSlots - s.from + 1);
  return s;
}

// A block's share of all quads: [x, x1), from quad pos of sequence b on.
template <int kWarps>
struct ShareScan {
  int64_t sums[kWarps];
  int64_t base;
  int b;
  Plan plan;
};

template <int NC, int kWarps>
struct Share {
  int64_t chunk, x, x1, pos;
  int b;
  Plan plan;

  // The quads of all sequences are counted (as many at a time as there are threads), then the sequence that the share starts in
  // is looked for.  All threads of the block take part; false, and the record says so, where nothing is left.
  __device__ __forceinline__ bool find(const AttendArgs& a, ShareScan<kWarps>& scan) {
    constexpr int kAt = kWarps * 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = a.step.B;
    int64_t own, upto;              // quads of this thread's sequence; of those up to it, within the round
    auto count = [&](int b0) {
      own = 0;
      if (b0 + tid < B) {
        plan = plan_of<NC>(a, b0 + tid);
        own = plan.quads * plan.ncb * a.c.H;
      }
      upto = own;
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      __syncthreads();
      if (lane == 31) scan.sums[warp] = upto;
      __syncthreads();
      int64_t sum = 0;
      for (int i = 0; i < kWarps; ++i) {
        if (i < warp) upto += scan.sums[i];
        sum += scan.sums[i];
      }
      return sum;
    };
    int64_t sum0 = count(0), all = sum0;
    for (int b0 = kAt; b0 < B; b0 += kAt) all += count(b0);
    chunk = (all + gridDim.x - 1) / gridDim.x;
    x = chunk * blockIdx.x;
    x1 = min(x + chunk, all);
    if (x >= x1) {
      if (tid == 0) a.rec[blockIdx.x].off = 0;
      return false;
    }
    int64_t base = 0;
    for (int b0 = 0;; b0 += kAt) {
      if (B > kAt) sum0 = count(b0);
      const int64_t lo = base + upto - own;
      if (lo <= x && x < lo + own) {
        scan.b = b0 + tid;
        scan.base = lo;
        scan.plan = plan;
      }
      base += sum0;
      if (base > x) break;          // the same for all threads
    }
    __syncthreads();
    b = scan.b;
    plan = scan.plan;
    pos = x - scan.base;
    return true;
  }

  // The sequence, head and column block at pos: quads [qa, qe) of the unit are this share's.
  __device__ __forceinline__ void unit(const AttendArgs& a, int& h, int& cb, int64_t& qa, int64_t& qe) {
    while (pos >= plan.quads * plan.ncb * a.c.H) {
      pos -= plan.quads * plan.ncb * a.c.H;
      plan = plan_of<NC>(a, ++b);
    }
    const int64_t u = pos / plan.quads;
    qa = pos - u * plan.quads;
    qe = min(plan.quads, qa + (x1 - x));
    h = static_cast<int>(u / plan.ncb);
    cb = static_cast<int>(u - static_cast<int64_t>(h) * plan.ncb);
  }
  __device__ __forceinline__ void advance(int64_t quads) {
    x += quads;
    pos += quads;
  }
  __device__ __forceinline__ AttendRecord record(int h, int cb, int64_t qa) const {
    return {static_cast<int>(min(chunk, static_cast<int64_t>(1) << 30)), static_cast<int>(qa), static_cast<int>(plan.quads),
            plan.r.first, plan.r.count, h, cb, static_cast<int>(blockIdx.x)};
  }
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

__device__ __forceinline__ void mma(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ float exp2_fast(float x) {      // 2 steps of fp32, zero below 2^-126
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }

// Two codes of `w` as fp16 whole numbers from -128 to 127: bytes `sel` placed below 0x64.
__device__ __forceinline__ uint32_t whole(uint32_t w, uint32_t sel) {
  const uint32_t v = __byte_perm(w, 0x64646464u, sel);
  const uint32_t bias = 0x64806480u;      // 1152
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&bias));
  return *reinterpret_cast<const uint32_t*>(&h);
}


template <typename T, int D, int NT>
struct Shape {
  static constexpr bool kF32 = sizeof(T) == 4;
  static constexpr int NC = 8 * NT, kParts = kF32 ? 2 : 1, kSteps = D / 16, kTiles = D / 16;
  static constexpr int kStep = NT <= 2 ? 2 : 1;                        // blocks of 16 slots taken at a time
  static constexpr int kBlocks = attend_blocks(kF32, D, NT), kStages = kBlocks == 3 && D == 128 ? 2 : 3;
  static constexpr bool kQReg = NT * kParts <= 2;                      // the queries' operand in registers, or in shared memory
  static constexpr int kRow = kBlockSlots * D;                         // bytes of a block of 16 rows
  static constexpr int kStage = 4 * kRow;                              // keys' two blocks, values' two blocks
  static constexpr int kRing = kAttendWarps * kStages * kStage;
  static constexpr int kQBytes = kQReg ? 0 : kSteps * NT * kParts * 256;
  static constexpr int kJoin = kAttendWarps * NC * D * 4;
  static constexpr int kBytes = (kRing > kJoin ? kRing : kJoin) + kQBytes;
};

// Where float pair i (dimensions 2 i, 2 i + 1) of a column lies in the join's rows: the four lanes of a row and the
// rows of a store fall on different banks.
template <int D>
__device__ __forceinline__ int join_at(int col, int i) {
  constexpr int kPer = D / 16;                 // pairs of a lane's row
  const int g = i / kPer, t = (col >> 1) & 3;
  return g * kPer + ((i % kPer) ^ (kPer == 8 ? ((g >> 1) & 1) | (t << 1) : t));
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kAttendWarps * 32, (attend_blocks(sizeof(T) == 4, D, NT))) attend_split_kernel(const AttendArgs a) {
  using S = Shape<T, D, NT>;
  constexpr int NC = S::NC, MT = S::kTiles, kStages = S::kStages;
  extern __shared__ __align__(128) char smem[];
  __shared__ ShareScan<kAttendWarps> scan;
  __shared__ float4 stage_ex[kAttendWarps][kStages];      // of the two blocks: 2^(key's exponent), 0 for an absent one; value's exponent
  __shared__ float3 warp_top[kAttendWarps][NC];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int H = a.c.H;

  Share<NC, kAttendWarps> share;
  if (!share.find(a, scan)) return;
  const Plan& plan = share.plan;
  const int& b = share.b;

  const uint32_t ring = smem_addr(smem) + warp * kStages * S::kStage;
  const uint32_t q_area = smem_addr(smem) + S::kBytes - S::kQBytes;
  // lane offsets within a block of 16 rows: copies, keys, values
  const int swap_w = D == 128 ? (((lane >> 3) >> 1 & 1) << 1) ^ (((lane >> 3) & 1) << 2) : (lane >> 3) << 1;
  const uint32_t to_a = (lane >> 3) * 128 + (((lane & 7) ^ swap_w) << 4);
  const uint32_t to_b = D == 128 ? to_a ^ 64 : to_a;
  const int swap_k = D == 128 ? ((g >> 1 & 3) << 1) ^ ((g & 1) << 2) : (g >> 1 & 3) << 1;
  const uint32_t k_at = D == 128 ? g * 128 : (g >> 1) * 128;
  const int k_chunk = D == 128 ? t : (g & 1) * 4 + t;

  bool begun = false;
  while (share.x < share.x1) {
    int h, cb;
    int64_t qa, qe;
    share.unit(a, h, cb, qa, qe);
    const Span sp = span_of<NC>(a, plan.r, cb);
    const Run run = plan.r;
    if (tid == 0 && !begun) a.rec[blockIdx.x] = share.record(h, cb, qa);
    begun = true;

    // ---- the warp's tiles: 4 q + warp for quads q in [qa, qe)
    const int n = max(0, static_cast<int>(min(qe, (static_cast<int64_t>(sp.tiles) - warp + 3) / 4) - qa));
    const int j0 = static_cast<int>(4 * qa) + warp;
    int blk0 = -1, blk1 = -1;
    float4 ex;
    auto slot_of = [&](int i) {
      const int j = j0 + 4 * i;
      return (j < sp.sunk ? j : j - sp.sunk + sp.from) * kTileSlots;
    };
    auto block_of = [&](int s) {
      if (s > sp.hi || !(s + kBlockSlots > sp.lo || s < a.sinks)) return -1;
      const int pg = a.c.page(b, s);
      return pg < 0 ? -1 : static_cast<int>(a.c.row(pg, h, s) / kBlockSlots);
    };
    auto issue = [&](int i) {
      if ((i & 31) == 0) {      // a lane looks up one tile of the next 32
        blk0 = blk1 = -1;
        ex = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (i + lane < n) {
          const int s = slot_of(i + lane);
          blk0 = block_of(s);
          blk1 = block_of(s + kBlockSlots);
          char2 e0 = make_char2(0, 0), e1 = e0;
          if (blk0 >= 0) e0 = *reinterpret_cast<const char2*>(a.c.ex + 2 * static_cast<size_t>(blk0));
          if (blk1 >= 0) e1 = *reinterpret_cast<const char2*>(a.c.ex + 2 * static_cast<size_t>(blk1));
          auto cut = [](int e) { return min(max(e, kExpLow), kExpHigh); };
          ex.x = blk0 >= 0 ? pow2(cut(e0.x)) : 0.0f;
          ex.y = blk1 >= 0 ? pow2(cut(e1.x)) : 0.0f;
          ex.z = static_cast<float>(cut(e0.y));
          ex.w = static_cast<float>(cut(e1.y));
        }
      }
      if (i < n) {
        const int stage = i % kStages;
        const int p0 = __shfl_sync(0xffffffffu, blk0, i & 31), p1 = __shfl_sync(0xffffffffu, blk1, i & 31);
        const uint32_t to = ring + stage * S::kStage;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int p = k ? p1 : p0;
          if (p >= 0) {
            const size_t at = static_cast<size_t>(p) * S::kRow + lane * 16;
#pragma unroll
            for (int i2 = 0; i2 < S::kRow / 512; ++i2) {
              copy16(to + k * S::kRow + i2 * 512 + (i2 & 1 ? to_b : to_a), a.c.kc + at + i2 * 512);
              copy16(to + (2 + k) * S::kRow + i2 * 512 + (i2 & 1 ? to_b : to_a), a.c.vc + at + i2 * 512);
            }
          }
        }
        if (lane == (i & 31)) stage_ex[warp][stage] = ex;      // behind the copies: it waits for the exponents
      }
      commit();
    };
    __syncthreads();              // the ring has been the last unit's join
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i);

    // ---- queries: lane (g, t) holds column g of each 8 at dimensions 64 k + 16 t .. + 15
    uint32_t qf[S::kQReg ? S::kSteps * NT * S::kParts * 2 : 1];
    float half_sum[NT][2], factor[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int64_t col = static_cast<int64_t>(cb) * NC + nt * 8 + g;
      const int token = static_cast<int>(col / a.G), head = static_cast<int>(col - static_cast<int64_t>(token) * a.G);
      const bool there = col < static_cast<int64_t>(run.count) * a.G;
      float q[D / 64][16];
      float most = 0.0f, sum = 0.0f;
#pragma unroll
      for (int k = 0; k < D / 64; ++k) {
        const T* from = static_cast<const T*>(a.Q) + ((static_cast<size_t>(run.first) + token) * H * a.G + static_cast<size_t>(h) * a.G + head) * D + 64 * k + 16 * t;
        if constexpr (S::kF32) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 v = there ? *reinterpret_cast<const float4*>(from + 4 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
            q[k][4 * i] = v.x; q[k][4 * i + 1] = v.y; q[k][4 * i + 2] = v.z; q[k][4 * i + 3] = v.w;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4 v = there ? *reinterpret_cast<const uint4*>(from + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              q[k][8 * i + 2 * j] = __uint_as_float(u[j] << 16);
              q[k][8 * i + 2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) most = fmaxf(most, fabsf(q[k][i]));
      }
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
      // times 2^x the largest lies in [2^14, 2^15)
      const int x2 = most > 0.0f ? min(141 - static_cast<int>(__float_as_uint(most) >> 23), 120) : 0;
      const float up = pow2(x2);
#pragma unroll
      for (int k = 0; k < D / 64; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] = q[k][4 * j + i] * up;
            sum += v[i];
          }
          uint32_t f0 = pack(v[0], v[1]), f1 = pack(v[2], v[3]);
#pragma unroll
          for (int part = 0; part < S::kParts; ++part) {
            if (part == 1) {
              const float2 r0 = unpack(f0), r1 = unpack(f1);
              f0 = pack(v[0] - r0.x, v[1] - r0.y);
              f1 = pack(v[2] - r1.x, v[3] - r1.y);
            }
            const int at = ((k * 4 + j) * NT + nt) * S::kParts + part;
            if constexpr (S::kQReg) {
              qf[2 * at] = f0;
              qf[2 * at + 1] = f1;
            } else if (warp == 0) {
              *reinterpret_cast<uint2*>(smem + S::kBytes - S::kQBytes + at * 256 + lane * 8) = make_uint2(f0, f1);
            }
          }
        }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const float fac = a.scale2 * pow2(-x2);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        half_sum[nt][i] = 0.5f * __shfl_sync(0xffffffffu, sum, 8 * t + 4 * i);
        factor[nt][i] = __shfl_sync(0xffffffffu, fac, 8 * t + 4 * i);
      }
    }
    if constexpr (!S::kQReg) __syncthreads();

    float acc[MT][NT][4], m[NT][2], M[NT][2], sum[NT][2], W[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) { m[nt][i] = M[nt][i] = kNone; sum[nt][i] = W[nt][i] = 0.0f; }
#pragma unroll
      for (int k = 0; k < MT; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[k][nt][i] = 0.0f;
    }
    // slots that every column sees, but for the sinks: (all_lo, all_hi]
    const int all_hi = run.len + sp.t0, all_lo = a.window > 0 ? run.len + sp.t1 - a.window : -1;

    for (int i = 0; i < n; ++i) {
      __syncwarp();               // the stage that is filled next has been read by all lanes
      issue(i + kStages - 1);
      wait_copies<kStages - 1>();
      __syncwarp();
      const int stage = i % kStages, s0 = slot_of(i);
      const uint32_t at = ring + stage * S::kStage;
      const float4 e2 = stage_ex[warp][stage];
      const bool plain = e2.x != 0.0f && e2.y != 0.0f && s0 + kTileSlots - 1 <= all_hi && (s0 > all_lo || s0 + kTileSlots <= a.sinks);
#pragma unroll
      for (int kb0 = 0; kb0 < 2; kb0 += S::kStep) {
        float z[S::kStep][NT][4];
        // ---- logits
#pragma unroll
        for (int kb = 0; kb < S::kStep; ++kb) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) z[kb][nt][c] = 0.0f;
          const uint32_t ka = at + (kb0 + kb) * S::kRow + k_at;
#pragma unroll
          for (int k = 0; k < D / 64; ++k) {
            const uint32_t piece = static_cast<uint32_t>((k_chunk + 4 * k) ^ swap_k) << 4;
            const uint4 r0 = lds128(ka + piece), r8 = lds128(ka + piece + S::kRow / 2);
            const uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w8[4] = {r8.x, r8.y, r8.z, r8.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t a0 = whole(w0[j], 0x4140), a1 = whole(w8[j], 0x4140), a2 = whole(w0[j], 0x4342), a3 = whole(w8[j], 0x4342);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int part = 0; part < S::kParts; ++part) {
                  const int qi = ((k * 4 + j) * NT + nt) * S::kParts + part;
                  if constexpr (S::kQReg) {
                    mma(z[kb][nt], a0, a1, a2, a3, qf[2 * qi], qf[2 * qi + 1]);
                  } else {
                    const uint2 qv = lds64(q_area + qi * 256 + lane * 8);
                    mma(z[kb][nt], a0, a1, a2, a3, qv.x, qv.y);
                  }
                }
            }
          }
        }
        // ---- weights
        float top[NT][2], topv[NT][2];
        bool over = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) top[nt][0] = top[nt][1] = topv[nt][0] = topv[nt][1] = -INFINITY;
#pragma unroll
        for (int kb = 0; kb < S::kStep; ++kb) {
          const float ek = kb0 + kb ? e2.y : e2.x, ev = kb0 + kb ? e2.w : e2.z;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int c = 0; c < 4; ++c) z[kb][nt][c] = (z[kb][nt][c] + half_sum[nt][c & 1]) * (factor[nt][c & 1] * ek);
            if (!plain) {
#pragma unroll
              for (int i2 = 0; i2 < 2; ++i2) {
                const int64_t col = static_cast<int64_t>(cb) * NC + nt * 8 + 2 * t + i2;
                const int own = run.len + static_cast<int>(col / a.G);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  const int s = s0 + (kb0 + kb) * kBlockSlots + g + 8 * r;
                  const bool seen = ek != 0.0f && s <= own && (a.window <= 0 || s > own - a.window || s < a.sinks);
                  if (!seen) z[kb][nt][2 * r + i2] = -INFINITY;
                }
              }
            }
#pragma unroll
            for (int i2 = 0; i2 < 2; ++i2) {
              const float v = fmaxf(z[kb][nt][i2], z[kb][nt][2 + i2]);
              top[nt][i2] = fmaxf(top[nt][i2], v);
              topv[nt][i2] = fmaxf(topv[nt][i2], v + ev);
            }
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i2 = 0; i2 < 2; ++i2) over |= top[nt][i2] > m[nt][i2] + kSlack || topv[nt][i2] > M[nt][i2] + kSlack;
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i2 = 0; i2 < 2; ++i2) {
              float u = fmaxf(top[nt][i2], m[nt][i2]), v = fmaxf(topv[nt][i2], M[nt][i2]);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) {
                u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, o));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
              }
              const float fm = exp2_fast(m[nt][i2] - u), fv = exp2_fast(M[nt][i2] - v);
              m[nt][i2] = u;
              M[nt][i2] = v;
              sum[nt][i2] *= fm;
              W[nt][i2] *= fv;
#pragma unroll
              for (int k = 0; k < MT; ++k) {
                acc[k][nt][i2] *= fv;
                acc[k][nt][2 + i2] *= fv;
              }
            }
        }
        uint32_t wf[S::kStep][NT][S::kParts][2];
#pragma unroll
        for (int kb = 0; kb < S::kStep; ++kb)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float w[2];
#pragma unroll
              for (int i2 = 0; i2 < 2; ++i2) {
                const float v = z[kb][nt][2 * r + i2];
                sum[nt][i2] += exp2_fast(v - m[nt][i2]);
                w[i2] = exp2_fast(v + ((kb0 + kb ? e2.w : e2.z) + kLift - M[nt][i2]));
                W[nt][i2] += w[i2];
              }
              const uint32_t hi = pack(w[0], w[1]);
              wf[kb][nt][0][r] = transposed(hi);
              if constexpr (S::kF32) {
                const float2 back = unpack(hi);
                wf[kb][nt][1][r] = transposed(pack(w[0] - back.x, w[1] - back.y));
              }
            }
        // ---- sums of values: fp32 outputs sum each step's products by themselves and add them with a rounding
        constexpr int kGroup = D / 32;           // words of a lane's dimensions in a row
        uint32_t v0[S::kStep][kGroup], v1[S::kStep][kGroup], v8[S::kStep][kGroup], v9[S::kStep][kGroup];
#pragma unroll
        for (int kb = 0; kb < S::kStep; ++kb) {
          const uint32_t va = at + (2 + kb0 + kb) * S::kRow;
          if constexpr (D == 128) {
            const uint32_t o0 = 2 * t * 128 + ((g ^ (t << 1)) << 4), o1 = (2 * t + 1) * 128 + ((g ^ (t << 1) ^ 4) << 4);
            const uint4 r0 = lds128(va + o0), r1 = lds128(va + o1), r8 = lds128(va + o0 + 1024), r9 = lds128(va + o1 + 1024);
            v0[kb][0] = r0.x; v0[kb][1] = r0.y; v0[kb][2] = r0.z; v0[kb][3] = r0.w;
            v1[kb][0] = r1.x; v1[kb][1] = r1.y; v1[kb][2] = r1.z; v1[kb][3] = r1.w;
            v8[kb][0] = r8.x; v8[kb][1] = r8.y; v8[kb][2] = r8.z; v8[kb][3] = r8.w;
            v9[kb][0] = r9.x; v9[kb][1] = r9.y; v9[kb][2] = r9.z; v9[kb][3] = r9.w;
          } else {
            const uint32_t o0 = t * 128 + (((g >> 1) ^ (t << 1)) << 4) + (g & 1) * 8, o1 = t * 128 + (((4 + (g >> 1)) ^ (t << 1)) << 4) + (g & 1) * 8;
            const uint2 r0 = lds64(va + o0), r1 = lds64(va + o1), r8 = lds64(va + o0 + 512), r9 = lds64(va + o1 + 512);
            v0[kb][0] = r0.x; v0[kb][1] = r0.y;
            v1[kb][0] = r1.x; v1[kb][1] = r1.y;
            v8[kb][0] = r8.x; v8[kb][1] = r8.y;
            v9[kb][0] = r9.x; v9[kb][1] = r9.y;
          }
        }
#pragma unroll
        for (int j = 0; j < kGroup; ++j)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float fresh[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 4; ++c) fresh[nt][c] = 0.0f;
#pragma unroll
            for (int kb = 0; kb < S::kStep; ++kb) {
              const uint32_t both0 = __byte_perm(v0[kb][j], v1[kb][j], half ? 0x7362 : 0x5140), both8 = __byte_perm(v8[kb][j], v9[kb][j], half ? 0x7362 : 0x5140);
              const uint32_t a0 = whole(both0, 0x4140), a1 = whole(both0, 0x4342), a2 = whole(both8, 0x4140), a3 = whole(both8, 0x4342);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int part = 0; part < S::kParts; ++part)
                  mma(S::kF32 ? fresh[nt] : acc[2 * j + half][nt], a0, a1, a2, a3, wf[kb][nt][part][0], wf[kb][nt][part][1]);
            }
            if constexpr (S::kF32) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[2 * j + half][nt][c] += fresh[nt][c];
            }
          }
      }
    }
    wait_copies<0>();

    // ---- the warps' sums joined
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i2 = 0; i2 < 2; ++i2) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          sum[nt][i2] += __shfl_xor_sync(0xffffffffu, sum[nt][i2], o);
          W[nt][i2] += __shfl_xor_sync(0xffffffffu, W[nt][i2], o);
        }
        if (g == 0) warp_top[warp][nt * 8 + 2 * t + i2] = make_float3(m[nt][i2], M[nt][i2], sum[nt][i2]);
      }
    __syncthreads();              // all rings have been read
    float2* join = reinterpret_cast<float2*>(smem);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i2 = 0; i2 < 2; ++i2) {
        const int col = nt * 8 + 2 * t + i2;
#pragma unroll
        for (int k = 0; k < MT; ++k)
          join[(warp * NC + col) * (D / 2) + join_at<D>(col, g * (D / 16) + k)] =
              make_float2(fmaf(0.5f, W[nt][i2], acc[k][nt][i2]), fmaf(0.5f, W[nt][i2], acc[k][nt][2 + i2]));
      }
    __syncthreads();
    const bool entire = qa == 0 && qe == plan.quads;
    const size_t place = (static_cast<size_t>(blockIdx.x) * 2 + (qa == 0 ? 1 : 0)) * NC;
    const int columns = static_cast<int>(min(static_cast<int64_t>(NC), static_cast<int64_t>(run.count) * a.G - static_cast<int64_t>(cb) * NC));
    for (int i = tid; i < columns * (D / 2); i += kAttendWarps * 32) {
      const int col = i / (D / 2), pair = i % (D / 2);
      float mt = kNone, Mt = kNone;
#pragma unroll
      for (int w = 0; w < kAttendWarps; ++w) {
        mt = fmaxf(mt, warp_top[w][col].x);
        Mt = fmaxf(Mt, warp_top[w][col].y);
      }
      float l = 0.0f;
      float2 o = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kAttendWarps; ++w) {
        const float3 tp = warp_top[w][col];
        l = fmaf(tp.z, exp2_fast(tp.x - mt), l);
        const float f = exp2_fast(tp.y - Mt);
        const float2 v = join[(w * NC + col) * (D / 2) + join_at<D>(col, pair)];
        o.x = fmaf(v.x, f, o.x);
        o.y = fmaf(v.y, f, o.y);
      }
      if (entire) {
        const float f = l == 0.0f ? 0.0f : 1.0f / l, up = exp2f(Mt - mt - kLift);
        const int64_t cc = static_cast<int64_t>(cb) * NC + col;
        const int token = static_cast<int>(cc / a.G), head = static_cast<int>(cc - static_cast<int64_t>(token) * a.G);
        T* to = static_cast<T*>(a.out) + ((static_cast<size_t>(run.first) + token) * H * a.G + static_cast<size_t>(h) * a.G + head) * D + 2 * pair;
        o.x = l == 0.0f ? 0.0f : o.x * f * up;
        o.y = l == 0.0f ? 0.0f : o.y * f * up;
        if constexpr (S::kF32) *reinterpret_cast<float2*>(to) = o;
        else *reinterpret_cast<__nv_bfloat162*>(to) = __floats2bfloat162_rn(o.x, o.y);
      } else {
        if (pair == 0) a.top[place + col] = make_float4(mt, Mt, l, 0.0f);
        *reinterpret_cast<float2*>(a.part + (place + col) * D + 2 * pair) = o;
      }
    }
    share.advance(qe - qa);
  }
}

template <typename T, int D, int NT>
cudaError_t launch_split(const AttendArgs& a, int ctas, cudaStream_t st) {
  using S = Shape<T, D, NT>;
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(attend_split_kernel<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_acq_rel);
  }
  attend_split_kernel<T, D, NT><<<ctas, kAttendWarps * 32, S::kBytes, st>>>(a);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_split_of(const AttendArgs& a, int nt, int ctas, cudaStream_t st) {
  return nt == 1 ? launch_split<T, D, 1>(a, ctas, st) : nt == 2 ? launch_split<T, D, 2>(a, ctas, st) : launch_split<T, D, 4>(a, ctas, st);
}

}  // namespace
#endif

}  // namespace tq
