// The split of tq_attend_int8 for pieces of prompts (bf16 queries, more columns a sequence than the warp-wide form takes):
// 256 columns a unit, products on tcgen05.
//
// Mathematics as in tq_int8_split.cuh, with the columns as rows: S = Q K^T (128 x 128 a tile, fp16 operands, fp32 sums in
// tensor memory), a thread owns a column, so that maxima and sums need no exchange.  Keys are the whole numbers c, values
// 2 c + 1, odd below 256 and exact in fp16, which saves the sum of weights.  The weights of 16 slots are p times
// one factor 2^(e - M + m).
//
// What bounds it: a tile of 128 slots is 2 x 2 products of 128 x 128 x D (2048 cycles of the tensor core for D = 128)
// and 32768 exponentials (2048 cycles at 16 a cycle).  What it takes is the way of one half from its logits to its next
// ones, some 4900 cycles: 1100 to 1500 for the maxima, 1900 to 2200 for the weights, the rest for the two products with the
// barriers between; the other half's runs beside it and the tensor core is busy for 34 % of them.  256 columns share a conversion of
// the codes (1000 cycles for keys, 700 for values).  1021 tokens over 8192 slots, 32 heads on 8: 187 us with the join (8), 690 TFLOP/s;
// the warp-wide form 700 us.  From an empty cache, where shares are uneven, 8192 tokens take 1.13 ms, 480 TFLOP/s.
// Weights with the maxima so far, kept in registers until they are known to hold, would read the logits once: slower by
// a fifth, as registers no longer suffice; so is one lane that waits and arrives for its warp.
//
// Warps: 0-3 and 4-7 the two halves' columns (weights, rescaling, output), 8-11 bring the codes from memory and lay them
// out as operands (128-byte swizzle; keys with the dimension, values with the slot as the outer index), 12 issues the
// products (13-15 only give up registers: 144 a thread for the columns, 112 for the others, 65536 in all; with fewer for the
// others their loops spill).  Weights go to tensor memory over the logits that they come from and are read there as an operand.
// Two stages of keys and of values; the next tile's codes are on their way in registers while a stage is waited for.  What is to be
// known of 16 tiles is a batch in a ring of four, which both halves follow and give back, with columns in the unit or without.
//
// Every wait gives up after the library's budget: the block then writes NaN for what it has not done, sets fault bit 128,
// lets the products in flight end, frees its tensor memory and returns.
#define TQ_INT8_SPLIT
#include "tq_int8_split.cuh"

namespace tq {
namespace {

constexpr int kHalf = 128, kNC = 2 * kHalf, kTileKeys = 128, kBatch = 16;
constexpr int kWarps = 16, kThreads = kWarps * 32, kMakers = 128;
constexpr unsigned int kFaultAttendWait = 128u;

__device__ __forceinline__ void bar_init(uint32_t bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void commit_to(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void operands_written() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 128-byte swizzle, rows of 128 bytes, 8 rows (1024 bytes) to the next group; `lbo` bytes to the next 64 columns of an operand
// whose columns are its outer index.
__device__ __forceinline__ uint64_t operand(uint32_t saddr, uint32_t lbo) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// fp16 operands, fp32 sums, 128 rows
__device__ __forceinline__ constexpr uint32_t shape_of(int N, bool b_outer) {
  return (1u << 4) | (b_outer ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(kHalf >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t shape, bool add) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a),
               "l"(b), "r"(shape), "r"(static_cast<uint32_t>(add))
               : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t shape, bool add) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a),
               "l"(b), "r"(shape), "r"(static_cast<uint32_t>(add))
               : "memory");
}
// The load is under way until tmem_loaded(), which its values have to pass.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
      "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]),
        "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]),
        "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]),
        "=f"(v[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_loaded(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]),
                 "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]),
                 "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]),
                 "+f"(v[28]));
  asm volatile("" : "+f"(v[29]), "+f"(v[30]), "+f"(v[31]));
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]),
        "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_loaded(float (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]),
                 "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
      "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two fp32 values an instruction.
__device__ __forceinline__ uint64_t two(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float2 apart(uint64_t v) {
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// What the columns' threads need of a tile's eight blocks: first slot, 2^(key's exponent) (0: absent), value's exponent.
struct alignas(16) BlockInfo {
  int slot;
  float ek, ev;
  int blk;
};
// Of all eight: lowest slot, highest (2^31 - 1 unless all are there), least and largest exponent of the values.
struct alignas(16) TileInfo {
  int lo, hi;
  float ev_lo, ev_hi;
};

template <int D>
struct PromptShape {
  static constexpr int kSide = kTileKeys * D * 2;          // bytes of an operand of 128 rows
  static constexpr int kPart = kTileKeys * 128;            // of its 64 columns
  static constexpr int kQ = 0, kK = 2 * kSide, kV = 4 * kSide, kBytes = 6 * kSide + 1024;
  static constexpr int kInfo = 4;                          // batches of block infos alive
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attend_prompt_kernel(const AttendArgs a) {
  using P = PromptShape<D>;
  extern __shared__ char smem_raw[];
  __shared__ ShareScan<kWarps> scan;
  __shared__ BlockInfo info[P::kInfo][kBatch * 8];
  __shared__ TileInfo tile_info[P::kInfo][kBatch];
  __shared__ __align__(8) uint64_t bars[25];
  __shared__ uint32_t tmem_slot;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  char* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const uint32_t base = smem_addr(smem);
  // barriers: keys full / free, values full / free (2 stages each), queries, logits, weights, products done (2 halves each),
  // infos full / free (4 each)
  const uint32_t bar0 = smem_addr(bars);
  const uint32_t k_full = bar0, k_free = bar0 + 16, v_full = bar0 + 32, v_free = bar0 + 48, q_full = bar0 + 64, s_full = bar0 + 80,
                 p_full = bar0 + 96, o_done = bar0 + 112, info_full = bar0 + 128, info_free = bar0 + 160, drained = bar0 + 192;

  Share<kNC, kWarps> share;
  if (!share.find(a, scan)) return;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      bar_init(k_full + 8 * i, kMakers);
      bar_init(k_free + 8 * i, 1);
      bar_init(v_full + 8 * i, kMakers);
      bar_init(v_free + 8 * i, 1);
      bar_init(q_full + 8 * i, kHalf);
      bar_init(s_full + 8 * i, 1);
      bar_init(p_full + 8 * i, kHalf);
      bar_init(o_done + 8 * i, 1);
    }
    bar_init(drained, 1);
    for (int i = 0; i < P::kInfo; ++i) {
      bar_init(info_full + 8 * i, kMakers);
      bar_init(info_free + 8 * i, 8);      // a lane of each of the columns' warps
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  before_sync();
  __syncthreads();
  after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);      // logits (and weights) of the halves at 0 and 128, sums at 256 and 384

  bool lost = false, begun = false;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (!lost) lost = !wait_parity_bounded(bar, parity & 1, kFaultAttendWait);
  };
  // A wait that ran out is the whole warp's: its lanes stay together for the votes and exchanges that follow.
  auto wait_all = [&](uint32_t bar, uint32_t parity) {
    wait(bar, parity);
    lost = __any_sync(0xffffffffu, lost);
  };
  uint32_t tiles_done = 0, batches_done = 0, units_done[2] = {0, 0}, half_tiles[2] = {0, 0};

  // The roles go through the same units, each in a loop of its own: registers are dealt out anew between them.
  int h, cb, b, columns, halves, n;
  int64_t qa, qe;
  Run run;
  Span sp;
  auto begin = [&]() {
    if (share.x >= share.x1) return false;
    share.unit(a, h, cb, qa, qe);
    run = share.plan.r;
    sp = span_of<kNC>(a, run, cb);
    b = share.b;
    if (tid == 0 && !begun) a.rec[blockIdx.x] = share.record(h, cb, qa);
    begun = true;
    columns = static_cast<int>(min(static_cast<int64_t>(kNC), static_cast<int64_t>(run.count) * a.G - static_cast<int64_t>(cb) * kNC));
    halves = columns > kHalf ? 2 : 1;
    n = max(0, static_cast<int>(min(qe, static_cast<int64_t>((sp.tiles + 3) / 4)) - qa));
    return true;
  };
  auto end = [&]() {
    __syncwarp();
    tiles_done += n;
    batches_done += (n + kBatch - 1) / kBatch;
    for (int half = 0; half < halves; ++half) {
      units_done[half] += n > 0;
      half_tiles[half] += n;
    }
    share.advance(qe - qa);
  };

  if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 112;");
    while (begin()) {
      // ---- the products: the whole warp keeps step, so that operands stay in its uniform registers; one lane issues
      if (warp == 12 && n > 0) {
        auto logits = [&](int i, int half) {
          const uint64_t kd = operand(base + P::kK + ((tiles_done + i) & 1) * P::kSide, 16), qd = operand(base + P::kQ + half * P::kSide, 16);
          after_sync();
          if (elected()) {
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
              const uint32_t at = ((s >> 2) * P::kPart + (s & 3) * 32) >> 4;      // operands are below 2^18: no carry
              mma_ss(tmem + half * 128, qd + at, kd + at, shape_of(kTileKeys, false), s > 0);
            }
            commit_to(s_full + 8 * half);
            if (half == halves - 1) commit_to(k_free + 8 * ((tiles_done + i) & 1));
          }
          __syncwarp();
        };
        auto k_there = [&](int i) { wait_all(k_full + 8 * ((tiles_done + i) & 1), (tiles_done + i) >> 1); };
        k_there(0);
        for (int half = 0; half < halves; ++half) {
          wait_all(q_full + 8 * half, units_done[half]);
          if (!lost) logits(0, half);
        }
        for (int i = 0; i < n && !lost; ++i) {
          const uint64_t vd = operand(base + P::kV + ((tiles_done + i) & 1) * P::kSide, P::kPart);
          wait_all(v_full + 8 * ((tiles_done + i) & 1), (tiles_done + i) >> 1);
          for (int half = 0; half < halves; ++half) {
            wait_all(p_full + 8 * half, half_tiles[half] + i);
            if (lost) break;
            after_sync();
            if (elected()) {
#pragma unroll
              for (int s = 0; s < kTileKeys / 16; ++s)
                mma_ts(tmem + 256 + half * 128, tmem + half * 128 + s * 8, vd + s * 128, shape_of(D, true), i > 0 || s > 0);
              commit_to(o_done + 8 * half);
              if (half == halves - 1) commit_to(v_free + 8 * ((tiles_done + i) & 1));
            }
            __syncwarp();
            if (i + 1 < n) {
              if (half == 0) k_there(i + 1);
              if (lost) break;
              logits(i + 1, half);
            }
          }
        }
      }
      end();
    }
  } else if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 112;");
    while (begin()) {
      // ---- codes to operands
      const int me = tid - 256;
      constexpr int kPieces = D / 16, kAt = kMakers / kPieces, kIt = kTileKeys / kAt;      // 16-byte pieces a row, rows at a time, times
      // a quarter warp's stores: four pieces of 64 columns of two rows, which the swizzle spreads over all banks
      const int col = D == 128 ? (me & 3) | (me >> 3 & 1) << 2 : me & 3, sub = D == 128 ? (me >> 2 & 1) | (me >> 4) << 1 : me >> 2;
      for (int i = 0; i < n && !lost; ++i) {
        const uint32_t tile = tiles_done + i, stage = tile & 1, batch = batches_done + i / kBatch;
        if (i % kBatch == 0) {
          wait_all(info_free + 8 * (batch & 3), (batch >> 2) + 1);
          if (lost) break;
          BlockInfo& to = info[batch & 3][me];
          const int64_t q = qa + i + me / 8;
          const int j = static_cast<int>(4 * q) + (me & 7) / 2;
          BlockInfo f = {0, 0.0f, 0.0f, -1};
          if (i + me / 8 < n && j < sp.tiles) {
            f.slot = (j < sp.sunk ? j : j - sp.sunk + sp.from) * kTileSlots + (me & 1) * kBlockSlots;
            if (f.slot <= sp.hi && (f.slot + kBlockSlots > sp.lo || f.slot < a.sinks)) {
              const int pg = a.c.page(b, f.slot);
              if (pg >= 0) {
                f.blk = static_cast<int>(a.c.row(pg, h, f.slot) / kBlockSlots);
                const char2 e = *reinterpret_cast<const char2*>(a.c.ex + 2 * static_cast<size_t>(f.blk));
                f.ek = pow2(min(max(static_cast<int>(e.x), kExpLow), kExpHigh));
                f.ev = static_cast<float>(min(max(static_cast<int>(e.y), kExpLow), kExpHigh));
              }
            }
          }
          to = f;
          int lo = f.slot, hi = f.ek != 0.0f ? f.slot + kBlockSlots - 1 : INT32_MAX;
          float ev_lo = f.ev, ev_hi = f.ev;
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) {
            lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
            ev_lo = fminf(ev_lo, __shfl_xor_sync(0xffffffffu, ev_lo, o));
            ev_hi = fmaxf(ev_hi, __shfl_xor_sync(0xffffffffu, ev_hi, o));
          }
          if ((me & 7) == 0) tile_info[batch & 3][me / 8] = {lo, hi, ev_lo, ev_hi};
          arrive(info_full + 8 * (batch & 3));
          wait_all(info_full + 8 * (batch & 3), batch >> 2);
        }
        uint4 k[kIt], v[kIt];
#pragma unroll
        for (int r = 0; r < kIt; ++r) {
          const int row = r * kAt + sub;
          const int blk = info[batch & 3][(i % kBatch) * 8 + row / kBlockSlots].blk;
          k[r] = v[r] = make_uint4(0u, 0u, 0u, 0u);
          if (blk >= 0) {
            const size_t at = (static_cast<size_t>(blk) * kBlockSlots + row % kBlockSlots) * D + col * 16;
            k[r] = __ldg(reinterpret_cast<const uint4*>(a.c.kc + at));
            v[r] = __ldg(reinterpret_cast<const uint4*>(a.c.vc + at));
          }
        }
        // 16 codes are two 16-byte chunks; rows of a thread are a multiple of 8 apart
        auto put = [&](int side, int r, const uint32_t (&w)[8]) {
          const uint32_t to = base + side + stage * P::kSide + (col >> 2) * P::kPart + (r * kAt + sub) * 128;
          const uint32_t c0 = static_cast<uint32_t>((2 * col & 7) ^ (sub & 7)) << 4;
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + c0), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + (c0 ^ 16)), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
        };
        wait_all(k_free + 8 * stage, (tile >> 1) + 1);
        if (lost) break;
#pragma unroll
        for (int r = 0; r < kIt; ++r) {
          const uint32_t c[4] = {k[r].x, k[r].y, k[r].z, k[r].w};
          uint32_t w[8];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            w[2 * u] = whole(c[u], 0x4140);
            w[2 * u + 1] = whole(c[u], 0x4342);
          }
          put(P::kK, r, w);
        }
        operands_written();
        arrive(k_full + 8 * stage);
        wait_all(v_free + 8 * stage, (tile >> 1) + 1);
        if (lost) break;
#pragma unroll
        for (int r = 0; r < kIt; ++r) {
          const uint32_t c[4] = {v[r].x, v[r].y, v[r].z, v[r].w};
          uint32_t w[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            // 2 u + 1 below 1024, minus 1280: 2 u - 255
            const uint32_t x = __byte_perm(c[u / 2], 0u, u & 1 ? 0x4342 : 0x4140) * 2 + 0x64016401u, bias = 0x65006500u;
            const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&bias));
            w[u] = *reinterpret_cast<const uint32_t*>(&y);
          }
          put(P::kV, r, w);
        }
        operands_written();
        arrive(v_full + 8 * stage);
      }
      end();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
    const int half = warp >> 2;
    // A batch of infos is given back when a half is done with it.
    auto give_back = [&](uint32_t batch) {
      __syncwarp();
      if ((tid & 31) == 0) arrive(info_free + 8 * (batch & 3));
    };
    while (begin()) {
      if (half >= halves) {
        // Nothing to do but to go along: a wait by parity tells only neighbouring phases apart, so that a half that had left the
        // batches of such units out would take an older one for the next unit's.
        for (int i = 0; i < n && !lost; i += kBatch) {
          const uint32_t batch = batches_done + i / kBatch;
          wait_all(info_full + 8 * (batch & 3), batch >> 2);
          if (!lost) give_back(batch);
        }
        end();
        continue;
      }
      // ---- a column: its query, weights, sums
      const int r = tid & 127;
      const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21);
      const uint32_t s_at = lanes + half * 128, o_at = lanes + 256 + half * 128;
      const int64_t cc = static_cast<int64_t>(cb) * kNC + half * kHalf + r;
      const bool there = cc < static_cast<int64_t>(run.count) * a.G;
      const int token = static_cast<int>(cc / a.G), head = static_cast<int>(cc - static_cast<int64_t>(token) * a.G);
      const int own = run.len + token;
      const size_t row = (static_cast<size_t>(run.first) + token) * a.c.H * a.G + static_cast<size_t>(h) * a.G + head;
      float m = kNone, M = kNone, sum = 0.0f, half_sum = 0.0f, factor = 0.0f;
      if (n > 0) {
        const uint4* from = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.Q) + row * D);
        const uint4 none = make_uint4(0u, 0u, 0u, 0u);
        float most = 0.0f;
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          const uint4 v = there ? __ldg(from + c) : none;
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int u = 0; u < 4; ++u) most = fmaxf(most, fmaxf(fabsf(__uint_as_float(w[u] << 16)), fabsf(__uint_as_float(w[u] & 0xffff0000u))));
        }
        const int x2 = most > 0.0f ? min(141 - static_cast<int>(__float_as_uint(most) >> 23), 120) : 0;
        // the scale's sign goes to the query: the largest product of a block is then its largest logit
        const float up = a.scale2 < 0.0f ? -pow2(x2) : pow2(x2);
        const uint32_t to = base + P::kQ + half * P::kSide + r * 128;
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          const uint4 v = there ? __ldg(from + c) : none;
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          uint32_t o[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float x = __uint_as_float(w[u] << 16) * up, y = __uint_as_float(w[u] & 0xffff0000u) * up;
            half_sum += 0.5f * x + 0.5f * y;
            o[u] = pack(x, y);
          }
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + (c >> 3) * P::kPart + (((c & 7) ^ (r & 7)) << 4)), "r"(o[0]), "r"(o[1]),
                       "r"(o[2]), "r"(o[3])
                       : "memory");
        }
        factor = fabsf(a.scale2) * pow2(-x2);
        operands_written();
        before_sync();            // the last unit's sums have been read
        arrive(q_full + 8 * half);
      }
      for (int i = 0; i < n && !lost; ++i) {
        const uint32_t batch = batches_done + i / kBatch;
        if (i % kBatch == 0) wait_all(info_full + 8 * (batch & 3), batch >> 2);
        const BlockInfo* f = info[batch & 3] + (i % kBatch) * 8;
        const TileInfo ti = tile_info[batch & 3][i % kBatch];
        bool plain = ti.hi <= own && (a.window <= 0 || ti.lo > own - a.window || ti.hi < a.sinks);
        plain = __all_sync(0xffffffffu, plain || !there);
        wait_all(s_full + 8 * half, half_tiles[half] + i);
        if (lost) break;
        after_sync();
        auto seen = [&](int k, int c) {
          const int s = f[k].slot + c;
          return f[k].ek != 0.0f && s <= own && (a.window <= 0 || s > own - a.window || s < a.sinks);
        };
        // largest logits of the blocks; the next block's are on their way meanwhile, its exponents read before they are waited
        // for.  (Loops are kept short: the warps' programs share an instruction cache.)
        auto exponents = [&](int k) { return make_float2(f[k].ek, f[k].ev); };
        float top = -INFINITY, topv = -INFINITY;
        float za[16], zb[16];
        auto largest = [&](const float (&z)[16], int k, float2 e) {
          float best = -INFINITY;
          if (plain) {
            float u[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) u[c] = fmaxf(fmaxf(z[c], z[4 + c]), fmaxf(z[8 + c], z[12 + c]));
            best = fmaxf(fmaxf(u[0], u[1]), fmaxf(u[2], u[3]));
          } else {
#pragma unroll
            for (int c = 0; c < 16; ++c) best = seen(k, c) ? fmaxf(best, z[c]) : best;
          }
          const float v = best == -INFINITY ? best : (best + half_sum) * (factor * e.x);
          top = fmaxf(top, v);
          topv = fmaxf(topv, v + e.y);
        };
        tmem_ld16(s_at, za);
#pragma unroll 1
        for (int k = 0; k < 8; k += 2) {
          const float2 e0 = exponents(k), e1 = exponents(k + 1);
          tmem_loaded(za);
          tmem_ld16(s_at + 16 * k + 16, zb);
          largest(za, k, e0);
          tmem_loaded(zb);
          tmem_ld16(s_at + (k < 6 ? 16 * k + 32 : 0), za);      // at the end the first again, for the weights
          largest(zb, k + 1, e1);
        }
        const bool over = top > m + kSlack || topv > M + kSlack;
        if (__any_sync(0xffffffffu, over)) {
          const float u = over ? fmaxf(top, m) : m, v = over ? fmaxf(topv, M) : M;
          const float fm = exp2_fast(m - u), fv = exp2_fast(M - v);
          m = u;
          M = v;
          sum *= fm;
          if (i > 0) {
            tmem_loaded(za);      // nothing is under way where the wait gives up
            wait_all(o_done + 8 * half, half_tiles[half] + i - 1);
            if (lost) break;
            after_sync();
#pragma unroll 1
            for (int c4 = 0; c4 < D / 32; ++c4) {
              float o[32];
              tmem_ld32(o_at + 32 * c4, o);
              tmem_loaded(o);
              uint32_t w[2][16];
#pragma unroll
              for (int c = 0; c < 32; ++c) w[c >> 4][c & 15] = __float_as_uint(o[c] * fv);
              tmem_st16(o_at + 32 * c4, w[0]);
              tmem_st16(o_at + 32 * c4 + 16, w[1]);
            }
          }
        }
        // where exponents of values are so far apart that a weight and its p do not fit one range, and where slots are hidden,
        // two exponentials a logit
        const float apart_by = m - M;
        const bool quick = plain && !__any_sync(0xffffffffu, apart_by + ti.ev_hi > 100.0f || apart_by + ti.ev_lo < -60.0f);
        auto weigh = [&](const float (&z)[16], float2 e, uint32_t* w) {
          const float scale = factor * e.x, up = e.y - M + kLift, shift = fmaf(half_sum, scale, up);
          const uint64_t scale2 = two(scale, scale), off = two(shift, shift);
          uint64_t all = two(0.0f, 0.0f);
#pragma unroll
          for (int c = 0; c < 16; c += 2) {
            const float2 v = apart(fma2(two(z[c], z[c + 1]), scale2, off));
            const float w0 = exp2_fast(v.x), w1 = exp2_fast(v.y);
            all = add2(all, two(w0, w1));
            w[c / 2] = pack(w0, w1);
          }
          const float2 sums = apart(all);
          sum = fmaf(sums.x + sums.y, exp2_fast(-m - up), sum);      // p is the weight less its block's factor
        };
        if (quick) {
#pragma unroll 1
          for (int k = 0; k < 8; k += 2) {
            const float2 e0 = exponents(k), e1 = exponents(k + 1);
            uint32_t w[16];
            tmem_loaded(za);
            tmem_ld16(s_at + 16 * k + 16, zb);
            weigh(za, e0, w);
            tmem_loaded(zb);
            if (k < 6) tmem_ld16(s_at + 16 * k + 32, za);
            weigh(zb, e1, w + 8);
            tmem_st16(s_at + 8 * k, w);      // over logits that have been read
          }
        } else {
          tmem_loaded(za);
#pragma unroll 1
          for (int k = 0; k < 8; k += 2) {
            uint32_t w[16];
#pragma unroll
            for (int k2 = 0; k2 < 2; ++k2) {
              if (k + k2 > 0) {
                tmem_ld16(s_at + 16 * (k + k2), za);
                tmem_loaded(za);
              }
              const float2 e = exponents(k + k2);
              const float scale = factor * e.x;
#pragma unroll
              for (int c = 0; c < 16; c += 2) {
                float q[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                  const float v = (za[c + u] + half_sum) * scale;
                  const bool on = seen(k + k2, c + u);
                  sum += on ? exp2_fast(v - m) : 0.0f;
                  q[u] = on ? exp2_fast(v + (e.y + kLift - M)) : 0.0f;
                }
                w[8 * k2 + c / 2] = pack(q[0], q[1]);
              }
            }
            tmem_st16(s_at + 8 * k, w);
          }
        }
        tmem_stored();
        before_sync();
        arrive(p_full + 8 * half);
        if (i % kBatch == kBatch - 1 || i == n - 1) give_back(batch);
      }
      // ---- out, or a part for the join
      if (n > 0) wait_all(o_done + 8 * half, half_tiles[half] + n - 1);
      after_sync();
      const bool entire = qa == 0 && qe == share.plan.quads;
      const size_t place = (static_cast<size_t>(blockIdx.x) * 2 + (qa == 0 ? 1 : 0)) * kNC + half * kHalf + r;
      // products were taken twice (2 c + 1) and weights 2^kLift times
      const float nan = __int_as_float(0x7fffffff);
      const float f = lost ? nan : sum == 0.0f ? 0.0f : exp2f(M - m - kLift - 1.0f) / sum;
      if (!entire && there) a.top[place] = make_float4(m, M, lost ? nan : sum, 0.0f);
#pragma unroll 1
      for (int c4 = 0; c4 < D / 32; ++c4) {
        float o[32];
        if (n > 0 && !lost) {
          tmem_ld32(o_at + 32 * c4, o);
          tmem_loaded(o);
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = 0.0f;
        }
        if (there && entire) {
          __nv_bfloat16* to = static_cast<__nv_bfloat16*>(a.out) + row * D + 32 * c4;
#pragma unroll
          for (int c = 0; c < 32; c += 8) {
            uint32_t w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const __nv_bfloat162 v = __floats2bfloat162_rn(sum == 0.0f && !lost ? 0.0f : o[c + 2 * u] * f, sum == 0.0f && !lost ? 0.0f : o[c + 2 * u + 1] * f);
              w[u] = *reinterpret_cast<const uint32_t*>(&v);
            }
            *reinterpret_cast<uint4*>(to + c) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else if (there) {
          float* to = a.part + place * D + 32 * c4;
#pragma unroll
          for (int c = 0; c < 32; c += 4)
            *reinterpret_cast<float4*>(to + c) = make_float4(0.5f * o[c], 0.5f * o[c + 1], 0.5f * o[c + 2], 0.5f * o[c + 3]);
        }
        __syncwarp();
      }
      end();
    }
  }
  if (warp == 12) {
    if (elected()) commit_to(drained);      // nothing is in flight, whatever ran out
    wait_parity_bounded(drained, 0, kFaultAttendWait);
    __syncwarp();
  }
  before_sync();
  __syncthreads();
  after_sync();
  if (warp == 12) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

template <int D>
cudaError_t launch(const AttendArgs& a, int ctas, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(attend_prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, PromptShape<D>::kBytes);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_acq_rel);
  }
  attend_prompt_kernel<D><<<ctas, kThreads, PromptShape<D>::kBytes, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend_prompt(const AttendArgs& a, int D, int ctas, cudaStream_t st) {
  return D == 64 ? launch<64>(a, ctas, st) : launch<128>(a, ctas, st);
}

cudaError_t take_faults_attend_prompt(unsigned int* bits) { return take_unit_faults(bits); }

}  // namespace tq
