// Eviction from the paged cache by accumulated attention weight (tq_evict_paged): two
// launches.
//
// select: a cluster of up to 8 CTAs per (sequence, head).  Each CTA keeps the keys (the order of
// preference as unsigned numbers) of its share of the slots in shared memory; the keep-th
// largest key is found by its digits from the top (11, 11 and 10 bits), the counts of a
// digit added up over the cluster through distributed shared memory; the keys that share the
// first digit are listed, so that the third pass reads few.  Where more slots are protected than
// are kept, the first digit is counted once more, by weight.  One pass in slot order then lists
// the slots given up below `keep` and the kept ones behind it (ballots; equal keys are counted
// only where the last one kept has equals that are not), and copies the weights that stay.
//
// move: the i-th listed row behind `keep` goes to the i-th listed slot below it.  Sources and
// targets are disjoint, so the rows move in any order; eight threads take a row.
//
// Bound: select by dependent latencies (16 x 8 rows of 4224 slots: some 40 loads, barriers and
// scans in a row, 15 us a call with the moves); move by DRAM's sectors: a row's 48 + 48 + 2 + 2 + 4 + 4
// bytes lie in scattered 32-byte sectors.  4 x 8 rows of 131072 slots to 32768: select 47 us, move
// 58 us for 314 MB of DRAM traffic (5.4 TB/s) where the rows' own bytes are 157 MB; 104 us a call.
// Measured on the way there (4 x 8 rows): one CTA a row 1853 us; 1024 threads a CTA (one an SM, two waves)
// 139 us, 512 threads 111 us; weights loaded eight deep 105 us; 128 rows a CTA of move 103 us.
#include <cooperative_groups.h>

#include "tq_paged.cuh"

namespace tq {
namespace {

namespace cg = cooperative_groups;

constexpr int kCluster = 8;             // CTAs of a cluster, at most
constexpr int kSel = 512;               // threads of a CTA of select (two or more CTAs an SM)
constexpr int kDigit = 2048;            // counts of the widest digit
constexpr int kCached = 48 * 1024;      // keys a CTA can keep in shared memory
constexpr int kListed = 4096;           // of them that share the first digit, listed for the last pass
constexpr int kMoves = 128;             // rows a CTA of move takes (256: 105 us instead of 103 for 4 x 131072)

// Order of preference as an unsigned number: the weight (its bits made monotone; -0 as 0, NaN
// as -inf), and protected slots above every weight.  `window`: where there are more of those than
// are kept, they go by weight and the others are below all.
__device__ __forceinline__ uint32_t rank_key(float m, int pos, long long oldest, bool window) {
  const bool safe = pos >= oldest;
  if (safe != window) return window ? 0u : 0xffffffffu;
  if (m != m) m = -INFINITY;
  const uint32_t u = __float_as_uint(m + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Exclusive prefix of v over the block, and the block's total.
__device__ __forceinline__ int block_scan(int v, int* red, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += t;
  }
  __syncthreads();
  if (lane == 31) red[warp] = x;
  __syncthreads();
  int t = lane < kSel / 32 ? red[lane] : 0;                // every warp adds up the warps' totals
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, t, o);
    if (lane >= o) t += u;
  }
  *total = __shfl_sync(0xffffffffu, t, 31);
  const int before = __shfl_sync(0xffffffffu, t, warp > 0 ? warp - 1 : 0);
  return x - v + (warp > 0 ? before : 0);
}

// This CTA's sum over the CTAs of lower rank of *mine, and the sum over all.
__device__ __forceinline__ int cluster_before(cg::cluster_group& cl, int* mine) {
  const int rank = cl.block_rank();
  int sum = 0;
#pragma unroll
  for (int r = 0; r < kCluster - 1; ++r)
    if (r < rank) sum += *cl.map_shared_rank(mine, r);
  return sum;
}

struct SelectArgs {
  const int* lengths;
  const int* seen;
  const float* mass;
  const int* positions;
  float* mass_out;
  int* pos_out;
  int* counts;                          // [B*H] moves
  int* lists;                           // [B*H][2][most] slots to fill, slots to take
  uint32_t* keys;                       // [B*H][S] where they do not fit shared memory
  int H, S, cap, budget, recent, most;
};

template <bool CACHED>
__global__ void __launch_bounds__(kSel, 2)
evict_select_kernel(const SelectArgs a) {
  extern __shared__ uint32_t cache[];
  __shared__ __align__(16) int hist[2][kDigit];
  __shared__ int red[32];
  __shared__ int pick[3];
  __shared__ int part[3];
  __shared__ int listed;
  __shared__ uint32_t list[kListed];
  cg::cluster_group cl = cg::this_cluster();
  const int C = cl.num_blocks(), rank = cl.block_rank(), t = threadIdx.x;
  const int unit = blockIdx.x / C, b = unit / a.H;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int n = a.lengths[b];
  if (n < 0 || n > a.cap) {
    if (t == 0) atomicOr(&g_wait_fault, static_cast<unsigned int>(kFaultPaged));
    n = n < 0 ? 0 : a.cap;
  }
  const int keep = min(n, a.budget);
  const int per = (n + C - 1) / C, first = min(n, rank * per), mine = min(n, first + per) - first;
  const size_t base = static_cast<size_t>(unit) * a.S + first;
  const float* m = a.mass + base;
  const int* ps = a.positions + base;
  float* mo = a.mass_out + base;
  int* po = a.pos_out + base;
  if (keep == n) {                                         // nothing to give up
    for (int s = t; s < mine; s += kSel) {
      mo[s] = m[s];
      po[s] = ps[s];
    }
    if (t == 0 && rank == 0) a.counts[unit] = 0;
    return;
  }
  uint32_t* key = CACHED ? cache : a.keys + base;
  const long long oldest = static_cast<long long>(a.seen[b]) - a.recent;
  for (int i = t; i < kDigit; i += kSel) hist[0][i] = 0;
  if (t == 0) listed = 0;
  __syncthreads();
  // the keep-th largest key; what shares its first digit is listed for the last pass
  uint32_t prefix = 0;
  int want = keep, equal = 0;
  // pick: the digit that the want-th largest has, which it is among those, and their number
  auto pick_digit = [&](int* hs, int width) {
    // four digits a thread, the largest first
    const int hi = (1 << width) - 1 - 4 * t;
    int4 v = make_int4(0, 0, 0, 0);
    if (hi > 0) {
      int4 x[kCluster];
#pragma unroll
      for (int r = 0; r < kCluster; ++r)                   // all ranks' counts in flight
        if (r < C) x[r] = *reinterpret_cast<const int4*>(cl.map_shared_rank(hs, r) + hi - 3);
#pragma unroll
      for (int r = 0; r < kCluster; ++r)
        if (r < C) v = make_int4(v.x + x[r].x, v.y + x[r].y, v.z + x[r].z, v.w + x[r].w);
    }
    int total;
    int above = block_scan(v.x + v.y + v.z + v.w, red, &total);
    const int at[4] = {v.w, v.z, v.y, v.x};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (above < want && want <= above + at[i]) {
        pick[0] = hi - i;
        pick[1] = want - above;
        pick[2] = at[i];
      }
      above += at[i];
    }
    __syncthreads();
  };
  // The top digit of all is that of protected slots alone (infinity's is 2044).  Where there are
  // more of them than are kept, the keys are made again, by weight among them.  (Two inlined
  // copies of this took 96 registers, one CTA an SM: 137 us instead of 104 for 4 x 131072.)
#pragma unroll 1
  for (bool window = false;; window = true) {
    constexpr int U = 8;                                   // loads of each array in flight, a thread
    for (int s0 = t; s0 < mine; s0 += U * kSel) {
      float x[U];
      int y[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int s = min(s0 + i * kSel, mine - 1);
        x[i] = m[s];
        y[i] = ps[s];
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int s = s0 + i * kSel;
        if (s < mine) {
          const uint32_t k = rank_key(x[i], y[i], oldest, window);
          key[s] = k;
          atomicAdd(&hist[0][k >> 21], 1);
        }
      }
    }
    cl.sync();
    for (int i = t; i < kDigit; i += kSel) hist[1][i] = 0;
    pick_digit(hist[0], 11);
    if (window || pick[0] != kDigit - 1 || pick[2] <= pick[1]) break;
    cl.sync();                                             // every CTA has read the counts
    for (int i = t; i < kDigit; i += kSel) hist[0][i] = 0;
    __syncthreads();
  }
  prefix = static_cast<uint32_t>(pick[0]) << 21;
  want = pick[1];
  __syncthreads();
#pragma unroll
  for (int pass = 1; pass < 3; ++pass) {
    const int shift = pass == 1 ? 10 : 0, width = pass == 2 ? 10 : 11;
    int* hs = hist[pass & 1];
    if (pass == 1) {
#pragma unroll 8
      for (int s = t; s < mine; s += kSel) {
        const uint32_t k = key[s];
        if ((k >> 21) == (prefix >> 21)) {
          atomicAdd(&hs[(k >> 10) & 2047u], 1);
          const int i = atomicAdd(&listed, 1);
          if (i < kListed) list[i] = k;
        }
      }
    } else {
      const bool all = listed > kListed;                   // more than the list holds: through all of them
      const uint32_t* from = all ? key : list;
      for (int s = t, e = all ? mine : listed; s < e; s += kSel)
        if ((from[s] >> 10) == (prefix >> 10)) atomicAdd(&hs[from[s] & 1023u], 1);
    }
    cl.sync();
    for (int i = t; i < kDigit; i += kSel) hist[(pass + 1) & 1][i] = 0;   // its readers are done: they have come to this sync
    pick_digit(hs, width);
    prefix |= static_cast<uint32_t>(pick[0]) << shift;
    want = pick[1];
    equal = pick[2];
    __syncthreads();
  }

  // Slots in order: a warp takes a run of them, 32 at a time.  Of the keys equal to the last one
  // kept (one, unless weights are the same) the first `want` are kept.
  const int lane = t & 31, warp = t >> 5;
  const uint32_t below = (1u << lane) - 1;
  const int run = ((mine + kSel - 1) / kSel) * 32;
  const int r0 = min(mine, warp * run), r1 = min(mine, r0 + run);
  int e0 = 0;                                              // equal keys before the run
  const bool ties = equal > want;
  if (ties) {
    int eq = 0, total;
    for (int s = r0 + lane; s < r1; s += 32) eq += key[s] == prefix;
    const int before = block_scan(eq, red, &total);
    e0 = __shfl_sync(0xffffffffu, before, 0);
    if (t == 0) part[0] = total;
    cl.sync();
    e0 += cluster_before(cl, &part[0]);
  }
  auto kept_now = [&](int s, int& e) {                     // is the slot kept; e: equal keys so far
    const uint32_t k = s < r1 ? key[s] : 0;
    bool kept = s < r1 && k >= prefix;
    if (ties) {
      const uint32_t same = __ballot_sync(0xffffffffu, s < r1 && k == prefix);
      if (k == prefix) kept = kept && e + __popc(same & below) < want;
      e += __popc(same);
    }
    return kept;
  };
  int holes = 0, extra = 0;
  {
    int e = e0;
#pragma unroll 8
    for (int s0 = r0; s0 < r1; s0 += 32) {
      const int s = s0 + lane;
      const bool kept = kept_now(s, e), low = first + s < keep;
      holes += s < r1 && low && !kept;
      extra += !low && kept;
    }
  }
  int total;
  int hi = block_scan(holes, red, &total);
  hi = __shfl_sync(0xffffffffu, hi, 0);
  if (t == 0) part[1] = total;
  int xi = block_scan(extra, red, &total);
  xi = __shfl_sync(0xffffffffu, xi, 0);
  if (t == 0) part[2] = total;
  cl.sync();
  hi += cluster_before(cl, &part[1]);
  xi += cluster_before(cl, &part[2]);
  if (rank == C - 1 && t == 0) a.counts[unit] = hi + part[1];   // thread 0: what the CTAs before have
  int* to = a.lists + static_cast<size_t>(unit) * 2 * a.most;
  int* from = to + a.most;
  {
    int e = e0;
    constexpr int V = 8;                                   // weights of slots that may stay: loads in flight
    for (int s0 = r0; s0 < r1; s0 += 32 * V) {
      float x[V];
      int y[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int s = s0 + 32 * i + lane;
        if (s < r1 && first + s < keep) {
          x[i] = m[s];
          y[i] = ps[s];
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (s0 + 32 * i >= r1) break;
        const int s = s0 + 32 * i + lane;
        const bool kept = kept_now(s, e), low = first + s < keep;
        const uint32_t hb = __ballot_sync(0xffffffffu, s < r1 && low && !kept), xb = __ballot_sync(0xffffffffu, !low && kept);
        if (kept && low) {
          mo[s] = x[i];
          po[s] = y[i];
        }
        if (hb >> lane & 1) to[hi + __popc(hb & below)] = first + s;
        if (xb >> lane & 1) from[xi + __popc(xb & below)] = first + s;
        hi += __popc(hb);
        xi += __popc(xb);
      }
    }
  }
  cl.sync();                                               // no CTA leaves while its counts may be read
}

// Eight threads of move take a row's 16-byte pieces (up to four of the key, up to four of the
// value), four rows each with all their loads in flight; a thread a row its two lengths, its
// weight and its position.
__global__ void __launch_bounds__(256)
evict_move_kernel(Paged pg, const float* __restrict__ mass, const int* __restrict__ positions, int S,
                  float* __restrict__ mass_out, int* __restrict__ pos_out, const int* __restrict__ counts,
                  const int* __restrict__ lists, int most, int chunks, int kbits, int vbits) {
  __shared__ long long rows[2][kMoves];
  const int unit = blockIdx.x / chunks, i0 = (blockIdx.x - unit * chunks) * kMoves;
  const int b = unit / pg.H, h = unit - b * pg.H, t = threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int cnt = min(kMoves, counts[unit] - i0);
  if (cnt <= 0) return;
  if (t < cnt) {
    const int* to = lists + static_cast<size_t>(unit) * 2 * most + i0;
    const int s = to[t], f = to[most + t];
    const int ps = pg.page(b, s), pf = pg.page(b, f);
    const size_t at = static_cast<size_t>(unit) * S;
    const float w = mass[at + f];                          // weights follow whether or not the rows can
    const int p = positions[at + f];
    const bool ok = ps >= 0 && pf >= 0;
    const size_t rt = ok ? pg.row(ps, h, s) : 0, rf = ok ? pg.row(pf, h, f) : 0;
    const uint16_t kn = pg.kn[rf], vn = pg.vn[rf];
    mass_out[at + s] = w;
    pos_out[at + s] = p;
    if (ok) {
      pg.kn[rt] = kn;
      pg.vn[rt] = vn;
    }
    rows[0][t] = ok ? static_cast<long long>(rt) : -1;
    rows[1][t] = static_cast<long long>(rf);
  }
  __syncthreads();
  const int c = t & 7;
  if (c >= kbits + vbits) return;
  const bool key = c < kbits;
  uint4* plane = reinterpret_cast<uint4*>(key ? pg.kp : pg.vp) + (key ? c : c - kbits);
  const int bits = key ? kbits : vbits;
  uint4 v[kMoves / 32];
  long long to[kMoves / 32];
#pragma unroll
  for (int k = 0; k < kMoves / 32; ++k) {
    const int i = k * 32 + (t >> 3);
    to[k] = i < cnt ? rows[0][i] : -1;
    if (to[k] >= 0) v[k] = plane[rows[1][i] * bits];
  }
#pragma unroll
  for (int k = 0; k < kMoves / 32; ++k)
    if (to[k] >= 0) plane[to[k] * bits] = v[k];
}

// Rows one (sequence, head) can move.
int most_moves(int S, int budget) { return budget >= S ? 0 : (budget < S - budget ? budget : S - budget); }

// CTAs of a cluster: as many as it takes to keep the keys in shared memory (where 8 do), and
// enough to fill the device from few rows.  Up to one CTA an SM a share is 2048 slots or more (8 x 8
// rows of 8191: 15.6 us a call with two CTAs a row, 17.3 with one; 1 row of 8191: 13.4 and 15.8, 1
// of 4224: 12.5 and 13.6), up to two 4096 or more (16 x 8 rows of 4224: 15.1 us with one, 17.4
// with two, 31 with four).
int cluster_size(int S, int64_t units, int sms) {
  int C = 1;
  while (C < kCluster && (S > C * kCached || (units * C * 2 <= sms && S / (2 * C) >= 2048) || (units * C <= sms && S / (2 * C) >= 4096))) C *= 2;
  return C;
}
bool keys_fit(int S) { return S <= kCluster * kCached; }

}  // namespace

size_t evict_paged_bytes(int B, int H, int S, int budget) {
  const size_t units = static_cast<size_t>(B) * H;
  return paged_round(units * 4) + paged_round(units * 2 * most_moves(S, budget) * 4) + (keys_fit(S) ? 0 : paged_round(units * S * 4));
}

cudaError_t launch_evict_paged(const tq_paged_cache& c, const int* table, const int* lengths, const int* seen,
                               int B, int max_pages, const float* mass, const int* positions, int S, int budget,
                               int recent, float* mass_out, int* positions_out, void* ws, cudaStream_t st) {
  static std::atomic<int> sms_cache[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int sms = sms_cache[dev & 63].load(std::memory_order_acquire);
  if (sms == 0) {
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(evict_select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kCached * 4);
    if (e != cudaSuccess) return e;
    sms_cache[dev & 63].store(sms, std::memory_order_release);
  }
  const int pages = max_pages * c.page_size;
  const int64_t units = static_cast<int64_t>(B) * c.H;
  const int most = most_moves(S, budget);
  SelectArgs a;
  a.lengths = lengths;
  a.seen = seen;
  a.mass = mass;
  a.positions = positions;
  a.mass_out = mass_out;
  a.pos_out = positions_out;
  a.counts = static_cast<int*>(ws);
  a.lists = reinterpret_cast<int*>(static_cast<char*>(ws) + paged_round(units * 4));
  a.keys = reinterpret_cast<uint32_t*>(reinterpret_cast<char*>(a.lists) + paged_round(units * 2 * most * 4));
  a.H = c.H;
  a.S = S;
  a.cap = S < pages ? S : pages;
  a.budget = budget;
  a.recent = recent;
  a.most = most;
  const int C = cluster_size(a.cap, units, sms);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units * C));
  cfg.blockDim = dim3(kSel);
  cfg.dynamicSmemBytes = keys_fit(S) ? (static_cast<size_t>(ceil_div(a.cap, C)) * 4 + 15) / 16 * 16 : 0;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = keys_fit(S) ? cudaLaunchKernelEx(&cfg, evict_select_kernel<true>, a) : cudaLaunchKernelEx(&cfg, evict_select_kernel<false>, a);
  if (e != cudaSuccess || most == 0) return e;
  const int chunks = ceil_div(most, kMoves);
  if (units * chunks > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t mv = {};
  mv.gridDim = dim3(static_cast<unsigned>(units * chunks));
  mv.blockDim = dim3(256);
  mv.stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  mv.attrs = attr;
  mv.numAttrs = 1;
  return cudaLaunchKernelEx(&mv, evict_move_kernel, paged_view(c, table, max_pages), mass, positions, S, mass_out,
                            positions_out, static_cast<const int*>(a.counts), static_cast<const int*>(a.lists), most,
                            chunks, c.k_bits, c.v_bits);
}

cudaError_t take_faults_evict(unsigned int* bits) { return take_unit_faults(bits); }

}  // namespace tq
