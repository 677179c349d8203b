// Eviction from the paged cache by accumulated attention weight (tq_evict_paged).
#include "tq_paged.cuh"

namespace tq {
namespace {

constexpr int kSel = 1024;

// Order of preference as an unsigned number: protected slots above every weight, then the
// weight (its bits made monotone; -0 as 0, NaN as -inf).
__device__ __forceinline__ uint32_t rank_key(float m, int pos, long long oldest) {
  if (pos >= oldest) return 0xffffffffu;
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
  if (warp == 0) {
    int t = lane < kSel / 32 ? red[lane] : 0;
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += u;
    }
    red[lane] = t;
  }
  __syncthreads();
  *total = red[kSel / 32 - 1];
  return x - v + (warp > 0 ? red[warp - 1] : 0);
}

// One block per (sequence, head).  The keep-th largest key is found by its digits from the
// top (256 counts a pass); then one pass in slot order lists the slots that are given up
// below `keep` and the kept ones behind it.
__global__ void __launch_bounds__(kSel)
evict_select_kernel(Paged pg, const int* __restrict__ lengths, const int* __restrict__ seen,
                    const float* __restrict__ mass, const int* __restrict__ positions, int S, int cap,
                    int budget, int recent, float* __restrict__ mass_out, int* __restrict__ pos_out,
                    int* __restrict__ counts, int* __restrict__ lists, int most) {
  __shared__ int hist[256];
  __shared__ int red[32];
  __shared__ int pick[2];
  const int b = blockIdx.x, h = blockIdx.y, t = threadIdx.x;
  const int n = pg.length(lengths, b, cap);
  const int keep = min(n, budget);
  const size_t unit = static_cast<size_t>(b) * pg.H + h;
  const float* m = mass + unit * S;
  const int* ps = positions + unit * S;
  const long long oldest = static_cast<long long>(seen[b]) - recent;
  uint32_t prefix = 0;
  int want = keep;
  if (keep < n) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (t < 256) hist[t] = 0;
      __syncthreads();
      for (int s = t; s < n; s += kSel) {
        const uint32_t k = rank_key(m[s], ps[s], oldest);
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      if (t == 0) {
        int left = want, v = 255;
        while (v > 0 && hist[v] < left) left -= hist[v--];
        pick[0] = v;
        pick[1] = left;
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(pick[0]) << shift;
      want = pick[1];
      __syncthreads();
    }
  }
  int* hole = lists + unit * 2 * most;
  int* sur = hole + most;
  int eq0 = 0, h0 = 0, s0 = 0, tot;
  for (int base = 0; base < n; base += kSel) {
    const int s = base + t;
    const uint32_t k = s < n ? rank_key(m[s], ps[s], oldest) : 0;
    const bool eq = s < n && keep < n && k == prefix;
    const int e = eq0 + block_scan(eq, red, &tot);
    eq0 += tot;
    const bool kept = s < n && (keep == n || k > prefix || (eq && e < want));
    const bool is_hole = s < keep && !kept, is_sur = s >= keep && kept;
    const int hi = h0 + block_scan(is_hole, red, &tot);
    h0 += tot;
    const int si = s0 + block_scan(is_sur, red, &tot);
    s0 += tot;
    if (is_hole) hole[hi] = s;
    if (is_sur) sur[si] = s;
    if (s < keep && kept) {
      mass_out[unit * S + s] = m[s];
      pos_out[unit * S + s] = ps[s];
    }
  }
  if (t == 0) counts[unit] = h0;
}

__global__ void evict_move_kernel(Paged pg, const float* __restrict__ mass, const int* __restrict__ positions,
                                  int S, float* __restrict__ mass_out, int* __restrict__ pos_out,
                                  const int* __restrict__ counts, const int* __restrict__ lists, int most,
                                  int kbits, int vbits) {
  const int b = blockIdx.x, h = blockIdx.y;
  const size_t unit = static_cast<size_t>(b) * pg.H + h;
  const int* hole = lists + unit * 2 * most;
  const int* sur = hole + most;
  const int cnt = counts[unit], parts = kbits + vbits + 1;
  for (int e = threadIdx.x; e < cnt * parts; e += blockDim.x) {
    const int i = e / parts, c = e % parts;
    const int to = hole[i], from = sur[i];
    const int pt = pg.page(b, to), pf = pg.page(b, from);
    if (pt < 0 || pf < 0) continue;
    const size_t rt = pg.row(pt, h, to), rf = pg.row(pf, h, from);
    if (c < kbits) {
      reinterpret_cast<uint4*>(pg.kp)[rt * kbits + c] = reinterpret_cast<const uint4*>(pg.kp)[rf * kbits + c];
    } else if (c < kbits + vbits) {
      reinterpret_cast<uint4*>(pg.vp)[rt * vbits + c - kbits] =
          reinterpret_cast<const uint4*>(pg.vp)[rf * vbits + c - kbits];
    } else {
      pg.kn[rt] = pg.kn[rf];
      pg.vn[rt] = pg.vn[rf];
      mass_out[unit * S + to] = mass[unit * S + from];
      pos_out[unit * S + to] = positions[unit * S + from];
    }
  }
}

// Rows one (sequence, head) can move.
int most_moves(int S, int budget) { return budget >= S ? 0 : (budget < S - budget ? budget : S - budget); }

}  // namespace

size_t evict_paged_bytes(int B, int H, int S, int budget) {
  const size_t units = static_cast<size_t>(B) * H;
  return paged_round(units * 4) + paged_round(units * 2 * most_moves(S, budget) * 4);
}

cudaError_t launch_evict_paged(const tq_paged_cache& c, const int* table, const int* lengths, const int* seen,
                               int B, int max_pages, const float* mass, const int* positions, int S, int budget,
                               int recent, float* mass_out, int* positions_out, void* ws, cudaStream_t st) {
  const int pages = max_pages * c.page_size;
  const int cap = S < pages ? S : pages;
  int* counts = static_cast<int*>(ws);
  int* lists = reinterpret_cast<int*>(static_cast<char*>(ws) + paged_round(static_cast<size_t>(B) * c.H * 4));
  const Paged pg = paged_view(c, table, max_pages);
  const int most = most_moves(S, budget);
  evict_select_kernel<<<dim3(B, c.H), kSel, 0, st>>>(pg, lengths, seen, mass, positions, S, cap, budget, recent,
                                                    mass_out, positions_out, counts, lists, most);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || most == 0) return e;
  evict_move_kernel<<<dim3(B, c.H), 256, 0, st>>>(pg, mass, positions, S, mass_out, positions_out, counts, lists,
                                                 most, c.k_bits, c.v_bits);
  return cudaGetLastError();
}

cudaError_t take_faults_evict(unsigned int* bits) { return take_unit_faults(bits); }

}  // namespace tq
