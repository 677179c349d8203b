// Attention of one new token over the paged cache (tq_decode_paged): four launches, each a
// programmatic dependent of the one before.
//   plan     a = Pi_k q for every query, and the tiles before each sequence
//   split    tq_paged_split.cuh: a partial (maximum, sum, value sum) per run and unit
//   combine  the partials of each query joined, out = Pi_v^T of it
//   mass     where asked for: every slot's weights from its logits, added to mass
//
// What each costs alone (16 ragged sequences of up to 8191 slots, 8 heads of 4 queries, with
// mass): plan 6.5 us, split 31, join 8.1, mass 7.2; 40 us a call, as the next one's launch and
// set-up overlap the one before.  The shortest call (1 sequence, 1021 slots) is 10.7 us, three
// launches of 2 to 3 us of dependent loads each.  The logits go through the workspace (16 bytes a slot at 4
// queries, written and read from L2): what a weight is divided by is known only after the join.
#include "tq_paged_split.cuh"

namespace tq {
namespace {

__device__ __forceinline__ float load_q(const float* q, size_t i) { return q[i]; }
__device__ __forceinline__ float load_q(const __nv_bfloat16* q, size_t i) { return __bfloat162float(q[i]); }
__device__ __forceinline__ void store_o(float* o, size_t i, float v) { o[i] = v; }
__device__ __forceinline__ void store_o(__nv_bfloat16* o, size_t i, float v) { o[i] = __float2bfloat16_rn(v); }

constexpr int kPlanThreads = 256;
constexpr int kPlanRows = 32;        // rows of Pi_k a block takes
constexpr int kPlanQ = 8;            // queries at a time

// Block (unit, quarter): 32 rows of Pi_k against the unit's queries; a warp per row, the
// row's 128 columns across its lanes.  The last block counts tiles.
template <typename T>
__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(const T* __restrict__ Q, const int* __restrict__ lengths, const float* __restrict__ Pik, int B, int H,
            int G, int rot, int cap, float* __restrict__ A, int* __restrict__ tiles, int* __restrict__ cut) {
  __shared__ __align__(16) float q[kPlanQ][kPD];
  __shared__ int red[kPlanThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (blockIdx.x == gridDim.x - 1) {
    int before = 0;
    for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
      const int b = b0 + tid;
      int n = 0;
      if (b < B) {
        n = lengths[b];
        if (n < 0 || n > cap) {
          atomicOr(&g_wait_fault, static_cast<unsigned int>(kFaultPaged));
          n = n < 0 ? 0 : cap;
        }
        cut[b] = n;
      }
      const int v = (n + kTile - 1) / kTile;
      int x = v;
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      __syncthreads();
      if (lane == 31) red[warp] = x;
      __syncthreads();
      int pre = 0, all = 0;
      for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < warp) pre += red[w];
        all += red[w];
      }
      if (b < B) tiles[b] = before + pre + x - v;
      before += all;
    }
    if (tid == 0) tiles[B] = before;
    return;
  }
  const int unit = blockIdx.x >> 2, row0 = (blockIdx.x & 3) * kPlanRows + warp * 4;
  const int h = unit % H;
  const float* P = Pik + (static_cast<size_t>(h % rot) * kPD + row0) * kPD + 4 * lane;
  float4 m[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) m[r] = __ldg(reinterpret_cast<const float4*>(P + r * kPD));
  for (int g0 = 0; g0 < G; g0 += kPlanQ) {
    const int ng = min(kPlanQ, G - g0);
    const size_t qo = (static_cast<size_t>(unit) * G + g0) * kPD;
    __syncthreads();
    for (int e = tid; e < ng * kPD; e += kPlanThreads) q[e / kPD][e % kPD] = load_q(Q, qo + e);
    __syncthreads();
    for (int i = 0; i < ng; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(&q[i][4 * lane]);
      float s[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) s[r] = fmaf(m[r].x, x.x, fmaf(m[r].y, x.y, fmaf(m[r].z, x.z, m[r].w * x.w)));
#pragma unroll
      for (int o = 16; o; o >>= 1) {
#pragma unroll
        for (int r = 0; r < 4; ++r) s[r] += __shfl_xor_sync(0xffffffffu, s[r], o);
      }
      if (lane == 0) *reinterpret_cast<float4*>(A + qo + i * kPD + row0) = make_float4(s[0], s[1], s[2], s[3]);
    }
  }
}

constexpr int kJoinThreads = 512;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kJoinQ = 8;
constexpr int kJoinSlots = 8;        // partials a warp has in flight

// Block (sequence and head, group of 1, 2, 4 or 8 of its queries).  Thread (r, d) of 4 x 128 holds
// rows 32r .. 32r+31 of column d of Pi_v, requested before the wait for the split.  The warps
// are shared out among the queries; a warp takes every (16 / group)-th partial of its query,
// eight in flight, four coordinates a lane.
template <typename T>
__global__ void __launch_bounds__(kJoinThreads)
join_kernel(const float* __restrict__ part, const int* __restrict__ tiles, const float* __restrict__ Piv, int B, int H,
            int G, int rot, int QT, int nqt, int W, int group, T* __restrict__ out, float* __restrict__ fin) {
  constexpr int kRows = kPD * kPD / kJoinThreads;
  __shared__ float wm[kJoinWarps], wl[kJoinWarps];
  __shared__ __align__(16) float wacc[kJoinWarps][kPD];
  __shared__ __align__(16) float norm[kJoinQ][kPD];
  __shared__ float sums[kJoinQ][kPD * kPD / (kPD * kRows)][kPD];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bh = blockIdx.x, b = bh / H, h = bh - b * H, q0 = blockIdx.y * group;
  const int nq = min(group, G - q0);
  const int d = tid & (kPD - 1), r = tid / kPD;
  const float* P = Piv + (static_cast<size_t>(h % rot) * kPD + r * kRows) * kPD + d;
  float pv[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) pv[k] = __ldg(P + k * kPD);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int per = H * nqt, T0 = tiles[b], nt = tiles[b + 1] - T0, total = tiles[B] * per;
  const int rq = total / W, rr = total - rq * W;
  const int mine = warp & (group - 1), each = kJoinWarps / group;   // this warp's query, and its warps
  {
    const int qi = min(q0 + mine, G - 1), j = qi / QT, c = qi - j * QT;
    const int unit = b * per + h * nqt + j, t0 = T0 * per + (h * nqt + j) * nt;
    float M = -INFINITY, Ls = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (nt > 0) {
      const int first = run_of(t0, rq, rr), last = run_of(t0 + nt - 1, rq, rr);
      for (int w = first + warp / group; w <= last; w += each * kJoinSlots) {
        float2 ml[kJoinSlots];
        float4 x[kJoinSlots];
#pragma unroll
        for (int k = 0; k < kJoinSlots; ++k) {
          const int wk = w + k * each;
          if (wk <= last) {
            const float* pp = part + (static_cast<size_t>(wk + unit) * QT + c) * kPartF;
            ml[k] = *reinterpret_cast<const float2*>(pp + kPD);
            x[k] = *reinterpret_cast<const float4*>(pp + 4 * lane);
          } else {
            ml[k] = make_float2(-INFINITY, 0.f);
            x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          }
        }
        float m = M;
#pragma unroll
        for (int k = 0; k < kJoinSlots; ++k) m = fmaxf(m, ml[k].x);
        const float ref = m > -INFINITY ? m : 0.f;
        const float f = exp2f(M - ref);                    // 0 while there is no weight
        Ls *= f;
        a.x *= f; a.y *= f; a.z *= f; a.w *= f;
#pragma unroll
        for (int k = 0; k < kJoinSlots; ++k) {
          const float e = exp2f(ml[k].x - ref);
          Ls = fmaf(ml[k].y, e, Ls);
          a.x = fmaf(x[k].x, e, a.x);
          a.y = fmaf(x[k].y, e, a.y);
          a.z = fmaf(x[k].z, e, a.z);
          a.w = fmaf(x[k].w, e, a.w);
        }
        M = m;
      }
    }
    if (lane == 0) {
      wm[warp] = M;
      wl[warp] = Ls;
    }
    *reinterpret_cast<float4*>(&wacc[warp][4 * lane]) = a;
  }
  __syncthreads();
  for (int i = r; i < nq; i += kJoinThreads / kPD) {       // a query for each 128 threads
    float m = -INFINITY;
    for (int w = i; w < kJoinWarps; w += group) m = fmaxf(m, wm[w]);
    const float ref = m > -INFINITY ? m : 0.f;
    float s = 0.f, l = 0.f;
    for (int w = i; w < kJoinWarps; w += group) {
      const float e = exp2f(wm[w] - ref);
      s = fmaf(wacc[w][d], e, s);
      l = fmaf(wl[w], e, l);
    }
    norm[i][d] = l != 0.f ? s / l : 0.f;                   // no slot at all: zeros
    if (fin != nullptr && d == 0)
      *reinterpret_cast<float2*>(fin + 2 * (static_cast<size_t>(bh) * G + q0 + i)) = make_float2(ref, l != 0.f ? 1.f / l : 0.f);
  }
  __syncthreads();
  for (int i = 0; i < nq; ++i) {
    float o = 0.f;
#pragma unroll
    for (int k = 0; k < kRows; k += 4) {
      const float4 v = *reinterpret_cast<const float4*>(&norm[i][r * kRows + k]);
      o = fmaf(v.x, pv[k], o);
      o = fmaf(v.y, pv[k + 1], o);
      o = fmaf(v.z, pv[k + 2], o);
      o = fmaf(v.w, pv[k + 3], o);
    }
    sums[i][r][d] = o;
  }
  __syncthreads();
  for (int i = r; i < nq; i += kJoinThreads / kPD)
    store_o(out, (static_cast<size_t>(bh) * G + q0 + i) * kPD + d, sums[i][0][d] + sums[i][1][d] + sums[i][2][d] + sums[i][3][d]);
}

// mass[b,h,s] += sum over the group's queries of 2^(z - M) / L.  Four slots a thread.
constexpr int kMassSlots = 1024;

__global__ void __launch_bounds__(256)
mass_kernel(const float* __restrict__ z, const float* __restrict__ fin, const int* __restrict__ cut, int H, int G,
            int QT, int nqt, int cap, int S, float* __restrict__ mass) {
  const int chunks = (cap + kMassSlots - 1) / kMassSlots;
  const int bh = blockIdx.x / chunks, s0 = (blockIdx.x - bh * chunks) * kMassSlots + threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n = cut[bh / H];
  if (s0 - static_cast<int>(threadIdx.x) >= n) return;
  float sum[4] = {0.f, 0.f, 0.f, 0.f}, old[4];
  float* to = mass + static_cast<size_t>(bh) * S;
#pragma unroll
  for (int k = 0; k < 4; ++k) old[k] = s0 + 256 * k < n ? to[s0 + 256 * k] : 0.f;
  for (int j = 0; j < nqt; ++j) {
    const float* zj = z + static_cast<size_t>(bh * nqt + j) * S * QT;
    for (int c0 = 0; c0 < QT; c0 += 4) {
      if (j * QT + c0 >= G) break;
      float4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        v[k] = s0 + 256 * k < n ? *reinterpret_cast<const float4*>(zj + static_cast<size_t>(s0 + 256 * k) * QT + c0)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int qi = j * QT + c0 + c;
        if (qi < G) {
          const float2 f = *reinterpret_cast<const float2*>(fin + 2 * (static_cast<size_t>(bh) * G + qi));
#pragma unroll
          for (int k = 0; k < 4; ++k) sum[k] = fmaf(exp2f((c == 0 ? v[k].x : c == 1 ? v[k].y : c == 2 ? v[k].z : v[k].w) - f.x), f.y, sum[k]);
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (s0 + 256 * k < n) to[s0 + 256 * k] = old[k] + sum[k];
}

// Workspace: rotated queries, tiles, cut lengths, maxima and sums, partials, logits.
struct Space {
  size_t A, tiles, cut, fin, part, z, all;
  Space(int B, int H, int G, int S, bool mass) {
    const size_t units = static_cast<size_t>(B) * H;
    size_t at = 0;
    auto take = [&at](size_t bytes) { const size_t o = at; at += paged_round(bytes); return o; };
    A = take(units * G * kPD * 4);
    tiles = take((static_cast<size_t>(B) + 1) * 4);
    cut = take(static_cast<size_t>(B) * 4);
    fin = take(units * G * 8);
    // query tiles of 8, or twice as many of 4: at most this many floats either way
    part = take((kMaxCtas * kSplitWarps + units * ((G + 7) / 8)) * 8 * kPartF * 4);
    z = take(mass ? units * (G <= 4 ? 4 : (G + 7) / 8 * 8) * static_cast<size_t>(S) * 4 : 0);
    all = at;
  }
};

template <typename T>
cudaError_t launch(const tq_paged_cache& c, const T* Q, const int* table, const int* lengths, int B, int G,
                   int max_pages, float scale, float* mass, int S, T* out, char* ws, cudaStream_t st) {
  static std::atomic<int> sms_cache[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int sms = sms_cache[dev & 63].load(std::memory_order_relaxed);
  if (sms == 0) {
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    sms_cache[dev & 63].store(sms, std::memory_order_relaxed);
  }
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  int cap = max_pages * c.page_size;
  if (mass != nullptr && S < cap) cap = S;
  const bool f32 = sizeof(T) == 4;
  const int variant = f32 ? kVarF32 : mass == nullptr ? kVarFast : G <= 4 ? kVarMass4 : kVarMass8;
  const int QT = variant == kVarFast || variant == kVarMass8 ? 8 : 4, nqt = (G + QT - 1) / QT;
  const Space sp(B, c.H, G, S, mass != nullptr);
  float* A = reinterpret_cast<float*>(ws + sp.A);
  int* tiles = reinterpret_cast<int*>(ws + sp.tiles);
  int* cut = reinterpret_cast<int*>(ws + sp.cut);
  float* fin = mass == nullptr ? nullptr : reinterpret_cast<float*>(ws + sp.fin);
  float* part = reinterpret_cast<float*>(ws + sp.part);
  float* z = mass == nullptr ? nullptr : reinterpret_cast<float*>(ws + sp.z);

  plan_kernel<T><<<B * c.H * 4 + 1, kPlanThreads, 0, st>>>(Q, lengths, c.Pi_k, B, c.H, G, c.rot_heads, cap, A, tiles, cut);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const Paged pg = paged_view(c, table, max_pages);
  const SplitArgs a = {c.k_plane, c.v_plane, c.k_norm, c.v_norm, table, c.n_pages, c.H, pg.shift, max_pages, A, tiles,
                       cut, c.k_codebook, c.v_codebook, part, z, B, G, nqt, S, scale * 1.4426950408889634f,
                       {1, 2, 4, 8, 16, 32, 64, 128}};
  switch (c.k_bits) {
    case 2: e = launch_split_k2(a, c.v_bits, variant, ctas, st); break;
    case 3: e = launch_split_k3(a, c.v_bits, variant, ctas, st); break;
    default: e = launch_split_k4(a, c.v_bits, variant, ctas, st); break;
  }
  if (e != cudaSuccess) return e;

  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // one query a block while that does not fill the SMs, up to 8 (Pi_v is then read once for them)
  const int64_t queries = static_cast<int64_t>(B) * c.H * G;
  int group = 1;
  while (group < kJoinQ && group < G && queries > static_cast<int64_t>(sms) * group) group *= 2;
  cfg.gridDim = dim3(B * c.H, (G + group - 1) / group);
  cfg.blockDim = dim3(kJoinThreads);
  e = cudaLaunchKernelEx(&cfg, join_kernel<T>, static_cast<const float*>(part), static_cast<const int*>(tiles), c.Pi_v,
                         B, c.H, G, c.rot_heads, QT, nqt, ctas * kSplitWarps, group, out, fin);
  if (e != cudaSuccess || mass == nullptr) return e;
  cfg.gridDim = dim3((cap + kMassSlots - 1) / kMassSlots * B * c.H);
  cfg.blockDim = dim3(256);
  return cudaLaunchKernelEx(&cfg, mass_kernel, static_cast<const float*>(z), static_cast<const float*>(fin),
                            static_cast<const int*>(cut), c.H, G, QT, nqt, cap, S, mass);
}

}  // namespace

cudaError_t take_faults_split_k2(unsigned int* bits);
cudaError_t take_faults_split_k3(unsigned int* bits);
cudaError_t take_faults_split_k4(unsigned int* bits);

size_t decode_paged_bytes(int B, int H, int G, int S, bool with_mass) { return Space(B, H, G, S, with_mass).all; }

cudaError_t launch_decode_paged(const tq_paged_cache& c, const void* Q, tq_qtype qtype, const int* table,
                                const int* lengths, int B, int G, int max_pages, float scale, float* mass,
                                int S, void* out, void* ws, cudaStream_t st) {
  if (qtype == TQ_Q_F32)
    return launch(c, static_cast<const float*>(Q), table, lengths, B, G, max_pages, scale, mass, S,
                  static_cast<float*>(out), static_cast<char*>(ws), st);
  return launch(c, static_cast<const __nv_bfloat16*>(Q), table, lengths, B, G, max_pages, scale, mass, S,
                static_cast<__nv_bfloat16*>(out), static_cast<char*>(ws), st);
}

cudaError_t take_faults_paged(unsigned int* bits) {
  cudaError_t e = take_unit_faults(bits);
  if (e == cudaSuccess) e = take_faults_split_k2(bits);
  if (e == cudaSuccess) e = take_faults_split_k3(bits);
  if (e == cudaSuccess) e = take_faults_split_k4(bits);
  return e;
}

}  // namespace tq
