// The routing step of a mixture-of-experts layer on FP32 router logits
// [M][E], forward and backward.
//
//   lse[m] = log sum_e exp(l[m][e]),  p[m][e] = exp(l[m][e] - lse[m])
//     (computed as exp(l - max) / sum exp(l - max): in a row masked with the
//     type's lowest value lse itself rounds the sum away)
//   experts[m] = the k largest logits (ties: lowest index; -inf never)
//   weights[m] = p at the experts, divided by their sum if asked
//   T = rows that take part, counts[e] = rows that chose e,
//   P[e] = sum_m p[m][e] / T
//   balance = E sum_e counts[e] / (k T) P[e],   z = sum_m lse[m]^2 / T
//
// A row takes part if it is valid and has a logit above -inf.  A NaN logit
// ranks first and makes the row's results NaN.
//
// Both kernels read the logits once: one warp per row, the row in registers,
// sums and statistics in FP32.  Each warp keeps the column sums of its rows
// in registers; blocks add their warps' sums and a second, small grid adds
// the blocks', both in a fixed order.
//
// Measured (top-8 of 256): one row 3.1 us forward, 1.8 us backward; 4510 rows
// 8.6 and 3.5 us; 65536 rows 37.4 us forward (40.0 with closed experts and
// padding rows; bound by issuing, 447 instructions a row there) and 26.6 us
// backward (5.2 TB/s of logits and gradients).
// A row is a chain of reductions about 2 us long, so small calls are bound by
// latency; up to kOneBlockRows rows one block does without the second grid.
#include <cuda_bf16.h>

#include <float.h>

#include <algorithm>
#include <atomic>

#include "internal.h"
#include "ptx.cuh"

namespace gb300 {
namespace {

constexpr int kWarps = 16;            // forward: rows in flight per block
constexpr int kMaxBlocks = 304;       // forward: two blocks per SM; bounds the partial sums
constexpr int kFinishCtas = 8;        // the cluster that adds the blocks' sums
constexpr int kFinishGroups = 16;
constexpr int kFinishThreads = 32 * (kFinishGroups + 1);
constexpr int kGradWarps = 8;         // backward: rows in flight per block
constexpr int kGradMaxBlocks = 608;   // four blocks per SM
constexpr int kOneBlockRows = 2 * kWarps;  // up to this many rows need no second grid

// Partial sums of one block: probabilities [E], z, then the counts [E], T.
__host__ __device__ constexpr int partial_words(int E) { return 2 * E + 2; }

// e^y, relative error below 2^-21 + 2^-23 |y|
__device__ __forceinline__ float fast_exp(float y) { return ptx::ex2(y * 1.4426950408889634f); }

// Order-preserving key of a logit: larger key = ranks earlier.  -0 = +0, NaN
// first; keys up to kNoKey (-inf) are never chosen.
constexpr uint32_t kNoKey = 0x007FFFFFu;
__device__ __forceinline__ uint32_t rank_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  if (v != v) return 0xFFFFFFFFu;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Value i of lane `lane` is column column_of(i, lane): groups of four
// consecutive columns, read and written 16 bytes at a time where kAligned says
// that rows start on 16 bytes and E % 4 == 0, value by value (through L1)
// otherwise.  The same columns either way, so results do not depend on it.
__device__ __forceinline__ int column_of(int i, int lane) {
  return ((i / 4) * 32 + lane) * 4 + i % 4;
}

// The lane's NV values of one row; -inf past column E.
template <int NV, bool kAligned>
__device__ __forceinline__ void load_row(const float* src, int E, int lane, float (&v)[NV]) {
#pragma unroll
  for (int i = 0; i < NV; i += 4) {
    const int e = column_of(i, lane);
    if constexpr (kAligned) {
      float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (e < E) q = __ldcg(reinterpret_cast<const float4*>(src + e));
      v[i] = q.x, v[i + 1] = q.y, v[i + 2] = q.z, v[i + 3] = q.w;
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) v[i + c] = e + c < E ? src[e + c] : -INFINITY;
    }
  }
}

struct RouteArgs {
  const float* logits;
  const unsigned char* valid;
  float* weights;
  int* experts;
  float* lse;
  int* counts;
  float* probs;
  float* losses;
  uint32_t* partial;
  int M, E, ld, k, normalize;
};

__device__ __forceinline__ float at_least_one(int T) { return float(T > 1 ? T : 1); }

// Sum over the block's threads, valid in thread 0; `red` holds one float per warp.
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  if (threadIdx.x == 0)
    for (int w = 0; w < int(blockDim.x >> 5); ++w) s += red[w];
  return s;
}

// NV: values per lane (E <= 32 NV)
template <int NV, bool kAligned>
__global__ void __launch_bounds__(32 * kWarps, NV <= 8 ? 2 : 1) route_kernel(const RouteArgs a) {
  extern __shared__ __align__(16) uint32_t sh[];
  float* sh_prob = reinterpret_cast<float*>(sh);             // [kWarps][E]
  int* sh_hits = reinterpret_cast<int*>(sh + kWarps * a.E);  // [E]
  // each warp's row, 32 NV values, 16-byte aligned
  __shared__ float sh_z[kWarps], red[kWarps];
  __shared__ int sh_t[kWarps];
  __shared__ __align__(16) unsigned long long sh_cand[kWarps][32];
  float* row_vals = reinterpret_cast<float*>(
      sh + (kWarps + 1) * ((a.E + 3) / 4 * 4) + (threadIdx.x >> 5) * 32 * NV);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) sh_hits[e] = 0;
  __syncthreads();
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();

  float acc[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) acc[i] = 0.0f;
  float z = 0.0f;
  int t = 0;
  unsigned long long* cand = sh_cand[warp];
  const long long step = (long long)gridDim.x * kWarps;
  for (long long row = (long long)blockIdx.x * kWarps + warp; row < a.M; row += step) {
    const bool valid = !a.valid || __ldcg(a.valid + row) != 0;
    float v[NV];
    load_row<NV, kAligned>(a.logits + row * a.ld, a.E, lane, v);
    float lane_max = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) lane_max = fmaxf(lane_max, v[i]);
    const float mx = ptx::redux_max(lane_max);
    const float ref = mx == -INFINITY ? 0.0f : mx;
    float s = 0.0f, p[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) s += p[i] = fast_exp(v[i] - ref);
    s = warp_sum(s);
    const float inv = ptx::rcp(s);
    const float l = ref + logf(s);
    if (lane == 0) a.lse[row] = l;
    // a sum of 0 is a row of -inf only (a NaN makes the sum NaN)
    const bool live = valid && s != 0.0f;
    if (live) {
      z += l * l;
      ++t;
#pragma unroll
      for (int i = 0; i < NV; ++i) acc[i] += p[i] * inv;
    }

    // Choice.  The k-th largest of the lanes' maxima (equal ones counted once)
    // bounds the k-th largest value from below, so only values that reach it
    // are candidates: usually little more than k, which rank themselves
    // against each other.
    int my_expert = -1, my_rank = lane;
    float my_weight = 0.0f;
    bool slow = live && s != s;  // NaN somewhere
    if (live && !slow) {
      float bound = mx, cur = lane_max;
      for (int r = 1; r < a.k; ++r) {
        if (cur == bound) cur = -INFINITY;
        bound = ptx::redux_max(cur);
      }
      // fewer than k lanes with a value: every value above -inf is a candidate
      bound = fmaxf(bound, -FLT_MAX);
      uint32_t mine = 0u;  // bit i: value i is a candidate
#pragma unroll
      for (int i = 0; i < NV; ++i) mine |= v[i] >= bound ? 1u << i : 0u;
      int n = __popc(mine), at = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int left = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += left;
      }
      at -= n;                                        // candidates of the lanes before
      n = __shfl_sync(0xffffffffu, at + n, 31);       // of all lanes
      slow = n > 32;
      if (!slow) {
        // the row goes through shared memory, where a lane can pick by index
#pragma unroll
        for (int i = 0; i < NV; i += 4)
          *reinterpret_cast<float4*>(row_vals + column_of(i, lane)) =
              make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        for (; mine; mine &= mine - 1u, ++at) {
          const int e = column_of(__ffs(int(mine)) - 1, lane);
          cand[at] = (static_cast<unsigned long long>(rank_key(row_vals[e])) << 32) |
                     (0xFFFFFFFFu - uint32_t(e));
        }
        if (lane == 0 && n % 2) cand[n] = 0ull;  // read in pairs below
        __syncwarp();
        const unsigned long long own = lane < n ? cand[lane] : 0ull;
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < n; j += 2) {
          const ulonglong2 other = *reinterpret_cast<const ulonglong2*>(cand + j);
          rank += int(other.x > own) + int(other.y > own);
        }
        __syncwarp();
        if (lane < n) {
          if (rank < a.k) {
            my_expert = int(0xFFFFFFFFu - uint32_t(own));
            my_weight = fast_exp(key_value(uint32_t(own >> 32)) - ref) * inv;
          }
          my_rank = rank;
        }
      }
    }
    if (slow) {  // NaN, or more than 32 candidates (ties): k rounds of the largest key
      uint32_t key[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) key[i] = rank_key(v[i]);
      my_rank = lane;
      for (int r = 0; r < a.k; ++r) {
        uint32_t best = 0u;
        int at = 0x7FFFFFFF;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (key[i] > best) {
            best = key[i];
            at = column_of(i, lane);
          }
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        if (top <= kNoKey) break;
        const int win = __reduce_min_sync(0xffffffffu, best == top ? at : 0x7FFFFFFF);
        float w = 0.0f;
        bool owner = false;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (column_of(i, lane) == win) {
            key[i] = 0u;
            w = p[i] * inv;
            owner = true;
          }
        w = __shfl_sync(0xffffffffu, w, __ffs(__ballot_sync(0xffffffffu, owner)) - 1);
        if (lane == r) {
          my_expert = win;
          my_weight = w;
        }
      }
    }
    if (a.normalize) {
      const float total = warp_sum(my_expert >= 0 ? my_weight : 0.0f);
      if (my_expert >= 0) my_weight *= ptx::rcp(total);
    }
    if (my_rank < a.k) {
      a.weights[row * a.k + my_rank] = my_weight;
      a.experts[row * a.k + my_rank] = my_expert;
      if (my_expert >= 0) atomicAdd(sh_hits + my_expert, 1);  // integers: any order
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = column_of(i, lane);
    if (e < a.E) sh_prob[warp * a.E + e] = acc[i];
  }
  if (lane == 0) {
    sh_z[warp] = z;
    sh_t[warp] = t;
  }
  __syncthreads();
  float zb = 0.0f;
  int tb = 0;
  for (int w = 0; w < kWarps; ++w) {
    zb += sh_z[w];
    tb += sh_t[w];
  }
  const bool alone = gridDim.x == 1;
  const float T = at_least_one(tb);
  uint32_t* out = alone ? nullptr : a.partial + size_t(blockIdx.x) * partial_words(a.E);
  float dot = 0.0f;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += sh_prob[w * a.E + e];
    const int c = sh_hits[e];
    if (alone) {
      a.probs[e] = sum / T;
      a.counts[e] = c;
      dot += float(c) / (float(a.k) * T) * (sum / T);
    } else {
      out[e] = __float_as_uint(sum);
      out[a.E + 1 + e] = uint32_t(c);
    }
  }
  if (alone) {
    dot = block_sum(dot, red);
    if (threadIdx.x == 0) {
      a.losses[0] = float(a.E) * dot;
      a.losses[1] = zb / T;
      a.counts[a.E] = tb;
    }
  } else if (threadIdx.x == 0) {
    out[a.E] = __float_as_uint(zb);
    out[2 * a.E + 1] = uint32_t(tb);
  }
}

// Adds the blocks' partial sums: one cluster, each CTA a slice of the columns,
// then the first CTA adds the slices' parts of the balance loss.  In a CTA,
// warp g of the first kFinishGroups takes the blocks b = g mod kFinishGroups,
// lane = column, and the groups are added in order; the last warp adds z and T
// (column E) meanwhile.  All loads of a thread are independent, so that one
// memory latency covers them.
__global__ void __cluster_dims__(kFinishCtas, 1, 1) __launch_bounds__(kFinishThreads)
    route_finish_kernel(const RouteArgs a, int blocks) {
  __shared__ float sum[kFinishGroups][33];
  __shared__ int hit[kFinishGroups][33];
  __shared__ float z_sum;
  __shared__ int T_sum;
  __shared__ float dots[kFinishCtas];
  ptx::cluster_sync();  // every CTA runs before its shared memory is written remotely
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int words = partial_words(a.E);
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int rank = int(ptx::cluster_ctarank());
  const int per = (a.E + kFinishCtas - 1) / kFinishCtas;
  const int e1 = min(a.E, (rank + 1) * per);
  float dot = 0.0f;
  for (int e0 = rank * per; e0 == rank * per || e0 < e1; e0 += 32) {
    const int e = e0 + lane;
    float fs = 0.0f;
    int ic = 0;
    if (g < kFinishGroups) {
      if (e < e1) {
        constexpr int kPer = (kMaxBlocks + kFinishGroups - 1) / kFinishGroups;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int b = g + i * kFinishGroups;
          if (b < blocks) {
            const uint32_t* src = a.partial + size_t(b) * words;
            fs += __uint_as_float(__ldcg(src + e));
            ic += int(__ldcg(src + a.E + 1 + e));
          }
        }
      }
      sum[g][lane] = fs;
      hit[g][lane] = ic;
    } else if (e0 == rank * per) {
      constexpr int kPer = (kMaxBlocks + 31) / 32;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int b = lane + i * 32;
        if (b < blocks) {
          const uint32_t* src = a.partial + size_t(b) * words;
          fs += __uint_as_float(__ldcg(src + a.E));
          ic += int(__ldcg(src + 2 * a.E + 1));
        }
      }
      fs = warp_sum(fs);
      ic = __reduce_add_sync(0xffffffffu, ic);
      if (lane == 0) {
        z_sum = fs;
        T_sum = ic;
      }
    }
    __syncthreads();
    if (g == 0 && e < e1) {
      float s = 0.0f;
      int c = 0;
#pragma unroll
      for (int i = 0; i < kFinishGroups; ++i) {
        s += sum[i][lane];
        c += hit[i][lane];
      }
      const float T = at_least_one(T_sum);
      const float P = s / T;
      a.probs[e] = P;
      a.counts[e] = c;
      dot += float(c) / (float(a.k) * T) * P;
    }
    __syncthreads();
  }
  if (g == 0) {
    dot = warp_sum(dot);
    if (lane == 0) ptx::st_cluster_f32(ptx::mapa_shared(ptx::smem_u32(&dots[rank]), 0), dot);
  }
  ptx::cluster_sync();
  if (rank == 0 && threadIdx.x == 0) {
    float d = 0.0f;
    for (int i = 0; i < kFinishCtas; ++i) d += dots[i];
    a.losses[0] = float(a.E) * d;
    a.losses[1] = z_sum / at_least_one(T_sum);
    a.counts[a.E] = T_sum;
  }
}

struct RouteGradArgs {
  const float* logits;
  const int* experts;
  const float* lse;
  const int* counts;
  const float* dweights;
  const float* dlosses;
  void* dlogits;
  int M, E, ld, k, normalize;
};

// With e = exp(l - lse) (lse only has to be near the row's maximum: e is
// divided by its own sum s, so that p keeps its precision in rows where lse
// has rounded the sum away) and, over the row, A = the taken experts:
//   dl[e] = p[e] (dp[e] - sum_f p[f] dp[f] + 2 d_z lse / T)
//   dp[e] = d_balance E counts[e] / (k T^2) + u[e],   u = 0 outside A
//   u[e]  = dw[e], or normalised (dw[e] - q) / a with a = sum_A p and
//           q = sum_A p dw / a; then sum_f p[f] u[f] = 0
// so one pass of four sums (s, sum e base, sum_A e, sum_A e dw) gives all that
// a row needs.  The k lanes that hold the gradients dw read their e from a row
// of shared memory and give u back through another, zero elsewhere.
template <int NV, bool kAligned, bool kBF16>
__global__ void __launch_bounds__(32 * kGradWarps, NV <= 8 ? 4 : 2)
    route_grad_kernel(const RouteGradArgs a) {
  extern __shared__ __align__(16) uint32_t sh[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int up_row = (a.E + 3) / 4 * 4;  // whole 16-byte groups
  float* base = reinterpret_cast<float*>(sh);  // [up_row] dp's first term
  float* up = base + (1 + 2 * warp) * up_row;  // [up_row] u
  float* er = up + up_row;                     // [up_row] e
  for (int e = lane; e < up_row; e += 32) up[e] = 0.0f;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const float t = at_least_one(a.counts[a.E]);
  const float db = a.dlosses ? a.dlosses[0] : 0.0f;
  const float dz = a.dlosses ? a.dlosses[1] : 0.0f;
  const float c0 = db * float(a.E) / (float(a.k) * t) / t;
  const float c1 = 2.0f * dz / t;
  // once per block: read by every row, these few lines of memory are the same
  // for the whole grid
  for (int e = threadIdx.x; e < up_row; e += blockDim.x)
    base[e] = e < a.E ? c0 * float(a.counts[e]) : 0.0f;
  __syncthreads();
  const long long step = (long long)gridDim.x * kGradWarps;
  for (long long row = (long long)blockIdx.x * kGradWarps + warp; row < a.M; row += step) {
    float p[NV];
    load_row<NV, kAligned>(a.logits + row * a.ld, a.E, lane, p);
    const float l = __ldcg(a.lse + row);
    int ex = -1;
    float g = 0.0f;
    if (lane < a.k) {
      ex = __ldcg(a.experts + row * a.k + lane);
      if (a.dweights) g = __ldcg(a.dweights + row * a.k + lane);
      if (ex >= a.E) ex = -1;  // not an expert: takes no part
    }
    const bool live = __shfl_sync(0xffffffffu, ex, 0) >= 0;
    float s = 0.0f, sb = 0.0f, sa = 0.0f, sg = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; i += 4) {
      const int e = column_of(i, lane);
#pragma unroll
      for (int c = i; c < i + 4; ++c) {
        p[c] = fast_exp(p[c] - l);
        s += p[c];
      }
      if (e < up_row) {
        const float4 b = *reinterpret_cast<const float4*>(base + e);
        sb += p[i] * b.x + p[i + 1] * b.y + p[i + 2] * b.z + p[i + 3] * b.w;
        *reinterpret_cast<float4*>(er + e) = make_float4(p[i], p[i + 1], p[i + 2], p[i + 3]);
      }
    }
    __syncwarp();
    if (ex >= 0) {
      sa = er[ex];
      sg = sa * g;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      sb += __shfl_xor_sync(0xffffffffu, sb, o);
      sa += __shfl_xor_sync(0xffffffffu, sa, o);
      sg += __shfl_xor_sync(0xffffffffu, sg, o);
    }
    const float inv = ptx::rcp(s);
    if (ex >= 0) {
      // q = sg / sa: the sum of the weights times their gradients; s / sa: 1 /
      // (the sum of the taken p)
      const float a1 = ptx::rcp(sa);
      up[ex] = a.normalize ? (g - sg * a1) * (s * a1) : g;
    }
    __syncwarp();
    const float shift = c1 * l - (sb + (a.normalize ? 0.0f : sg)) * inv;
#pragma unroll
    for (int i = 0; i < NV; i += 4) {
      const int e = column_of(i, lane);
      float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (live && e < up_row) {
        const float4 b = *reinterpret_cast<const float4*>(base + e);
        const float4 u = *reinterpret_cast<const float4*>(up + e);
        d[0] = p[i] * inv * (b.x + u.x + shift);
        d[1] = p[i + 1] * inv * (b.y + u.y + shift);
        d[2] = p[i + 2] * inv * (b.z + u.z + shift);
        d[3] = p[i + 3] * inv * (b.w + u.w + shift);
      }
      const size_t off = size_t(row) * a.E + e;
      // BF16: one rounding, for a gradient that goes into a BF16 product
      if constexpr (kBF16) {
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.dlogits) + off;
        if constexpr (kAligned) {
          const __nv_bfloat162 lo = __floats2bfloat162_rn(d[0], d[1]);
          const __nv_bfloat162 hi = __floats2bfloat162_rn(d[2], d[3]);
          if (e < a.E)
            *reinterpret_cast<uint2*>(out) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                                        *reinterpret_cast<const uint32_t*>(&hi));
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (e + c < a.E) out[c] = __float2bfloat16_rn(d[c]);
        }
      } else {
        float* out = static_cast<float*>(a.dlogits) + off;
        if constexpr (kAligned) {
          if (e < a.E) *reinterpret_cast<float4*>(out) = make_float4(d[0], d[1], d[2], d[3]);
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (e + c < a.E) out[c] = d[c];
        }
      }
    }
    __syncwarp();
    if (ex >= 0) up[ex] = 0.0f;
  }
}

int route_blocks(int M) {
  if (M <= kOneBlockRows) return 1;
  return int(std::min<long long>(kMaxBlocks, ((long long)M + kWarps - 1) / kWarps));
}

template <class Kernel, class... Args>
int launch(Kernel kernel, int grid, int threads, size_t shared, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  return GEMM_OK;
}

// Dynamic shared memory of a launch.
constexpr size_t route_shared(int E, int NV) {
  return (size_t(kWarps + 1) * ((E + 3) / 4 * 4) + size_t(kWarps) * 32 * NV) * 4;
}
constexpr size_t route_grad_shared(int E) {
  return size_t(2 * kGradWarps + 1) * ((E + 3) / 4 * 4) * 4;
}

// Past the default limit (together with the static arrays) a kernel has to be
// allowed its dynamic shared memory.  The attribute belongs to the kernel and
// its last value counts, so it is set once per device, to the most that any E
// of the kernel needs: a value per call could be lowered by another host thread
// before the launch.
template <auto kKernel, size_t kMost>
bool allow_shared(const DeviceInfo& dev) {
  if constexpr (kMost > 40 * 1024) {
    static std::atomic<bool> allowed[64];
    std::atomic<bool>& done = allowed[dev.device & 63];
    if (done.load()) return true;
    if (cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMost)) !=
        cudaSuccess) {
      cudaGetLastError();
      return false;
    }
    done.store(true);
  }
  return true;
}

template <int NV, bool kAligned>
int run_route(const RouteArgs& a, int blocks, const DeviceInfo& dev, cudaStream_t stream) {
  if (!allow_shared<route_kernel<NV, kAligned>, route_shared(32 * NV, NV)>(dev))
    return GEMM_ERR_LAUNCH;
  return launch(route_kernel<NV, kAligned>, blocks, 32 * kWarps, route_shared(a.E, NV), stream, a);
}

template <int NV, bool kAligned, bool kBF16>
int run_route_grad(const RouteGradArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  if (!allow_shared<route_grad_kernel<NV, kAligned, kBF16>, route_grad_shared(32 * NV)>(dev))
    return GEMM_ERR_LAUNCH;
  const int blocks = int(
      std::min<long long>(kGradMaxBlocks, ((long long)a.M + kGradWarps - 1) / kGradWarps));
  return launch(route_grad_kernel<NV, kAligned, kBF16>, blocks, 32 * kGradWarps,
                route_grad_shared(a.E), stream, a);
}

// The smallest row buffer that holds E columns.
template <bool kAligned>
int pick_route(const RouteArgs& a, int blocks, const DeviceInfo& dev, cudaStream_t stream) {
  if (a.E <= 128) return run_route<4, kAligned>(a, blocks, dev, stream);
  if (a.E <= 256) return run_route<8, kAligned>(a, blocks, dev, stream);
  if (a.E <= 512) return run_route<16, kAligned>(a, blocks, dev, stream);
  return run_route<32, kAligned>(a, blocks, dev, stream);
}

template <bool kAligned, bool kBF16>
int pick_route_grad(const RouteGradArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  if (a.E <= 128) return run_route_grad<4, kAligned, kBF16>(a, dev, stream);
  if (a.E <= 256) return run_route_grad<8, kAligned, kBF16>(a, dev, stream);
  if (a.E <= 512) return run_route_grad<16, kAligned, kBF16>(a, dev, stream);
  return run_route_grad<32, kAligned, kBF16>(a, dev, stream);
}

bool aligned_to(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace

size_t router_topk_workspace(int M, int E) {
  const int b = route_blocks(M);
  return b > 1 ? size_t(b) * partial_words(E) * 4 : 0;
}

int launch_router_topk(const RouterTopk& r, const DeviceInfo& dev, cudaStream_t stream) {
  const RouteArgs a{r.logits, r.valid, r.weights, r.experts, r.lse, r.counts, r.probs, r.losses,
                    static_cast<uint32_t*>(r.workspace), r.M, r.E, r.ld, r.k, r.normalize};
  const int blocks = route_blocks(r.M);
  const bool aligned = r.E % 4 == 0 && (r.ld % 4 == 0 || r.M == 1) && aligned_to(r.logits, 16);
  const int rc = aligned ? pick_route<true>(a, blocks, dev, stream)
                         : pick_route<false>(a, blocks, dev, stream);
  if (rc != GEMM_OK || blocks == 1) return rc;
  return launch(route_finish_kernel, kFinishCtas, kFinishThreads, 0, stream, a, blocks);
}

int launch_router_topk_backward(const RouterTopkBackward& r, const DeviceInfo& dev,
                                cudaStream_t stream) {
  const RouteGradArgs a{r.logits, r.experts, r.lse, r.counts, r.dweights, r.dlosses, r.dlogits,
                        r.M, r.E, r.ld, r.k, r.normalize};
  const bool aligned = r.E % 4 == 0 && (r.ld % 4 == 0 || r.M == 1) && aligned_to(r.logits, 16) &&
                   aligned_to(r.dlogits, r.bf16 ? 8 : 16);
  if (r.bf16)
    return aligned ? pick_route_grad<true, true>(a, dev, stream)
                   : pick_route_grad<false, true>(a, dev, stream);
  return aligned ? pick_route_grad<true, false>(a, dev, stream)
                 : pick_route_grad<false, false>(a, dev, stream);
}

}  // namespace gb300
