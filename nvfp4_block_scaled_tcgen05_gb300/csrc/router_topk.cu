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
// Both kernels read the logits once: one warp per row, the row in registers
// (element e of a row in lane e % 32), sums and statistics in FP32.
#include <cuda_bf16.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace gb300 {
namespace {

constexpr int kWarps = 8;            // rows in flight per block
constexpr int kMaxBlocks = 304;      // two blocks per SM; bounds the partial sums
constexpr int kFinishThreads = 1024;

// Partial sums of one block: probabilities [E], z, then the counts [E], T.
__host__ __device__ constexpr size_t partial_words(int E) { return 2 * size_t(E) + 2; }

// Order-preserving key of a logit: larger key = ranks earlier.  -0 = +0, NaN
// first; keys up to kNoKey (-inf) are never chosen.
constexpr uint32_t kNoKey = 0x007FFFFFu;
__device__ __forceinline__ uint32_t rank_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  if (v != v) return 0xFFFFFFFFu;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
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

// balance, z, P and counts from the sums over all rows.  Called by one whole
// block; prob(e), hits(e) give column e's sums.
template <class Prob, class Hits>
__device__ void finish(const RouteArgs& a, float z_sum, int T, Prob prob, Hits hits) {
  __shared__ float red[32];
  const float t = float(T > 1 ? T : 1);
  float dot = 0.0f;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    const float P = prob(e) / t;
    const int c = hits(e);
    a.probs[e] = P;
    a.counts[e] = c;
    dot += float(c) / (float(a.k) * t) * P;
  }
  dot = warp_sum(dot);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = dot;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.0f;
    for (int w = 0; w < int(blockDim.x >> 5); ++w) s += red[w];
    a.losses[0] = float(a.E) * s;
    a.losses[1] = z_sum / t;
    a.counts[a.E] = T;
  }
}

// NV: values per lane (E <= 32 NV)
template <int NV>
__global__ void __launch_bounds__(32 * kWarps) route_kernel(const RouteArgs a) {
  extern __shared__ uint32_t sh[];
  float* sh_prob = reinterpret_cast<float*>(sh);            // [kWarps][E]
  int* sh_hits = reinterpret_cast<int*>(sh + kWarps * a.E); // [E]
  __shared__ float sh_z[kWarps];
  __shared__ int sh_t[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) sh_hits[e] = 0;
  __syncthreads();
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();

  float acc[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) acc[j] = 0.0f;
  float z = 0.0f;
  int t = 0;
  for (long long row = (long long)blockIdx.x * kWarps + warp; row < a.M;
       row += (long long)gridDim.x * kWarps) {
    const float* src = a.logits + row * a.ld;
    const bool valid = !a.valid || a.valid[row] != 0;
    float v[NV];
    float mx = -INFINITY;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = j * 32 + lane;
      v[j] = e < a.E ? __ldcg(src + e) : -INFINITY;
      mx = fmaxf(mx, v[j]);
    }
    mx = warp_max(mx);
    const float ref = mx == -INFINITY ? 0.0f : mx;
    float s = 0.0f, p[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) s += p[j] = expf(v[j] - ref);
    s = warp_sum(s);
    const float inv = 1.0f / s;
    const float l = ref + logf(s);
    if (lane == 0) a.lse[row] = l;
    // a sum of 0 is a row of -inf only (a NaN makes the sum NaN)
    const bool live = valid && s != 0.0f;
    if (live) {
      z += l * l;
      ++t;
#pragma unroll
      for (int j = 0; j < NV; ++j) acc[j] += p[j] * inv;
    }
    uint32_t key[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) key[j] = live ? rank_key(v[j]) : 0u;
    // k rounds of: the largest key of the warp, lowest index among equals
    int my_expert = -1;
    float my_weight = 0.0f, total = 0.0f;
    for (int r = 0; r < a.k; ++r) {
      uint32_t best = 0u;
      int at = 0;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (key[j] > best) {
          best = key[j];
          at = j * 32 + lane;
        }
      const uint32_t top = __reduce_max_sync(0xffffffffu, best);
      if (top <= kNoKey) break;
      const int win = __reduce_min_sync(0xffffffffu, best == top ? at : 0x7FFFFFFF);
      float w = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (j * 32 + lane == win) {
          key[j] = 0u;
          w = p[j] * inv;
        }
      w = __shfl_sync(0xffffffffu, w, win & 31);
      total += w;
      if (lane == r) {
        my_expert = win;
        my_weight = w;
      }
    }
    if (a.normalize && my_expert >= 0) my_weight = my_weight / total;
    if (lane < a.k) {
      a.weights[row * a.k + lane] = my_weight;
      a.experts[row * a.k + lane] = my_expert;
      if (my_expert >= 0) atomicAdd(sh_hits + my_expert, 1);  // integers: any order
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (j * 32 + lane < a.E) sh_prob[warp * a.E + j * 32 + lane] = acc[j];
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
  auto prob = [&](int e) {
    float s = 0.0f;
    for (int w = 0; w < kWarps; ++w) s += sh_prob[w * a.E + e];
    return s;
  };
  if (gridDim.x == 1) {
    finish(a, zb, tb, prob, [&](int e) { return sh_hits[e]; });
    return;
  }
  uint32_t* out = a.partial + size_t(blockIdx.x) * partial_words(a.E);
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    out[e] = __float_as_uint(prob(e));
    out[a.E + 1 + e] = uint32_t(sh_hits[e]);
  }
  if (threadIdx.x == 0) {
    out[a.E] = __float_as_uint(zb);
    out[2 * a.E + 1] = uint32_t(tb);
  }
}

// Adds the blocks' partial sums in block order.
__global__ void __launch_bounds__(kFinishThreads) route_finish_kernel(const RouteArgs a, int blocks) {
  extern __shared__ uint32_t sh[];
  float* sh_prob = reinterpret_cast<float*>(sh);       // [E + 1]
  int* sh_hits = reinterpret_cast<int*>(sh) + a.E + 1; // [E + 1]
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const size_t words = partial_words(a.E);
  for (int c = threadIdx.x; c < int(words); c += blockDim.x) {
    const uint32_t* src = a.partial + c;
    if (c <= a.E) {
      float s = 0.0f;
#pragma unroll 8
      for (int b = 0; b < blocks; ++b) s += __uint_as_float(__ldcg(src + size_t(b) * words));
      sh_prob[c] = s;
    } else {
      int s = 0;
#pragma unroll 8
      for (int b = 0; b < blocks; ++b) s += int(__ldcg(src + size_t(b) * words));
      sh_hits[c - a.E - 1] = s;
    }
  }
  __syncthreads();
  finish(a, sh_prob[a.E], sh_hits[a.E], [&](int e) { return sh_prob[e]; },
         [&](int e) { return sh_hits[e]; });
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

// dl[e] = p[e] (dp[e] - sum_f p[f] dp[f] + 2 d_z lse / T) with
// dp[e] = d_balance E counts[e] / (k T^2) + (the weight's gradient at a taken
// expert).  The k entries of the second term go through a zeroed row of
// shared memory, which every lane reads at its own columns.
template <int NV, bool kBF16>
__global__ void __launch_bounds__(32 * kWarps) route_grad_kernel(const RouteGradArgs a) {
  extern __shared__ uint32_t sh[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* up = reinterpret_cast<float*>(sh) + warp * a.E;
  for (int e = lane; e < a.E; e += 32) up[e] = 0.0f;
  __syncwarp();
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int T = a.counts[a.E];
  const float t = float(T > 1 ? T : 1);
  const float db = a.dlosses ? a.dlosses[0] : 0.0f, dz = a.dlosses ? a.dlosses[1] : 0.0f;
  const float c0 = db * float(a.E) / (float(a.k) * t) / t;
  const float c1 = 2.0f * dz / t;
  float base[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = j * 32 + lane;
    base[j] = e < a.E ? c0 * float(a.counts[e]) : 0.0f;
  }
  for (long long row = (long long)blockIdx.x * kWarps + warp; row < a.M;
       row += (long long)gridDim.x * kWarps) {
    const float* src = a.logits + row * a.ld;
    const float l = a.lse[row];
    int ex = lane < a.k ? a.experts[row * a.k + lane] : -1;
    if (ex >= a.E) ex = -1;  // not an expert: takes no part
    const bool live = __shfl_sync(0xffffffffu, ex, 0) >= 0;
    float p[NV];
    float mx = -INFINITY;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = j * 32 + lane;
      p[j] = (live && e < a.E) ? __ldcg(src + e) : -INFINITY;
      mx = fmaxf(mx, p[j]);
    }
    mx = warp_max(mx);
    const float ref = mx == -INFINITY ? 0.0f : mx;
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) s += p[j] = expf(p[j] - ref);
    s = warp_sum(s);
    const float inv = s > 0.0f ? 1.0f / s : s;  // 0 in a row that takes no part, NaN stays
#pragma unroll
    for (int j = 0; j < NV; ++j) p[j] *= inv;
    float g = (ex >= 0 && a.dweights) ? a.dweights[row * a.k + lane] : 0.0f;
    if (a.normalize) {
      const float q = ex >= 0 ? expf(__ldcg(src + ex) - ref) * inv : 0.0f;
      const float sum = warp_sum(q);
      const float gq = warp_sum(g * q);
      if (ex >= 0) g = (g - gq / sum) / sum;
    }
    if (ex >= 0) up[ex] = g;
    __syncwarp();
    float dp[NV];
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = j * 32 + lane;
      dp[j] = e < a.E ? base[j] + up[e] : 0.0f;
      dot += p[j] * dp[j];
    }
    dot = warp_sum(dot);
    const float shift = (live ? c1 * l : 0.0f) - dot;
    __syncwarp();
    if (ex >= 0) up[ex] = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = j * 32 + lane;
      if (e >= a.E) continue;
      const float d = live ? p[j] * (dp[j] + shift) : 0.0f;
      const size_t off = size_t(row) * a.E + e;
      // BF16: one rounding, for a gradient that goes into a BF16 product
      if constexpr (kBF16) static_cast<__nv_bfloat16*>(a.dlogits)[off] = __float2bfloat16_rn(d);
      else static_cast<float*>(a.dlogits)[off] = d;
    }
    __syncwarp();
  }
}

int route_blocks(int M) { return int(std::min<long long>(kMaxBlocks, ((long long)M + kWarps - 1) / kWarps)); }

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

}  // namespace

size_t router_topk_workspace(int M, int E) {
  const int b = route_blocks(M);
  return b > 1 ? size_t(b) * partial_words(E) * 4 : 0;
}

int launch_router_topk(const RouterTopk& r, const DeviceInfo&, cudaStream_t stream) {
  const RouteArgs a{r.logits, r.valid, r.weights, r.experts, r.lse, r.counts, r.probs, r.losses,
                    static_cast<uint32_t*>(r.workspace), r.M, r.E, r.ld, r.k, r.normalize};
  const int blocks = route_blocks(r.M);
  const size_t shared = size_t(kWarps + 1) * r.E * 4;
  const int threads = 32 * kWarps;
  int rc;
  if (r.E <= 64) rc = launch(route_kernel<2>, blocks, threads, shared, stream, a);
  else if (r.E <= 256) rc = launch(route_kernel<8>, blocks, threads, shared, stream, a);
  else rc = launch(route_kernel<32>, blocks, threads, shared, stream, a);
  if (rc != GEMM_OK || blocks == 1) return rc;
  return launch(route_finish_kernel, 1, kFinishThreads, partial_words(r.E) * 4, stream, a, blocks);
}

int launch_router_topk_backward(const RouterTopkBackward& r, const DeviceInfo&,
                                cudaStream_t stream) {
  const RouteGradArgs a{r.logits, r.experts, r.lse, r.counts, r.dweights, r.dlosses, r.dlogits,
                        r.M, r.E, r.ld, r.k, r.normalize};
  const int blocks = route_blocks(r.M);
  const size_t shared = size_t(kWarps) * r.E * 4;
  const int threads = 32 * kWarps;
  if (r.bf16) {
    if (r.E <= 64) return launch(route_grad_kernel<2, true>, blocks, threads, shared, stream, a);
    if (r.E <= 256) return launch(route_grad_kernel<8, true>, blocks, threads, shared, stream, a);
    return launch(route_grad_kernel<32, true>, blocks, threads, shared, stream, a);
  }
  if (r.E <= 64) return launch(route_grad_kernel<2, false>, blocks, threads, shared, stream, a);
  if (r.E <= 256) return launch(route_grad_kernel<8, false>, blocks, threads, shared, stream, a);
  return launch(route_grad_kernel<32, false>, blocks, threads, shared, stream, a);
}

}  // namespace gb300
