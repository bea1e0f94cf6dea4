// Residual step of a block: for each row of D values, with r(v) = 1 / sqrt(mean(v^2) + eps)
//   c = b * r(b) * w_post      (norm after the block; c = b without w_post)
//   y = x + scale * gate * c   (rounded to the stream's type)
//   n = y * r(y) * w_pre       (norm before the next block, of y as it is stored)
// and its gradient, from dy (at y) and dn (at n):
//   t  = dy + r_y (dn w_pre - yh mean(dn w_pre yh)),   yh = y r_y      dx = t
//   q  = scale * gate * t * w_post,                    bh = b r_b
//   db = r_b (q - bh mean(q bh))
//   dw_pre = sum dn yh,  dw_post = sum scale gate t bh,  dgate = sum scale t bh w_post
// The second mean needs t, which needs the first: with q = p t, p = scale gate w_post,
//   sum q bh = sum p bh (dy + r_y dn w_pre) - r_y mean(dn w_pre yh) sum p bh yh,
// so one joint reduction of three sums serves both.
//
// Bound by memory: forward x, b read and y, n written once, backward dy, dn, y, b
// read and dx, db written once; a row lives in registers between its read and its
// write.  Sums are FP32 in a fixed order (results repeat bit for bit).
#include <algorithm>

#include "epilogue_math.cuh"
#include "chain.cuh"

namespace gb300 {

namespace {

// Eight values of a row.
struct Vec8 {
  float v[8];
};

__device__ __forceinline__ Vec8 unpack8(uint4 a) {
  Vec8 r;
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = bf16_lo(w[i]);
    r.v[2 * i + 1] = bf16_hi(w[i]);
  }
  return r;
}
__device__ __forceinline__ uint4 pack8(const Vec8& a) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = pack_bf16x2(__float_as_uint(a.v[2 * i]), __float_as_uint(a.v[2 * i + 1]));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// What a thread has read of eight values of the stream (BF16 or FP32).
template <bool kF32>
struct Raw8;
template <>
struct Raw8<false> {
  uint4 a;
  __device__ __forceinline__ void load(const void* p, size_t i) {
    a = __ldcg(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ Vec8 get() const { return unpack8(a); }
};
template <>
struct Raw8<true> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p, size_t i) {
    a = __ldcg(reinterpret_cast<const float4*>(p) + 2 * i);
    b = __ldcg(reinterpret_cast<const float4*>(p) + 2 * i + 1);
  }
  __device__ __forceinline__ Vec8 get() const { return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}}; }
};
// Stores eight values and returns them as they are stored.
template <bool kF32>
__device__ __forceinline__ Vec8 store8(void* p, size_t i, const Vec8& v) {
  if constexpr (kF32) {
    reinterpret_cast<float4*>(p)[2 * i] = make_float4(v.v[0], v.v[1], v.v[2], v.v[3]);
    reinterpret_cast<float4*>(p)[2 * i + 1] = make_float4(v.v[4], v.v[5], v.v[6], v.v[7]);
    return v;
  } else {
    const uint4 w = pack8(v);
    reinterpret_cast<uint4*>(p)[i] = w;
    return unpack8(w);
  }
}

// Sums of N values over the block's threads; every thread gets them.  `part`
// holds N floats per warp and is free again after the next barrier.
template <int N>
__device__ __forceinline__ void block_sum(float (&s)[N], float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
  const int warps = int(blockDim.x) >> 5;
  if (warps == 1) return;
  const int warp = int(threadIdx.x) >> 5;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) part[warp * N + k] = s[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) s[k] = 0.0f;
  for (int w = 0; w < warps; ++w)
#pragma unroll
    for (int k = 0; k < N; ++k) s[k] += part[w * N + k];
}

__device__ __forceinline__ float inverse_rms(float sum, int D, float eps) {
  return 1.0f / sqrtf(sum / float(D) + eps);
}

// ---------------------------------------------------------------- forward
template <bool kF32, int V>
__global__ void __launch_bounds__(512)
    residual_norm_kernel(const ResidualNorm a) {
  __shared__ float part[2][32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int pieces = a.D / 8;
  for (int row = int(blockIdx.x); row < a.M; row += int(gridDim.x)) {
    const size_t base = size_t(row) * pieces;
    Vec8 y[V];
    uint4 b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = int(threadIdx.x) + i * int(blockDim.x);
      y[i] = Vec8{};
      b[i] = make_uint4(0, 0, 0, 0);
      if (c < pieces) {
        Raw8<kF32> x;
        x.load(a.x, base + c);
        if (a.block) b[i] = __ldcg(static_cast<const uint4*>(a.block) + base + c);
        y[i] = x.get();
      }
    }
    float r = 1.0f;
    if (a.w_post) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const Vec8 v = unpack8(b[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[0] += v.v[j] * v.v[j];
      }
      block_sum(s, part[0]);
      r = inverse_rms(s[0], a.D, a.eps);
      if (threadIdx.x == 0 && a.rstd_post) a.rstd_post[row] = r;
    }
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = int(threadIdx.x) + i * int(blockDim.x);
      if (c >= pieces) break;
      if (a.block) {
        const Vec8 v = unpack8(b[i]);
        const Vec8 w = a.w_post ? unpack8(__ldg(static_cast<const uint4*>(a.w_post) + c)) : Vec8{};
        const Vec8 g = a.gate ? unpack8(__ldg(static_cast<const uint4*>(a.gate) +
                                              size_t(row / a.rows_per_gate) * pieces + c))
                              : Vec8{};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float u = v.v[j];
          if (a.w_post) u *= r * w.v[j];
          if (a.gate) u *= g.v[j];
          y[i].v[j] += a.scale * u;
        }
        y[i] = store8<kF32>(a.y, base + c, y[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] += y[i].v[j] * y[i].v[j];
    }
    if (a.w_pre) {
      block_sum(s, part[1]);
      const float ry = inverse_rms(s[0], a.D, a.eps);
      if (threadIdx.x == 0 && a.rstd_pre) a.rstd_pre[row] = ry;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = int(threadIdx.x) + i * int(blockDim.x);
        if (c >= pieces) break;
        const Vec8 w = unpack8(__ldg(static_cast<const uint4*>(a.w_pre) + c));
        Vec8 n;
#pragma unroll
        for (int j = 0; j < 8; ++j) n.v[j] = y[i].v[j] * ry * w.v[j];
        static_cast<uint4*>(a.n)[base + c] = pack8(n);
      }
    }
    __syncthreads();  // `part` is free for the next row
  }
}

// ---------------------------------------------------------------- backward
// Rows are divided among the blocks in runs; a run lies within one gate group, or
// holds whole groups.  A thread keeps its columns' weight gradients of the run in
// registers and writes them to the block's place in the workspace; dgate of groups
// that lie within a run goes straight to the output.
template <bool kF32, int V>
__global__ void __launch_bounds__(512)
    residual_norm_backward_kernel(const ResidualNormBackward a) {
  __shared__ float part[2][3 * 32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int pieces = a.D / 8;
  const int run = int(blockIdx.x);
  int row0, row1;
  if (a.parts_per_gate) {  // a run is a part of one group
    const int group = run / a.parts_per_gate, k = run % a.parts_per_gate;
    row0 = group * a.rows_per_gate + k * a.rows_per_run;
    row1 = min(row0 + a.rows_per_run, (group + 1) * a.rows_per_gate);
  } else {
    row0 = run * a.rows_per_run;
    row1 = min(row0 + a.rows_per_run, a.M);
  }
  Vec8 dwi[V], dwo[V], dg[V];
#pragma unroll
  for (int i = 0; i < V; ++i) dwi[i] = dwo[i] = dg[i] = Vec8{};
  int buf = 0;
  for (int row = row0; row < row1; ++row) {
    const size_t base = size_t(row) * pieces;
    const float ry = a.w_pre ? a.rstd_pre[row] : 0.0f;
    const float rb = a.w_post ? a.rstd_post[row] : 1.0f;
    Vec8 t[V], yh[V], bh[V], p[V];
    float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = int(threadIdx.x) + i * int(blockDim.x);
      t[i] = yh[i] = bh[i] = p[i] = Vec8{};
      if (c >= pieces) continue;
      if (a.dy) {
        Raw8<kF32> r;
        r.load(a.dy, base + c);
        t[i] = r.get();
      }
      if (a.w_pre) {
        Raw8<kF32> r;
        r.load(a.y, base + c);
        yh[i] = r.get();
        const Vec8 d = unpack8(__ldcg(static_cast<const uint4*>(a.dn) + base + c));
        const Vec8 w = unpack8(__ldg(static_cast<const uint4*>(a.w_pre) + c));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          yh[i].v[j] *= ry;
          dwi[i].v[j] += d.v[j] * yh[i].v[j];
          const float e = d.v[j] * w.v[j];
          s[0] += e * yh[i].v[j];
          t[i].v[j] += ry * e;
        }
      }
      if (a.block) {
        bh[i] = unpack8(__ldcg(static_cast<const uint4*>(a.block) + base + c));
        const Vec8 w = a.w_post ? unpack8(__ldg(static_cast<const uint4*>(a.w_post) + c)) : Vec8{};
        const Vec8 g = a.gate ? unpack8(__ldg(static_cast<const uint4*>(a.gate) +
                                              size_t(row / a.rows_per_gate) * pieces + c))
                              : Vec8{};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float f = a.scale;
          if (a.gate) f *= g.v[j];
          p[i].v[j] = f;
          if (a.w_post) {
            bh[i].v[j] *= rb;
            s[1] += f * w.v[j] * bh[i].v[j] * t[i].v[j];
            s[2] += f * w.v[j] * bh[i].v[j] * yh[i].v[j];
          }
        }
      }
    }
    if (a.w_pre || a.w_post) block_sum(s, part[buf]);
    buf ^= 1;
    const float m1 = ry * s[0] / float(a.D);
    const float m2 = (s[1] - m1 * s[2]) / float(a.D);
    const bool flush = a.dgate && !a.parts_per_gate && (row + 1) % a.rows_per_gate == 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = int(threadIdx.x) + i * int(blockDim.x);
      if (c >= pieces) break;
#pragma unroll
      for (int j = 0; j < 8; ++j) t[i].v[j] -= m1 * yh[i].v[j];
      store8<kF32>(a.dx, base + c, t[i]);
      if (a.block) {
        const Vec8 w = a.w_post ? unpack8(__ldg(static_cast<const uint4*>(a.w_post) + c)) : Vec8{};
        Vec8 db;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float dc = p[i].v[j] * t[i].v[j];  // at the norm's output
          const float cv = a.w_post ? bh[i].v[j] * w.v[j] : bh[i].v[j];
          dg[i].v[j] += a.scale * t[i].v[j] * cv;
          if (a.w_post) {
            dwo[i].v[j] += dc * bh[i].v[j];
            db.v[j] = rb * (dc * w.v[j] - bh[i].v[j] * m2);
          } else {
            db.v[j] = dc;
          }
        }
        static_cast<uint4*>(a.dblock)[base + c] = pack8(db);
        if (flush) {
          store8<true>(a.dgate, size_t(row / a.rows_per_gate) * pieces + c, dg[i]);
          dg[i] = Vec8{};
        }
      }
    }
  }
  // the run's parts: [run][kinds][D]
  const int kinds = a.kinds;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = int(threadIdx.x) + i * int(blockDim.x);
    if (c >= pieces) break;
    size_t at = size_t(run) * kinds * pieces + c;
    if (a.dw_pre) {
      store8<true>(a.parts, at, dwi[i]);
      at += pieces;
    }
    if (a.dw_post) {
      store8<true>(a.parts, at, dwo[i]);
      at += pieces;
    }
    if (a.dgate && a.parts_per_gate) store8<true>(a.parts, at, dg[i]);
  }
}

// Sums the runs' parts in order.  blockIdx.y: dw_pre, dw_post (all runs), then the
// gate's groups (each its own runs).  A block takes 32 columns; 8 warps share the
// runs and are joined in a fixed order.
constexpr int kJoinWarps = 8;
__global__ void __launch_bounds__(32 * kJoinWarps)
    residual_norm_join_kernel(const ResidualNormBackward a) {
  __shared__ float sum[kJoinWarps][32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int norms = (a.dw_pre != nullptr) + (a.dw_post != nullptr);
  const int kind = min(int(blockIdx.y), norms), group = int(blockIdx.y) - norms;
  float* out = kind == norms ? a.dgate + size_t(group) * a.D
                             : (kind == 0 && a.dw_pre ? a.dw_pre : a.dw_post);
  const int first = kind == norms ? group * a.parts_per_gate : 0;
  const int count = kind == norms ? a.parts_per_gate : a.runs;
  const int col = int(blockIdx.x) * 32 + int(threadIdx.x & 31), warp = int(threadIdx.x) >> 5;
  float s = 0.0f;
  if (col < a.D) {
    const float* src = a.parts + (size_t(first) * a.kinds + kind) * a.D + col;
    const size_t step = size_t(a.kinds) * a.D;
#pragma unroll 4
    for (int r = warp; r < count; r += kJoinWarps) s += __ldcg(src + r * step);
  }
  sum[warp][threadIdx.x & 31] = s;
  __syncthreads();
  if (warp == 0 && col < a.D) {
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) s += sum[w][threadIdx.x];
    out[col] = s;
  }
}

// Threads of a row: 8 V values each.
struct RowShape {
  int threads, V;
};
RowShape row_shape(int D, int most_threads, int most_v) {
  const int pieces = D / 8;
  int v = 1;
  while (v < most_v && (pieces + v - 1) / v > most_threads / 2) v *= 2;
  const int threads = ((pieces + v - 1) / v + 31) / 32 * 32;
  return {threads, v};
}

// Backward: runs of rows, about two per SM.
constexpr int kRuns = 304;
struct RunPlan {
  int runs, rows_per_run, kinds, parts_per_gate;
};
RunPlan make_runs(int M, int rows_per_gate, int weights, bool gates) {
  RunPlan q{};
  q.kinds = weights;
  int rows = (M + kRuns - 1) / kRuns;
  if (gates && rows_per_gate >= rows) {
    const int parts = (rows_per_gate + rows - 1) / rows;
    rows = (rows_per_gate + parts - 1) / parts;
    q.parts_per_gate = (rows_per_gate + rows - 1) / rows;
    q.runs = M / rows_per_gate * q.parts_per_gate;
    ++q.kinds;
  } else {
    if (gates) rows = (rows + rows_per_gate - 1) / rows_per_gate * rows_per_gate;
    q.runs = (M + rows - 1) / rows;
  }
  q.rows_per_run = rows;
  return q;
}

}  // namespace

size_t residual_norm_backward_workspace(int M, int D, int rows_per_gate, int weights, bool gates) {
  const RunPlan q = make_runs(M, rows_per_gate, weights, gates);
  return size_t(q.runs) * q.kinds * D * sizeof(float);
}

int launch_residual_norm(const ResidualNorm& a, const DeviceInfo& dev, cudaStream_t stream) {
  const RowShape s = row_shape(a.D, 1024, 4);
  const int per_sm = std::max(1, 2048 / s.threads);
  const dim3 grid(std::min(a.M, dev.num_sms * per_sm));
  auto go = [&](auto kernel) { return launch_dependent(kernel, grid, s.threads, stream, a); };
  if (a.x_f32)
    return s.V == 1 ? go(residual_norm_kernel<true, 1>)
                    : s.V == 2 ? go(residual_norm_kernel<true, 2>) : go(residual_norm_kernel<true, 4>);
  return s.V == 1 ? go(residual_norm_kernel<false, 1>)
                  : s.V == 2 ? go(residual_norm_kernel<false, 2>) : go(residual_norm_kernel<false, 4>);
}

int launch_residual_norm_backward(const ResidualNormBackward& args, const DeviceInfo& dev,
                                  cudaStream_t stream) {
  ResidualNormBackward a = args;
  const int weights = (a.dw_pre != nullptr) + (a.dw_post != nullptr);
  const RunPlan q = make_runs(a.M, a.rows_per_gate, weights, a.dgate != nullptr);
  a.runs = q.runs;
  a.rows_per_run = q.rows_per_run;
  a.kinds = q.kinds;
  a.parts_per_gate = q.parts_per_gate;
  const RowShape s = row_shape(a.D, 1024, 4);
  (void)dev;
  auto go = [&](auto kernel) {
    return launch_dependent(kernel, dim3(a.runs), s.threads, stream, a);
  };
  int rc;
  if (a.x_f32)
    rc = s.V == 1 ? go(residual_norm_backward_kernel<true, 1>)
                  : s.V == 2 ? go(residual_norm_backward_kernel<true, 2>)
                             : go(residual_norm_backward_kernel<true, 4>);
  else
    rc = s.V == 1 ? go(residual_norm_backward_kernel<false, 1>)
                  : s.V == 2 ? go(residual_norm_backward_kernel<false, 2>)
                             : go(residual_norm_backward_kernel<false, 4>);
  const int joins = weights + (a.parts_per_gate ? a.M / a.rows_per_gate : 0);
  if (rc != GEMM_OK || joins == 0) return rc;
  return launch_dependent(residual_norm_join_kernel, dim3((a.D + 31) / 32, joins), 32 * kJoinWarps,
                          stream, a);
}

}  // namespace gb300
