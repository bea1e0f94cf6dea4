// Products of few tokens (M <= 16) with NVFP4 weights:
//   C[m][n] = bf16( scale2 sum_k A[m][k] w[n][k] ),  w = e2m1(b[n][k]) e4m3(sfb[n][k/16])
// and, for the two projections of a gated block at once,
//   H[m][n] = bf16( act(scale2_g sum_k A wg) * (scale2_u sum_k A wu) ).
//
// Bound by reading the weights, 9/16 byte each, once.  A warp multiplies 16 weight
// rows by the tokens with mma.m16n8k16 (the weights as the 16-row operand, tokens as
// the 8 columns: a tcgen05 tile would spend 128 rows on what one warp streams), from
// registers: per 256 K a lane reads 32 code bytes of each of two rows, straight from
// memory.  Which k a lane's operand slots stand for is free as long as both operands
// agree, so each lane multiplies its own consecutive k.
//
// The operands are FP16, both exact: a weight has six significant bits and lies in
// [2^-10, 2688], and one instruction turns two codes into FP16 (to BF16 it takes table
// lookups, five instructions a weight in all, which bound the kernel: 2048 x 11008,
// one token 14.4 us).  A BF16 token value is exact in FP16 after a power of two that
// brings a block's largest to 2^15, if it is at least 2^-32 of that (its eight bits are
// then multiples of 2^-24).  Values below that wait for another pass over the weights
// with a scale of their own: one pass for tokens as they come, up to eight for tokens
// that span the whole BF16 range.  So products are exact and sums FP32.
//
// A block takes RT tiles of 16 weight rows (gated: half of them of each matrix), KS
// warps to a tile, which take its 256-K steps in turn; the blocks of a cluster divide
// K further where there are few rows, and add their sums through distributed shared
// memory.  Sums are joined in a fixed order.
#include <algorithm>

#include "chain.cuh"
#include "e2m1.cuh"
#include "gate_act.cuh"

namespace gb300 {

namespace {

constexpr int kThreads = 256;    // RT * KS = 8 warps
constexpr int kDepth = 2;        // 256-K steps that a warp has in flight
constexpr int kMaxCluster = 8;
constexpr int kTokenBytes = 96 << 10;  // of A in shared memory at a time, at most

__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The e2m1 codes of byte kByte of w times s: FP16 k = even, odd.
template <int kByte>
__device__ __forceinline__ uint32_t weights2(uint32_t w, uint32_t s) {
  uint32_t q;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b%2;\n\t}"
      : "=r"(q)
      : "r"(w), "n"(kByte));
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&q), *reinterpret_cast<const __half2*>(&s));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// BF16 values as biased exponents: the place that the lowest of their eight bits has.
__device__ __forceinline__ uint32_t place(uint32_t bf16) { return max((bf16 >> 7) & 0xFFu, 1u); }
constexpr uint32_t kSpan = 32;

// Four token values in [low, high] of place() (and infinities and NaN with `special`)
// times `scale` as FP16, zeros for the others.
__device__ __forceinline__ uint2 to_f16(uint2 v, uint32_t low, uint32_t high, bool special, float scale) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = ((i < 2 ? v.x : v.y) >> (16 * (i & 1))) & 0xFFFFu;
    const uint32_t p = place(b);
    const bool take = p == 255u ? special : p >= low && p <= high;
    o[i] = take ? b << 16 : 0u;
  }
  const __half2 lo = __floats2half2_rn(__uint_as_float(o[0]) * scale, __uint_as_float(o[1]) * scale);
  const __half2 hi = __floats2half2_rn(__uint_as_float(o[2]) * scale, __uint_as_float(o[3]) * scale);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// A lane's part of a 256-K step of 16 rows: of rows g and g + 8, two runs of 32 codes
// (k 128 j + 32 t ..) with their two block scales each.
struct Step {
  uint4 c[2][2];
  uint16_t s[2][2];
};

// NT: groups of 8 tokens.
template <int NT, int RT, bool kGated>
__global__ void __launch_bounds__(kThreads, 2)
    gemv_w4a16_kernel(const GemvW4 a, int splits, int chunk) {
  constexpr int KS = kThreads / 32 / RT, kRows = 16 * RT, kOuts = kGated ? kRows / 2 : kRows;
  static_assert(!kGated || RT % 2 == 0, "tiles of both matrices");
  extern __shared__ uint2 tokens[];  // [step][i][token group][t][token]: 4 k of a token
  __shared__ float sums[KS][kRows][8 * NT + 1];
  __shared__ uint32_t range[2][kThreads / 32];
  const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
  const int g = lane >> 2, t = lane & 3, tile = warp % RT, part = warp / RT;
  const int rank = splits > 1 ? int(ptx::cluster_ctarank()) : 0;
  const int first = int(blockIdx.x) / splits * kOuts;
  // this warp's rows: matrix, and first row of the tile
  const bool which = kGated && tile >= RT / 2;
  const int row0 = first + 16 * (kGated ? tile % (RT / 2) : tile);
  const int steps = a.K / 256;
  const int s0 = int((long long)steps * rank / splits), s1 = int((long long)steps * (rank + 1) / splits);

  // rows past the end read the last row again; nothing of them is stored
  const uint8_t *pb[2], *ps[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const size_t row = size_t(min(row0 + g + 8 * h, a.N - 1));
    pb[h] = (which ? a.b[1] : a.b[0]) + row * size_t(a.K / 2) + t * 16;
    ps[h] = (which ? a.sf[1] : a.sf[0]) + row * size_t(a.K / 16) + t * 2;
  }
  auto load = [&](Step& x, int s) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        x.c[h][j] = __ldcs(reinterpret_cast<const uint4*>(pb[h] + size_t(s) * 128 + j * 64));
        x.s[h][j] = *reinterpret_cast<const uint16_t*>(ps[h] + size_t(s) * 16 + j * 8);
      }
  };

  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  Step ring[kDepth];
#pragma unroll
  for (int d = 0; d < kDepth; ++d)
    if (s0 + part + KS * d < s1) load(ring[d], s0 + part + KS * d);

  float total_acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) total_acc[n][i] = 0.0f;
  // tokens of each group of 8
  const int m0 = min(a.M, 8), m1 = a.M - m0;
  // this block's part of the tokens
  const uint16_t* A = static_cast<const uint16_t*>(a.A) + size_t(s0) * 256;
  const int part_k = (s1 - s0) * 256;

  uint32_t below = 255;  // places that are still due: below this one
  for (bool first_pass = true;; first_pass = false) {
    // the largest and the smallest place among them, zeros aside
    uint32_t high = 0, low = 255;
    for (int m = 0; m < a.M; ++m) {
      const uint4* src = reinterpret_cast<const uint4*>(A + size_t(m) * a.K);
#pragma unroll 4
      for (int q = int(threadIdx.x); q < part_k / 8; q += kThreads) {
        const uint4 v = src[q];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t b = (w[i / 2] >> (16 * (i & 1))) & 0x7FFFu, p = place(b);
          if (b != 0 && p < below) {
            high = max(high, p);
            low = min(low, p);
          }
        }
      }
    }
    high = __reduce_max_sync(0xffffffffu, high);
    low = __reduce_min_sync(0xffffffffu, low);
    if (!first_pass) __syncthreads();
    if (lane == 0) {
      range[0][warp] = high;
      range[1][warp] = low;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
      high = max(high, range[0][i]);
      low = min(low, range[1][i]);
    }
    if (!first_pass && high == 0) break;
    const uint32_t from = high > kSpan ? high - kSpan : 0u;
    // 2^(142 - high) brings the largest to 2^15; at most 2^127
    const int e = min(142 - int(high), 127);
    const float scale = __uint_as_float(uint32_t(max(e + 127, 1)) << 23);
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
    if (!first_pass) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d)
        if (s0 + part + KS * d < s1) load(ring[d], s0 + part + KS * d);
    }

    // `chunk` is a multiple of KS * kDepth: a chunk ends where the ring starts over
    for (int c0 = s0; c0 < s1; c0 += chunk) {
      const int here = min(chunk, s1 - c0);
      if (c0 > s0) __syncthreads();
      for (int m = 0; m < a.M; ++m) {
        const uint2* src = reinterpret_cast<const uint2*>(A + size_t(m) * a.K + size_t(c0 - s0) * 256);
        const int col = m < 8 ? m : 4 * m0 + m - 8, cols = m < 8 ? m0 : m1;
#pragma unroll 4
        for (int q = int(threadIdx.x); q < here * 64; q += kThreads) {
          // 4 k of 128-K half step q / 32
          const int blk = q >> 5, qt = (q >> 3) & 3, i = q & 7;
          tokens[(blk * 8 + i) * 4 * a.M + qt * cols + col] = to_f16(src[q], from, high, first_pass, scale);
        }
      }
      __syncthreads();
#pragma unroll 1
      for (int sb = c0 + part; sb < c0 + here; sb += KS * kDepth) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
          const int s = sb + KS * d;
          if (s >= c0 + here) break;
          const Step x = ring[d];
          if (s + KS * kDepth < s1) load(ring[d], s + KS * kDepth);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t sc[2][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t s16;
              asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s16) : "h"(x.s[h][j]));
              sc[h][0] = prmt(s16, 0u, 0x1010u);
              sc[h][1] = prmt(s16, 0u, 0x3232u);
            }
            const uint2* tok = tokens + ((s - c0) * 2 + j) * 32 * a.M;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              uint32_t w[2][2];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t word = (&x.c[h][j].x)[i >> 1];
                w[h][0] = i & 1 ? weights2<2>(word, sc[h][i >> 2]) : weights2<0>(word, sc[h][i >> 2]);
                w[h][1] = i & 1 ? weights2<3>(word, sc[h][i >> 2]) : weights2<1>(word, sc[h][i >> 2]);
              }
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                uint2 v = make_uint2(0, 0);
                if (g < (n ? m1 : m0)) v = tok[i * 4 * a.M + (n ? 4 * m0 + t * m1 : t * m0) + g];
                mma_16x8x16(acc[n], w[0][0], w[1][0], w[0][1], w[1][1], v.x, v.y);
              }
            }
          }
        }
      }
    }
    // 2^-e in two factors, since it may lie below the FP32 range, and scale2, so that
    // a sum that lies above it comes back before it is stored
    const float back = __uint_as_float(uint32_t(127 - e / 2) << 23);
    const float back2 = __uint_as_float(uint32_t(127 - (e - e / 2)) << 23) * (which ? a.scale2[1] : a.scale2[0]);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) total_acc[n][i] += acc[n][i] * back * back2;
    if (low >= from || from == 0) break;
    below = from;
    __syncthreads();
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      sums[part][16 * tile + g + 8 * (i >> 1)][8 * n + 2 * t + (i & 1)] = total_acc[n][i];
  if (splits > 1) ptx::cluster_sync();
  else __syncthreads();

  // the blocks of a cluster share the outputs; sums in the order of the splits
  const int per = kOuts / splits;
  for (int i = int(threadIdx.x); i < per * a.M; i += kThreads) {
    const int r = rank * per + i % per, m = i / per;
    auto total = [&](int row) {
      float s = 0.0f;
      for (int c = 0; c < splits; ++c)
#pragma unroll
        for (int h = 0; h < KS; ++h) {
          const float* p = &sums[h][row][m];
          s += splits > 1 ? ptx::ld_cluster_f32(ptx::mapa_shared(ptx::smem_u32(p), uint32_t(c))) : *p;
        }
      return s;
    };
    float v = total(r);
    if constexpr (kGated) {
      v = a.act == GEMM_ACT_SILU ? gate_act<GEMM_ACT_SILU>(v) : gate_act<GEMM_ACT_GELU_TANH>(v);
      v *= total(r + kOuts);
    }
    if (first + r < a.N)
      static_cast<__nv_bfloat16*>(a.C)[size_t(m) * a.N + first + r] = __float2bfloat16_rn(v);
  }
  // a block's sums are read by the others until here
  if (splits > 1) ptx::cluster_sync();
}

// How a product is divided: 16-row tiles per block and blocks per cluster.
struct Plan {
  int rt, splits;
};
// The SM that gets the most blocks takes their weights and tokens and, per block, what
// an SM could read while one starts and ends.
Plan make_plan(const GemvW4& a) {
  const bool gated = a.b[1] != nullptr;
  const int steps = a.K / 256;
  Plan best{4, 1};
  double best_cost = 1e300;
  for (int rt = gated ? 2 : 1; rt <= 4; rt *= 2)
    for (int splits = 1; splits <= kMaxCluster && splits <= steps; splits *= 2) {
      const int outs = gated ? 8 * rt : 16 * rt;
      const long long blocks = ((long long)a.N + outs - 1) / outs * splits;
      const double k = double((steps + splits - 1) / splits) * 256;
      const double bytes = k * (16 * rt * 0.5625 + 2.0 * a.M);
      const double cost = double((blocks + 151) / 152) * (bytes + 40e3) + (splits > 1 ? 20e3 : 0.0);
      if (cost < best_cost) {
        best_cost = cost;
        best = {rt, splits};
      }
    }
  return best;
}

template <int NT, int RT, bool kGated>
int run(const GemvW4& a, int splits, const DeviceInfo& dev, cudaStream_t stream) {
  constexpr int kOuts = kGated ? 8 * RT : 16 * RT, kGroup = kThreads / 32 / RT * kDepth;
  const int tiles = (a.N + kOuts - 1) / kOuts;
  const int steps = (a.K / 256 + splits - 1) / splits;
  const int step_bytes = 512 * a.M;
  int chunk = std::max(1, kTokenBytes / step_bytes / kGroup) * kGroup;
  const size_t smem = size_t(std::min(steps, chunk)) * step_bytes;
  auto kernel = gemv_w4a16_kernel<NT, RT, kGated>;
  static std::atomic<bool> ready[64];
  if (!ready[dev.device & 63].load()) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             std::max(kTokenBytes, kGroup * 512 * 8 * NT)) != cudaSuccess) {
      cudaGetLastError();
      return GEMM_ERR_LAUNCH;
    }
    ready[dev.device & 63].store(true);
  }
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = splits;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(unsigned(tiles) * splits);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = splits > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, a, splits, chunk) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  return GEMM_OK;
}

}  // namespace

int launch_gemv_w4a16(const GemvW4& a, const DeviceInfo& dev, cudaStream_t stream) {
  const Plan q = make_plan(a);
  auto go = [&](auto nt) {
    constexpr int NT = decltype(nt)::value;
    if (a.b[1])
      return q.rt == 2 ? run<NT, 2, true>(a, q.splits, dev, stream)
                       : run<NT, 4, true>(a, q.splits, dev, stream);
    return q.rt == 1   ? run<NT, 1, false>(a, q.splits, dev, stream)
           : q.rt == 2 ? run<NT, 2, false>(a, q.splits, dev, stream)
                       : run<NT, 4, false>(a, q.splits, dev, stream);
  };
  return a.M <= 8 ? go(std::integral_constant<int, 1>{}) : go(std::integral_constant<int, 2>{});
}

}  // namespace gb300
