// Products of few tokens (M <= 16) with NVFP4 weights:
//   C[m][n] = bf16( scale2 sum_k A[m][k] w[n][k] ),  w = e2m1(b[n][k]) e4m3(sfb[n][k/16])
// and, for the two projections of a gated block at once,
//   H[m][n] = bf16( act(scale2_g sum_k A wg) * (scale2_u sum_k A wu) ).
//
// Bound by reading the weights, 9/16 byte each, once.  A warp multiplies 16 weight
// rows by the tokens with mma.m16n8k16 (the weights as the 16-row operand, tokens as
// the 8 columns: a tcgen05 tile would spend 128 rows on what one warp streams), from
// registers: a lane reads 16 code bytes of two rows per 128 K, straight from memory.
// Which k a lane's operand slots stand for is free as long as both operands agree,
// so each lane multiplies its own 32 consecutive k.  The weights become BF16 exactly
// (six significant bits), so products are exact and sums FP32.
//
// A block takes 64 weight rows (gated: 32 of each matrix), four 16-row tiles by two
// interleaved halves of K; the blocks of a cluster divide K where there are few rows,
// and add their sums through distributed shared memory in a fixed order.
#include <algorithm>

#include "chain.cuh"
#include "e2m1.cuh"
#include "gate_act.cuh"

namespace gb300 {

namespace {

constexpr int kRows = 64;      // weight rows per block
constexpr int kThreads = 256;  // 4 row tiles x 2 halves of K
constexpr int kDepth = 4;      // K blocks of 128 that a warp has in flight
constexpr int kMaxCluster = 8;
constexpr int kChunk = 16;     // K blocks of A in shared memory at a time

__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, __nv_bfloat162 s) {
  const __nv_bfloat162 q = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), s);
  return *reinterpret_cast<const uint32_t*>(&q);
}

// A lane's part of one 128-deep K block of 16 rows: 32 codes and two block scales
// of rows g and g + 8.
struct Block {
  uint4 c[2];
  uint16_t s[2];
};

// NT: groups of 8 tokens.
template <int NT, bool kGated>
__global__ void __launch_bounds__(kThreads)
    gemv_w4a16_kernel(const GemvW4 a, int splits) {
  extern __shared__ uint2 tokens[];  // [K block][i][token group][t][token]: 4 k of a token
  __shared__ float sums[2][kRows][8 * NT + 1];
  const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
  const int g = lane >> 2, t = lane & 3, tile = warp & 3, half = warp >> 2;
  const int rank = splits > 1 ? int(ptx::cluster_ctarank()) : 0;
  const int first = int(blockIdx.x) / splits * (kGated ? kRows / 2 : kRows);
  // this warp's rows: matrix, and first row of the tile
  const int which = kGated ? tile >> 1 : 0;
  const int row0 = first + 16 * (kGated ? tile & 1 : tile);
  const int nkb = a.K / 128;
  const int kb0 = int((long long)nkb * rank / splits), kb1 = int((long long)nkb * (rank + 1) / splits);

  // rows past the end read the last row again; nothing of them is stored
  const uint8_t *pb[2], *ps[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const size_t row = size_t(min(row0 + g + 8 * h, a.N - 1));
    pb[h] = a.b[which] + row * size_t(a.K / 2) + t * 16;
    ps[h] = a.sf[which] + row * size_t(a.K / 16) + t * 2;
  }
  auto load = [&](Block& x, int kb) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      x.c[h] = __ldcs(reinterpret_cast<const uint4*>(pb[h] + size_t(kb) * 64));
      x.s[h] = __ldg(reinterpret_cast<const unsigned short*>(ps[h] + size_t(kb) * 8));
    }
  };

  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  Block ring[kDepth];
#pragma unroll
  for (int d = 0; d < kDepth; ++d)
    if (kb0 + half + 2 * d < kb1) load(ring[d], kb0 + half + 2 * d);

  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
  // tokens of each group of 8
  const int m0 = min(a.M, 8), m1 = a.M - m0;

  for (int c0 = kb0; c0 < kb1; c0 += kChunk) {
    const int blocks = min(kChunk, kb1 - c0);
    if (c0 > kb0) __syncthreads();
    for (int m = 0; m < a.M; ++m) {
      const uint2* src = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.A) +
                                                        size_t(m) * a.K + size_t(c0) * 128);
      const int col = m < 8 ? m : m - 8, cols = m < 8 ? m0 : m1;
      for (int q = int(threadIdx.x); q < blocks * 32; q += kThreads) {
        const int kb = q >> 5, qt = (q >> 3) & 3, i = q & 7;
        tokens[(kb * 8 + i) * 4 * a.M + (m < 8 ? 0 : 4 * m0) + qt * cols + col] = __ldcg(src + q);
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int kb = c0 + half; kb < c0 + blocks; kb += 2 * kDepth) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        const int k = kb + 2 * d;
        if (k >= c0 + blocks) break;
        const Block x = ring[d];
        if (k + 2 * kDepth < kb1) load(ring[d], k + 2 * kDepth);
        __nv_bfloat162 sc[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t s16;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s16) : "h"(x.s[h]));
          const float2 sf = __half22float2(*reinterpret_cast<const __half2*>(&s16));
          sc[h][0] = __float2bfloat162_rn(sf.x);
          sc[h][1] = __float2bfloat162_rn(sf.y);
        }
        const uint2* tok = tokens + (k - c0) * 32 * a.M;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t w[2][2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t word = (&x.c[h].x)[i >> 1];
            e2m1x4_to_bf16(i & 1 ? word >> 16 : word & 0xFFFFu, w[h][0], w[h][1]);
            w[h][0] = mul_bf16x2(w[h][0], sc[h][i >> 2]);
            w[h][1] = mul_bf16x2(w[h][1], sc[h][i >> 2]);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            uint2 v = make_uint2(0, 0);
            if (g < (n ? m1 : m0))
              v = tok[i * 4 * a.M + (n ? 4 * m0 + t * m1 : t * m0) + g];
            mma_16x8x16(acc[n], w[0][0], w[1][0], w[0][1], w[1][1], v.x, v.y);
          }
        }
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      sums[half][16 * tile + g + 8 * (i >> 1)][8 * n + 2 * t + (i & 1)] = acc[n][i];
  if (splits > 1) ptx::cluster_sync();
  else __syncthreads();

  // the blocks of a cluster share the rows; sums in the order of the splits
  const int outs = kGated ? kRows / 2 : kRows;
  const int per = outs / splits;
  for (int i = int(threadIdx.x); i < per * a.M; i += kThreads) {
    const int r = rank * per + i % per, m = i / per;
    auto total = [&](int row) {
      float s = 0.0f;
      for (int c = 0; c < splits; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float* p = &sums[h][row][m];
          s += splits > 1 ? ptx::ld_cluster_f32(ptx::mapa_shared(ptx::smem_u32(p), uint32_t(c))) : *p;
        }
      return s;
    };
    float v = a.scale2[0] * total(r);
    if constexpr (kGated) {
      v = a.act == GEMM_ACT_SILU ? gate_act<GEMM_ACT_SILU>(v) : gate_act<GEMM_ACT_GELU_TANH>(v);
      v *= a.scale2[1] * total(r + kRows / 2);
    }
    if (first + r < a.N)
      static_cast<__nv_bfloat16*>(a.C)[size_t(m) * a.N + first + r] = __float2bfloat16_rn(v);
  }
  // a block's sums are read by the others until here
  if (splits > 1) ptx::cluster_sync();
}

template <int NT, bool kGated>
int run(const GemvW4& a, const DeviceInfo& dev, cudaStream_t stream) {
  const int tiles = (a.N + (kGated ? kRows / 2 : kRows) - 1) / (kGated ? kRows / 2 : kRows);
  const int nkb = a.K / 128;
  int splits = 1;
  while (splits < kMaxCluster && tiles * splits < 2 * dev.num_sms && nkb >= 8 * splits) splits *= 2;
  const int blocks = std::min(kChunk, (nkb + splits - 1) / splits);
  const size_t smem = size_t(blocks) * 256 * a.M;
  auto kernel = gemv_w4a16_kernel<NT, kGated>;
  static std::atomic<bool> ready[64];
  if (!ready[dev.device & 63].load()) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kChunk * 256 * 8 * NT) != cudaSuccess) {
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
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kernel, a, splits) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  return GEMM_OK;
}

}  // namespace

int launch_gemv_w4a16(const GemvW4& a, const DeviceInfo& dev, cudaStream_t stream) {
  if (a.b[1]) return a.M <= 8 ? run<1, true>(a, dev, stream) : run<2, true>(a, dev, stream);
  return a.M <= 8 ? run<1, false>(a, dev, stream) : run<2, false>(a, dev, stream);
}

}  // namespace gb300
