// The gated projection of a few tokens (M <= 32) and its gradient's elementwise part:
//   G = X Wg^T,  U = X Wu^T (FP32),  H = bf16(act(G) U)   or, from dH,
//   dG = bf16(dH U act'(G)),  dU = bf16(dH act(G)).
//
// Bound by reading the weights once.  A warp multiplies 8 rows of each matrix (the two
// products of 8 outputs, in one lane's accumulators) by the tokens with mma.m16n8k16,
// from registers: the weights come straight from memory, 16 bytes of two rows a lane.
// Which k a lane's operand slots stand for is free as long as both operands agree, so
// each lane multiplies its own consecutive k.  One block per SM takes a run of tiles;
// its warps share the run's 128-K steps evenly, each a consecutive part of (tile, step),
// so that all stream to the end whatever the sizes.  A warp that began a tile joins the
// parts of those that went on with it, in order, at the end.
//
// 11008 x 2048, one token: 15.0 us, 90 MB at 6.0 TB/s (tcgen05 tiles of 128 weight rows,
// whose rounds do not fit the sizes, 20.8); 1024 x 1024, 4 tokens: 3.2 (7.1); 512 x 4096,
// 16 tokens: 5.9 (17.1).  What shared memory takes, the first-level cache lacks for the
// loads in flight (16 x 4096 x 5120 with 35 KB more of it: 29 us, as it is 19).
#include <algorithm>
#include <type_traits>

#include "chain.cuh"
#include "gate_act.cuh"

namespace gb300 {

namespace {

constexpr int kInFlight = 32;  // 128-K steps that a block's warps have in flight
constexpr int kTokenBytes = 184 << 10;

// A lane's part of a step: of its gate and its up row, k 32 j + 8 t .. + 7.
struct Step {
  uint4 v[2][4];
};

struct FewTokens {
  const void *X, *Wg, *Wu;
  const uint16_t* dH;  // the gradient's form: dG and dU to out
  uint16_t *out, *gates;
  int act, M, F, K;
};

__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16-byte pieces of a token in shared memory, its K rounded up to steps; four more, so
// that eight lanes of two tokens read different banks.
__host__ __device__ constexpr int token_pieces(int steps) { return steps * 16 + 4; }

template <int NT, int kWarps, bool kGrad>
__global__ void __launch_bounds__(32 * kWarps, 1)
    gated_few_kernel(const FewTokens a, unsigned int* status, unsigned long long timeout_ns) {
  __shared__ alignas(8) unsigned long long token_bar;
  __shared__ volatile uint32_t abort;
  constexpr int kThreads = 32 * kWarps, kDepth = kInFlight / kWarps;
  __shared__ float4 parts[kWarps][NT][32];  // a warp's sums of a tile that another one began
  extern __shared__ uint4 tokens[];
  const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
  const int g = lane >> 2, t = lane & 3;
  const int steps = (a.K + 127) / 128, pitch = token_pieces(steps);
  const int tile0 = int((long long)(a.F / 8) * blockIdx.x / gridDim.x);
  const int tiles = int((long long)(a.F / 8) * (blockIdx.x + 1) / gridDim.x) - tile0;
  const long long all = (long long)tiles * steps;
  auto begin = [&](int w) { return all * w / kWarps; };  // of warp w's part
  const long long u0 = begin(warp), u1 = begin(warp + 1);

  // where the lane's rows of the next step lie
  const uint16_t *row_g = nullptr, *row_u = nullptr;
  int tile_in = int(u0 / steps), step_in = int(u0 - (long long)tile_in * steps);
  auto go_to = [&](int tile) {
    const size_t at = (size_t(tile0 + tile) * 8 + g) * a.K + 8 * t;
    row_g = static_cast<const uint16_t*>(a.Wg) + at;
    row_u = static_cast<const uint16_t*>(a.Wu) + at;
  };
  auto load_next = [&](Step& x) {
    const int k = step_in * 128;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool in = k + 32 * j + 8 * t < a.K;  // past the end: zeros
      x.v[0][j] = in ? __ldcs(reinterpret_cast<const uint4*>(row_g + k + 32 * j)) : make_uint4(0, 0, 0, 0);
      x.v[1][j] = in ? __ldcs(reinterpret_cast<const uint4*>(row_u + k + 32 * j)) : make_uint4(0, 0, 0, 0);
    }
    if (++step_in == steps) {
      step_in = 0;
      go_to(++tile_in);
    }
  };
  // the outputs of row f and token m
  auto store = [&](int f, int m, float gate, float up) {
    if (m >= a.M) return;
    const size_t at = size_t(m) * a.F + f, mf = size_t(a.M) * a.F;
    if constexpr (kGrad) {
      const float2 s = a.act == GEMM_ACT_SILU ? gate_act_slope<GEMM_ACT_SILU>(gate)
                                              : gate_act_slope<GEMM_ACT_GELU_TANH>(gate);
      const float d = __uint_as_float(uint32_t(__ldcg(a.dH + at)) << 16);
      const uint32_t two = pack_bf16x2(__float_as_uint(d * up * s.y), __float_as_uint(d * s.x));
      a.out[at] = uint16_t(two);
      a.out[mf + at] = uint16_t(two >> 16);
    } else {
      if (a.gates) {
        const uint32_t two = pack_bf16x2(__float_as_uint(gate), __float_as_uint(up));
        a.gates[at] = uint16_t(two);
        a.gates[mf + at] = uint16_t(two >> 16);
      }
      const float s = a.act == GEMM_ACT_SILU ? gate_act<GEMM_ACT_SILU>(gate) : gate_act<GEMM_ACT_GELU_TANH>(gate);
      a.out[at] = uint16_t(pack_bf16x2(__float_as_uint(s * up), 0u));
    }
  };

  // K rounded up to steps: zeros
  const int rest = steps * 16 - a.K / 8;
  for (int i = int(threadIdx.x); i < a.M * rest; i += kThreads)
    tokens[i / rest * pitch + a.K / 8 + i % rest] = make_uint4(0, 0, 0, 0);
  const uint32_t bar = ptx::smem_u32(&token_bar);
  if (threadIdx.x == 0) {
    ptx::mbar_init(bar, 1);
    abort = 0u;
  }
  ptx::fence_mbar_init();
  __syncthreads();
  // The weights' first steps on their way into L2 while the previous grid ends (11008 x
  // 2048, one token 16.2 -> 14.9 us; three steps 15.0, four 15.7).  Rows that do not begin
  // on a cache line lose by it (5512 x 2056 10.0 -> 10.5), and the shortest runs (1024 x
  // 1024, 4 tokens 3.2 -> 3.4).
  if (a.K % 64 == 0 && u1 - u0 >= kDepth) {
    const long long end = u0 + kDepth;
    for (long long u = u0; u < end;) {
      const int k = int(u / steps), st = int(u - (long long)k * steps), n = int(min((long long)(steps - st), end - u));
      const void* W = lane & 8 ? a.Wu : a.Wg;
      if (lane < 16)
        ptx::bulk_prefetch(static_cast<const uint16_t*>(W) + (size_t(tile0 + k) * 8 + (lane & 7)) * a.K + st * 128,
                           uint32_t(min(n * 128, a.K - st * 128)) * 2u);
      u += n;
    }
  }
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  // The weights' first loads, then the tokens: the weights are what takes long (16 x 2048
  // x 4096: 12.7 us, tokens first 15).
  Step ring[kDepth];
  if (u0 < u1) go_to(tile_in);
#pragma unroll
  for (int d = 0; d < kDepth; ++d)
    if (u0 + d < u1) load_next(ring[d]);
  if (warp == 0) {
    if (lane == 0) ptx::mbar_arrive_expect_tx(bar, uint32_t(a.M) * uint32_t(a.K) * 2u);
    __syncwarp();
    if (lane < a.M)
      ptx::bulk_load(ptx::smem_u32(tokens + lane * pitch), static_cast<const uint16_t*>(a.X) + size_t(lane) * a.K,
                     uint32_t(a.K) * 2u, bar);
  }
  const Watch watch{&abort, status, timeout_ns};
  // (a wait that runs out is recorded; the kernel goes on over what is there, once the
  // copies have had time to land)
  if (!wait_bar(bar, 0, watch, 14)) spin_ns(2000000ull);

  // the lane's tokens 8 n + g; past the last one the last again, which is not stored
  const uint4* mine[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) mine[n] = tokens + min(8 * n + g, a.M - 1) * pitch + t;
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
  int tile = int(u0 / steps), step = int(u0 - (long long)tile * steps);
  // stores the tile's outputs
  auto store_all = [&]() {
    const int f = (tile0 + tile) * 8 + g;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      store(f, 8 * n + 2 * t, acc[n][0], acc[n][2]);
      store(f, 8 * n + 2 * t + 1, acc[n][1], acc[n][3]);
    }
  };
  bool begun = step == 0;  // this warp has the tile from its start
#pragma unroll 1
  for (long long ub = u0; ub < u1; ub += kDepth) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      if (ub + d >= u1) break;
      Step& x = ring[d];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 v = mine[n][step * 16 + 4 * j];
          mma_16x8x16(acc[n], x.v[0][j].x, x.v[1][j].x, x.v[0][j].y, x.v[1][j].y, v.x, v.y);
          mma_16x8x16(acc[n], x.v[0][j].z, x.v[1][j].z, x.v[0][j].w, x.v[1][j].w, v.z, v.w);
        }
      }
      if (ub + d + kDepth < u1) load_next(x);
      const bool end = ++step == steps;
      if (!begun && (end || ub + d + 1 == u1)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) parts[warp][n][lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
      }
      if (end) {
        if (begun) store_all();
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
        begun = true;
        step = 0;
        ++tile;
      }
    }
  }
  __syncthreads();
  // A tile of several warps is joined by the one that has its start, in order.
  if (u0 == u1 || !begun || step == 0) return;
  const long long to = (long long)(tile + 1) * steps;
  for (int w = warp + 1; w < kWarps && begin(w) < to; ++w) {
    if (begin(w) == begin(w + 1)) continue;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float4 v = parts[w][n][lane];
      acc[n][0] += v.x;
      acc[n][1] += v.y;
      acc[n][2] += v.z;
      acc[n][3] += v.w;
    }
  }
  store_all();
}

template <int NT, int kWarps, bool kGrad>
int run(const FewTokens& a, const DeviceInfo& dev, cudaStream_t stream) {
  static std::atomic<int> ready[64];
  auto kernel = gated_few_kernel<NT, kWarps, kGrad>;
  if (!ready[dev.device & 63].load()) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTokenBytes) != cudaSuccess) {
      cudaGetLastError();
      return GEMM_ERR_LAUNCH;
    }
    ready[dev.device & 63].store(1);
  }
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(std::min(a.F / 8, dev.num_sms));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.dynamicSmemBytes = size_t(a.M) * token_pieces((a.K + 127) / 128) * 16;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, a, dev.status, wait_timeout_ns()) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  return GEMM_OK;
}

// Whether a block's run has 64 steps: 16 warps then have two each in flight; else 8 have
// four (4 x 1024 x 1024 3.8 -> 3.1 us, 16 x 512 x 4096 7.1 -> 6.3; 11008 x 2048, 145
// steps, one token 16.6 -> 17.6).
bool long_run(int F, int K) {
  return (long long)(F / 8) * ((K + 127) / 128) >= 64ll * 2 * kPairs;
}

template <bool kGrad>
int run(const FewTokens& a, const DeviceInfo& dev, cudaStream_t stream) {
  const bool many = long_run(a.F, a.K);
  if (a.M <= 8) return many ? run<1, 16, kGrad>(a, dev, stream) : run<1, 8, kGrad>(a, dev, stream);
  if (a.M <= 16) return many ? run<2, 16, kGrad>(a, dev, stream) : run<2, 8, kGrad>(a, dev, stream);
  return run<4, 8, kGrad>(a, dev, stream);
}

}  // namespace

// Up to 16 tokens that fit in shared memory; up to 32 where the runs are short (17 tokens:
// 2752 x 2048 11.8 us on the tcgen05 tiles, here 8.4; 14336 x 2816 30.2, here 31.0).
bool gated_few_takes(int M, int F, int K) {
  return M <= 32 && (M <= 16 || !long_run(F, K)) && (long long)M * token_pieces(K / 128 + 1) * 16 <= kTokenBytes;
}

int launch_gated_few(const GatedForward& a, const DeviceInfo& dev, cudaStream_t stream) {
  return run<false>({a.X, a.Wg, a.Wu, nullptr, static_cast<uint16_t*>(a.H), static_cast<uint16_t*>(a.gates),
                     a.act, a.M, a.F, a.K}, dev, stream);
}
int launch_gated_few_grad(const GatedBackward& a, uint16_t* grad, const DeviceInfo& dev, cudaStream_t stream) {
  return run<true>({a.X, a.Wg, a.Wu, static_cast<const uint16_t*>(a.dH), grad, nullptr, a.act, a.M, a.F, a.K},
                   dev, stream);
}

}  // namespace gb300
