// Gated projection of a feed-forward block: for X [M][K], Wg and Wu [F][K]
//   G = X Wg^T,  U = X Wu^T (FP32),   H = bf16(act(G) * U)
// and its gradient, from dH [M][F]:
//   dG = dH * U * act'(G),  dU = dH * act(G)
//   dX = dG Wg + dU Wu,     dWg = dG^T X,  dWu = dU^T X;
// and C = A^T B, the weight gradient of a plain product (the down projection's).
//
// Forward: 256-row tiles whose accumulator holds 128 gate columns beside the 128
// up columns of the same outputs (GatedCfg), so the two products, the activation
// and their product take one pass over X and the weights.  Bound by the tensor cores:
// 5120 x 11008 x 2048 with the gates stored 249 us, 1860 TFLOP/s (280 us where calls
// follow each other and the power limit lowers the clock).
//
// Backward: dG and dU as BF16 (the operand type of the products that follow: one
// rounding of relative size at most 2^-8 per term), from the stored gates by a
// streaming kernel, or from X by the forward kernel with another epilogue; then
// dX as one K loop over both weight matrices (DualKCfg) and both weight gradients
// as one grid (DualOutCfg).  Order of the grids: dX's grid waits for dG and dU and
// only then lets the weight gradients' grid start, on the SM pairs that dX's last
// round leaves idle; that grid reads what was complete before it could start, and
// waits for dX at its end.  5120 x 11008 x 2048 from the stored gates: 571 us, 77 of
// them the streaming kernel's, the products 1870 TFLOP/s.
//
// C = A^T B: both operands with their K as the rows, as dWg and dWu have them; 2048 x
// 11008 x 5120 129 us, 1800 TFLOP/s.
//
// Rows of an odd multiple of 16 bytes take five 32-byte sectors per 128 bytes on the way
// from L2.  1016 tokens, forward: 5504 x 2048 33.7 us, 5512 x 2048 34.0, 5504 x 2056 42.6;
// gradients from X: 100.9, 110.8 (dG and dU, whose rows in the workspace are F long) and
// 115.5, both odd 129.7.
#include <algorithm>

#include "chain.cuh"

namespace gb300 {

namespace {

using FwdPair = GatedCfg<TileCfg<Operand::kBF16, 2, 256, 3, 4, 2, true, false, 2>>;
// Few tokens that gated_few.cu does not take: the weights on the MMA's M side, half of a
// tile's rows of each matrix, the tokens on the N side, so that the kernel streams the
// weights.  (11008 x 2048: 32 tokens 20.4 us, 128 tokens 23.6, 129 on the tiles above 26.)
// Their gradient reads dH two bytes at a time, which pays up to 32 tokens (5504 x 2048,
// all gradients from X: 17 tokens 49 -> 41 us, 128 50.8 -> 52.8).
constexpr int kFewTokens = 128, kFewTokensGrad = 32;
template <int BN, int STAGES>
using Few = PairedRowsCfg<
    FewTokensCfg<TileCfg<Operand::kBF16, 2, BN, STAGES, 4, 1, true, false, 2>, true>>;
using Few64 = Few<64, 5>;
using Few128 = Few<128, 4>;
template <bool kAmn>
using ChainPair =
    TrimCfg<TileCfg<Operand::kBF16, 2, 256, 3, 4, 2, true, false, 2, true, false, kAmn, true>>;
using DxPair = DualKCfg<ChainPair<false>>;
using DwPair = DualOutCfg<ChainPair<true>>;
using TnPair = ChainPair<true>;

// Tensor map of two BF16 matrices [2][rows][cols], boxes of 64 columns.
int encode_two(CUtensorMap* m, const void* base, int rows, int cols, int box_rows) {
  return encode_tmap_3d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, uint64_t(cols),
                        uint64_t(rows), 2, 64, uint32_t(box_rows), CU_TENSOR_MAP_SWIZZLE_128B);
}

// N blocks of full width (128 outputs) of `mb` M blocks, the rest being of 64: so that
// the pair with the most tiles has the least.  A tile of half the width takes about 0.6
// of the time.
constexpr double kNarrowTile = 0.6;
int wide_blocks(int mb, int F) {
  const int all = (F + 127) / 128;
  int best = all;
  double best_cost = 1e300;
  // whole rounds of wide tiles, from all of them downward
  for (long long rounds = ((long long)mb * all + kPairs - 1) / kPairs; rounds >= 0; --rounds) {
    const int wide = int(std::min<long long>(all, rounds * kPairs / mb));
    const long long tw = (long long)mb * wide;
    const long long tn = (long long)mb * ((std::max(0, F - wide * 128) + 63) / 64);
    double cost = 0.0;
    for (int c = 0; c < kPairs; ++c) {
      const long long w = (tw - c + kPairs - 1) / kPairs, t = (tw + tn - c + kPairs - 1) / kPairs;
      cost = std::max(cost, double(w) + kNarrowTile * double(t - w));
    }
    if (cost < best_cost - 0.05) {
      best_cost = cost;
      best = wide;
    }
    if (rounds + 2 < ((long long)mb * all + kPairs - 1) / kPairs) break;
  }
  return best;
}

// Maps and schedule of the gated tiles: X, both weight matrices.
template <class Cfg>
int setup_gated(const void* X, const void* Wg, const void* Wu, int act, int M, int F, int K,
                const DeviceInfo& dev, CUtensorMap& tx, CUtensorMap& tg, CUtensorMap& tu,
                GemmParams& p) {
  int rc = encode_rows(&tx, X, M, K, Cfg::BM);
  if (rc == GEMM_OK) rc = encode_rows(&tg, Wg, F, K, Cfg::BN / 4);
  if (rc == GEMM_OK) rc = encode_rows(&tu, Wu, F, K, Cfg::BN / 4);
  p = base_params<Cfg>(M, F, K, dev);
  p.n_wide = wide_blocks(p.num_m_blocks, F);
  p.num_n_blocks = p.n_wide + (std::max(0, F - p.n_wide * 128) + 63) / 64;
  p.total_tiles = p.num_m_blocks * p.num_n_blocks;
  p.act = act;
  return rc;
}

// The few tokens' form of both: H (and the gates), or with dH the two gradients.
template <class Cfg, Epilogue EPI>
int run_few(const void* X, const void* Wg, const void* Wu, const void* dH, void* out, void* gates,
            int act, int M, int F, int K, const DeviceInfo& dev, cudaStream_t stream) {
  CUtensorMap tx, tg, tu;
  const int rows = few_rows(2 * F, Cfg::BN) / 2;  // of each matrix, per CTA and tile
  int rc = encode_rows(&tx, X, M, K, Cfg::B_ROWS);
  if (rc == GEMM_OK) rc = encode_rows(&tg, Wg, F, K, rows);
  if (rc == GEMM_OK) rc = encode_rows(&tu, Wu, F, K, rows);
  if (rc != GEMM_OK) return rc;
  GemmParams p = base_params<Cfg>(F, M, K, dev);
  set_few_rows(p, rows);
  p.act = act;
  p.c_ptr = out;
  p.dh = static_cast<const uint16_t*>(dH);
  p.gates_ptr = static_cast<uint16_t*>(gates);
  return launch_tcgen05<Cfg, EPI>(tg, tx, tg, tu, tg, p, dev, stream);
}

// dG and dU [2][n] from the stored gates [2][n]: three values read and two written
// per output, bound by memory (5120 x 11008: 564 MB, 77 us,
// part of them still in the second-level cache).
constexpr int kGradThreads = 256;
template <int kAct>
__global__ void __launch_bounds__(kGradThreads)
    gated_grad_kernel(const uint16_t* gates, const uint16_t* dh, uint16_t* out, size_t n) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const size_t pieces = n / 8, stride = size_t(gridDim.x) * kGradThreads;
  for (size_t i = size_t(blockIdx.x) * kGradThreads + threadIdx.x; i < pieces; i += stride) {
    const uint4 g4 = __ldcs(reinterpret_cast<const uint4*>(gates) + i);
    const uint4 u4 = __ldcs(reinterpret_cast<const uint4*>(gates + n) + i);
    const uint4 d4 = __ldcs(reinterpret_cast<const uint4*>(dh) + i);
    const uint32_t g[4] = {g4.x, g4.y, g4.z, g4.w}, u[4] = {u4.x, u4.y, u4.z, u4.w},
                   d[4] = {d4.x, d4.y, d4.z, d4.w};
    uint32_t og[4], ou[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = gate_act_slope<kAct>(bf16_lo(g[j])), b = gate_act_slope<kAct>(bf16_hi(g[j]));
      const float da = bf16_lo(d[j]), db = bf16_hi(d[j]);
      og[j] = pack_bf16x2(__float_as_uint(da * bf16_lo(u[j]) * a.y),
                          __float_as_uint(db * bf16_hi(u[j]) * b.y));
      ou[j] = pack_bf16x2(__float_as_uint(da * a.x), __float_as_uint(db * b.x));
    }
    reinterpret_cast<uint4*>(out)[i] = make_uint4(og[0], og[1], og[2], og[3]);
    reinterpret_cast<uint4*>(out + n)[i] = make_uint4(ou[0], ou[1], ou[2], ou[3]);
  }
}

// A weight gradient's tile in K blocks: its K loop, or 2.3 blocks' time to write it.
double dw_tile_kb(int M) { return std::max((M + 127) / 128 + 0.5, 2.3); }

// The backward pass's workspace: dG and dU, then dX's FP32 parts.
struct GatedPlan {
  size_t grad_bytes, dx_bytes;
  int splits;  // parts that dX's K loop is divided in
};

// dX has (M / 256) x (K / 256) tiles, often few rounds of CTA pairs; its K loop
// (2 F) is divided so that the rounds fill, and the parts are summed in order.
// Cost in K blocks (0.68 us of a pair's MMAs): the rounds' K loops, two more per
// tile for filling the pipeline and handing over, writing and adding the parts at
// 5 TB/s, and the weight gradients' grid from dX's last round on.
GatedPlan make_plan(int M, int F, int K) {
  GatedPlan q{};
  q.grad_bytes = (size_t(M) * F * 4 + 255) / 256 * 256;
  q.splits = 1;
  const long long mb = (M + 255) / 256, kb = (K + 255) / 256, tiles = mb * kb;
  const int nkb = 2 * ((F + DxPair::BK - 1) / DxPair::BK);
  double best = 1e300;
  const int most = std::max<int>(4, int(2 * kPairs / std::min<long long>(tiles, kPairs)));
  for (int want = 1; want <= most && want <= std::max(1, nkb / 4); ++want) {
    const int per = (nkb + want - 1) / want;
    const int s = (nkb + per - 1) / per;
    const double parts = s > 1 ? double(s) * M * double(K) * 8.0 / 3.4e6 : 0.0;
    const long long dw_tiles = 2ll * ((F + 255) / 256) * kb;
    const double cost = double(tiles * s / kPairs) * (per + 2) + parts +
                        head_start({tiles * s, per + 2.0}, dw_tiles, dw_tile_kb(M), kPairs).end;
    if (cost < best) {
      best = cost;
      q.splits = s;
    }
  }
  q.dx_bytes = q.splits == 1 ? 0 : size_t(q.splits) * M * size_t(K) * 4;
  return q;
}

// Divides the K loop in `splits` parts, none of them empty, that are summed later.
void split_k(GemmParams& p, int splits) {
  p.kb_per_split = (p.num_k_blocks + splits - 1) / splits;
  p.k_splits = p.L = splits;
  p.total_tiles *= splits;
}

// Parts of A^T B's K loop, where its tiles leave CTA pairs idle: cost in K blocks as in
// make_plan, four for the second grid.
int tn_splits(int M, int N, int K) {
  const long long tiles = (long long)((M + 255) / 256) * ((N + 255) / 256);
  const int nkb = (K + TnPair::BK - 1) / TnPair::BK;
  int splits = 1;
  double best = 1e300;
  for (int want = 1; want <= std::max(1, nkb / 4) && want * tiles <= 2 * kPairs + tiles; ++want) {
    const int per = (nkb + want - 1) / want, s = (nkb + per - 1) / per;
    const double parts = s > 1 ? double(s) * M * double(N) * 8.0 / 3.4e6 + 4.0 : 0.0;
    const double cost = double((tiles * s + kPairs - 1) / kPairs) * (per + 2) + parts;
    if (cost < 0.95 * best) {
      best = cost;
      splits = s;
    }
  }
  return splits;
}

int run_grad(const GatedBackward& a, uint16_t* grad, const DeviceInfo& dev, cudaStream_t stream) {
  if (a.gates) {
    const size_t n = size_t(a.M) * a.F;
    const int grid = int(std::min<size_t>((n / 8 + kGradThreads - 1) / kGradThreads,
                                          size_t(dev.num_sms) * 16));
    const auto kernel = a.act == GEMM_ACT_SILU ? gated_grad_kernel<GEMM_ACT_SILU>
                                               : gated_grad_kernel<GEMM_ACT_GELU_TANH>;
    return launch_dependent(kernel, dim3(grid), kGradThreads, stream,
                            static_cast<const uint16_t*>(a.gates),
                            static_cast<const uint16_t*>(a.dH), grad, n);
  }
  if (gated_few_takes(a.M, a.F, a.K)) return launch_gated_few_grad(a, grad, dev, stream);
  if (a.M <= kFewTokensGrad)
    return run_few<Few64, Epilogue::kGatedGradTBF16>(a.X, a.Wg, a.Wu, a.dH, grad, nullptr, a.act, a.M,
                                                     a.F, a.K, dev, stream);
  using Cfg = FwdPair;
  CUtensorMap tx, tg, tu, tc;
  GemmParams p;
  int rc = setup_gated<Cfg>(a.X, a.Wg, a.Wu, a.act, a.M, a.F, a.K, dev, tx, tg, tu, p);
  if (rc == GEMM_OK) rc = encode_two(&tc, grad, a.M, a.F, 32);
  if (rc != GEMM_OK) return rc;
  p.dh = static_cast<const uint16_t*>(a.dH);
  return launch_tcgen05<Cfg, Epilogue::kGatedGradBF16>(tx, tg, tc, tx, tu, p, dev, stream);
}

// dX = dG Wg + dU Wu, whole or in FP32 parts.
int run_dx(const GatedBackward& a, const GatedPlan& q, const uint16_t* grad, float* parts,
           GridTiles* grid, const DeviceInfo& dev, cudaStream_t stream) {
  using Cfg = DxPair;
  CUtensorMap tdg, tdu, tg, tu, tc;
  int rc = encode_rows(&tdg, grad, a.M, a.F, Cfg::BM);
  if (rc == GEMM_OK) rc = encode_rows(&tdu, grad + size_t(a.M) * a.F, a.M, a.F, Cfg::BM);
  if (rc == GEMM_OK) rc = encode_rows(&tg, a.Wg, a.F, a.K, Cfg::BK);
  if (rc == GEMM_OK) rc = encode_rows(&tu, a.Wu, a.F, a.K, Cfg::BK);
  if (rc != GEMM_OK) return rc;
  GemmParams p = base_params<Cfg>(a.M, a.K, a.F, dev);
  p.k_half = p.num_k_blocks;
  p.num_k_blocks *= 2;
  p.K = p.k_half * Cfg::BK + a.F;  // the end of the second product
  p.group_m = raster_group_m(p.num_m_blocks, (long long)Cfg::TILE_M * a.F * 4);
  p.kb_per_split = p.num_k_blocks;
  p.trigger_late = 1;
  if (q.splits == 1) {
    rc = encode_rows(&tc, a.dX, a.M, a.K, 32);
    if (rc != GEMM_OK) return rc;
    *grid = {p.total_tiles, p.num_k_blocks + 2.0};
    return launch_tcgen05<Cfg, Epilogue::kStoreBF16>(tdg, tg, tc, tdu, tu, p, dev, stream);
  }
  rc = encode_tmap_3d(&tc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, parts, uint64_t(a.K),
                      uint64_t(a.M), uint64_t(q.splits), 32, 32, CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc != GEMM_OK) return rc;
  split_k(p, q.splits);
  *grid = {p.total_tiles, p.kb_per_split + 2.0};
  return launch_tcgen05<Cfg, Epilogue::kAddF32>(tdg, tg, tc, tdu, tu, p, dev, stream);
}

// dWg = dG^T X and dWu = dU^T X.  Their K loop, the tokens, is not divided: with few weight
// tiles and many tokens most pairs are idle (8192 tokens, 512 x 512: 43 us of both, where
// gemm_bf16_tn, which divides it, takes 12.5 us of each).
int run_dw(const GatedBackward& a, const uint16_t* grad, bool after_dx, GridTiles before,
           const DeviceInfo& dev, cudaStream_t stream) {
  using Cfg = DwPair;
  CUtensorMap td, tx, tcg, tcu;
  int rc = encode_two(&td, grad, a.M, a.F, Cfg::BK);
  if (rc == GEMM_OK) rc = encode_rows(&tx, a.X, a.M, a.K, Cfg::BK);
  if (rc == GEMM_OK) rc = encode_rows(&tcg, a.dWg, a.F, a.K, 32);
  if (rc == GEMM_OK) rc = encode_rows(&tcu, a.dWu, a.F, a.K, 32);
  if (rc != GEMM_OK) return rc;
  GemmParams p = base_params<Cfg>(a.F, a.K, a.M, dev);
  p.L = 2;
  p.total_tiles *= 2;
  p.late_wait = after_dx;
  if (after_dx) set_head_start<Cfg, Epilogue::kStoreBF16>(p, before, dw_tile_kb(a.M), dev);
  return launch_tcgen05<Cfg, Epilogue::kStoreBF16>(td, tx, tcg, tcu, td, p, dev, stream);
}

}  // namespace

size_t gated_backward_workspace(int M, int F, int K) {
  const GatedPlan q = make_plan(M, F, K);
  return q.grad_bytes + q.dx_bytes;
}

int launch_gated_forward(const GatedForward& a, const DeviceInfo& dev, cudaStream_t stream) {
  if (gated_few_takes(a.M, a.F, a.K)) return launch_gated_few(a, dev, stream);
  if (a.M <= kFewTokens) {
    const auto few = a.M <= 64 ? run_few<Few64, Epilogue::kGatedTBF16> : run_few<Few128, Epilogue::kGatedTBF16>;
    return few(a.X, a.Wg, a.Wu, nullptr, a.H, a.gates, a.act, a.M, a.F, a.K, dev, stream);
  }
  using Cfg = FwdPair;
  CUtensorMap tx, tg, tu, th, tk;
  GemmParams p;
  int rc = setup_gated<Cfg>(a.X, a.Wg, a.Wu, a.act, a.M, a.F, a.K, dev, tx, tg, tu, p);
  if (rc == GEMM_OK) rc = encode_rows(&th, a.H, a.M, a.F, 32);
  tk = tx;
  if (rc == GEMM_OK && a.gates) rc = encode_two(&tk, a.gates, a.M, a.F, 32);
  if (rc != GEMM_OK) return rc;
  p.gates_out = a.gates != nullptr;
  return launch_tcgen05<Cfg, Epilogue::kGatedBF16>(tx, tg, th, tk, tu, p, dev, stream);
}

int launch_gated_backward(const GatedBackward& a, const DeviceInfo& dev, cudaStream_t stream) {
  const GatedPlan q = make_plan(a.M, a.F, a.K);
  uint16_t* grad = static_cast<uint16_t*>(a.workspace);
  float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + q.grad_bytes);
  GridTiles before{0, 0.0};
  int rc = run_grad(a, grad, dev, stream);
  if (rc == GEMM_OK && a.dX) rc = run_dx(a, q, grad, parts, &before, dev, stream);
  if (rc == GEMM_OK && a.dWg) rc = run_dw(a, grad, a.dX != nullptr, before, dev, stream);
  if (rc == GEMM_OK && a.dX && q.splits > 1)
    rc = launch_sum_slots(parts, a.dX, size_t(a.M) * a.K, q.splits, dev, stream);
  return rc;
}

size_t gemm_bf16_tn_workspace(int M, int N, int K) {
  const int splits = tn_splits(M, N, K);
  return splits == 1 ? 0 : size_t(splits) * M * size_t(N) * 4;
}

int launch_gemm_bf16_tn(const void* A, const void* B, void* C, void* workspace, int M, int N, int K,
                        const DeviceInfo& dev, cudaStream_t stream) {
  using Cfg = TnPair;
  CUtensorMap ta, tb, tc;
  const int splits = tn_splits(M, N, K);
  int rc = encode_rows(&ta, A, K, M, Cfg::BK);
  if (rc == GEMM_OK) rc = encode_rows(&tb, B, K, N, Cfg::BK);
  if (rc == GEMM_OK)
    rc = splits == 1 ? encode_rows(&tc, C, M, N, 32)
                     : encode_tmap_3d(&tc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, workspace, uint64_t(N),
                                      uint64_t(M), uint64_t(splits), 32, 32, CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc != GEMM_OK) return rc;
  GemmParams p = base_params<Cfg>(M, N, K, dev);
  if (splits == 1) return launch_tcgen05<Cfg, Epilogue::kStoreBF16>(ta, tb, tc, ta, ta, p, dev, stream);
  split_k(p, splits);
  rc = launch_tcgen05<Cfg, Epilogue::kAddF32>(ta, tb, tc, ta, ta, p, dev, stream);
  if (rc != GEMM_OK) return rc;
  return launch_sum_slots(static_cast<const float*>(workspace), C, size_t(M) * N, splits, dev, stream);
}

}  // namespace gb300
