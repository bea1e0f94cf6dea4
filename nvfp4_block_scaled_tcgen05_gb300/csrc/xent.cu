// Linear cross entropy of a language-model head: for X [M][K], W [V][K]
//   z[m][v]  = sum_k X[m][k] W[v][k]                 (FP32, never stored)
//   lse[m]   = log sum_v exp(z[m][v]),   loss[m] = lse[m] - z[m][target[m]]
// and its gradient, with d[m] = dL/dloss[m]:
//   G[m][v]  = d[m] (exp(z[m][v] - lse[m]) - [v = target[m]])
//   dX = G . W,   dW = G^T . X.
//
// Forward: the NT GEMM with an epilogue that folds a row's 128 columns of a
// tile into (maximum, sum of exponentials); a second kernel joins the groups of
// a row in a fixed order.  Per row and 128 logits 8 bytes leave the chip
// instead of 256.  Bound by the MMAs (8192 x 65536 x 4096: 2220 us in a burst,
// 1981 TFLOP/s; 2390-2470 under the power cap) or, with few tokens, by reading
// W (64 x 131072 x 4096: 158 us, 6.8 TB/s; one token and 32768 x 2048, where
// the grids' ramps weigh more: 26.4 us, 5.1 TB/s).  Rows whose pitch is not a
// multiple of 32 bytes cost a fifth sector per 128 bytes on the way from L2:
// 1016 x 32003 x 2056 takes 103 us where 1024 x 32768 x 2048 takes 82.
//
// Backward: pieces of the vocabulary.  Per piece one GEMM forms the logits
// again, in the forward pass's chunks of K, and writes G as BF16 (the operand
// type of the products that follow: one rounding of relative size at most 2^-8
// per term), one adds G . W into FP32, one computes the piece's rows of dW:
// three times the forward's products, since the logits are not kept.  The grids of a piece are chained so that one
// without a data dependency on its predecessor starts on the SMs the
// predecessor's last round leaves idle (launch_xent_backward).  4096 x 131072 x
// 4096: 6850-7260 us in a burst (1818-1927 TFLOP/s), 7660-7710 under the power
// cap; 37 x 32768 x 2048: 75.5 us, of which reading W twice and writing dW take
// 60.
#include <algorithm>

#include "chain.cuh"

namespace gb300 {

// Forward, tokens on the MMA's M side: 256 x 256 pair tiles; 8 epilogue warps
// hold a tile's sums over the K chunks, 128 columns each, in registers.
using XentFwdPair = ChunkedCfg<TileCfg<Operand::kBF16, 2, 256, 3, 8, 0, true, false, 2>>;
// Forward of few tokens: the vocabulary on the M side (256 rows per CTA pair),
// the tokens on the N side, so that the MMA's time shrinks with the tokens and
// the kernel streams W at the rate of memory (64 x 131072 x 4096: 160 us, 6.7
// TB/s).  Pairs halve each CTA's share of the tokens; single CTAs took 209 us
// with one token.
template <int BN, int STAGES>
using XentFwdT = FewTokensCfg<
    ChunkedCfg<TileCfg<Operand::kBF16, 2, BN, STAGES, 4, 1, true, false, 2>>, true>;
template <int CG, int STAGES, int KSUB, bool BMN, bool AMN>
using XentCfg =
    TileCfg<Operand::kBF16, CG, 256, STAGES, 4, 2, true, false, KSUB, BMN, false, AMN, true>;
// G: 8 epilogue warps (one box each), since an exponential per logit takes
// longer than the MMAs of a short K loop.  One chunk of K needs no sum in
// registers, and streams (1024 x 32768 x 256: 55.9 us, through the sums 58.9).
using XentGradStream =
    TileCfg<Operand::kBF16, 2, 256, 3, 8, 1, true, false, 2, false, false, false, true>;
using XentGradPair = ChunkedCfg<XentGradStream>;
// dX and dW have K columns, often few tiles of 256: the last one is trimmed.
using XentDxPair = TrimCfg<XentCfg<2, 3, 2, true, false>>;
using XentDwPair = TrimCfg<XentCfg<2, 3, 2, true, true>>;
// Few tokens: G is formed transposed ([vocabulary][tokens]) by the roles of
// XentFwdT, so dX reads it MN-major and dW K-major.
template <int BN, int STAGES>
using XentGradT = FewTokensCfg<
    ChunkedCfg<
        TileCfg<Operand::kBF16, 2, BN, STAGES, 4, 3, true, false, 2, false, false, false, true>>,
    false>;
// The second and last read of the weights (37 x 32768 x 2048: 80 -> 76.5 us
// with G keeping them in L2 and dX letting them go).
template <class Base>
struct LastRead : Base {
  static constexpr bool STREAM_B = true;
};
using XentDxFew = LastRead<XentCfg<1, 4, 1, true, true>>;
// dW of few tokens is bound by writing it: 8 epilogue warps with 4 boxes each
// keep more of that stream in flight (with 256 tokens the two are even).
using XentDwFew =
    TileCfg<Operand::kBF16, 2, 256, 3, 8, 4, true, false, 1, true, false, false, true>;

namespace {

constexpr int kRowsFew = 128;  // up to this many tokens, they take the MMA's N side

// K per accumulator, see ChunkedCfg.  8192 x 65536 x 4096 under the power cap:
// 2530 us with 512 (lse off by 3e-7 of its value), 2470 with 1024 (6e-7, 1e-6 in
// well-learned rows; a plain FP32 evaluation is off by 3e-7 to 6e-7), 2445 with
// 2048 (1.3e-6): the extra reads of the accumulators cost power.  Few tokens
// have it to spare, and a single row's loss lse - z[target] cancels: 37 x 32768
// x 2048 takes 27.0 us with 512, 27.3 with 256, 28.2 with 128.
constexpr int kChunkK = 1024, kChunkKFew = 256;

// Joins the groups' statistics of each row.  A block takes `rows` (a power of
// two) rows; thread t takes row t % rows and the groups t / rows,
// t / rows + threads / rows, ...; the threads of a row are then joined
// pairwise.  The order depends on the sizes alone.
constexpr int kJoinThreads = 512;
__device__ __forceinline__ float2 join2(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x);
  const float ref = (m == -INFINITY) ? 0.0f : m;
  return make_float2(m, a.y * fast_exp(a.x - ref) + b.y * fast_exp(b.x - ref));
}

__global__ void __launch_bounds__(kJoinThreads)
    xent_join_kernel(const float2* __restrict__ stats, const long long* __restrict__ target,
                     float* __restrict__ loss, float* __restrict__ lse, int M, int V, int groups,
                     int rows) {
  __shared__ float2 part[kJoinThreads];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int t = int(threadIdx.x);
  const int row = int(blockIdx.x) * rows + t % rows;
  const int per = kJoinThreads / rows;
  float2 s = make_float2(-INFINITY, 0.0f);
  if (row < M) {
#pragma unroll 4
    for (int i = t / rows; i < groups; i += per) s = join2(s, __ldcg(stats + size_t(i) * M + row));
  }
  part[t] = s;
  __syncthreads();
  for (int h = kJoinThreads / 2; h >= rows; h >>= 1) {
    if (t < h) part[t] = join2(part[t], part[t + h]);
    __syncthreads();
  }
  if (t >= rows || row >= M) return;
  s = part[t];
  const float l = ((s.x == -INFINITY) ? 0.0f : s.x) + logf(s.y);
  lse[row] = l;
  const long long y = target[row];
  // loss[row] holds the target's logit, written by the tile that has it
  loss[row] = y < 0 ? 0.0f : (y >= V ? NAN : l - loss[row]);
}

// X's rows with a pitch that is a multiple of 32 bytes, K + 8 elements: see
// pads_x.  One 16-byte piece per thread.
constexpr int kPadThreads = 128;
__global__ void __launch_bounds__(kPadThreads)
    xent_pad_kernel(const uint4* X, uint4* out, int M, int pieces) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  for (int row = int(blockIdx.y); row < M; row += int(gridDim.y)) {
    const uint4* src = X + size_t(row) * pieces;
    uint4* dst = out + size_t(row) * (pieces + 1);
    const int i = int(blockIdx.x) * kPadThreads + int(threadIdx.x);
    if (i < pieces) dst[i] = __ldcg(src + i);
  }
}

int run_forward(const XentForward& a, const DeviceInfo& dev, cudaStream_t stream) {
  using Cfg = XentFwdPair;
  CUtensorMap tx, tw;
  int rc = encode_rows(&tx, a.X, a.M, a.K, Cfg::BM);
  if (rc == GEMM_OK) rc = encode_rows(&tw, a.W, a.V, a.K, Cfg::B_ROWS);
  if (rc != GEMM_OK) return rc;
  GemmParams p = base_params<Cfg>(a.M, a.V, a.K, dev);
  set_chunks<Cfg>(p, kChunkK);
  p.target = a.target;
  p.stats = static_cast<float2*>(a.workspace);
  p.picked = a.loss;
  return launch_tcgen05<Cfg, Epilogue::kXentStats>(tx, tw, tx, tx, tx, p, dev, stream);
}

template <class Cfg>
int run_forward_few(const XentForward& a, int* groups, const DeviceInfo& dev,
                    cudaStream_t stream) {
  CUtensorMap tx, tw;
  const int rows = few_rows(a.V, Cfg::BN);
  int rc = encode_rows(&tw, a.W, a.V, a.K, rows);
  if (rc == GEMM_OK) rc = encode_rows(&tx, a.X, a.M, a.K, Cfg::B_ROWS);
  if (rc != GEMM_OK) return rc;
  GemmParams p = base_params<Cfg>(a.V, a.M, a.K, dev);
  set_few_rows(p, rows);
  set_chunks<Cfg>(p, kChunkKFew);
  p.target = a.target;
  p.stats = static_cast<float2*>(a.workspace);
  p.picked = a.loss;
  // fewer clusters where the device holds fewer than the workspace allows for
  const int clusters =
      std::min({*groups / (4 * Cfg::CLUSTER), p.total_tiles,
                tcgen05_cluster_capacity<Cfg, Epilogue::kXentStatsT>(dev)});
  if (clusters <= 0) return GEMM_ERR_LAUNCH;
  *groups = clusters * 4 * Cfg::CLUSTER;
  return launch_tcgen05<Cfg, Epilogue::kXentStatsT>(tw, tx, tw, tw, tw, p, dev, stream, clusters);
}

// Column groups that the forward statistics come in: one per 128 columns,
// or (few rows) four per CTA, of at most kFewCtas CTAs.
constexpr int kFewCtas = 152;
int few_ctas(int V) { return std::min(kFewCtas, 2 * ((V + 63) / 64)); }
int stat_groups(int M, int V) {
  return M <= kRowsFew ? 4 * few_ctas(V) : (V + 127) / 128;
}

// How the backward pass is divided.
struct XentPlan {
  int piece;      // vocabulary columns per piece
  int pieces;
  int splits;     // FP32 slots that dX is summed in (split K of its GEMM)
  size_t g_bytes; // one piece's G
  int g_bufs;
  size_t dx_bytes;
};

// G of one piece, at most; two are held at a time.  Larger pieces mean fewer
// FP32 additions into dX and fewer changes of grid, for more memory: 4096 x
// 131072 x 4096 under the power cap takes 7970 us with 64 MB, 7730 with 128,
// 7660 with 256, 7640 with 512.  At least kMinPiece columns, which keeps those
// additions hidden behind the MMAs.
constexpr long long kPieceBytes = 128ll << 20;
constexpr int kMinPiece = 4096;

// A dW tile in K blocks: its K loop, or 2.3 blocks' time to write it.
double dw_tile_kb(int M) { return std::max((M + 127) / 128 + 0.5, 2.3); }

XentPlan make_plan(int M, int V, int K) {
  XentPlan q{};
  const int mb = (M + 255) / 256, vb = (V + 255) / 256;
  long long cols = kPieceBytes / (2ll * M);
  if (cols < kMinPiece) cols = kMinPiece;
  int nb = int(std::min<long long>(vb, cols / 256));
  if (nb < vb) {
    // equal pieces, then a block count whose tiles fill whole rounds of CTA pairs
    const int pieces = (vb + nb - 1) / nb;
    const int even = (vb + pieces - 1) / pieces;
    int best = nb;
    double best_cost = 1e300;
    for (int c = std::max(1, even - even / 8); c <= nb; ++c) {
      const long long n = (vb + c - 1) / c;
      const long long last = vb - (n - 1) * c;
      const double rounds = double(n - 1) * double(((long long)mb * c + kPairs - 1) / kPairs) +
                            double(((long long)mb * last + kPairs - 1) / kPairs);
      if (rounds + 0.2 * double(n) < best_cost) {
        best_cost = rounds + 0.2 * double(n);
        best = c;
      }
    }
    nb = best;
  }
  q.piece = int(std::min<long long>(V, (long long)nb * 256));
  q.pieces = (V + q.piece - 1) / q.piece;
  q.g_bytes = M <= kRowsFew ? size_t(q.piece) * size_t(round64(M)) * 2
                            : size_t(M) * size_t(round64(q.piece)) * 2;
  q.g_bytes = (q.g_bytes + 255) / 256 * 256;
  q.g_bufs = q.pieces > 1 ? 2 : 1;
  // dX has (M / rows) x (K / 256) tiles, often few rounds of CTA pairs with
  // the last one part empty.  Its K loop (the vocabulary) is divided so that
  // the rounds fill; the parts are summed in order.  Cost in K blocks (0.68 us
  // of a pair's MMAs): the rounds' K loops, two more per tile for filling the
  // pipeline and handing over, and writing and adding the parts at 5 TB/s
  // (4096 x 131072 x 4096: 256 tiles in 4 rounds took 7406 us, 512 in 7 7217).
  const bool few = M <= kRowsFew;
  const int units = few ? 2 * kPairs : kPairs;
  const long long tiles = (long long)(few ? 1 : mb) * ((K + 255) / 256);
  const int bk = few ? XentDxFew::BK : XentDxPair::BK;
  const int nkb = (q.piece + bk - 1) / bk;
  q.splits = 1;
  double best = 1e300;
  // (more than two rounds of parts fill no better)
  const int most = std::max<int>(4, int(2 * units / std::min<long long>(tiles, units)));
  for (int want = 1; want <= most && want <= std::max(1, nkb / 4); ++want) {
    const int per = (nkb + want - 1) / want;
    const int s = (nkb + per - 1) / per;
    const double parts = double(s) * M * double(K) * 8.0 / 3.4e6;
    double cost = double((tiles * s + units - 1) / units) * (per + 2) + parts;
    if (!few) {
      const long long dw_tiles = (long long)((q.piece + 255) / 256) * ((K + 255) / 256);
      cost = double(tiles * s / units) * (per + 2) + parts +
             head_start({tiles * s, per + 2.0}, dw_tiles, dw_tile_kb(M), units).end;
    }
    if (cost < best) {
      best = cost;
      q.splits = s;
    }
  }
  q.dx_bytes = (q.pieces == 1 && q.splits == 1) ? 0 : size_t(q.splits) * M * size_t(K) * 4;
  return q;
}

// A piece of the vocabulary and its G: [M][ld], or with few tokens transposed,
// [cols][ld].
struct Piece {
  void* G;
  int v0, cols, ld;
};

// G of one piece.
template <class Cfg, bool kT>
int run_grad(const XentBackward& a, const Piece& pc, bool late, GridTiles before,
             const DeviceInfo& dev, cudaStream_t stream) {
  CUtensorMap tx, tw, tg;
  const uint16_t* W = static_cast<const uint16_t*>(a.W) + size_t(pc.v0) * a.K;
  int rc = encode_rows(&tx, a.X, a.M, a.K, a.ldx, kT ? Cfg::B_ROWS : Cfg::BM);
  const int rows = kT ? few_rows(pc.cols, Cfg::BN) : 0;
  if (rc == GEMM_OK) rc = encode_rows(&tw, W, pc.cols, a.K, kT ? rows : Cfg::B_ROWS);
  if (rc == GEMM_OK) rc = encode_rows(&tg, pc.G, kT ? pc.cols : a.M, pc.ld, 32);
  if (rc != GEMM_OK) return rc;
  GemmParams p = kT ? base_params<Cfg>(pc.cols, a.M, a.K, dev)
                    : base_params<Cfg>(a.M, pc.cols, a.K, dev);
  if constexpr (kT) set_few_rows(p, rows);
  // the forward pass's chunks, see ChunkedCfg
  if constexpr (Cfg::CHUNKED) set_chunks<Cfg>(p, kT ? kChunkKFew : kChunkK);
  p.target = a.target;
  p.row_lse = a.lse;
  p.row_scale = a.dloss;
  p.col_offset = pc.v0;
  p.col_total = a.V;
  p.late_wait = late;
  constexpr Epilogue kEpi = kT ? Epilogue::kXentGradTBF16 : Epilogue::kXentGradBF16;
  if (late) set_head_start<Cfg, kEpi>(p, before, p.num_k_blocks + 1.0, dev);
  if constexpr (kT)
    return launch_tcgen05<Cfg, kEpi>(tw, tx, tg, tw, tw, p, dev, stream);
  else
    return launch_tcgen05<Cfg, kEpi>(tx, tw, tg, tx, tx, p, dev, stream);
}

// One piece's term of dX: G [M][cols] . W_piece [cols][K].
template <class Cfg>
int run_dx(const XentBackward& a, const XentPlan& q, const Piece& pc, float* acc,
           GridTiles* grid, const DeviceInfo& dev, cudaStream_t stream) {
  CUtensorMap tg, tw, tc;
  const uint16_t* W = static_cast<const uint16_t*>(a.W) + size_t(pc.v0) * a.K;
  int rc = Cfg::A_MN ? encode_rows(&tg, pc.G, pc.cols, pc.ld, Cfg::BK)
                     : encode_rows(&tg, pc.G, a.M, pc.ld, Cfg::BM);
  if (rc == GEMM_OK) rc = encode_rows(&tw, W, pc.cols, a.K, Cfg::BK);
  if (rc != GEMM_OK) return rc;
  GemmParams p = base_params<Cfg>(a.M, a.K, pc.cols, dev);
  p.trigger_late = 1;
  *grid = {p.total_tiles, p.num_k_blocks + 2.0};
  if (q.dx_bytes == 0) {
    rc = encode_rows(&tc, a.dX, a.M, a.K, 32);
    if (rc != GEMM_OK) return rc;
    return launch_tcgen05<Cfg, Epilogue::kStoreBF16>(tg, tw, tc, tg, tg, p, dev, stream);
  }
  rc = encode_tmap_3d(&tc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, acc, uint64_t(a.K), uint64_t(a.M),
                      uint64_t(q.splits), 32, 32, CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc != GEMM_OK) return rc;
  // every part holds at least one K block: a shorter last piece may use fewer
  // slots than the first, whose plain store fills them all
  const int s = std::min(q.splits, p.num_k_blocks);
  p.kb_per_split = (p.num_k_blocks + s - 1) / s;
  p.k_splits = (p.num_k_blocks + p.kb_per_split - 1) / p.kb_per_split;
  p.L = p.k_splits;
  p.total_tiles *= p.k_splits;
  *grid = {p.total_tiles, p.kb_per_split + 2.0};
  p.accumulate = pc.v0 > 0;
  return launch_tcgen05<Cfg, Epilogue::kAddF32>(tg, tw, tc, tg, tg, p, dev, stream);
}

// The piece's rows of dW: G^T [cols][M] . X [M][K].
template <class Cfg>
int run_dw(const XentBackward& a, const Piece& pc, bool after_dx, const float* sum, int slots,
           GridTiles before, GridTiles* grid, const DeviceInfo& dev, cudaStream_t stream) {
  CUtensorMap tg, tx, tc;
  uint16_t* dW = static_cast<uint16_t*>(a.dW) + size_t(pc.v0) * a.K;
  int rc = Cfg::A_MN ? encode_rows(&tg, pc.G, a.M, pc.ld, Cfg::BK)
                     : encode_rows(&tg, pc.G, pc.cols, pc.ld, Cfg::BM);
  if (rc == GEMM_OK) rc = encode_rows(&tx, a.X, a.M, a.K, a.ldx, Cfg::BK);
  if (rc == GEMM_OK) rc = encode_rows(&tc, dW, pc.cols, a.K, 32);
  if (rc != GEMM_OK) return rc;
  GemmParams p = base_params<Cfg>(pc.cols, a.K, a.M, dev);
  p.late_wait = after_dx;
  p.trigger_late = !after_dx;
  p.sum_src = sum;
  p.sum_dst = a.dX;
  p.sum_n = size_t(a.M) * a.K;
  p.sum_slots = slots;
  if (after_dx) set_head_start<Cfg, Epilogue::kStoreBF16>(p, before, dw_tile_kb(a.M), dev);
  *grid = p.extra ? GridTiles{0, 0.0} : GridTiles{p.total_tiles, dw_tile_kb(a.M)};
  return launch_tcgen05<Cfg, Epilogue::kStoreBF16>(tg, tx, tc, tg, tg, p, dev, stream);
}

// The sum of dX's parts as a grid of its own, where no dW follows to do it or
// its threads would take longer (37 x 32768 x 2048, 1.4 M values: 75.8 us with
// a grid, 73.2 within dW; 1024 x 32768 x 2048, 4 M values: 247 against 252).
constexpr size_t kSumInDw = size_t(3) << 20;  // values of all parts

// Rows whose pitch is an odd multiple of 16 bytes (K % 16 == 8) take five
// 32-byte sectors per 128 bytes on the way from L2, which then paces the MMAs.
// The backward pass first copies X to rows of K + 8 elements, where the
// vocabulary is long enough to repay it: 1016 x 32003 x 2056 283.6 -> 276 us,
// 2048 x 40000 x 4104 1262 -> 1202, 300 x 32003 x 2056 159 -> 154, but 1016 x
// 9000 x 2056 90.8 -> 92.5.  (W would cost more than it gains.)
constexpr int kPadColumns = 12288;
bool pads_x(int M, int V, int K) { return K % 16 != 0 && M > kRowsFew && V >= kPadColumns; }
size_t pad_bytes(int M, int V, int K) {
  return pads_x(M, V, K) ? (size_t(M) * (size_t(K) + 8) * 2 + 255) / 256 * 256 : 0;
}
int pad_x(XentBackward& a, void* to, cudaStream_t stream) {
  const int pieces = a.K / 8;
  const int rc = launch_dependent(
      xent_pad_kernel, dim3((pieces + kPadThreads - 1) / kPadThreads, std::min(a.M, 4096)),
      kPadThreads, stream, static_cast<const uint4*>(a.X), static_cast<uint4*>(to), a.M, pieces);
  a.X = to;
  a.ldx = a.K + 8;
  return rc;
}

}  // namespace

size_t xent_forward_workspace(int M, int V) {
  return size_t(M) * size_t(stat_groups(M, V)) * sizeof(float2);
}

size_t xent_backward_workspace(int M, int V, int K) {
  const XentPlan q = make_plan(M, V, K);
  return pad_bytes(M, V, K) + q.g_bytes * q.g_bufs + q.dx_bytes;
}

int launch_xent_forward(const XentForward& a, const DeviceInfo& dev, cudaStream_t stream) {
  int groups = stat_groups(a.M, a.V);
  int rc;
  if (a.M > kRowsFew) rc = run_forward(a, dev, stream);
  else if (a.M <= 64) rc = run_forward_few<XentFwdT<64, 4>>(a, &groups, dev, stream);
  else rc = run_forward_few<XentFwdT<128, 3>>(a, &groups, dev, stream);
  if (rc != GEMM_OK) return rc;
  // few rows: more threads per row
  const int rows = a.M >= 2048 ? 32 : a.M >= 256 ? 8 : 1;
  return launch_dependent(xent_join_kernel, dim3((a.M + rows - 1) / rows), kJoinThreads, stream,
                          static_cast<const float2*>(a.workspace), a.target, a.loss, a.lse, a.M,
                          a.V, groups, rows);
}

// Order of the grids, and why each may start when it does ("waits" = its
// programmatic wait for the end of the previous grid comes first):
//   G_0 waits: everything before the call is complete from here on.
//   The first product of piece i (dX, or dW if there is no dX) waits: G_i is
//     complete, and with it, through the late waits below, all of piece i-1.
//     It lets the next grid start only once it has waited.
//   dW_i after dX_i reads G_i, complete when it starts, and waits at its end.
//   G_{i+1} writes the other G buffer, whose readers (piece i-1) are complete
//     when a product of piece i has started, and waits at its end.
// A grid that ends after its predecessor keeps the chain: whoever waits for it
// also has everything before it.
int launch_xent_backward(const XentBackward& args, const DeviceInfo& dev, cudaStream_t stream) {
  XentBackward a = args;
  a.ldx = a.K;
  if (const size_t pad = pad_bytes(a.M, a.V, a.K)) {
    const int rc = pad_x(a, a.workspace, stream);
    if (rc != GEMM_OK) return rc;
    a.workspace = static_cast<uint8_t*>(a.workspace) + pad;
  }
  const XentPlan q = make_plan(a.M, a.V, a.K);
  const bool few = a.M <= kRowsFew;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  float* acc = reinterpret_cast<float*>(ws + q.g_bytes * q.g_bufs);
  const bool sum_in_dw =
      a.dX && a.dW && q.dx_bytes && size_t(a.M) * a.K * q.splits <= kSumInDw;
  GridTiles before{0, 0.0};  // the latest grid, for the next one's head start
  for (int i = 0; i < q.pieces; ++i) {
    Piece pc;
    pc.G = ws + q.g_bytes * (i & (q.g_bufs - 1));
    pc.v0 = i * q.piece;
    pc.cols = std::min(q.piece, a.V - pc.v0);
    pc.ld = round64(few ? a.M : pc.cols);
    int rc;
    if (!few && a.K <= kChunkK) rc = run_grad<XentGradStream, false>(a, pc, i > 0, before, dev, stream);
    else if (!few) rc = run_grad<XentGradPair, false>(a, pc, i > 0, before, dev, stream);
    else if (a.M <= 64) rc = run_grad<XentGradT<64, 4>, true>(a, pc, i > 0, before, dev, stream);
    else rc = run_grad<XentGradT<128, 3>, true>(a, pc, i > 0, before, dev, stream);
    if (rc == GEMM_OK && a.dX)
      rc = few ? run_dx<XentDxFew>(a, q, pc, acc, &before, dev, stream)
               : run_dx<XentDxPair>(a, q, pc, acc, &before, dev, stream);
    // (the few tokens' dX runs on single CTAs: its last round frees no pairs in order)
    if (few) before = {0, 0.0};
    // the last dW grid, which ends after dX's, also adds dX's parts
    const int slots = (sum_in_dw && i + 1 == q.pieces) ? q.splits : 0;
    if (rc == GEMM_OK && a.dW)
      rc = few ? run_dw<XentDwFew>(a, pc, a.dX != nullptr, acc, slots, before, &before, dev, stream)
               : run_dw<XentDwPair>(a, pc, a.dX != nullptr, acc, slots, before, &before, dev, stream);
    if (rc != GEMM_OK) return rc;
  }
  if (a.dX && q.dx_bytes && !sum_in_dw)
    return launch_sum_slots(acc, a.dX, size_t(a.M) * a.K, q.splits, dev, stream);
  return GEMM_OK;
}

}  // namespace gb300
