// Host-side helpers of operators that are sequences of grids (the linear cross
// entropy, the gated projection): tensor maps of row-major matrices, schedules,
// programmatic dependent launches, and the head start that a chained grid gets
// on the SM pairs its predecessor's last round leaves idle.
#pragma once

#include <algorithm>

#include "launch.cuh"

namespace gb300 {

constexpr int kPairs = 76;  // CTA pairs of a GB300

// Tensor map of a BF16 matrix [rows][cols] with row pitch ld (all in
// elements): boxes of 64 columns and box_rows rows, 128-byte swizzle.
inline int encode_rows(CUtensorMap* m, const void* base, int rows, int cols, int ld, int box_rows) {
  return encode_tmap_3d_strided(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, uint64_t(cols),
                                uint64_t(rows), 1, uint64_t(ld) * 2,
                                uint64_t(ld) * 2 * uint64_t(rows), 64, uint32_t(box_rows), 1,
                                CU_TENSOR_MAP_SWIZZLE_128B);
}
inline int encode_rows(CUtensorMap* m, const void* base, int rows, int cols, int box_rows) {
  return encode_rows(m, base, rows, cols, cols, box_rows);
}

template <class Cfg>
GemmParams base_params(int M, int N, int K, const DeviceInfo& dev) {
  GemmParams p{};
  p.M = M;
  p.N = N;
  p.K = K;
  p.L = 1;
  p.num_m_blocks = (M + Cfg::TILE_M - 1) / Cfg::TILE_M;
  p.num_n_blocks = (N + Cfg::BN - 1) / Cfg::BN;
  p.num_k_blocks = (K + Cfg::BK - 1) / Cfg::BK;
  p.total_tiles = p.num_m_blocks * p.num_n_blocks;
  p.group_m = raster_group_m(p.num_m_blocks, (long long)Cfg::TILE_M * K * 2);
  p.k_splits = 1;
  p.kb_per_split = p.num_k_blocks;
  p.n_last = (N - (p.num_n_blocks - 1) * Cfg::BN + 31) / 32 * 32;
  p.status = dev.status;
  p.timeout_ns = wait_timeout_ns();
  return p;
}

template <class Cfg>
void set_chunks(GemmParams& p, int k) {
  p.k_chunk = std::max(1, k / Cfg::BK);
  p.chunks = (p.num_k_blocks + p.k_chunk - 1) / p.k_chunk;
}

// Rows per CTA and tile of the few tokens' kernels (FewTokensCfg): whole
// rounds of tiles stream at the rate of memory, shared by the pairs; a last
// round of n tiles takes n / pairs of a round's time, but no less than 0.44,
// since a pair alone draws no more than about 200 GB/s.  Below 46 (79) rows
// the MMAs of 64 (128) tokens take longer than the rows; 8 rows' time per
// tile for its change.
inline int few_rows(int V, int BN) {
  int best = 128;
  double best_cost = 1e300;
  for (int h = 128; h >= 32; h -= 32) {
    const int tiles = (V + 2 * h - 1) / (2 * h), last = tiles % kPairs;
    const double rounds = tiles / kPairs + (last ? std::max(double(last) / kPairs, 0.44) : 0.0);
    const double cost = rounds * (std::max(double(h), BN == 64 ? 46.0 : 79.0) + 8.0);
    if (cost < best_cost) {
      best_cost = cost;
      best = h;
    }
  }
  return best;
}
inline void set_few_rows(GemmParams& p, int rows) {
  p.m_rows = rows;
  p.num_m_blocks = (p.M + 2 * rows - 1) / (2 * rows);
  p.total_tiles = p.num_m_blocks * p.num_n_blocks;
}

inline int round64(int n) { return (n + 63) / 64 * 64; }

// A grid of the backward chain may start while the last round of its
// predecessor's tiles runs on part of the SM pairs.  Clusters are started in
// order, so the first ones get the free pairs: they take `extra` more tiles,
// chosen so that all end together.  `before`: the predecessor's tiles and the
// K blocks' time of each; then `tiles` tiles of `tile_kb`; `end`: from the
// start of the predecessor's last round to the end.  Measured: 2048 x 40000 x
// 2560 744 -> 700 us, 1024 x 32768 x 2048 253 -> 246 us.  (A start that comes
// later than assumed costs time, not results.)
struct GridTiles {
  long long tiles;
  double kb;
};
struct HeadStart {
  int early, extra;
  double end;
};
inline HeadStart head_start(GridTiles before, long long tiles, double tile_kb, int pairs) {
  const int busy = int(before.tiles % pairs);
  HeadStart h{0, 0, double((tiles + pairs - 1) / pairs) * tile_kb};
  if (busy == 0) return h;
  const int early = pairs - busy;
  h.end += before.kb;
  // the early clusters' end grows with x and the others' falls; they meet near
  // the head start's worth of tiles
  const long long even =
      std::min(static_cast<long long>(before.kb / tile_kb), tiles / early);
  for (long long x = std::max(0ll, even - 1); x <= even + 1 && x * early <= tiles; ++x) {
    const long long rest = tiles - x * early;
    const double end_early = double(x + (rest + pairs - 1) / pairs) * tile_kb;
    const double end_late =
        before.kb + double(std::max(0ll, (rest - early + pairs - 1) / pairs)) * tile_kb;
    if (std::max(end_early, end_late) < h.end)
      h = {early, int(x), std::max(end_early, end_late)};
  }
  return h;
}
template <class Cfg, Epilogue EPI>
static void set_head_start(GemmParams& p, GridTiles before, double tile_kb, const DeviceInfo& dev) {
  const int pairs = tcgen05_cluster_capacity<Cfg, EPI>(dev);
  if (before.tiles == 0 || pairs <= 0 || p.total_tiles < pairs) return;
  const HeadStart h = head_start(before, p.total_tiles, tile_kb, pairs);
  p.early = h.early;
  p.extra = h.extra;
}

// out[i] = bf16(sum of the slots' acc[slot][i]) as a grid of its own.
constexpr int kSumThreads = 128;
static __global__ void __launch_bounds__(kSumThreads)
    sum_slots_kernel(const float* acc, uint16_t* out, size_t n, int slots) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  sum_slots(acc, out, n, slots, size_t(blockIdx.x) * kSumThreads + threadIdx.x,
            size_t(gridDim.x) * kSumThreads);
}

template <class Kernel, class... Args>
int launch_dependent(Kernel kernel, dim3 grid, int threads, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  return GEMM_OK;
}

static inline int launch_sum_slots(const float* acc, void* out, size_t n, int slots, const DeviceInfo& dev,
                            cudaStream_t stream) {
  const long long grid = std::min<long long>((n / 4 + kSumThreads - 1) / kSumThreads,
                                             (long long)dev.num_sms * 16);
  return launch_dependent(sum_slots_kernel, dim3(unsigned(grid)), kSumThreads, stream, acc,
                          static_cast<uint16_t*>(out), n, slots);
}

}  // namespace gb300
