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
// with a scale of their own: one pass for normally distributed tokens, up to eight for
// tokens that span the whole BF16 range.  So products are exact and sums FP32; they are
// scaled back, and by scale2, before they are stored, so that a sum beyond the FP32 range
// whose result is not comes back; the largest token may be another one than the sum's, so
// the factors alone stay within the range too.
//
// The output of a gated projection spans more the larger its negative gates are, and one
// value is enough for another pass of the blocks whose K holds it.  2048 x 11008, one token
// (11): normal tokens 6.9 us (11.7), SiLU of normal gates 6.9 (14.7), GELU 6.9 (15.5), SiLU
// of gates of eight times that size 15.5 (35.8), GELU of four times 27.8 (65).
//
// A tile is 16 weight rows (gated: 8 of each matrix, so that a lane gets both products
// of its outputs).  One block per SM takes a run of tiles; it turns its tokens into FP16
// in shared memory once, then its 16 warps share the run's 256-K steps evenly, each a
// consecutive part of (tile, step), and stream without meeting.  Their sums of a tile
// are joined at the end in a fixed order.  Where there are few tiles, or the tokens do
// not fit, the blocks of a cluster divide K and join through distributed shared memory.
//
// Measured: 2048 x 11008, one token 6.8 us (12.7 MB; 4 us of it are the launch, the
// tokens and the first loads' way, before and after the stream); both of 8192 x 7168,
// 11 tokens 24.3 us (66 MB, 2.7 TB/s: turning codes into operands keeps the warps busy).
// Warps and steps in flight, the latter call: 16 and 2 24.3 us, 12 and 3 24.8, 24 and 1
// 39.7, 20 and 2 41 (their registers no longer hold the loads).
#include <algorithm>

#include "chain.cuh"
#include "e2m1.cuh"
#include "gate_act.cuh"

namespace gb300 {

namespace {

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kDepth = 2;          // 256-K steps that a warp has in flight
constexpr int kMaxCluster = 8;
constexpr int kBatch = 16;         // tiles of a block at a time
constexpr int kTokenBytes = 160 << 10;  // of tokens in shared memory at a time, at most

__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
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

// A lane's part of a 256-K step of 16 rows: of rows g and g + 8, two runs of 32 codes
// (k 128 j + 32 t ..) with their two block scales each.
struct Step {
  uint4 c[2][2];
  uint16_t s[2][2];
};

// A BF16 value's place: that of the lowest of its eight bits, as a biased exponent.
__device__ __forceinline__ uint32_t place(uint32_t magnitude) { return max(magnitude >> 7, 1u); }
constexpr uint32_t kSpan = 32;          // places that FP16 holds exactly
constexpr uint32_t kInf = 0x7F80u;      // BF16 infinity; NaN above

// Joins the magnitudes below `below` of eight token values into the largest and the
// smallest so far, zeros aside (the smallest less 1, so that zeros come last); two values
// per word.
__device__ __forceinline__ void span_of(uint4 v, uint32_t below, uint32_t& high2, uint32_t& low2) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t b = w[i] & 0x7FFF7FFFu;
    if (below != 0x8000u) b &= __vcmpltu2(b, below | below << 16);
    high2 = __vmaxu2(high2, b);
    low2 = __vminu2(low2, __vsub2(b, 0x00010001u));
  }
}

// Eight token values times `scale` as FP16.  kAll: all of them; else those whose
// magnitude is in [low, high] (infinities and NaN with `special`), zeros for the others.
template <bool kAll>
__device__ __forceinline__ uint4 to_f16(uint4 v, uint32_t low, uint32_t high, bool special, float scale) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (!kAll) {
      auto keep = [&](uint32_t b) { return b >= kInf ? special : b >= low && b <= high; };
      w[i] &= (keep(w[i] & 0x7FFFu) ? 0xFFFFu : 0u) | (keep(w[i] >> 16 & 0x7FFFu) ? 0xFFFF0000u : 0u);
    }
    const __half2 h = __floats2half2_rn(bf16_lo(w[i]) * scale, bf16_hi(w[i]) * scale);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// acc * back0 * back1 * scale2, in an order in which nothing leaves the FP32 range unless the
// result does: 2^-34 <= |acc| <= 2^57, the factors back both in [2^-64, 1] or in [1, 2^56],
// and back1 and scale2 are multiplied with each other where one grows and one shrinks.
__device__ __forceinline__ float scaled_back(float acc, float back0, float back1, float scale2) {
  const bool together = (back1 <= 1.0f) == (fabsf(scale2) >= 1.0f);
  const float first = together ? back1 * scale2 : scale2, second = together ? 1.0f : back1;
  return acc * back0 * first * second;
}

// A tile's sums: [16 rows][8 NT tokens], one more for the banks.
template <int NT>
struct Tile {
  float v[16][8 * NT + 1];
};

// NT: groups of 8 tokens.  `chunk`: steps whose tokens shared memory holds.
template <int NT, bool kGated>
__global__ void __launch_bounds__(kThreads, 1)
    gemv_w4a16_kernel(const GemvW4 a, int splits, int chunk) {
  constexpr int kOuts = kGated ? 8 : 16;
  __shared__ Tile<NT> joined[kBatch];
  __shared__ uint32_t range[2][kWarps], with[kBatch];
  // [tile + warp]: a warp's part of a tile's sums (warps take parts in order, so two of
  // them share at most one tile and no two pairs have the same place); then the tokens,
  // [128 K][token][t][chunk]: the 32 k of lane column t in four chunks of 8, chunk c at
  // c ^ (place / 2 % 4) of place 4 token + t, so that eight lanes read different banks
  extern __shared__ uint4 dynamic[];
  Tile<NT>* parts = reinterpret_cast<Tile<NT>*>(dynamic);
  const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
  const int g = lane >> 2, t = lane & 3;
  const int rank = splits > 1 ? int(ptx::cluster_ctarank()) : 0;
  const int cluster = int(blockIdx.x) / splits, clusters = int(gridDim.x) / splits;
  const int all_tiles = (a.N + kOuts - 1) / kOuts;
  const int tile0 = int((long long)all_tiles * cluster / clusters);
  const int tile1 = int((long long)all_tiles * (cluster + 1) / clusters);
  uint4* tokens = reinterpret_cast<uint4*>(parts + (min(kBatch, tile1 - tile0) + kWarps - 1));
  const int all_steps = a.K / 256;
  const int s0 = int((long long)all_steps * rank / splits);
  const int s1 = int((long long)all_steps * (rank + 1) / splits);

  // This lane's place in each 128 K of the tokens, of token 8 n + g; past the last
  // token the last one again: those columns of the product are not stored.
  int mine[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int at = 4 * min(8 * n + g, a.M - 1) + t;
#pragma unroll
    for (int c = 0; c < 4; ++c) mine[n][c] = at * 4 + (c ^ (at >> 1 & 3));
  }
  // The lane's rows of a tile: g and g + 8, or row g of both matrices; where their next
  // step lies.  Rows past the end read the last row again; nothing of them is stored.
  const uint8_t *codes[2], *scales[2];
  auto go_to = [&](int tile, int s) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const size_t row = size_t(min(tile * kOuts + g + (kGated ? 0 : 8 * h), a.N - 1));
      codes[h] = (kGated && h ? a.b[1] : a.b[0]) + row * size_t(a.K / 2) + size_t(s) * 128 + t * 16;
      scales[h] = (kGated && h ? a.sf[1] : a.sf[0]) + row * size_t(a.K / 16) + size_t(s) * 16 + t * 2;
    }
  };
  auto load = [&](Step& x) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        x.c[h][j] = __ldcs(reinterpret_cast<const uint4*>(codes[h] + j * 64));
        x.s[h][j] = *reinterpret_cast<const uint16_t*>(scales[h] + j * 8);
      }
      codes[h] += 128;
      scales[h] += 16;
    }
  };

  // the output of row r of tile k and token m, from its sum (gated: both)
  auto store = [&](int k, int r, int m, float v, float u, int batch) {
    if constexpr (kGated)
      v = u * (a.act == GEMM_ACT_SILU ? gate_act<GEMM_ACT_SILU>(v) : gate_act<GEMM_ACT_GELU_TANH>(v));
    const int n = (batch + k) * kOuts + r;
    if (n < a.N) static_cast<__nv_bfloat16*>(a.C)[size_t(m) * a.N + n] = __float2bfloat16_rn(v);
  };

  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  bool ready = false;  // shared memory holds the tokens of a single pass
  float scale_back[2] = {1.0f, 1.0f};  // of the pass
  for (int batch = tile0; batch < tile1; batch += kBatch) {
    const int tiles = min(kBatch, tile1 - batch);
    bool first_pass = true, done = false;  // of this batch
    for (int c0 = s0; c0 < s1; c0 += chunk) {
      const int steps = min(chunk, s1 - c0);
      // this warp's part of the (tile, step) pairs, and its first loads
      const int u0 = tiles * steps * warp / kWarps, u1 = tiles * steps * (warp + 1) / kWarps;
      // the warps that have a step of each tile (one lane per warp), for the join
      for (int k = warp; k < tiles; k += kWarps) {
        const int from_u = tiles * steps * lane / kWarps, to_u = tiles * steps * (lane + 1) / kWarps;
        const uint32_t b = __ballot_sync(0xffffffffu, lane < kWarps && from_u < to_u &&
                                                          from_u < (k + 1) * steps && to_u > k * steps);
        if (lane == 0) with[k] = b;
      }
      Step ring[kDepth];
      int tile_in = 0, step_in = 0;  // of the next load
      auto load_next = [&](Step& x) {
        load(x);
        if (++step_in == steps) {
          step_in = 0;
          go_to(batch + ++tile_in, c0);
        }
      };
      // (the first loads go out between the steps of the tokens' preparation: all at once
      // they would hold up the tokens)
      auto start = [&](int d0, int d1) {
        if (d0 == 0) {
          tile_in = u0 / steps;
          step_in = u0 - tile_in * steps;
          go_to(batch + tile_in, c0 + step_in);
        }
#pragma unroll
        for (int d = 0; d < kDepth; ++d)
          if (d >= d0 && d < d1 && u0 + d < u1) load_next(ring[d]);
      };
      const uint16_t* A = static_cast<const uint16_t*>(a.A) + size_t(c0) * 256;
      const int per_token = steps * 32, pieces = per_token * a.M;  // of 8 k
      // what(place, piece of token m) for this thread's pieces, kAhead at a time: `get`
      // first for all of them
      auto each_piece = [&](auto get, auto what) {
        constexpr int kAhead = 4;
        int q = int(threadIdx.x), m = 0;
        while (true) {
          int at[kAhead];
#pragma unroll
          for (int b = 0; b < kAhead; ++b) {
            while (q >= per_token && m < a.M) q -= per_token, ++m;
            at[b] = -1;
            if (m < a.M) {
              // q / 16: 128 K, q / 4 % 4: t, q % 4: chunk
              const int row = 4 * m + (q >> 2 & 3);
              at[b] = ((q >> 4) * 4 * a.M + row) * 4 + ((q & 3) ^ (row >> 1 & 3));
              get(b, at[b], reinterpret_cast<const uint4*>(A + size_t(m) * a.K) + q);
            }
            q += kThreads;
          }
#pragma unroll
          for (int b = 0; b < kAhead; ++b)
            if (at[b] >= 0) what(b, at[b]);
          if (m >= a.M) break;
        }
      };
      uint32_t below = 0x8000u;  // magnitudes that are still due: below this one
      bool more = true;
      for (int plane = 0; more; ++plane) {
        uint32_t from = 0;
        const bool first_plane = plane == 0;
        more = false;
        if (ready) {
          start(0, kDepth);
        } else if (first_plane) {
          // Tokens as they come are zero or between 2^-25 and 2^8: converted on their
          // way, with one scale.  A value outside is seen at the end, and the tokens then
          // go the long way.
          constexpr uint32_t kLeast = (127 - 25) << 7, kMost = ((127 + 8) << 7) - 1;
          start(0, 1);
          uint32_t high2 = 0, low2 = 0xFFFFFFFFu;
          uint4 v[4];
          each_piece([&](int b, int, const uint4* src) { v[b] = __ldcg(src); },
                     [&](int b, int at) {
                       span_of(v[b], 0x8000u, high2, low2);
                       tokens[at] = to_f16<true>(v[b], 0u, 0u, false, 256.0f);
                     });
          start(1, kDepth);
          scale_back[0] = 1.0f / 256.0f;
          scale_back[1] = 1.0f;
          more = __syncthreads_or(max(high2 & 0xFFFFu, high2 >> 16) > kMost ||
                                  min(low2 & 0xFFFFu, low2 >> 16) < kLeast - 1);
        }
        if (!ready && (more || !first_plane)) {
          if (!first_plane) start(0, kDepth);
          // the tokens as they are
          each_piece([&](int, int at, const uint4* src) { ptx::cp_async_16(&tokens[at], src); }, [](int, int) {});
          ptx::cp_async_wait_all();
          __syncthreads();
          uint32_t high2 = 0, low2 = 0xFFFFFFFFu;
          for (int q = int(threadIdx.x); q < pieces; q += kThreads) span_of(tokens[q], below, high2, low2);
          uint32_t high = __reduce_max_sync(0xffffffffu, max(high2 & 0xFFFFu, high2 >> 16));
          uint32_t low = __reduce_min_sync(0xffffffffu, min(low2 & 0xFFFFu, low2 >> 16));
          if (lane == 0) {
            range[0][warp] = high;
            range[1][warp] = low;
          }
          __syncthreads();
#pragma unroll
          for (int i = 0; i < kWarps; ++i) {
            high = max(high, range[0][i]);
            low = min(low, range[1][i]);
          }
          if (high >= kInf) high = kInf - 1;
          // the magnitudes of this pass: [from, high]
          const uint32_t top = place(high);
          from = top > kSpan + 1 ? (top - kSpan) << 7 : 0u;
          more = low != 0xFFFFu && low + 1 < from;
          // 2^(142 - top) brings the largest to 2^15; at most 2^127
          const int e = min(142 - int(top), 127);
          const float scale = __uint_as_float(uint32_t(e + 127) << 23);
          // 2^-e in two factors, since it may lie below the FP32 range
          scale_back[0] = __uint_as_float(uint32_t(127 - e / 2) << 23);
          scale_back[1] = __uint_as_float(uint32_t(127 - (e - e / 2)) << 23);
          for (int q = int(threadIdx.x); q < pieces; q += kThreads)
            tokens[q] = to_f16<false>(tokens[q], from, high, first_plane, scale);
          __syncthreads();
        }

        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
        int tile = u0 / steps, step = u0 - tile * steps;
#pragma unroll 1
        for (int ub = u0; ub < u1; ub += kDepth) {
#pragma unroll
          for (int d = 0; d < kDepth; ++d) {
            if (ub + d >= u1) break;
            Step& x = ring[d];
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
              const uint4* tok = tokens + (step * 2 + j) * 16 * a.M;
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                uint4 v[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) v[n] = tok[mine[n][c]];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  uint32_t w[2][2];
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    const uint32_t word = (&x.c[h][j].x)[c], s2 = sc[h][c >> 1];
                    w[h][0] = i ? weights2<2>(word, s2) : weights2<0>(word, s2);
                    w[h][1] = i ? weights2<3>(word, s2) : weights2<1>(word, s2);
                  }
#pragma unroll
                  for (int n = 0; n < NT; ++n)
                    mma_16x8x16(acc[n], w[0][0], w[1][0], w[0][1], w[1][1], i ? v[n].z : v[n].x,
                                i ? v[n].w : v[n].y);
                }
              }
            }
            if (ub + d + kDepth < u1) load_next(x);
            if (++step == steps || ub + d + 1 == u1) {  // the warp's part of this tile is done
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  parts[tile + warp].v[g + 8 * (i >> 1)][8 * n + 2 * t + (i & 1)] =
                      scaled_back(acc[n][i], scale_back[0], scale_back[1], kGated && i >= 2 ? a.scale2[1] : a.scale2[0]);
                  acc[n][i] = 0.0f;
                }
              step = 0;
              ++tile;
            }
          }
        }
        __syncthreads();
        // Joins the warps' parts of each tile in order.  The sums are the result where
        // nothing else is added, and wait in `joined` otherwise.
        const bool whole = first_plane && !more && splits == 1 && s1 - s0 <= chunk;
        const int rows = whole ? kOuts : 16;
        for (int i = int(threadIdx.x); i < tiles * rows * 8 * NT; i += kThreads) {
          const int r = i % rows, m = i / rows % (8 * NT), k = i / rows / (8 * NT);
          if (m >= a.M) continue;
          auto sum = [&](int row) {
            float s = first_pass ? 0.0f : joined[k].v[row][m];
            for (uint32_t b = with[k]; b; b &= b - 1) s += parts[k + __ffs(int(b)) - 1].v[row][m];
            return s;
          };
          if (whole) store(k, r, m, sum(r), kGated ? sum(r + 8) : 0.0f, batch);
          else joined[k].v[r][m] = sum(r);
        }
        done = whole;
        first_pass = false;
        if (more) below = from;
        else if (first_plane && s1 - s0 <= chunk) ready = true;
        __syncthreads();
      }
    }
    if (done) continue;
    if (splits > 1) ptx::cluster_sync();
    // the blocks of a cluster share the outputs; sums in the order of the splits
    for (int i = int(threadIdx.x) * splits + rank; i < tiles * kOuts * 8 * NT; i += kThreads * splits) {
      const int r = i % kOuts, m = i / kOuts % (8 * NT), k = i / kOuts / (8 * NT);
      if (m >= a.M) continue;
      auto total = [&](int row) {
        const float* p = &joined[k].v[row][m];
        if (splits == 1) return *p;
        float v[kMaxCluster], s = 0.0f;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c)
          v[c] = c < splits ? ptx::ld_cluster_f32(ptx::mapa_shared(ptx::smem_u32(p), uint32_t(c))) : 0.0f;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) s += v[c];
        return s;
      };
      store(k, r, m, total(r), kGated ? total(r + 8) : 0.0f, batch);
    }
    // `joined` is read until here, by the other blocks too
    if (splits > 1) ptx::cluster_sync();
    else __syncthreads();
  }
}

template <int NT, bool kGated>
int run(const GemvW4& a, const DeviceInfo& dev, cudaStream_t stream) {
  constexpr int kOuts = kGated ? 8 : 16;
  const int tiles = (a.N + kOuts - 1) / kOuts, steps = a.K / 256, step_bytes = 512 * a.M;
  // K is divided where the tokens do not fit, or the tiles leave SMs without work that
  // have a step for each warp
  int splits = 1;
  while (splits < kMaxCluster && ((steps + splits - 1) / splits * step_bytes > kTokenBytes ||
                                  (tiles * splits * 2 <= dev.num_sms && steps >= 2 * splits * kWarps)))
    splits *= 2;
  auto kernel = gemv_w4a16_kernel<NT, kGated>;
  const int parts = int(sizeof(Tile<NT>)) * (kBatch + kWarps - 1);
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = splits;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = parts + kTokenBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // clusters of each size that the device holds at a time
  static std::atomic<int> capacity[64][4];
  const int log2 = splits == 1 ? 0 : splits == 2 ? 1 : splits == 4 ? 2 : 3;
  int cap = capacity[dev.device & 63][log2].load();
  if (cap == 0) {
    cfg.gridDim = dim3(dev.num_sms / splits * splits);
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, parts + kTokenBytes) !=
        cudaSuccess) {
      cudaGetLastError();
      return GEMM_ERR_LAUNCH;
    }
    if (cudaOccupancyMaxActiveClusters(&cap, kernel, &cfg) != cudaSuccess || cap <= 0) {
      cudaGetLastError();
      cap = dev.num_sms / splits;
    }
    capacity[dev.device & 63][log2].store(cap);
  }
  const int clusters = std::min(tiles, cap);
  const int chunk = std::max(1, std::min((steps + splits - 1) / splits, kTokenBytes / step_bytes));
  const int most = std::min(kBatch, (tiles + clusters - 1) / clusters);
  cfg.gridDim = dim3(unsigned(clusters) * splits);
  cfg.dynamicSmemBytes = sizeof(Tile<NT>) * (most + kWarps - 1) + size_t(chunk) * step_bytes;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kernel, a, splits, chunk) != cudaSuccess) {
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
