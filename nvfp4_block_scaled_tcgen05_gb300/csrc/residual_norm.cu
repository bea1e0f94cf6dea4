// Residual step of a block: for each row of D values, with r(v) = 1 / sqrt(mean(v^2) + eps)
//   c = b * r(b) * w_post      (norm after the block; c = b without w_post)
//   y = x + scale * gate * c   (rounded to the stream's type)
//   n = y * r(y) * w_pre       (norm before the next block, of y as it is stored)
// and its gradient, from dy (at y) and dn (at n), with yh = y r_y, bh = b r_b:
//   t  = dy + r_y (dn w_pre - yh mean(dn w_pre yh)),                  dx = t
//   db = r_b (p t - bh mean(p t bh)),  p = scale * gate * w_post
//   dw_pre = sum dn yh,  dw_post = sum scale gate t bh,  dgate = sum scale t bh w_post
// The second mean needs t, which needs the first; with u = dy + r_y dn w_pre,
//   sum p t bh = sum p bh u - r_y mean(dn w_pre yh) sum p bh yh,
// so one joint reduction of three sums serves both.  dw_post and dgate are both
// multiples of T = sum t bh over a gate group's rows, the one sum that is kept.
//
// Bound by memory: forward x, b read and y, n written once, backward dy, dn, y, b
// read and dx, db written once.  A unit of warps takes a row at a time; the rows
// ahead are on their way into its ring in shared memory by bulk copies, so that the
// bytes in flight do not depend on how many threads wait.  Sums are FP32 in a fixed
// order (results repeat bit for bit).
//
// Forward 16384 x 4096 with an FP32 stream 126 us (805 MB at 6.4 TB/s; without
// the ring 184 us), 8192 x 4096 BF16 46 us; backward 8128 x 4104 74.6 us (400 MB, 5.4 TB/s).
#include <algorithm>

#include "chain.cuh"
#include "epilogue_math.cuh"

namespace gb300 {

namespace {

// Eight values of a row, two FP32 operations per instruction.
struct Vec8 {
  float2 v[4];
};
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ Vec8 zero8() {
  Vec8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = make_float2(0.0f, 0.0f);
  return r;
}
__device__ __forceinline__ Vec8 unpack8(uint4 a) {
  Vec8 r;
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = make_float2(bf16_lo(w[i]), bf16_hi(w[i]));
  return r;
}
__device__ __forceinline__ uint4 pack8(const Vec8& a) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = pack_bf16x2(__float_as_uint(a.v[i].x), __float_as_uint(a.v[i].y));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight values of the stream, BF16 or FP32, as they lie in memory.
template <bool kF32>
struct Raw8;
template <>
struct Raw8<false> {
  uint4 a;
  __device__ __forceinline__ void read(const uint8_t* row, int c) {
    a = reinterpret_cast<const uint4*>(row)[c];
  }
  __device__ __forceinline__ Vec8 get() const { return unpack8(a); }
};
template <>
struct Raw8<true> {
  Vec8 a;
  __device__ __forceinline__ void read(const uint8_t* row, int c) {
    const float4 lo = reinterpret_cast<const float4*>(row)[2 * c];
    const float4 hi = reinterpret_cast<const float4*>(row)[2 * c + 1];
    a.v[0] = make_float2(lo.x, lo.y);
    a.v[1] = make_float2(lo.z, lo.w);
    a.v[2] = make_float2(hi.x, hi.y);
    a.v[3] = make_float2(hi.z, hi.w);
  }
  __device__ __forceinline__ Vec8 get() const { return a; }
};
// Stores piece i of eight values, where `live`, and returns them as they are stored.
template <bool kF32>
__device__ __forceinline__ Vec8 store8(void* p, size_t i, const Vec8& v, bool live = true) {
  if constexpr (kF32) {
    float4* q = static_cast<float4*>(p) + 2 * i;
    if (live) {
      q[0] = make_float4(v.v[0].x, v.v[0].y, v.v[1].x, v.v[1].y);
      q[1] = make_float4(v.v[2].x, v.v[2].y, v.v[3].x, v.v[3].y);
    }
    return v;
  } else {
    const uint4 w = pack8(v);
    if (live) static_cast<uint4*>(p)[i] = w;
    return unpack8(w);
  }
}
__device__ __forceinline__ Vec8 weights8(const void* w, size_t i) {
  return unpack8(static_cast<const uint4*>(w)[i]);
}

__device__ __forceinline__ Vec8 weighted(Vec8 v, const Vec8& w) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v.v[j] = ptx::mul2(v.v[j], w.v[j]);
  return v;
}
__device__ __forceinline__ Vec8 scaled(float scale, Vec8 v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v.v[j] = ptx::mul2(both(scale), v.v[j]);
  return v;
}
// Piece `at` of a gate (ones where there is none) times `scale`; piece c of a weight
// (ones) times v.
__device__ __forceinline__ Vec8 scaled_gate(float scale, const void* gate, size_t at) {
  if (gate) return scaled(scale, weights8(gate, at));
  Vec8 f;
#pragma unroll
  for (int j = 0; j < 4; ++j) f.v[j] = both(scale);
  return f;
}
__device__ __forceinline__ Vec8 times_weight(const Vec8& v, const void* weight, int c) {
  return weight ? weighted(v, weights8(weight, c)) : v;
}

__device__ __forceinline__ float inverse_rms(float sum, int D, float eps) {
  return 1.0f / sqrtf(sum / float(D) + eps);
}

// How a kernel's blocks are laid out: `units` of `warps` warps each, a unit with a
// ring of `stages` rows of stage_bytes; a thread has V pieces of eight values.
struct Shape {
  int V, warps, units, stages;
  int stage_bytes;
  int threads() const { return 32 * warps * units; }
  int smem() const { return 128 + units * stages * (stage_bytes + 8); }
};

constexpr int kMaxWarps = 16;  // of a unit: D = 16384 with V = 4

// Rows of up to five matrices through a unit's ring.
struct Source {
  const void* p;
  uint32_t bytes;  // per row; 0: no such matrix
  int rows = 1;    // that share a row of it
};
template <int N>
struct Ring {
  Source src[N];
  uint8_t* mem;
  uint32_t bars, base;
  int stage_bytes, stages, unit, warps, tid;
  int next_stage, stage;
  uint32_t phase;
  Watch w;

  // `smem`: the block's dynamic shared memory.  Every thread of the block calls it.
  __device__ __forceinline__ void init(uint8_t* smem, const Shape& s, unsigned int* status,
                                       unsigned long long timeout_ns) {
    volatile uint32_t* abort = reinterpret_cast<volatile uint32_t*>(smem);
    warps = s.warps;
    stages = s.stages;
    stage_bytes = s.stage_bytes;
    unit = int(threadIdx.x) / (32 * warps);
    tid = int(threadIdx.x) - unit * 32 * warps;
    const uint32_t at = ptx::smem_u32(smem);
    mem = smem + 128 + size_t(unit) * stages * stage_bytes;
    base = ptx::smem_u32(mem);
    bars = at + 128 + s.units * stages * stage_bytes + unit * stages * 8;
    if (tid == 0)
      for (int i = 0; i < stages; ++i) ptx::mbar_init(bars + 8 * i, 1);
    if (threadIdx.x == 0) *abort = 0u;
    ptx::fence_mbar_init();
    __syncthreads();
    w = Watch{abort, status, timeout_ns};
    next_stage = stage = 0;
    phase = 0;
  }
  // The unit's first thread: the row's copies into the next stage.
  __device__ __forceinline__ void fill(int row) {
    uint32_t total = 0, dst = base + uint32_t(next_stage) * stage_bytes;
#pragma unroll
    for (int i = 0; i < N; ++i) total += src[i].bytes;
    const uint32_t bar = bars + 8 * next_stage;
    ptx::mbar_arrive_expect_tx(bar, total);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (src[i].bytes) {
        const int of = src[i].rows == 1 ? row : row / src[i].rows;
        ptx::bulk_load(dst, static_cast<const uint8_t*>(src[i].p) + size_t(of) * src[i].bytes, src[i].bytes, bar);
        dst += src[i].bytes;
      }
    if (++next_stage == stages) next_stage = 0;
  }
  // Waits for the current stage.  A wait that runs out is recorded and the kernel
  // goes on over what is there (every thread makes the same steps either way).
  __device__ __forceinline__ const uint8_t* wait() {
    wait_bar(bars + 8 * stage, phase, w, 12);
    return mem + size_t(stage) * stage_bytes;
  }
  __device__ __forceinline__ void advance() {
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  // After a wait that ran out: time for the copies in flight to land.
  __device__ __forceinline__ void settle() const {
    if (*w.abort) spin_ns(2000000ull);
  }
  __device__ __forceinline__ void sync() const {
    if (warps == 1) __syncwarp();
    else ptx::named_barrier(1 + unit, 32 * warps);
  }
  // Sums of K values over the unit; every thread gets them.  A barrier of the unit's
  // threads lies within.  `part`: K floats per warp, free again two calls later.
  template <int K>
  __device__ __forceinline__ void sum(float (&s)[K], float* part) const {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < K; ++k) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
    if (warps == 1) {
      __syncwarp();
      return;
    }
    if ((tid & 31) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) part[k * kMaxWarps + (tid >> 5)] = s[k];
    sync();
    // every warp adds the parts in the same tree
    const int lane = tid & 31;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      s[k] = lane < warps ? part[k * kMaxWarps + lane] : 0.0f;
#pragma unroll
      for (int o = kMaxWarps / 2; o > 0; o >>= 1) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
      s[k] = __shfl_sync(0xffffffffu, s[k], 0);
    }
  }
};

// ---------------------------------------------------------------- forward
// kFull: there are a block and both norms, the usual call, whose choices are then made
// at compile time (below: `has_*`).  kGates: and nearly every row of a unit has another
// gate, which then comes through the ring (8192 x 4096, a gate for each row: 74 -> 55 us).
template <bool kF32, int V, int kThreads, bool kFull, bool kGates>
__global__ void __launch_bounds__(kThreads, 1)
    residual_norm_kernel(const ResidualNorm a, const Shape shape, unsigned int* status,
                         unsigned long long timeout_ns) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float parts[kMaxWarps][2][2][kMaxWarps];
  const bool has_block = kFull || a.block, has_post = kFull || a.w_post, has_pre = kFull || a.w_pre;
  Ring<kGates ? 3 : 2> ring;
  ring.src[0] = {a.x, uint32_t(a.D) * (kF32 ? 4u : 2u)};
  ring.src[1] = {a.block, has_block ? uint32_t(a.D) * 2u : 0u};
  if constexpr (kGates) ring.src[2] = {a.gate, uint32_t(a.D) * 2u, a.rows_per_gate};
  ring.init(smem, shape, status, timeout_ns);
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int pieces = a.D / 8, step = int(gridDim.x) * shape.units, threads = 32 * shape.warps;
  const int first = int(blockIdx.x) * shape.units + ring.unit;
  if (ring.tid == 0)
    for (int i = 0, row = first; i < shape.stages && row < a.M; ++i, row += step) ring.fill(row);
  // This thread's pieces.  A place past the row's end reads the last piece again; its
  // values are set to zero before each sum (an infinite weight or gate makes them NaN in
  // between), and not stored.
  int at[V];
  uint4 w_pre[V], w_post[V];
  Vec8 p[V];  // scale * gate * w_post
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = ring.tid + i * threads;
    at[i] = min(c, pieces - 1);
    w_pre[i] = has_pre ? static_cast<const uint4*>(a.w_pre)[at[i]] : make_uint4(0, 0, 0, 0);
    p[i] = has_block && !a.gate ? times_weight(scaled_gate(a.scale, nullptr, 0), a.w_post, at[i]) : zero8();
    if (kGates) w_post[i] = static_cast<const uint4*>(a.w_post)[at[i]];
  }
  auto live = [&](int i) { return ring.tid + i * threads < pieces; };
  int gate_row = -1;
  float(*part)[2][kMaxWarps] = parts[ring.unit];
  int odd = 0;
  for (int row = first; row < a.M; row += step, odd ^= 1) {
    const size_t base = size_t(row) * pieces;
    if (!kGates && a.gate && row / a.rows_per_gate != gate_row) {
      gate_row = row / a.rows_per_gate;
#pragma unroll
      for (int i = 0; i < V; ++i)
        p[i] = times_weight(scaled_gate(a.scale, a.gate, size_t(gate_row) * pieces + at[i]), a.w_post, at[i]);
    }
    const uint8_t* mem = ring.wait();
    Vec8 y[V], b[V];
    uint4 gate[V];
    float2 s2 = both(0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      Raw8<kF32> x;
      x.read(mem, at[i]);
      y[i] = x.get();
      b[i] = zero8();
      if (has_block) b[i] = unpack8(reinterpret_cast<const uint4*>(mem + ring.src[0].bytes)[at[i]]);
      if constexpr (kGates)
        gate[i] = reinterpret_cast<const uint4*>(mem + ring.src[0].bytes + ring.src[1].bytes)[at[i]];
      if (!live(i)) b[i] = zero8();
#pragma unroll
      for (int j = 0; j < 4; ++j) s2 = ptx::fma2(b[i].v[j], b[i].v[j], s2);
    }
    // the row is in registers: after the next barrier its stage takes another
    ptx::fence_proxy_async_smem();
    const int ahead = row + shape.stages * step;
    const bool refill = ring.tid == 0 && ahead < a.M && ahead > row;
    float r = 1.0f;
    if (has_post) {
      float s[1] = {s2.x + s2.y};
      ring.sum(s, part[odd][0]);
      if (refill) ring.fill(ahead);
      r = inverse_rms(s[0], a.D, a.eps);
      if (ring.tid == 0 && a.rstd_post) a.rstd_post[row] = r;
    }
    s2 = both(0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (has_block) {
        if constexpr (kGates) p[i] = weighted(scaled(a.scale, unpack8(gate[i])), unpack8(w_post[i]));
#pragma unroll
        for (int j = 0; j < 4; ++j)
          y[i].v[j] = ptx::fma2(ptx::mul2(b[i].v[j], both(r)), p[i].v[j], y[i].v[j]);
        y[i] = store8<kF32>(a.y, base + at[i], y[i], live(i));
      }
      if (!live(i)) y[i] = zero8();
#pragma unroll
      for (int j = 0; j < 4; ++j) s2 = ptx::fma2(y[i].v[j], y[i].v[j], s2);
    }
    if (has_pre) {
      float s[1] = {s2.x + s2.y};
      ring.sum(s, part[odd][1]);
      if (refill && !has_post) ring.fill(ahead);
      const float ry = inverse_rms(s[0], a.D, a.eps);
      if (ring.tid == 0 && a.rstd_pre) a.rstd_pre[row] = ry;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const Vec8 w = unpack8(w_pre[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[i].v[j] = ptx::mul2(ptx::mul2(y[i].v[j], both(ry)), w.v[j]);
        store8<false>(a.n, base + at[i], y[i], live(i));
      }
    } else if (!has_post) {
      ring.sync();
      if (refill) ring.fill(ahead);
    }
    ring.advance();
  }
  ring.settle();
}

// ---------------------------------------------------------------- backward
// Each unit takes a run of consecutive rows.  Where a gate's gradient is summed and
// its rows are many, a block's runs lie within one gate group (parts_per_gate blocks
// to a group); else a run holds whole groups and writes their dgate itself.  A
// thread keeps its columns' sums of the run in registers; a block's units are added
// in order and go to the block's place in the workspace, [block][kinds][D]: dn yh,
// and T, which the join multiplies, or (several gate groups in a run, kMulti) dw_post.
// kGates: every row has its own gate, which comes through the ring, and T is the row's
// (8192 x 4096: read when at hand 165 us, so 107; FP32 stream 196 and 148).
template <bool kF32, int V, int kThreads, bool kMulti, bool kFull, bool kGates>
__global__ void __launch_bounds__(kThreads, 1)
    residual_norm_backward_kernel(const ResidualNormBackward a, const Shape shape,
                                  unsigned int* status, unsigned long long timeout_ns) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float parts[kMaxWarps][2][3 * kMaxWarps];
  const bool has_dy = kFull || a.dy, has_block = kFull || a.block, has_post = kFull || a.w_post,
             has_pre = kFull || a.w_pre;
  static_assert(!kGates || (kMulti && kFull), "a run of many gates, every part");
  Ring<kGates ? 5 : 4> ring;
  const uint32_t wide = uint32_t(a.D) * (kF32 ? 4u : 2u), narrow = uint32_t(a.D) * 2u;
  ring.src[0] = {a.dy, has_dy ? wide : 0u};
  ring.src[1] = {a.y, has_pre ? wide : 0u};
  ring.src[2] = {a.dn, has_pre ? narrow : 0u};
  ring.src[3] = {a.block, has_block ? narrow : 0u};
  if constexpr (kGates) ring.src[4] = {a.gate, narrow};
  ring.init(smem, shape, status, timeout_ns);
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int pieces = a.D / 8, threads = 32 * shape.warps;
  int row, end;
  {
    int first, last;  // the block's rows
    if (a.parts_per_gate) {
      const int group = int(blockIdx.x) / a.parts_per_gate, k = int(blockIdx.x) % a.parts_per_gate;
      first = group * a.rows_per_gate + k * a.rows_per_run * shape.units;
      last = (group + 1) * a.rows_per_gate;
    } else {
      first = int(blockIdx.x) * a.rows_per_run * shape.units;
      last = a.M;
    }
    row = min(first + ring.unit * a.rows_per_run, last);
    end = min(row + a.rows_per_run, last);
  }
  const int begin = row;
  if (ring.tid == 0)
    for (int i = 0; i < shape.stages && row + i < end; ++i) ring.fill(row + i);
  // This thread's pieces.  A place past the row's end reads the last piece again, and
  // neither joins the row's sums nor is stored.
  int at[V];
  auto live = [&](int i) { return ring.tid + i * threads < pieces; };
  uint4 w_pre[V], w_post[V];
  Vec8 dwi[V], T[V], dwo[kMulti ? V : 1];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    at[i] = min(ring.tid + i * threads, pieces - 1);
    w_pre[i] = has_pre && live(i) ? static_cast<const uint4*>(a.w_pre)[at[i]] : make_uint4(0, 0, 0, 0);
    if (kGates) w_post[i] = static_cast<const uint4*>(a.w_post)[at[i]];
    dwi[i] = T[i] = zero8();
    if constexpr (kMulti) dwo[i] = zero8();
  }
  Vec8 p[V];
  int gate_row = -1;
  auto read_gate = [&](int gate) {
    gate_row = gate;
#pragma unroll
    for (int i = 0; i < V; ++i)
      p[i] = has_block && live(i)
                 ? times_weight(scaled_gate(a.scale, a.gate, size_t(gate) * pieces + at[i]), a.w_post, at[i])
                 : zero8();
  };
  if (!kMulti) read_gate(row < end ? row / a.rows_per_gate : 0);
  float(*part)[3 * kMaxWarps] = parts[ring.unit];
  float ry = 0.0f, rb = 1.0f;
  auto read_rstd = [&](int of) {
    if (has_pre) ry = __ldcg(a.rstd_pre + of);
    if (has_post) rb = __ldcg(a.rstd_post + of);
  };
  if (row < end) read_rstd(row);
  int odd = 0;
  for (; row < end; ++row, odd ^= 1) {
    const size_t base = size_t(row) * pieces;
    if (kMulti && !kGates && row / a.rows_per_gate != gate_row) read_gate(row / a.rows_per_gate);
    const float r_y = ry, r_b = rb;
    const uint8_t* mem = ring.wait();
    if (row + 1 < end) read_rstd(row + 1);  // a row ahead
    const uint8_t *mem_y = mem + (has_dy ? wide : 0u), *mem_n = mem_y + wide;
    const uint8_t* mem_b = has_pre ? mem_n + narrow : mem_y;
    // piece i of the row's gate, and of scale * gate * w_post
    auto own_gate = [&](int i) { return scaled(a.scale, unpack8(reinterpret_cast<const uint4*>(mem_b + narrow)[at[i]])); };
    auto factor = [&](int i) {
      if constexpr (kGates) return weighted(own_gate(i), unpack8(w_post[i]));
      else return p[i];
    };
    Vec8 u[V];
    float2 s0 = both(0.0f), s1 = s0, s2 = s0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      u[i] = zero8();
      Vec8 yh = zero8();
      float2 q0 = both(0.0f), q1 = q0, q2 = q0;
      if (has_dy) {
        Raw8<kF32> d;
        d.read(mem, at[i]);
        u[i] = d.get();
      }
      if (has_pre) {
        Raw8<kF32> y;
        y.read(mem_y, at[i]);
        yh = y.get();
        const Vec8 d = unpack8(reinterpret_cast<const uint4*>(mem_n)[at[i]]), w = unpack8(w_pre[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          yh.v[j] = ptx::mul2(yh.v[j], both(r_y));
          dwi[i].v[j] = ptx::fma2(d.v[j], yh.v[j], dwi[i].v[j]);
          const float2 e = ptx::mul2(d.v[j], w.v[j]);
          q0 = ptx::fma2(e, yh.v[j], q0);
          u[i].v[j] = ptx::fma2(e, both(r_y), u[i].v[j]);
        }
      }
      if (has_post) {
        const Vec8 b = unpack8(reinterpret_cast<const uint4*>(mem_b)[at[i]]), f = factor(i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // p bh, its factor r_b left for the sums
          const float2 pb = ptx::mul2(f.v[j], b.v[j]);
          q1 = ptx::fma2(pb, u[i].v[j], q1);
          q2 = ptx::fma2(pb, yh.v[j], q2);
        }
      }
      if (live(i)) {
        s0 = ptx::add2(s0, q0);
        s1 = ptx::add2(s1, q1);
        s2 = ptx::add2(s2, q2);
      }
    }
    // Behind the next barrier every thread is done with the previous row, whose stage
    // then takes another (with one stage: at the end of the row).
    ptx::fence_proxy_async_smem();
    float s[3] = {s0.x + s0.y, s1.x + s1.y, s2.x + s2.y};
    if (has_pre || has_post) ring.sum(s, part[odd]);
    else ring.sync();
    if (ring.tid == 0 && shape.stages > 1 && row > begin && shape.stages - 1 < end - row)
      ring.fill(row - 1 + shape.stages);
    const float m1 = r_y * s[0] / float(a.D);  // r_y mean(dn w_pre yh)
    const float m2 = r_b * (s[1] - m1 * s[2]) / float(a.D);
    const float2 ny = both(-m1 * r_y), nb = both(-m2 * r_b * r_b);
    const bool last = kGates || (kMulti && ((row + 1) % a.rows_per_gate == 0 || row + 1 == end));
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (has_pre) {
        Raw8<kF32> y;
        y.read(mem_y, at[i]);
        const Vec8 v = y.get();
#pragma unroll
        for (int j = 0; j < 4; ++j) u[i].v[j] = ptx::fma2(v.v[j], ny, u[i].v[j]);
      }
      store8<kF32>(a.dx, base + at[i], u[i], live(i));
      if (has_block) {
        const Vec8 b = unpack8(reinterpret_cast<const uint4*>(mem_b)[at[i]]), f = factor(i);
        Vec8 db;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          T[i].v[j] = ptx::fma2(u[i].v[j], ptx::mul2(b.v[j], both(r_b)), T[i].v[j]);
          db.v[j] = ptx::mul2(f.v[j], u[i].v[j]);
          if (has_post) db.v[j] = ptx::fma2(b.v[j], nb, ptx::mul2(db.v[j], both(r_b)));
        }
        store8<false>(a.dblock, base + at[i], db, live(i));
        if (last) {  // the gate group's end
          const size_t to = kGates ? base : size_t(gate_row) * pieces;
          const Vec8 gate = kGates ? own_gate(i) : scaled_gate(a.scale, a.gate, to + at[i]);
          Vec8 dg = scaled(a.scale, T[i]);
          dg = kGates ? weighted(dg, unpack8(w_post[i])) : times_weight(dg, a.w_post, at[i]);
          if (a.dgate) store8<true>(a.dgate, to + at[i], dg, live(i));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (kMulti) dwo[i].v[j] = ptx::fma2(gate.v[j], T[i].v[j], dwo[i].v[j]);
            T[i].v[j] = make_float2(0.0f, 0.0f);
          }
        }
      }
    }
    if (shape.stages == 1 && row + 1 < end) {
      ptx::fence_proxy_async_smem();
      ring.sync();
      if (ring.tid == 0) ring.fill(row + 1);
    }
    ring.advance();
  }
  ring.settle();
  if (a.kinds == 0) return;
  // the block's sums; the units after the first hand theirs over in the rings' place,
  // free once every unit is done
  __syncthreads();
  float* hand = reinterpret_cast<float*>(smem + 128);
  auto give = [&](Vec8* v, int kind) {
    if (ring.unit > 0)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = ring.tid + i * threads;
        if (c < pieces) store8<true>(hand, size_t(ring.unit - 1) * pieces + c, v[i]);
      }
    __syncthreads();
    if (ring.unit == 0)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = ring.tid + i * threads;
        if (c >= pieces) continue;
        for (int n = 1; n < shape.units; ++n) {
          Raw8<true> other;
          other.read(reinterpret_cast<const uint8_t*>(hand), (n - 1) * pieces + c);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[i].v[j] = ptx::add2(v[i].v[j], other.a.v[j]);
        }
        store8<true>(a.parts, (size_t(blockIdx.x) * a.kinds + kind) * pieces + c, v[i]);
      }
    __syncthreads();
  };
  if (a.dw_pre) give(dwi, 0);
  if (a.kinds > (a.dw_pre != nullptr)) give(kMulti ? dwo : T, a.dw_pre != nullptr);
}

// Adds the blocks' parts in a fixed order.  A block takes 32 columns; blockIdx.y 0:
// dw_pre (or, without it, what 1 does); 1: dw_post and dgate, from T of each gate
// group's parts, or dw_post from its own parts (multi).  The warps are shared
// out among the groups (8128 x 4104, 8 groups of 19 parts: one group after the other,
// all warps on each, 15 us).
constexpr int kJoinWarps = 16;
__global__ void __launch_bounds__(32 * kJoinWarps)
    residual_norm_join_kernel(const ResidualNormBackward a, int blocks, int multi) {
  __shared__ float sum[kJoinWarps][32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = int(threadIdx.x) & 31, warp = int(threadIdx.x) >> 5;
  const int col = int(blockIdx.x) * 32 + lane;
  const bool live = col < a.D;
  const int kind = int(blockIdx.y);
  const size_t step = size_t(a.kinds) * a.D;
  const float* src = a.parts + size_t(kind) * a.D + col;
  auto range = [&](int from, int to, int by) {
    float s = 0.0f;
    if (live) {
#pragma unroll 8
      for (int r = from; r < to; r += by) s += __ldcg(src + size_t(r) * step);
    }
    return s;
  };
  // the warps' values, added in order; warp 0 gets the sum
  auto join = [&](float s) {
    __syncthreads();
    sum[warp][lane] = s;
    __syncthreads();
    if (warp == 0)
      for (int w = 1; w < kJoinWarps; ++w) s += sum[w][lane];
    return s;
  };
  if ((kind == 0 && a.dw_pre) || multi) {
    const float s = join(range(warp, blocks, kJoinWarps));
    if (warp == 0 && live) (kind == 0 && a.dw_pre ? a.dw_pre : a.dw_post)[col] = s;
    return;
  }
  const int per = a.parts_per_gate ? a.parts_per_gate : blocks, groups = blocks / per;
  const float w = live && a.w_post ? __uint_as_float(uint32_t(static_cast<const uint16_t*>(a.w_post)[col]) << 16) : 1.0f;
  float dwo = 0.0f;
  auto group_done = [&](int g, float s) {
    if (!live) return;
    if (a.dgate) a.dgate[size_t(g) * a.D + col] = a.scale * w * s;
    const float f = a.gate ? __uint_as_float(uint32_t(static_cast<const uint16_t*>(a.gate)[size_t(g) * a.D + col]) << 16) : 1.0f;
    dwo += a.scale * f * s;
  };
  // `share` warps to a group
  int share = kJoinWarps;
  while (share > 1 && share * groups > kJoinWarps) share /= 2;
  for (int g0 = 0; g0 < groups; g0 += kJoinWarps / share) {
    const int g = g0 + warp / share, sub = warp % share;
    float s = g < groups ? range(g * per + sub, (g + 1) * per, share) : 0.0f;
    if (share > 1) {
      __syncthreads();
      sum[warp][lane] = s;
      __syncthreads();
      if (sub == 0)
        for (int j = 1; j < share; ++j) s += sum[warp + j][lane];
    }
    if (sub == 0 && g < groups) group_done(g, s);
  }
  dwo = join(dwo);
  if (warp == 0 && live && a.dw_post) a.dw_post[col] = dwo;
}

// ---------------------------------------------------------------- host
// A row of D / 8 pieces with V pieces a thread.  One block per SM, of as many units
// as the registers of V pieces leave warps for; two units or more where two or three
// pieces a thread allow it, so that one works while another waits at its barrier.
// (One unit of two pieces a thread: backward 76 us at 6553 x 5120 and 5461 x 6144, 74 at
// 4096 x 8192; two units of four pieces, which spill, took 139 us at the first.  Rows of more
// than 8192 values need four pieces, and spill: 2736 x 12288 forward 80, backward 167 us,
// floors 40 and 59.)
constexpr int kBlocks = 152;
// Rows on their way, per SM: the backward pass needs the 200 KB (100 KB: 8192 x 4096
// 76 -> 106 us), the forward pass was a little faster with half of it (56 -> 54 us, before
// the choices at compile time).
constexpr int kThreadsOf[5] = {0, 512, 512, 384, 512};
constexpr int kForwardBytes = 104 << 10, kBackwardBytes = 208 << 10;
Shape make_shape(int D, int row_bytes, bool forward) {
  const int ring_bytes = forward ? kForwardBytes : kBackwardBytes;
  Shape s{};
  const int pieces = D / 8;
  auto take = [&](int v) {
    s.V = v;
    s.warps = (pieces + 32 * v - 1) / (32 * v);
    s.units = std::min(kMaxWarps, kThreadsOf[v] / (32 * s.warps));
    return s.units >= 2;
  };
  if (pieces <= 32) {
    take(1);
  } else if (!take(2) && !take(3)) {
    // the forward pass needs fewer registers: two units of three pieces a thread still
    // fit, spilling a little (6553 x 5120: 64 us with one unit, 46 with two)
    if (forward && s.warps <= 8) s.units = 2;
    else take(pieces <= 1024 ? 2 : 4);
  }
  s.units = std::max(1, s.units);
  s.stage_bytes = (row_bytes + 127) / 128 * 128;
  s.stages = std::min(8, std::max(1, ring_bytes / (s.units * (s.stage_bytes + 8))));
  return s;
}

// How the backward pass's rows are divided; depends on the sizes alone.  Where a gate's
// gradient is summed, no run crosses a group's end unless it holds whole groups, whatever
// that leaves of the SMs.  8192 x 4096: one to eight gates 74 us (8 x 19 blocks), 16 and 32
// gates 107 (160 blocks: a second round for eight of them), 64 99 (192); 32768 x 1024 with
// 128 rows to a gate 439 us (each unit a whole group, on 32 SMs), 65536 x 512 with 256 rows
// 817 (16 SMs), against 80 with one gate.
struct RunPlan {
  int blocks, rows_per_run, parts_per_gate;
  bool multi;
};
RunPlan make_runs(int M, int rows_per_gate, bool gates, const Shape& s) {
  RunPlan q{};
  const int most = kBlocks * s.units;
  int rows = (M + most - 1) / most;
  const int per_block = rows * s.units;
  // one group for all rows needs no care
  if (rows_per_gate >= M) {
    q.blocks = (M + per_block - 1) / per_block;
  } else if (gates && rows_per_gate >= per_block) {
    q.parts_per_gate = (rows_per_gate + per_block - 1) / per_block;
    const int units = q.parts_per_gate * s.units;
    rows = (rows_per_gate + units - 1) / units;
    q.parts_per_gate = (rows_per_gate + rows * s.units - 1) / (rows * s.units);
    q.blocks = M / rows_per_gate * q.parts_per_gate;
  } else {
    q.multi = true;
    if (gates) rows = (rows + rows_per_gate - 1) / rows_per_gate * rows_per_gate;
    q.blocks = (M + rows * s.units - 1) / (rows * s.units);
  }
  q.rows_per_run = rows;
  return q;
}

template <class Kernel, class... Args>
int launch_rows(Kernel kernel, const Shape& s, int blocks, std::atomic<int> (&ready)[64],
                const DeviceInfo& dev, cudaStream_t stream, Args... args) {
  if (!ready[dev.device & 63].load()) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 << 10) !=
        cudaSuccess) {
      cudaGetLastError();
      return GEMM_ERR_LAUNCH;
    }
    ready[dev.device & 63].store(1);
  }
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(s.threads());
  cfg.dynamicSmemBytes = s.smem();
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args..., s, dev.status, wait_timeout_ns()) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  return GEMM_OK;
}

template <bool kF32, int V, bool kFull, bool kGates, int kThreads = kThreadsOf[V]>
int run_forward(const ResidualNorm& a, const Shape& s, const DeviceInfo& dev, cudaStream_t stream) {
  static std::atomic<int> ready[64];
  const int blocks = std::min((a.M + s.units - 1) / s.units, kBlocks);
  return launch_rows(residual_norm_kernel<kF32, V, kThreads, kFull, kGates>, s, blocks, ready, dev, stream, a);
}

template <bool kF32, int V, bool kMulti, bool kFull, bool kGates>
int run_backward(const ResidualNormBackward& a, const Shape& s, int blocks, const DeviceInfo& dev,
                 cudaStream_t stream) {
  static std::atomic<int> ready[64];
  return launch_rows(residual_norm_backward_kernel<kF32, V, kThreadsOf[V], kMulti, kFull, kGates>, s, blocks,
                     ready, dev, stream, a);
}

int backward_row_bytes(int D, bool f32, bool dy, bool pre, bool block) {
  const int wide = D * (f32 ? 4 : 2);
  return (dy ? wide : 0) + (pre ? wide + 2 * D : 0) + (block ? 2 * D : 0);
}

}  // namespace

// The shape's units and blocks do not depend on the stages, so the matrices that a
// call has make no difference here.
size_t residual_norm_backward_workspace(int M, int D, int rows_per_gate, int weights, bool gates) {
  const Shape s = make_shape(D, 128, false);
  const RunPlan q = make_runs(M, rows_per_gate, gates, s);
  return size_t(q.blocks) * (weights + (gates && !q.multi)) * D * sizeof(float);
}

int launch_residual_norm(const ResidualNorm& a, const DeviceInfo& dev, cudaStream_t stream) {
  // (a unit's rows are at most kBlocks units apart; with V = 4 the kernel has no registers
  // for choices made at compile time)
  const bool full = a.block && a.w_post && a.w_pre && a.D <= 8192;
  const int row_bytes = a.D * (a.x_f32 ? 4 : 2) + (a.block ? 2 * a.D : 0);
  Shape s = make_shape(a.D, row_bytes, true);
  const bool gates = full && a.gate && a.rows_per_gate < kBlocks * s.units;
  if (gates) s = make_shape(a.D, row_bytes + 2 * a.D, true);
  auto go = [&](auto f32, auto kind) {
    constexpr bool kF32 = decltype(f32)::value, kFull = decltype(kind)::value > 0, kGates = decltype(kind)::value > 1;
    if (s.V == 1) return run_forward<kF32, 1, kFull, kGates>(a, s, dev, stream);
    if (s.V == 2) return run_forward<kF32, 2, kFull, kGates>(a, s, dev, stream);
    if (s.V == 3)
      return s.threads() <= kThreadsOf[3] ? run_forward<kF32, 3, kFull, kGates>(a, s, dev, stream)
                                          : run_forward<kF32, 3, kFull, kGates, 512>(a, s, dev, stream);
    return run_forward<kF32, 4, false, false>(a, s, dev, stream);
  };
  auto go_kind = [&](auto f32) {
    if (gates) return go(f32, std::integral_constant<int, 2>{});
    return full ? go(f32, std::integral_constant<int, 1>{}) : go(f32, std::integral_constant<int, 0>{});
  };
  return a.x_f32 ? go_kind(std::true_type{}) : go_kind(std::false_type{});
}

int launch_residual_norm_backward(const ResidualNormBackward& args, const DeviceInfo& dev,
                                  cudaStream_t stream) {
  ResidualNormBackward a = args;
  const bool full = a.dy && a.block && a.w_post && a.w_pre && a.D <= 8192;
  const bool gates = full && a.gate && a.rows_per_gate == 1 && a.M > 1;
  const Shape s = make_shape(a.D, backward_row_bytes(a.D, a.x_f32, a.dy, a.w_pre, a.block) + (gates ? 2 * a.D : 0), false);
  const RunPlan q = make_runs(a.M, a.rows_per_gate, a.dgate != nullptr, s);
  a.rows_per_run = q.rows_per_run;
  a.parts_per_gate = q.parts_per_gate;
  a.kinds = (a.dw_pre != nullptr) + (a.dw_post != nullptr || (a.dgate && !q.multi));
  // kinds: any call; every part (0, 1), of one gate or (2) several per run; 3: a gate per row
  auto go = [&](auto f32, auto kind) {
    constexpr int k = decltype(kind)::value;
    constexpr bool kF32 = decltype(f32)::value, kMulti = k >= 2, kFull = k == 1 || k == 3, kGates = k == 3;
    if (s.V == 1) return run_backward<kF32, 1, kMulti, kFull, kGates>(a, s, q.blocks, dev, stream);
    if (s.V == 2) return run_backward<kF32, 2, kMulti, kFull, kGates>(a, s, q.blocks, dev, stream);
    if (s.V == 3) return run_backward<kF32, 3, kMulti, kFull, kGates>(a, s, q.blocks, dev, stream);
    return run_backward<kF32, 4, kMulti, false, false>(a, s, q.blocks, dev, stream);
  };
  auto go_kind = [&](auto f32) {
    if (q.multi)
      return gates ? go(f32, std::integral_constant<int, 3>{}) : go(f32, std::integral_constant<int, 2>{});
    return full ? go(f32, std::integral_constant<int, 1>{}) : go(f32, std::integral_constant<int, 0>{});
  };
  const int rc = a.x_f32 ? go_kind(std::true_type{}) : go_kind(std::false_type{});
  if (rc != GEMM_OK || a.kinds == 0) return rc;
  return launch_dependent(residual_norm_join_kernel, dim3((a.D + 31) / 32, a.kinds),
                          32 * kJoinWarps, stream, a, q.blocks, int(q.multi));
}

}  // namespace gb300
