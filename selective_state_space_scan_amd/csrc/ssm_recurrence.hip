// The gated recurrence, for MI355X (gfx950): forward, backward, and one step on
// a cache of states.
//
// For every batch row b, channel d and step t < valid_len[b], with r =
// sigmoid(a_gate), i = sigmoid(x_gate) and s = exp(A_log[d]) r:
//
//     a[t] = exp(-s),  c[t] = sqrt(1 - a[t]^2),  h[t] = a[t] h[t-1] + c[t] i[t] x[t],  y[t] = h[t]
//
// Backward, g[t] the gradient of h[t]:
//
//     g[t] = dy[t] + a[t+1] g[t+1]  (dh_last behind the last step),
//     dx = g c i,  dx_gate = g c i x (1 - i),  q = s dL/ds = (s a^2 / c) g i x - s a g h[t-1],
//     da_gate = q (1 - r),  dA_log = sum over b, t of q,  dh0 = a[0] g[0]
//
// (s enters through exp(A_log) and through r, so its own gradient is wanted
// only as s dL/ds; s a^2 / c goes to 0 with s.)
//
// Both recurrences are affine, h -> a h + u, and affine maps compose: (P, S)
// behind (P', S') is (P P', P S' + S).  A lane folds the steps it holds into
// one pair, a workgroup's waves join theirs in LDS, and every step is then
// known from the state in front of its lane.
//
// 40 vector operations a step and channel forward and 75 backward, 6 of them
// transcendental, on 8 and 14 bytes of bf16: about as long as the bytes take (us, 8 x
// 4096 x 1024 bf16: 61 to 65 forward for 53 of bytes, 123 backward for 92; 1 x 32768 x
// 2048: 108 for 104, 233 for 183; 8 x 4096 x 512 f32: 55 for 53, 95.5 for 92).

#include <hip/hip_runtime.h>

#include <cstdint>

#include "ssm_block.h"

namespace {

constexpr int kChunk = 64;  // steps between kept states

struct GatedParams {
  const void* x;
  const void* ag;
  const void* xg;
  const float* A_log;
  const int32_t* valid_len;
  const float* h0;
  void* y;
  float* h_last;
  float* states;
  int64_t x_bs, x_ts, ag_bs, ag_ts, xg_bs, xg_ts, y_bs, y_ts;
  int64_t L;
  int32_t nd, n_cg, n_states;
};

struct GatedBwdParams {
  const void* x;
  const void* ag;
  const void* xg;
  const float* A_log;
  const int32_t* valid_len;
  const float* h0;
  const void* dy;
  const float* dh_last;
  const float* states;
  void* dx;
  void* dag;
  void* dxg;
  float* dh0;
  float* ws;
  int64_t x_bs, x_ts, ag_bs, ag_ts, xg_bs, xg_ts, dy_bs, dy_ts, dx_bs, dx_ts, dag_bs, dag_ts, dxg_bs, dxg_ts;
  int64_t L;
  int32_t nd, n_cg, n_states;
};

// 1 - a^2 for a = 2^-s2.  Near s2 = 0, where the difference would cancel, s2 times a
// polynomial: the one of degree 4 nearest to (1 - 2^-2x) / x on [0, 0.36] by its
// largest relative error (1.44 U with these coefficients, U = 2^-24; found by
// exchange of its extrema).  From there on, 1 - a^2 >= 0.39, the difference loses
// at most 1.5 times a^2's own rounding.
__device__ __forceinline__ float one_minus_square(float a, float s2) {
  float p = __builtin_fmaf(s2, 0.0346816927f, -0.151441112f);
  p = __builtin_fmaf(s2, p, 0.443718821f);
  p = __builtin_fmaf(s2, p, -0.960891724f);
  p = __builtin_fmaf(s2, p, 1.38629425f) * s2;
  return s2 < 0.36f ? p : __builtin_fmaf(-a, a, 1.0f);
}

// A gate's sigmoid.  sigmoid_exact cuts its argument, and a NaN there comes out as
// a bound; a gate that is no number has to show in the state.
template <typename IO>
__device__ __forceinline__ float gate_sigmoid(float v) {
  const float s = sigmoid_for<IO>(v);
  return sizeof(IO) == 2 || v == v ? s : v;
}

// A step's gates.  rate2 = exp(A_log) log2(e), so that a = 2^-s2 with s2 = s log2(e).
struct Gate {
  float r, i, s2, a, c;
};
template <typename IO>
__device__ __forceinline__ Gate gate_of(float ag, float xg, float rate2) {
  Gate g;
  g.r = gate_sigmoid<IO>(ag);
  g.i = gate_sigmoid<IO>(xg);
  g.s2 = rate2 * g.r;
  g.a = fast_exp2(-g.s2);
  g.c = __builtin_amdgcn_sqrtf(one_minus_square(g.a, g.s2));
  return g;
}

// A channel's rate2.  Finite, so that it times r = 0, or s2 times a = 0, is no NaN.
__device__ __forceinline__ float rate2_of(float a_log) {
  const float r = expf(a_log) * kLog2e;
  return r > 0x1p127f ? 0x1p127f : r;
}

// What the backward takes of a step besides a and u: with g the state's gradient, h the
// state in front and rate = exp(A_log),
//     dx = g kx,  dx_gate = g u ki,  q = rate g (k1 - r a h),  da_gate = q (1 - r)
// k1 = r a^2 i x / c, and 0 where c is.
struct Back {
  float a, u, kx, ki, k1, r;
};
template <typename IO>
__device__ __forceinline__ Back back_of(float x, float ag, float xg, float rate2) {
  Back b;
  const float r = gate_sigmoid<IO>(ag), i = gate_sigmoid<IO>(xg), s2 = rate2 * r;
  b.a = fast_exp2(-s2);
  const float c2 = one_minus_square(b.a, s2);
  // the forward's square root takes a subnormal c2 as 0
  const float rc = c2 < 0x1p-126f ? 0.0f : __builtin_amdgcn_rsqf(c2), c = c2 * rc, ix = i * x;
  b.u = c * ix;
  b.kx = c * i;
  b.ki = 1.0f - i;
  b.k1 = r * b.a * b.a * (rc * ix);
  b.r = r;
  return b;
}

// A row's valid length, the same row for the whole wave: by a scalar load, which does
// not wait for the vector loads and stores in flight.
__device__ __forceinline__ int32_t length_of(const int32_t* valid_len, int32_t b, int64_t L) {
  if (valid_len == nullptr) return static_cast<int32_t>(L);
  typedef const __attribute__((address_space(4))) int32_t* scalar;
  const int32_t n = ((scalar)(uintptr_t)valid_len)[__builtin_amdgcn_readfirstlane(b)];
  return n < 0 ? 0 : (n > L ? static_cast<int32_t>(L) : n);
}

// V elements at a lane's byte offset from an address that is the same for the wave.
template <typename IO>
__device__ __forceinline__ const IO* lane_at(const IO* p, uint32_t off) {
  return reinterpret_cast<const IO*>(reinterpret_cast<const char*>(p) + off);
}
template <typename IO>
__device__ __forceinline__ IO* lane_at(IO* p, uint32_t off) {
  return reinterpret_cast<IO*>(reinterpret_cast<char*>(p) + off);
}

__device__ __forceinline__ int wave_index() { return __builtin_amdgcn_readfirstlane(threadIdx.x / 64); }

// V channels of a wave's steps of one tensor, loaded one step after another.  Unless
// all of them are steps of the row (FULL), those past the last one read it again
// (their values are not used).  ONCE: past the caches, where pieces are whole lines.
template <typename IO, int V, bool FULL, bool ONCE>
struct Feed {
  const IO* p;  // the same for the wave, where all its lanes take the same steps
  int64_t ts;
  int32_t left;
  __device__ __forceinline__ Feed(const void* base, int64_t bs, int64_t step, int32_t b, int32_t t0, int32_t last)
      : p(static_cast<const IO*>(base) + b * bs + (FULL || t0 < last ? t0 : last) * step), ts(step), left(last - t0) {}
  __device__ __forceinline__ RawVec<IO, V> next(int t, int32_t d) {
    RawVec<IO, V> raw;
    const IO* at = lane_at(p, static_cast<uint32_t>(d) * static_cast<uint32_t>(sizeof(IO)));
    if constexpr (ONCE)
      raw.load_once(at);
    else
      raw.load(at);
    p += FULL || t < left ? ts : 0;
    return raw;
  }
};

// A wave's steps of both gates and x.  Loads come back in order: what the first step
// takes is asked for first.
template <bool FULL, bool ONCE, typename IO, int V, int T, typename P>
__device__ __forceinline__ void load_steps(const P& prm, int32_t b, int32_t t0, int32_t last, int32_t d,
                                           RawVec<IO, V> (&ra)[T], RawVec<IO, V> (&rg)[T], RawVec<IO, V> (&rx)[T]) {
  Feed<IO, V, FULL, ONCE> fa(prm.ag, prm.ag_bs, prm.ag_ts, b, t0, last), fg(prm.xg, prm.xg_bs, prm.xg_ts, b, t0, last),
      fx(prm.x, prm.x_bs, prm.x_ts, b, t0, last);
#pragma unroll
  for (int t = 0; t < T; ++t) ra[t] = fa.next(t, d), rg[t] = fg.next(t, d), rx[t] = fx.next(t, d);
}

// A kernel's parameters, read again where they are used: held in scalar registers
// from turn to turn, some fifty pointers and strides were spilled to vector ones.
// The parameters are the kernel's first argument.
template <typename P>
__device__ __forceinline__ const __attribute__((address_space(4))) P& params_again() {
  auto p = (const __attribute__((address_space(4))) P*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *p;
}

// ---- rows cut into tiles ----------------------------------------------------
//
// Where (row, channel) work alone does not fill the GPU, tiles of T W steps of one
// chain (a row's 64 V channels) run on different workgroups.  A tile folds its
// steps into one pair per channel, needs the state in front of it, and leaves the
// one behind.  kSpan tiles make a span.  The state goes from span to span, from
// the last tile of one to all of the next; within a span every tile publishes its
// pair as soon as its inputs have come, and composes those of the tiles in front
// of it, in order, behind the span's state.  What a tile computes does not depend
// on when the others come, so results are the same bits from run to run, and only
// every kSpan-th tile is a step of the serial chain.
//
// Tiles are dealt by a counter, in runs of one or more, all chains' first tiles first: a
// tile waits only for tiles with smaller numbers, a workgroup takes its own in order, so
// the smallest unfinished one is always at work and never waits for one that is not:
// every wait ends.
//
// Published words tell by themselves that they are there: a fill kernel sets all
// to kEmpty, a NaN that is never published (it is replaced by another), and words
// are stored and read whole, relaxed, at agent scope.

constexpr int kSpan = 16;
constexpr uint32_t kEmpty = 0xffffffffu;
// Far more polls than any wait takes: should one end here all the same, the
// states that hang on it become NaN.
constexpr int kPolls = 1 << 21;

template <int V>
struct Words;
template <>
struct Words<1> {
  typedef uint32_t type;
};
template <>
struct Words<2> {
  typedef unsigned long long type;
};

template <int V>
__device__ __forceinline__ void publish(float* at, const float (&v)[V]) {
  typedef typename Words<V>::type W;
  W w = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v[i]);
    w |= static_cast<W>(u == kEmpty ? 0x7fc00000u : u) << (i * 32 % (8 * sizeof(W)));
  }
  __hip_atomic_store(reinterpret_cast<W*>(at), w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// K published vectors, once all of them are there.
template <int V, int K>
__device__ __forceinline__ void await(const float* const (&at)[K], float (&v)[K][V]) {
  typedef typename Words<V>::type W;
  for (int polls = 0;; ++polls) {
    bool there = true;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const W w = __hip_atomic_load(reinterpret_cast<const W*>(at[k]), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint32_t u = static_cast<uint32_t>(w >> (i * 32 % (8 * sizeof(W))));
        there = there && u != kEmpty;
        v[k][i] = __builtin_bit_cast(float, u);
      }
    }
    if (__all(there) || polls == kPolls) return;  // kEmpty itself is a NaN
    __builtin_amdgcn_s_sleep(1);
  }
}

// A product of decays that underflowed would make NaN of an infinite state.
__device__ __forceinline__ float above_zero(float p) { return __builtin_fmaxf(p, 0x1p-149f); }

// The chains' workspace: a counter, then the tiles' pairs and the spans' states.
struct ChainSpace {
  uint32_t* counter;
  float* pairs;   // [tile][chain][P, S][64 V]
  float* states;  // [span][chain][64 V]
  uint32_t chains;
  uint32_t run;  // the logarithm of the tickets drawn at once
  __device__ __forceinline__ bool last_of_run(uint32_t ticket) const { return (ticket + 1) >> run << run == ticket + 1; }
  __device__ __forceinline__ uint32_t draw() const { return atomicAdd(counter, 1u) << run; }
  template <int V>
  __device__ __forceinline__ float* pair(uint32_t pos, uint32_t chain) const {
    return pairs + ((static_cast<int64_t>(pos) * chains + chain) * 2 * 64 + threadIdx.x % 64) * V;
  }
  template <int V>
  __device__ __forceinline__ float* state(uint32_t span, uint32_t chain) const {
    return states + ((static_cast<int64_t>(span) * chains + chain) * 64 + threadIdx.x % 64) * V;
  }
};

// LDS of the waves of a tile, and of the tiles in front of it.
template <int V, int W>
struct ChainLds {
  float waves[2][W][2 * V][64];
  float front[kSpan][2 * V][64];
  float state[V][64];
  uint32_t ticket;
};

// Joining a tile to its chain, in two halves, each with a barrier.  The first takes
// every wave's pair (P, S) and publishes the tile's; it is called with the chain's
// initial state in `h` for its first tile, which takes it into its pair, and zero
// for the others.  The second waits for the pairs in front and the span's state, and
// leaves in `h` the state in front of the wave's steps and, in the wave of the tile's
// last ones, in `out` the one behind the tile.  pos: the tile's place in its chain; more: whether another follows.  The
// workgroup's next ticket is drawn here, where all wait anyway.
template <int V, int W, bool REVERSE>
__device__ __forceinline__ void join_begin(ChainLds<V, W>& lds, const ChainSpace& sp, int buf, int wave, uint32_t pos,
                                           uint32_t chain, bool more, const float (&P)[V], const float (&S)[V],
                                           float (&h)[V]) {
  const int lane = threadIdx.x % 64;
  auto& mine = lds.waves[buf];
#pragma unroll
  for (int v = 0; v < V; ++v) asm volatile("" : "+v"(h[v]));  // the initial state has come before one is written
#pragma unroll
  for (int v = 0; v < V; ++v) mine[wave][v][lane] = above_zero(P[v]), mine[wave][V + v][lane] = S[v];
  __syncthreads();
  __builtin_amdgcn_s_setprio(3);  // others wait for what this workgroup publishes
  if (wave == W - 1 && more && pos % kSpan != kSpan - 1) {
    float p[V], s[V];
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = 1.0f, s[v] = h[v];
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const int w = REVERSE ? W - 1 - k : k;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float a = mine[w][v][lane];
        s[v] = __builtin_fmaf(a, s[v], mine[w][V + v][lane]);
        p[v] *= a;
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = above_zero(p[v]);
    float* at = sp.pair<V>(pos, chain);
    publish<V>(at, p);
    publish<V>(at + 64 * V, s);
  }
}

template <int V, int W, bool REVERSE>
__device__ __forceinline__ void join_end(ChainLds<V, W>& lds, const ChainSpace& sp, int buf, int wave, uint32_t pos,
                                         uint32_t chain, bool more, float (&h)[V], float (&out)[V], uint32_t& ticket) {
  const int lane = threadIdx.x % 64;
  auto& mine = lds.waves[buf];
  const uint32_t span = pos / kSpan;
  const int before = static_cast<int>(pos % kSpan);  // tiles of the span in front of this one
  const bool draw = sp.last_of_run(ticket);
  if (draw && threadIdx.x == 0) lds.ticket = sp.draw();
  for (int j = wave; j <= before; j += W) {
    if (j < before) {
      const float* at = sp.pair<V>(span * kSpan + j, chain);
      const float* const two[2] = {at, at + 64 * V};
      float v2[2][V];
      await<V, 2>(two, v2);
#pragma unroll
      for (int v = 0; v < V; ++v) lds.front[j][v][lane] = v2[0][v], lds.front[j][V + v][lane] = v2[1][v];
    } else if (span > 0) {
      const float* const one[1] = {sp.state<V>(span, chain)};
      float v1[1][V];
      await<V, 1>(one, v1);
#pragma unroll
      for (int v = 0; v < V; ++v) lds.state[v][lane] = v1[0][v];
    }
  }
  __syncthreads();
  ticket = draw ? __builtin_amdgcn_readfirstlane(lds.ticket) : ticket + 1;
  if (span > 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = lds.state[v][lane];
  }
  for (int j = 0; j < before; ++j) {
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = __builtin_fmaf(lds.front[j][v][lane], h[v], lds.front[j][V + v][lane]);
  }
  // through the waves in front, four pairs read at a time
  const int mine_at = REVERSE ? W - 1 - wave : wave;
#pragma unroll
  for (int k0 = 0; k0 < W; k0 += 4) {
    if (k0 >= mine_at) break;
    float a[4][V], u[4][V];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int w = REVERSE ? W - 1 - (k0 + k) : k0 + k;
#pragma unroll
      for (int v = 0; v < V; ++v) a[k][v] = mine[w][v][lane], u[k][v] = mine[w][V + v][lane];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k0 + k < mine_at) {
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = __builtin_fmaf(a[k][v], h[v], u[k][v]);
      }
    }
  }
  if (mine_at == W - 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) out[v] = __builtin_fmaf(mine[wave][v][lane], h[v], mine[wave][V + v][lane]);
    if (more && before == kSpan - 1) publish<V>(sp.state<V>(span + 1, chain), out);
  }
  __builtin_amdgcn_s_setprio(0);
}

// Zeros in the 64 V channels (`left` are there) of some rows, 16 bytes a lane, by
// WAVES waves from the second on.
template <typename IO, int V, int WAVES>
__device__ __forceinline__ void zero_rows(IO* p, int64_t ts, int64_t rows, int64_t left) {
  constexpr int K = VecIO<IO>::kWide, kPieces = 64 * V / K;
  for (int i = threadIdx.x - 64; i < rows * kPieces; i += 64 * WAVES) {
    const int c = i % kPieces * K;
    const float zero[K] = {};
    store_n<IO, K>(p + i / kPieces * ts + c, left - c < K ? static_cast<int>(left - c) : K, zero);
  }
}

__global__ void chain_fill_kernel(uint32_t* p, int64_t n) {
  typedef uint32_t vec4 __attribute__((ext_vector_type(4), aligned(8)));
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  // the first 16 bytes are the counter's
  if (i < n) *reinterpret_cast<vec4*>(p + i) = i == 0 ? vec4(0u) : vec4(kEmpty);
}

// ---- rows that one workgroup holds ----------------------------------------------
//
// Short rows: W waves of G groups of 64 / G lanes, each lane V channels and T steps, and
// G W T steps hold the row.  With G = 1 rows are read 128 or 256 bytes at a time; with
// G = 4 a few long rows are spread over four times as many workgroups, which are then
// done sooner.

// The pairs of the groups, and the states in front of them.
template <int V, int G, int W>
struct RowLds {
  float pair[G * W][64 / G][2 * V];
  float front[G * W][64 / G][V];
};

// From the pairs, in the order of the steps (REVERSE: from the last), to the states;
// `h`, the state in front of all, becomes the one behind.  By one wave, each row of
// 64 / G lanes W groups; all rows hold h.
template <int V, int G, int W, bool REVERSE>
__device__ __forceinline__ void scan_groups(RowLds<V, G, W>& lds, float (&h)[V]) {
  static_assert(G == 1 || G == 4, "the whole wave, or rows of 16 lanes");
  const int lane = threadIdx.x % 64, sub = lane / (64 / G), cl = lane % (64 / G);
  const auto at = [&](int k) { return REVERSE ? G * W - 1 - (sub * W + k) : sub * W + k; };
  if constexpr (G == 4) {
    float P[V], S[V];
#pragma unroll
    for (int v = 0; v < V; ++v) P[v] = 1.0f, S[v] = 0.0f;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const float* g = lds.pair[at(k)][cl];
#pragma unroll
      for (int v = 0; v < V; ++v) S[v] = __builtin_fmaf(g[v], S[v], g[V + v]), P[v] *= g[v];
    }
    // rows 0, 1 and rows 2, 3 join, then the halves: what is in front of a row
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float p0, p1, s0, s1, ph, sh, back;
      rows_swap16(above_zero(P[v]), p0, p1);
      rows_swap16(S[v], s0, s1);
      rows_swap32(above_zero(p0 * p1), ph, back);
      rows_swap32(__builtin_fmaf(p1, s0, s1), sh, back);
      if (sub >= 2) h[v] = __builtin_fmaf(ph, h[v], sh);
      if (sub % 2 == 1) h[v] = __builtin_fmaf(p0, h[v], s0);
    }
  }
#pragma unroll
  for (int k = 0; k < W; ++k) {
    const float* g = lds.pair[at(k)][cl];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      lds.front[at(k)][cl][v] = h[v];
      h[v] = __builtin_fmaf(g[v], h[v], g[V + v]);
    }
  }
  if constexpr (G == 4) {  // the last row's to all
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float lo, hi;
      rows_swap32(h[v], lo, hi);
      rows_swap16(hi, lo, h[v]);
    }
  }
}

// Where a lane works.  Lanes past the last channel repeat the last V of the row
// (which a lane whose V would reach past it takes too: both compute and write the
// same).
struct RowAt {
  int32_t b, d, q, t0;
  bool mine;
};
template <int V, int G, int T>
__device__ __forceinline__ RowAt row_place(int32_t nd, int32_t n_cg) {
  constexpr int LPG = 64 / G;
  RowAt at;
  const int lane = threadIdx.x % 64;
  at.b = blockIdx.x / n_cg;
  const int32_t first = (static_cast<int32_t>(blockIdx.x % n_cg) * LPG + lane % LPG) * V;
  at.d = first < nd - V ? first : nd - V;
  at.mine = first < nd;
  at.q = wave_index() * G + (G == 1 ? 0 : lane / LPG);
  at.t0 = at.q * T;
  return at;
}

template <typename IO, int V, int G, int T, int W>
__global__ __launch_bounds__(64 * W) void gated_fwd_row_kernel(const GatedParams prm) {
  __shared__ RowLds<V, G, W> lds;
  static_assert(kChunk % T == 0, "chunks are whole groups of steps");
  const RowAt at = row_place<V, G, T>(prm.nd, prm.n_cg);
  const int cl = threadIdx.x % (64 / G);
  const int32_t n = length_of(prm.valid_len, at.b, prm.L), d = at.d, t0 = at.t0;
  const int64_t bd = static_cast<int64_t>(at.b) * prm.nd + d;
  float al[V], rate2[V], a[T][V], u[T][V], P[V], S[V], h[V] = {};
  VecIO<float>::load(prm.A_log + d, al);
  if (wave_index() == 0 && prm.h0 != nullptr) VecIO<float>::load(prm.h0 + bd, h);
  RawVec<IO, V> ra[T], rg[T], rx[T];
  if (n > 0) load_steps<false, false>(prm, at.b, t0, n - 1, d, ra, rg, rx);
#pragma unroll
  for (int v = 0; v < V; ++v) rate2[v] = rate2_of(al[v]), P[v] = 1.0f, S[v] = 0.0f;
#pragma unroll
  for (int t = 0; t < T; ++t) {
    float xv[V], av[V], gv[V];
    rx[t].unpack(xv);
    ra[t].unpack(av);
    rg[t].unpack(gv);
    const bool valid = t0 + t < n;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const Gate g = gate_of<IO>(av[v], gv[v], rate2[v]);
      a[t][v] = valid ? g.a : 1.0f;
      u[t][v] = valid ? g.c * g.i * xv[v] : 0.0f;
      P[v] *= a[t][v];
      S[v] = __builtin_fmaf(a[t][v], S[v], u[t][v]);
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) lds.pair[at.q][cl][v] = above_zero(P[v]), lds.pair[at.q][cl][V + v] = S[v];
  __syncthreads();
  if (wave_index() == 0) {
    scan_groups<V, G, W, false>(lds, h);
    if (at.mine && threadIdx.x < 64 / G) {
      if (prm.h_last != nullptr) VecIO<float>::store(prm.h_last + bd, h);
      // chunks that end behind the last group
      if (prm.states != nullptr)
        for (int32_t c = G * W * T / kChunk; c < prm.n_states; ++c)
          VecIO<float>::store(prm.states + (static_cast<int64_t>(at.b) * prm.n_states + c) * prm.nd + d, h);
    }
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = lds.front[at.q][cl][v];
  if (!at.mine) return;
  const IO* out = static_cast<IO*>(prm.y) + at.b * prm.y_bs + t0 * prm.y_ts;
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const bool valid = t0 + t < n;
    float o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      h[v] = __builtin_fmaf(a[t][v], h[v], u[t][v]);
      o[v] = valid ? h[v] : 0.0f;
    }
    if (t0 + t < prm.L)
      VecIO<IO>::store(const_cast<IO*>(lane_at(out, static_cast<uint32_t>(d) * static_cast<uint32_t>(sizeof(IO)))), o);
    out += prm.y_ts;
  }
  if (prm.states != nullptr && (t0 + T) % kChunk == 0 && (t0 + T) / kChunk <= prm.n_states)
    VecIO<float>::store(prm.states + (static_cast<int64_t>(at.b) * prm.n_states + (t0 + T) / kChunk - 1) * prm.nd + d, h);
}

// The same with the row's tiles on different workgroups.
template <typename IO, int V, int T, int W, bool ONCE>
__global__ __launch_bounds__(64 * W, 4) void gated_fwd_chain_kernel(const GatedParams, const ChainSpace sp,
                                                                 uint32_t tickets) {
  __shared__ ChainLds<V, W> lds;
  const int wave = wave_index(), lane = threadIdx.x % 64;
  if (threadIdx.x == 0) lds.ticket = sp.draw();
  __syncthreads();
  uint32_t ticket = __builtin_amdgcn_readfirstlane(lds.ticket);
  __syncthreads();
  for (int buf = 0; ticket < tickets;) {
    const auto& prm = params_again<GatedParams>();
    const uint32_t pos = ticket / sp.chains, chain = ticket - pos * sp.chains;
    const int32_t b = chain / prm.n_cg, cg = chain % prm.n_cg, tile = pos * (T * W), t0 = tile + wave * T;
    const int32_t first = (cg * 64 + lane) * V, d = first < prm.nd - V ? first : prm.nd - V;
    const bool mine = first < prm.nd;
    const int32_t n = length_of(prm.valid_len, b, prm.L);
    const int64_t bd = static_cast<int64_t>(b) * prm.nd + d;
    float h[V] = {}, out[V];
    if (pos == 0 && prm.h0 != nullptr) VecIO<float>::load(prm.h0 + bd, h);
    const auto body = [&]<bool FULL>() __attribute__((always_inline)) {
      float al[V], rate2[V], a[T][V], u[T][V], P[V], S[V];
      RawVec<IO, V> ra[T], rg[T], rx[T];
      VecIO<float>::load(prm.A_log + d, al);
      load_steps<FULL, ONCE>(prm, b, t0, n - 1, d, ra, rg, rx);
#pragma unroll
      for (int v = 0; v < V; ++v) rate2[v] = rate2_of(al[v]), P[v] = 1.0f, S[v] = 0.0f;
#pragma unroll
      for (int t = 0; t < T; ++t) {
        float xv[V], av[V], gv[V];
        rx[t].unpack(xv);
        ra[t].unpack(av);
        rg[t].unpack(gv);
        const bool valid = FULL || t0 + t < n;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const Gate g = gate_of<IO>(av[v], gv[v], rate2[v]);
          a[t][v] = valid ? g.a : 1.0f;
          u[t][v] = valid ? g.c * g.i * xv[v] : 0.0f;
          P[v] *= a[t][v];
          S[v] = __builtin_fmaf(a[t][v], S[v], u[t][v]);
        }
      }
      join_begin<V, W, false>(lds, sp, buf, wave, pos, chain, tile + T * W < n, P, S, h);
      join_end<V, W, false>(lds, sp, buf, wave, pos, chain, tile + T * W < n, h, out, ticket);
      buf ^= 1;
      const auto& prm = params_again<GatedParams>();
      if (!mine) return;
      // a new value, zero-extended here: stores at scalar addresses
      uint32_t off = static_cast<uint32_t>(d) * static_cast<uint32_t>(sizeof(IO));
      asm volatile("" : "+v"(off));
      IO* y = static_cast<IO*>(prm.y) + b * prm.y_bs + t0 * prm.y_ts;
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const bool valid = FULL || t0 + t < n;
        float o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          h[v] = __builtin_fmaf(a[t][v], h[v], u[t][v]);
          o[v] = valid ? h[v] : 0.0f;
        }
        if (FULL || t0 + t < prm.L) VecIO<IO>::store(lane_at(y, off), o);
        y += prm.y_ts;
      }
      if (prm.states != nullptr && (t0 + T) % kChunk == 0 && (t0 + T) / kChunk <= prm.n_states)
        VecIO<float>::store(prm.states + (static_cast<int64_t>(b) * prm.n_states + (t0 + T) / kChunk - 1) * prm.nd + d, h);
    };
    if (tile + T * W <= n) {
      body.template operator()<true>();
    } else if (tile < n) {
      body.template operator()<false>();
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) out[v] = h[v];
      const int64_t at = static_cast<int64_t>(cg) * (64 * V);
      __syncthreads();  // this turn's ticket has been read
      const bool draw = sp.last_of_run(ticket);
      if (draw && threadIdx.x == 0) lds.ticket = sp.draw();
      if (wave > 0)  // the first one would wait for its stores before it knows the ticket
        zero_rows<IO, V, W - 1>(static_cast<IO*>(prm.y) + b * prm.y_bs + tile * prm.y_ts + at, prm.y_ts,
                                prm.L - tile < T * W ? prm.L - tile : T * W, prm.nd - at);
      __syncthreads();
      ticket = draw ? __builtin_amdgcn_readfirstlane(lds.ticket) : ticket + 1;
    }
    const auto& end = params_again<GatedParams>();
    // the row's last tile (its first where it has no step) leaves the state
    if (wave == W - 1 && mine && (tile < n ? tile + T * W >= n : tile == 0)) {
      if (end.h_last != nullptr) VecIO<float>::store(end.h_last + bd, out);
      if (end.states != nullptr) {
        for (int32_t c = tile < n ? (tile + T * W) / kChunk : 0; c < end.n_states; ++c)
          VecIO<float>::store(end.states + (static_cast<int64_t>(b) * end.n_states + c) * end.nd + d, out);
      }
    }
  }
}

// The same from the row's end; the states come again from the row's first.
template <typename IO, int V, int G, int T, int W>
__global__ __launch_bounds__(64 * W) void gated_bwd_row_kernel(const GatedBwdParams prm) {
  __shared__ RowLds<V, G, W> lds, back;
  const RowAt at = row_place<V, G, T>(prm.nd, prm.n_cg);
  const int cl = threadIdx.x % (64 / G), wave = wave_index();
  const int32_t n = length_of(prm.valid_len, at.b, prm.L), d = at.d, t0 = at.t0;
  const int64_t bd = static_cast<int64_t>(at.b) * prm.nd + d;
  float al[V], rate2[V], a[T][V], u[T][V], kx[T][V], ki[T][V], k1[T][V], r[T][V], P[V], S[V], h[V] = {}, g[V] = {};
  VecIO<float>::load(prm.A_log + d, al);
  if (wave == 0 && prm.h0 != nullptr) VecIO<float>::load(prm.h0 + bd, h);
  if (wave == W - 1 && prm.dh_last != nullptr) VecIO<float>::load(prm.dh_last + bd, g);
  RawVec<IO, V> ra[T], rg[T], rx[T], rd[T];
  if (n > 0) {
    load_steps<false, false>(prm, at.b, t0, n - 1, d, ra, rg, rx);
    Feed<IO, V, false, false> fd(prm.dy, prm.dy_bs, prm.dy_ts, at.b, t0, n - 1);
#pragma unroll
    for (int t = 0; t < T; ++t) rd[t] = fd.next(t, d);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) rate2[v] = rate2_of(al[v]), P[v] = 1.0f, S[v] = 0.0f;
#pragma unroll
  for (int t = 0; t < T; ++t) {
    float xv[V], av[V], gv[V];
    rx[t].unpack(xv);
    ra[t].unpack(av);
    rg[t].unpack(gv);
    const bool valid = t0 + t < n;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const Back q = back_of<IO>(xv[v], av[v], gv[v], rate2[v]);
      a[t][v] = valid ? q.a : 1.0f;
      u[t][v] = valid ? q.u : 0.0f;
      kx[t][v] = q.kx, ki[t][v] = q.ki, k1[t][v] = q.k1, r[t][v] = q.r;
      P[v] *= a[t][v];
      S[v] = __builtin_fmaf(a[t][v], S[v], u[t][v]);
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    lds.pair[at.q][cl][v] = back.pair[at.q][cl][v] = above_zero(P[v]);
    lds.pair[at.q][cl][V + v] = S[v], S[v] = 0.0f;
  }
  // what comes into a group from behind leaves it as a (dy + .) of its first step
#pragma unroll
  for (int t = T - 1; t >= 0; --t) {
    float dv[V];
    rd[t].unpack(dv);
    const bool valid = t0 + t < n;
#pragma unroll
    for (int v = 0; v < V; ++v) S[v] = a[t][v] * (S[v] + (valid ? dv[v] : 0.0f));
  }
#pragma unroll
  for (int v = 0; v < V; ++v) back.pair[at.q][cl][V + v] = S[v];
  __syncthreads();
  if (wave == 0) scan_groups<V, G, W, false>(lds, h);
  if (wave == W - 1) {
    scan_groups<V, G, W, true>(back, g);
    if (at.mine && threadIdx.x % 64 < 64 / G && prm.dh0 != nullptr) VecIO<float>::store(prm.dh0 + bd, g);
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = lds.front[at.q][cl][v], g[v] = back.front[at.q][cl][v];
  // k1 becomes k1 - r a h
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      k1[t][v] = __builtin_fmaf(-(r[t][v] * a[t][v]), h[v], k1[t][v]);
      h[v] = __builtin_fmaf(a[t][v], h[v], u[t][v]);
    }
  float dA[V] = {}, rate[V];
#pragma unroll
  for (int v = 0; v < V; ++v) rate[v] = rate2[v] * kLn2;
  const uint32_t off = static_cast<uint32_t>(d) * static_cast<uint32_t>(sizeof(IO));
  IO* px = static_cast<IO*>(prm.dx) + at.b * prm.dx_bs + (t0 + T - 1) * prm.dx_ts;
  IO* pa = static_cast<IO*>(prm.dag) + at.b * prm.dag_bs + (t0 + T - 1) * prm.dag_ts;
  IO* pg = static_cast<IO*>(prm.dxg) + at.b * prm.dxg_bs + (t0 + T - 1) * prm.dxg_ts;
#pragma unroll
  for (int t = T - 1; t >= 0; --t) {
    float dv[V], ox[V], oa[V], og[V];
    rd[t].unpack(dv);
    const bool valid = t0 + t < n;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float gt = g[v] + dv[v], q = gt * k1[t][v];
      ox[v] = valid ? gt * kx[t][v] : 0.0f;
      og[v] = valid ? gt * u[t][v] * ki[t][v] : 0.0f;
      oa[v] = valid ? q * __builtin_fmaf(-rate[v], r[t][v], rate[v]) : 0.0f;
      dA[v] += valid ? q : 0.0f;
      g[v] = valid ? gt * a[t][v] : g[v];
    }
    if (at.mine && t0 + t < prm.L) {
      VecIO<IO>::store(lane_at(px, off), ox);
      VecIO<IO>::store(lane_at(pa, off), oa);
      VecIO<IO>::store(lane_at(pg, off), og);
    }
    px -= prm.dx_ts, pa -= prm.dag_ts, pg -= prm.dxg_ts;
  }
  // the groups' sums of q, in order (every group has read its states by now, from
  // places of its own)
#pragma unroll
  for (int v = 0; v < V; ++v) lds.front[at.q][cl][v] = dA[v] * rate[v];
  __syncthreads();
  if (at.mine && threadIdx.x < 64 / G) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      dA[v] = 0.0f;
      for (int q = 0; q < G * W; ++q) dA[v] += lds.front[q][cl][v];
    }
    VecIO<float>::store(prm.ws + bd, dA);
  }
}

// The same with the row's tiles on different workgroups, the last ones first.  What
// a step needs of the forward pass comes from its own tile alone; the chain carries
// the state's gradient.  A wave's product of decays is one for both directions.
template <typename IO, int V, int T, int W, bool ONCE>
__global__ __launch_bounds__(64 * W, 4) void gated_bwd_chain_kernel(const GatedBwdParams, const ChainSpace sp,
                                                                 uint32_t tickets, uint32_t tiles) {
  static_assert(T * W % kChunk == 0, "a tile begins behind a kept state");
  __shared__ ChainLds<V, W> lds;
  __shared__ float sums[2][W][V][64], dsum[2][W][V][64];
  const int wave = wave_index(), lane = threadIdx.x % 64;
  // A tile's sums of q, one a wave, wait for the next barrier; then the last wave
  // adds them in order.
  float* sum_to = nullptr;
  int sum_buf = 0;
  const auto flush = [&]() __attribute__((always_inline)) {
    if (wave == W - 1 && sum_to != nullptr) {
      float t[V] = {};
#pragma unroll
      for (int w = 0; w < W; ++w)
#pragma unroll
        for (int v = 0; v < V; ++v) t[v] += dsum[sum_buf][w][v][lane];
      VecIO<float>::store(sum_to, t);
    }
  };
  if (threadIdx.x == 0) lds.ticket = sp.draw();
  __syncthreads();
  uint32_t ticket = __builtin_amdgcn_readfirstlane(lds.ticket);
  __syncthreads();
  for (int buf = 0; ticket < tickets;) {
    const auto& prm = params_again<GatedBwdParams>();
    const uint32_t turn = ticket / sp.chains, chain = ticket - turn * sp.chains, k = tiles - 1 - turn;
    const int32_t b = chain / prm.n_cg, cg = chain % prm.n_cg, tile = k * (T * W), t0 = tile + wave * T;
    const int32_t first = (cg * 64 + lane) * V, d = first < prm.nd - V ? first : prm.nd - V;
    const bool mine = first < prm.nd;
    const int32_t n = length_of(prm.valid_len, b, prm.L);
    const int64_t bd = static_cast<int64_t>(b) * prm.nd + d;
    const uint32_t pos = (n + T * W - 1) / (T * W) - 1 - k;  // from the row's last tile with a step
    float g[V] = {}, out[V], dA[V] = {};
    if ((tile < n ? pos == 0 : k == 0) && prm.dh_last != nullptr) VecIO<float>::load(prm.dh_last + bd, g);
    const auto body = [&]<bool FULL>() __attribute__((always_inline)) {
      float al[V], rate2[V], a[T][V], u[T][V], kx[T][V], ki[T][V], k1[T][V], r[T][V], P[V], S[V], h[V] = {};
      RawVec<IO, V> ra[T], rg[T], rx[T], rd[T];
      VecIO<float>::load(prm.A_log + d, al);
      load_steps<FULL, ONCE>(prm, b, t0, n - 1, d, ra, rg, rx);
      Feed<IO, V, FULL, ONCE> fd(prm.dy, prm.dy_bs, prm.dy_ts, b, t0, n - 1);
#pragma unroll
      for (int t = 0; t < T; ++t) rd[t] = fd.next(t, d);
      if (tile > 0)
        VecIO<float>::load(prm.states + (static_cast<int64_t>(b) * prm.n_states + tile / kChunk - 1) * prm.nd + d, h);
      else if (prm.h0 != nullptr)
        VecIO<float>::load(prm.h0 + bd, h);
#pragma unroll
      for (int v = 0; v < V; ++v) rate2[v] = rate2_of(al[v]), P[v] = 1.0f, S[v] = 0.0f;
#pragma unroll
      for (int t = 0; t < T; ++t) {
        float xv[V], av[V], gv[V];
        rx[t].unpack(xv);
        ra[t].unpack(av);
        rg[t].unpack(gv);
        const bool valid = FULL || t0 + t < n;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const Back q = back_of<IO>(xv[v], av[v], gv[v], rate2[v]);
          a[t][v] = valid ? q.a : 1.0f;
          u[t][v] = valid ? q.u : 0.0f;
          kx[t][v] = q.kx, ki[t][v] = q.ki, k1[t][v] = q.k1, r[t][v] = q.r;
          P[v] *= a[t][v];
          S[v] = __builtin_fmaf(a[t][v], S[v], u[t][v]);
        }

      }
#pragma unroll
      for (int v = 0; v < V; ++v) sums[buf][wave][v][lane] = S[v], S[v] = 0.0f;
      // what comes into a wave from behind leaves it as a (dy + .) of its first step
#pragma unroll
      for (int t = T - 1; t >= 0; --t) {
        float dv[V];
        rd[t].unpack(dv);
        const bool valid = FULL || t0 + t < n;
#pragma unroll
        for (int v = 0; v < V; ++v) S[v] = a[t][v] * (S[v] + (valid ? dv[v] : 0.0f));
      }
      join_begin<V, W, true>(lds, sp, buf, wave, pos, chain, k > 0, P, S, g);
      flush();
      for (int w = 0; w < wave; ++w) {
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = __builtin_fmaf(lds.waves[buf][w][v][lane], h[v], sums[buf][w][v][lane]);
      }
      // k1 becomes k1 - r a h
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          k1[t][v] = __builtin_fmaf(-(r[t][v] * a[t][v]), h[v], k1[t][v]);
          h[v] = __builtin_fmaf(a[t][v], h[v], u[t][v]);
        }
      join_end<V, W, true>(lds, sp, buf, wave, pos, chain, k > 0, g, out, ticket);
      buf ^= 1;
      const auto& prm = params_again<GatedBwdParams>();
      if (!mine) return;
      // a new value, zero-extended here: stores at scalar addresses
      uint32_t off = static_cast<uint32_t>(d) * static_cast<uint32_t>(sizeof(IO));
      asm volatile("" : "+v"(off));
      IO* px = static_cast<IO*>(prm.dx) + b * prm.dx_bs + (t0 + T - 1) * prm.dx_ts;
      IO* pa = static_cast<IO*>(prm.dag) + b * prm.dag_bs + (t0 + T - 1) * prm.dag_ts;
      IO* pg = static_cast<IO*>(prm.dxg) + b * prm.dxg_bs + (t0 + T - 1) * prm.dxg_ts;
      float rate[V];
#pragma unroll
      for (int v = 0; v < V; ++v) rate[v] = rate2[v] * kLn2;
#pragma unroll
      for (int t = T - 1; t >= 0; --t) {
        float dv[V], ox[V], oa[V], og[V];
        rd[t].unpack(dv);
        const bool valid = FULL || t0 + t < n;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float gt = g[v] + dv[v], q = gt * k1[t][v];
          ox[v] = valid ? gt * kx[t][v] : 0.0f;
          og[v] = valid ? gt * u[t][v] * ki[t][v] : 0.0f;
          oa[v] = valid ? q * __builtin_fmaf(-rate[v], r[t][v], rate[v]) : 0.0f;
          dA[v] += valid ? q : 0.0f;
          g[v] = valid ? gt * a[t][v] : g[v];
        }
        if (FULL || t0 + t < prm.L) {
          VecIO<IO>::store(lane_at(px, off), ox);
          VecIO<IO>::store(lane_at(pa, off), oa);
          VecIO<IO>::store(lane_at(pg, off), og);
        }
        px -= prm.dx_ts, pa -= prm.dag_ts, pg -= prm.dxg_ts;
      }
#pragma unroll
      for (int v = 0; v < V; ++v) dA[v] *= rate[v];
    };
    if (tile + T * W <= n) {
      body.template operator()<true>();
    } else if (tile < n) {
      body.template operator()<false>();
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) out[v] = g[v];
      const int64_t at = static_cast<int64_t>(cg) * (64 * V), rows = prm.L - tile < T * W ? prm.L - tile : T * W;
      __syncthreads();  // this turn's ticket has been read
      flush();
      const bool draw = sp.last_of_run(ticket);
      if (draw && threadIdx.x == 0) lds.ticket = sp.draw();
      if (wave > 0) {  // the first one would wait for its stores before it knows the ticket
        zero_rows<IO, V, W - 1>(static_cast<IO*>(prm.dx) + b * prm.dx_bs + tile * prm.dx_ts + at, prm.dx_ts, rows,
                                prm.nd - at);
        zero_rows<IO, V, W - 1>(static_cast<IO*>(prm.dag) + b * prm.dag_bs + tile * prm.dag_ts + at, prm.dag_ts, rows,
                                prm.nd - at);
        zero_rows<IO, V, W - 1>(static_cast<IO*>(prm.dxg) + b * prm.dxg_bs + tile * prm.dxg_ts + at, prm.dxg_ts, rows,
                                prm.nd - at);
      }
      __syncthreads();
      ticket = draw ? __builtin_amdgcn_readfirstlane(lds.ticket) : ticket + 1;
    }
    const auto& end = params_again<GatedBwdParams>();
    if (wave == 0 && mine && k == 0 && end.dh0 != nullptr) VecIO<float>::store(end.dh0 + bd, out);
    sum_buf ^= 1;
    sum_to = mine ? end.ws + (static_cast<int64_t>(k) * (sp.chains / end.n_cg) + b) * end.nd + d : nullptr;
#pragma unroll
    for (int v = 0; v < V; ++v) dsum[sum_buf][wave][v][lane] = dA[v];
  }
  __syncthreads();
  flush();
}

struct GatedGrads {
  float* dA;
  __device__ __forceinline__ void operator()(int64_t col, float v) const { dA[col] = v; }
};

__global__ void gated_copy_kernel(const float* from, float* to, int64_t n) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) to[i] = from == nullptr ? 0.0f : from[i];
}

// ---- single tokens ---------------------------------------------------------

struct GatedStepParams {
  const void* x;
  const void* ag;
  const void* xg;
  const float* A_log;
  const int32_t* slots;
  const float* h0;
  float* h_last;
  void* y;
  int64_t x_rs, ag_rs, xg_rs, y_rs, n_slots;
  int32_t nb, nd;
};

// A lane takes V channels of one row: 16 bytes of states.
template <typename IO, int V>
__global__ __launch_bounds__(256) void gated_step_kernel(const GatedStepParams prm) {
  const int32_t b = blockIdx.y;
  const int64_t d = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * V;
  const int m = d >= prm.nd ? 0 : (prm.nd - d < V ? static_cast<int>(prm.nd - d) : V);
  const int32_t slot[1] = {prm.slots == nullptr ? b : prm.slots[b]};
  const int64_t at = static_cast<int64_t>(slot[0]) * prm.nd + d;
  float h[V] = {}, x[V] = {}, ag[V] = {}, xg[V] = {}, al[V];
  // a row that turns out idle is read all the same, inside its bounds
  const int k = slot[0] >= 0 && slot[0] < prm.n_slots ? m : 0;
  load_n<float, V>(prm.h0 + at, k, h);
  load_n<IO, V>(static_cast<const IO*>(prm.x) + b * prm.x_rs + d, k, x);
  load_n<IO, V>(static_cast<const IO*>(prm.ag) + b * prm.ag_rs + d, k, ag);
  load_n<IO, V>(static_cast<const IO*>(prm.xg) + b * prm.xg_rs + d, k, xg);
  load_n<float, V>(prm.A_log + d, m, al);
  bool active[1];
  step_rows_active<1>(prm.slots, b, prm.nb, slot, prm.n_slots, active);
  float o[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const Gate g = gate_of<IO>(ag[v], xg[v], rate2_of(al[v]));
    h[v] = __builtin_fmaf(g.a, h[v], g.c * g.i * x[v]);
    o[v] = active[0] ? h[v] : 0.0f;
  }
  if (active[0]) store_n<float, V>(prm.h_last + at, m, h);
  store_n<IO, V>(static_cast<IO*>(prm.y) + b * prm.y_rs + d, m, o);
}

// ---- host ------------------------------------------------------------------

constexpr int64_t kMaxGatedDim = 1 << 29;

int check_gated_dims(const ssm_gated_dims* dims) {
  if (dims == nullptr || dims->batch < 0 || dims->seqlen < 0 || dims->dim < 0) return SSM_ERR_INVALID_ARG;
  if (dims->io_dtype != SSM_IO_F32 && dims->io_dtype != SSM_IO_BF16) return SSM_ERR_INVALID_ARG;
  // a row's steps are counted in 32 bits, a tile's beyond its end among them
  if (dims->dim >= kMaxGatedDim || dims->batch > kMaxSize || dims->seqlen > kMaxSize - 65536) return SSM_ERR_UNSUPPORTED;
  if (static_cast<__int128>(dims->batch) * (dims->seqlen + 1) * dims->dim * 4 >= (static_cast<__int128>(1) << 62))
    return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

int64_t n_states(const ssm_gated_dims* dims) { return (dims->seqlen + kChunk - 1) / kChunk; }

// Steps of a lane, and the most channels of one.
constexpr int kFwdSteps = 16, kFwdWide = 2;
constexpr int kBwdSteps = 8, kBwdWide = 1;

// Whether every piece of 64 channels begins and ends with a line of 128 bytes.  Tiles
// read those past the caches (us, bf16 but for the last: 8 x 4096 x 1024 forward 66.2 for
// 67.5 and backward 128 for 134, 16 x 8192 x 512 ragged 81 for 86, 8 x 4096 x 512 f32 58
// for 62 and 97 for 110); a line that two pieces share is better kept (16 x 2048 x 1001:
// 71.5 and 166 for 75 and 184).
bool whole_lines(const Rows& r) {
  return aligned(r.p, 128) && (r.n1 == 1 || r.s1 * r.e % 128 == 0) && (r.n0 == 1 || r.s0 * r.e % 128 == 0);
}

// How a call is cut up, and the workspace that takes.
struct Cut {
  int64_t V, groups, chains, waves, tiles, tickets, run, words;
  bool shared;
};

// Up to kFew workgroups of 16 channels take whole short rows (us forward / backward:
// 1 x 512 x 64 7.2 / 9.1 where tiles of a chain take 11 / 15.9, 1 x 512 x 2048 9.0 / 13.1
// and 11.1 / 16.3; at 1024 of them, 8 x 512 x 2048, their 32-byte pieces cost 44 / 80
// where tiles take 23 / 44).  Up to 256 of them gain everywhere (2 x 512 x 2048: bf16 12.2
// / 20.0 for 13.5 / 23, f32 12.3 / 19.8 for 13.8 / 25); from there to kFew they gain and
// lose: 4 x 256 x 2048 bf16 12.0 / 20.0 for 9.0 / 22.3, f32 12.6 / 19.8 for 10.7 / 24.6; 3 x
// 512 x 2048 bf16 18.8 / 30.7 for 16.8 / 26.8, f32 17.4 / 31.0 for 18.5 / 31.7; 4 x 512 x
// 2048 bf16 22.3 / 35.2 for 19.8 / 29.8, f32 20.3 / 46.0 for 23.0 / 36.0.  Forward, half as
// many take rows of up to 1024 steps, 16 a lane (1 x 600 x 64 8.1 for 11.8, 4 x 1024 x
// 1024 f32 20.6 for 23.6; at 2 x 1024 x 2048 bf16 20.7 for 20.5; 504 of them, 8 x 1000 x
// 1000, 41 for 24.5).  Wider ones take rows of up to 16 waves' steps (256 x 129
// x 512 forward 45.3, tiles 54).  Two bf16 channels a lane read pieces of 256 bytes, 65 us
// for 78.5 at 8 x 4096 x 1024, but for kFill tiles of 128 x 128 and more; two of fp32
// cost more registers than they give (102 us at one, 107 at two).
// Tiles of 16 waves halve the chain's length where there are kMany of them at least (us
// at 16 / 8 waves, bf16: 8 x 4096 x 1024, 1024 of them, 65 / 68, 1 x 32768 x 2048, 2048,
// 108 / 132; but with 64 of them, 1 x 4096 x 256, 16.7 / 13.3; none measured between).
// Backward, their registers leave one workgroup a CU, which took 15 and 8 % longer.
constexpr int64_t kFew = 512, kFill = 512, kMany = 512;
Cut cut_of(const ssm_gated_dims* dims, int64_t steps, int64_t wide, int64_t most_waves) {
  Cut c;
  const int64_t nb = dims->batch, L = dims->seqlen, nd = dims->dim;
  c.tiles = 1, c.tickets = 0, c.run = 0, c.words = 0, c.waves = 1, c.shared = false;
  if (nb * ((nd + 15) / 16) <= (L <= 4 * 16 * 8 ? kFew : (L <= 4 * 16 * steps ? kFew / 2 : 0))) {
    c.groups = 4, c.V = 1, c.chains = nb * ((nd + 15) / 16);
    while (c.waves < 16 && 4 * 8 * c.waves < L) c.waves *= 2;
    return c;
  }
  c.groups = 1;
  // one channel a lane where two would leave half of a wave idle, or half of the GPU, or
  // make two workgroups share a channel
  const int64_t blocks = nb * ((nd + 127) / 128) * ((L + 127) / 128);
  c.V = dims->io_dtype == SSM_IO_F32 || nd <= 64 || nd % 128 == 1 || blocks < kFill ? 1 : wide;
  c.chains = nb * ((nd + 64 * c.V - 1) / (64 * c.V));
  if (L <= 16 * steps) {
    while (c.waves < 16 && steps * c.waves < L) c.waves *= 2;
    return c;
  }
  c.shared = true;
  for (c.waves = most_waves;; c.waves = 8) {
    c.tiles = (L + steps * c.waves - 1) / (steps * c.waves);
    c.tickets = c.tiles * c.chains;
    if (c.waves == 8 || c.tickets >= kMany) break;
  }
  c.words = 4 + 64 * c.V * c.chains * (2 * c.tiles + c.tiles / kSpan + 1);
  return c;
}
Cut fwd_cut(const ssm_gated_dims* dims) { return cut_of(dims, kFwdSteps, kFwdWide, 16); }
Cut bwd_cut(const ssm_gated_dims* dims) {
  Cut c = cut_of(dims, kBwdSteps, kBwdWide, 8);
  // One counter deals a run every 13 ns, whatever the tiles take: many are dealt in
  // pairs (us, bf16: 1 x 32768 x 2048 234 for 256, 16 x 8192 x 512 ragged 169 for 220; with
  // fewer, 8 x 4096 x 512 f32 97 for 96, 16 x 2048 x 1001 174 for 164).
  c.run = c.tickets > 8192 ? 1 : 0;
  return c;
}

// Whether the sums for dA_log take a second pass.  A workgroup that holds a whole row has
// all of its sums: with one row, they are the result (1 x 512 x 64 bf16 9.1 us, with the
// second pass 12.6).
bool sums_apart(const Cut& c, const ssm_gated_dims* dims) { return c.shared || dims->batch > 1; }

// Calls f.template operator()<IO, V>().
template <int WIDE, typename F>
void for_gated(const ssm_gated_dims* dims, int64_t V, const F& f) {
  if (dims->io_dtype == SSM_IO_F32)
    f.template operator()<float, 1>();
  else
    V == 1 ? f.template operator()<uint16_t, 1>() : f.template operator()<uint16_t, WIDE>();
}

// Calls f.template operator()<W>().
template <typename F>
void for_waves(int64_t waves, const F& f) {
  switch (waves) {
    case 1:
      return f.template operator()<1>();
    case 2:
      return f.template operator()<2>();
    case 4:
      return f.template operator()<4>();
    case 8:
      return f.template operator()<8>();
    default:
      return f.template operator()<16>();
  }
}

// Workgroups that take tiles: as many as the GPU holds at 128 registers a lane, 16
// waves a CU.  More start only when others end, to find no tile left (three times
// as many: backward 132 us where these take 125, 8 x 4096 x 1024 bf16).
int64_t takers(const Cut& c, int64_t cus) {
  const int64_t held = 16 / c.waves * cus, runs = ((c.tickets - 1) >> c.run) + 1;
  return runs < held ? runs : held;
}

ChainSpace chain_space(void* workspace, const Cut& c, int64_t V) {
  ChainSpace sp;
  sp.counter = static_cast<uint32_t*>(workspace);
  sp.pairs = static_cast<float*>(workspace) + 4;
  sp.states = sp.pairs + 2 * 64 * V * c.chains * c.tiles;
  sp.chains = static_cast<uint32_t>(c.chains);
  sp.run = static_cast<uint32_t>(c.run);
  return sp;
}
int64_t fill_blocks(const Cut& c) { return (c.words / 4 + 255) / 256; }
void launch_fill(void* workspace, const Cut& c, hipStream_t s) {
  hipLaunchKernelGGL(chain_fill_kernel, dim3(static_cast<unsigned>(fill_blocks(c))), dim3(256), 0, s,
                     static_cast<uint32_t*>(workspace), c.words);
}

// Whether a call that is cut up like this can be launched: its grids, and tickets that
// stay in 32 bits with those that are drawn behind the last.
bool launchable(const Cut& c) {
  return c.shared ? c.tickets < (1 << 28) && grid_fits(fill_blocks(c), 256) : grid_fits(c.chains, 64 * c.waves);
}

}  // namespace

extern "C" {

int64_t ssm_gated_recurrence_chunk_len(void) { return kChunk; }

int64_t ssm_gated_recurrence_fwd_workspace_bytes(const ssm_gated_dims* dims) {
  if (check_gated_dims(dims) != SSM_OK) return -1;
  return fwd_cut(dims).words * 4;
}

int ssm_gated_recurrence_fwd(ssm_scan_t handle, const ssm_gated_dims* dims, const ssm_gated_fwd_io* io, void* stream) {
  const int bad = check_gated_dims(dims);
  if (bad != SSM_OK) return bad;
  if (io == nullptr || io->workspace_bytes < 0) return SSM_ERR_INVALID_ARG;
  const int64_t nb = dims->batch, L = dims->seqlen, nd = dims->dim, ns = n_states(dims);
  const int64_t e = dims->io_dtype == SSM_IO_BF16 ? 2 : 4;
  const int64_t need = ssm_gated_recurrence_fwd_workspace_bytes(dims);
  const bool empty = nb == 0 || nd == 0;
  const Cut cut = fwd_cut(dims);
  if (!empty && L > 0 && !launchable(cut)) return SSM_ERR_UNSUPPORTED;
  // no steps: the state is copied
  if (!empty && L == 0 && io->h_last != nullptr && io->h_last != io->h0 && !grid_fits((nb * nd + 255) / 256, 256))
    return SSM_ERR_UNSUPPORTED;
  bool lines = false;
  if (!empty) {
    if (L > 0 && (io->x == nullptr || io->a_gate == nullptr || io->x_gate == nullptr || io->A_log == nullptr ||
                  io->y == nullptr))
      return SSM_ERR_INVALID_ARG;
    if (need > 0 && (io->workspace == nullptr || io->workspace_bytes < need)) return SSM_ERR_INVALID_ARG;
    const Rows x{io->x, nb, io->x_batch_stride, L, io->x_time_stride, nd, e};
    const Rows ag{io->a_gate, nb, io->a_gate_batch_stride, L, io->a_gate_time_stride, nd, e};
    const Rows xg{io->x_gate, nb, io->x_gate_batch_stride, L, io->x_gate_time_stride, nd, e};
    const Rows y{io->y, nb, io->y_batch_stride, L, io->y_time_stride, nd, e};
    if (x.bytes() < 0 || ag.bytes() < 0 || xg.bytes() < 0 || y.bytes() < 0 || !y.disjoint()) return SSM_ERR_INVALID_ARG;
    if (!aligned(io->x, e) || !aligned(io->a_gate, e) || !aligned(io->x_gate, e) || !aligned(io->y, e) ||
        !aligned(io->A_log, 4) || !aligned(io->valid_len, 4) || !aligned(io->h0, 4) || !aligned(io->h_last, 4) ||
        !aligned(io->chunk_states, 4) || !aligned(io->workspace, 8))
      return SSM_ERR_UNSUPPORTED;
    lines = whole_lines(x) && whole_lines(ag) && whole_lines(xg);
    // the state may be updated in place: it is read before it is written
    const Rows in[] = {x, ag, xg, flat(io->A_log, nd * 4), flat(io->valid_len, nb * 4),
                       flat(io->h0, io->h0 == io->h_last ? 0 : nb * nd * 4)};
    const Rows out[] = {y, flat(io->h_last, nb * nd * 4), flat(io->chunk_states, nb * ns * nd * 4),
                        flat(io->workspace, io->workspace_bytes)};
    if (any_overlap(in, out)) return SSM_ERR_ALIAS;
  }
  const int rc = check_handle(handle);
  if (rc != SSM_OK || empty) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (L == 0) {
    if (io->h_last == nullptr || io->h_last == io->h0) return SSM_OK;
    hipLaunchKernelGGL(gated_copy_kernel, dim3(static_cast<unsigned>((nb * nd + 255) / 256)), dim3(256), 0, s, io->h0,
                       io->h_last, nb * nd);
    return launched();
  }

  GatedParams p;
  p.x = io->x, p.ag = io->a_gate, p.xg = io->x_gate, p.A_log = io->A_log, p.valid_len = io->valid_len, p.h0 = io->h0;
  p.y = io->y, p.h_last = io->h_last, p.states = io->chunk_states;
  p.x_bs = io->x_batch_stride, p.x_ts = io->x_time_stride, p.ag_bs = io->a_gate_batch_stride;
  p.ag_ts = io->a_gate_time_stride, p.xg_bs = io->x_gate_batch_stride, p.xg_ts = io->x_gate_time_stride;
  p.y_bs = io->y_batch_stride, p.y_ts = io->y_time_stride;
  p.L = L, p.nd = static_cast<int32_t>(nd), p.n_states = static_cast<int32_t>(ns);
  p.n_cg = static_cast<int32_t>(cut.chains / nb);
  if (cut.shared) launch_fill(io->workspace, cut, s);
  for_gated<kFwdWide>(dims, cut.V, [&]<typename IO, int V>() {
    if (cut.shared) {
      const auto kernel = cut.waves == 16 ? (lines ? gated_fwd_chain_kernel<IO, V, kFwdSteps, 16, true>
                                                   : gated_fwd_chain_kernel<IO, V, kFwdSteps, 16, false>)
                                          : (lines ? gated_fwd_chain_kernel<IO, V, kFwdSteps, 8, true>
                                                   : gated_fwd_chain_kernel<IO, V, kFwdSteps, 8, false>);
      hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(takers(cut, handle->cu_count))),
                         dim3(static_cast<unsigned>(64 * cut.waves)), 0, s, p, chain_space(io->workspace, cut, V),
                         static_cast<uint32_t>(cut.tickets));
      return;
    }
    for_waves(cut.waves, [&]<int W>() {
      auto kernel = cut.groups == 4 ? gated_fwd_row_kernel<IO, 1, 4, 8, W> : gated_fwd_row_kernel<IO, V, 1, kFwdSteps, W>;
      if constexpr (W == 16)
        if (cut.groups == 4 && L > 4 * 16 * 8) kernel = gated_fwd_row_kernel<IO, 1, 4, kFwdSteps, W>;
      hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(cut.chains)), dim3(64 * W), 0, s, p);
    });
  });
  return launched();
}

int64_t ssm_gated_recurrence_bwd_workspace_bytes(const ssm_gated_dims* dims) {
  if (check_gated_dims(dims) != SSM_OK) return -1;
  // the chains' words, then a row of sums for every tile that a workgroup took
  const Cut c = bwd_cut(dims);
  return sums_apart(c, dims) ? (c.words + c.tiles * dims->batch * dims->dim) * 4 : 0;
}

int ssm_gated_recurrence_bwd(ssm_scan_t handle, const ssm_gated_dims* dims, const ssm_gated_bwd_io* io, void* stream) {
  const int bad = check_gated_dims(dims);
  if (bad != SSM_OK) return bad;
  if (io == nullptr || io->workspace_bytes < 0) return SSM_ERR_INVALID_ARG;
  const int64_t nb = dims->batch, L = dims->seqlen, nd = dims->dim, ns = n_states(dims);
  const int64_t e = dims->io_dtype == SSM_IO_BF16 ? 2 : 4;
  const int64_t need = ssm_gated_recurrence_bwd_workspace_bytes(dims);
  const bool some = nb > 0 && L > 0;
  const Cut cut = bwd_cut(dims);
  const bool sums = sums_apart(cut, dims);
  if (some && nd > 0 && (!launchable(cut) || (sums && !reduce_fits(nd)))) return SSM_ERR_UNSUPPORTED;
  if (nb > 0 && nd > 0 && L == 0 && io->dh0 != nullptr && !grid_fits((nb * nd + 255) / 256, 256))
    return SSM_ERR_UNSUPPORTED;
  bool lines = false;
  if (nd > 0) {
    if (io->dA_log == nullptr) return SSM_ERR_INVALID_ARG;
    if (some && (io->x == nullptr || io->a_gate == nullptr || io->x_gate == nullptr || io->A_log == nullptr ||
                 io->dy == nullptr || io->dx == nullptr || io->da_gate == nullptr || io->dx_gate == nullptr ||
                 (io->chunk_states == nullptr && L > kChunk) ||
                 (need > 0 && (io->workspace == nullptr || io->workspace_bytes < need))))
      return SSM_ERR_INVALID_ARG;
    const Rows x{io->x, nb, io->x_batch_stride, L, io->x_time_stride, nd, e};
    const Rows ag{io->a_gate, nb, io->a_gate_batch_stride, L, io->a_gate_time_stride, nd, e};
    const Rows xg{io->x_gate, nb, io->x_gate_batch_stride, L, io->x_gate_time_stride, nd, e};
    const Rows dy{io->dy, nb, io->dy_batch_stride, L, io->dy_time_stride, nd, e};
    const Rows dx{io->dx, nb, io->dx_batch_stride, L, io->dx_time_stride, nd, e};
    const Rows dag{io->da_gate, nb, io->da_gate_batch_stride, L, io->da_gate_time_stride, nd, e};
    const Rows dxg{io->dx_gate, nb, io->dx_gate_batch_stride, L, io->dx_gate_time_stride, nd, e};
    for (const Rows* r : {&x, &ag, &xg, &dy, &dx, &dag, &dxg})
      if (r->bytes() < 0) return SSM_ERR_INVALID_ARG;
    if (!dx.disjoint() || !dag.disjoint() || !dxg.disjoint()) return SSM_ERR_INVALID_ARG;
    for (const Rows* r : {&x, &ag, &xg, &dy, &dx, &dag, &dxg})
      if (!aligned(r->p, e)) return SSM_ERR_UNSUPPORTED;
    if (!aligned(io->A_log, 4) || !aligned(io->valid_len, 4) || !aligned(io->h0, 4) || !aligned(io->dh_last, 4) ||
        !aligned(io->chunk_states, 4) || !aligned(io->dA_log, 4) || !aligned(io->dh0, 4) || !aligned(io->workspace, 8))
      return SSM_ERR_UNSUPPORTED;
    lines = whole_lines(x) && whole_lines(ag) && whole_lines(xg) && whole_lines(dy);
    const Rows in[] = {x, ag, xg, dy, flat(io->A_log, nd * 4), flat(io->valid_len, nb * 4), flat(io->h0, nb * nd * 4),
                       flat(io->dh_last, nb * nd * 4), flat(io->chunk_states, nb * ns * nd * 4)};
    const Rows out[] = {dx, dag, dxg, flat(io->dA_log, nd * 4), flat(io->dh0, nb * nd * 4),
                        flat(io->workspace, io->workspace_bytes)};
    if (any_overlap(in, out)) return SSM_ERR_ALIAS;
  }
  const int rc = check_handle(handle);
  if (rc != SSM_OK || nd == 0) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (!some) {  // sums over nothing; the state's gradient passes through
    hipLaunchKernelGGL(gated_copy_kernel, dim3(static_cast<unsigned>((nd + 255) / 256)), dim3(256), 0, s, nullptr,
                       io->dA_log, nd);
    if (nb > 0 && io->dh0 != nullptr)
      hipLaunchKernelGGL(gated_copy_kernel, dim3(static_cast<unsigned>((nb * nd + 255) / 256)), dim3(256), 0, s,
                         io->dh_last, io->dh0, nb * nd);
    return launched();
  }
  GatedBwdParams p;
  p.x = io->x, p.ag = io->a_gate, p.xg = io->x_gate, p.A_log = io->A_log, p.valid_len = io->valid_len, p.h0 = io->h0;
  p.dy = io->dy, p.dh_last = io->dh_last, p.states = io->chunk_states;
  p.dx = io->dx, p.dag = io->da_gate, p.dxg = io->dx_gate, p.dh0 = io->dh0, p.ws = static_cast<float*>(io->workspace);
  p.x_bs = io->x_batch_stride, p.x_ts = io->x_time_stride, p.ag_bs = io->a_gate_batch_stride;
  p.ag_ts = io->a_gate_time_stride, p.xg_bs = io->x_gate_batch_stride, p.xg_ts = io->x_gate_time_stride;
  p.dy_bs = io->dy_batch_stride, p.dy_ts = io->dy_time_stride, p.dx_bs = io->dx_batch_stride;
  p.dx_ts = io->dx_time_stride, p.dag_bs = io->da_gate_batch_stride, p.dag_ts = io->da_gate_time_stride;
  p.dxg_bs = io->dx_gate_batch_stride, p.dxg_ts = io->dx_gate_time_stride;
  p.L = L, p.nd = static_cast<int32_t>(nd), p.n_states = static_cast<int32_t>(ns);
  p.ws = sums ? p.ws + cut.words : io->dA_log;
  p.n_cg = static_cast<int32_t>(cut.chains / nb);
  if (cut.shared) launch_fill(io->workspace, cut, s);
  for_gated<kBwdWide>(dims, cut.V, [&]<typename IO, int V>() {
    if (cut.shared) {
      const auto kernel =
          lines ? gated_bwd_chain_kernel<IO, V, kBwdSteps, 8, true> : gated_bwd_chain_kernel<IO, V, kBwdSteps, 8, false>;
      hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(takers(cut, handle->cu_count))),
                         dim3(static_cast<unsigned>(64 * cut.waves)), 0, s, p, chain_space(io->workspace, cut, V),
                         static_cast<uint32_t>(cut.tickets), static_cast<uint32_t>(cut.tiles));
      return;
    }
    for_waves(cut.waves, [&]<int W>() {
      const auto kernel = cut.groups == 4 ? gated_bwd_row_kernel<IO, 1, 4, 8, W> : gated_bwd_row_kernel<IO, V, 1, kBwdSteps, W>;
      hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(cut.chains)), dim3(64 * W), 0, s, p);
    });
  });
  if (launched() != SSM_OK) return SSM_ERR_HIP;
  if (!sums) return SSM_OK;
  launch_reduce(p.ws, cut.tiles * nb, nd, GatedGrads{io->dA_log}, s);
  return launched();
}

int ssm_gated_recurrence_step(ssm_scan_t handle, const ssm_gated_dims* dims, const ssm_gated_step_io* io,
                              void* stream) {
  const int bad = check_gated_dims(dims);
  if (bad != SSM_OK) return bad;
  if (io == nullptr || dims->seqlen != 1 || io->n_slots < 0) return SSM_ERR_INVALID_ARG;
  const int64_t nb = dims->batch, nd = dims->dim, rows = io->slots == nullptr ? nb : io->n_slots;
  if (nb > 65535 || rows > kMaxSize) return SSM_ERR_UNSUPPORTED;
  const int64_t e = dims->io_dtype == SSM_IO_BF16 ? 2 : 4;
  const bool empty = nb == 0 || nd == 0;
  if (!empty) {
    if (io->x == nullptr || io->a_gate == nullptr || io->x_gate == nullptr || io->A_log == nullptr ||
        io->y == nullptr || (rows > 0 && (io->h0 == nullptr || io->h_last == nullptr)))
      return SSM_ERR_INVALID_ARG;
    const Rows x{io->x, nb, io->x_row_stride, 1, 0, nd, e}, ag{io->a_gate, nb, io->a_gate_row_stride, 1, 0, nd, e};
    const Rows xg{io->x_gate, nb, io->x_gate_row_stride, 1, 0, nd, e}, y{io->y, nb, io->y_row_stride, 1, 0, nd, e};
    if (x.bytes() < 0 || ag.bytes() < 0 || xg.bytes() < 0 || y.bytes() < 0 || !y.disjoint()) return SSM_ERR_INVALID_ARG;
    const int64_t bh = span_bytes(rows, nd, 1, 0, nd, 4);
    if (bh < 0) return SSM_ERR_UNSUPPORTED;
    if (!aligned(io->x, e) || !aligned(io->a_gate, e) || !aligned(io->x_gate, e) || !aligned(io->y, e) ||
        !aligned(io->A_log, 4) || !aligned(io->slots, 4) || !aligned(io->h0, 4) || !aligned(io->h_last, 4))
      return SSM_ERR_UNSUPPORTED;
    const Rows in[] = {x, ag, xg, flat(io->A_log, nd * 4), flat(io->slots, nb * 4),
                       flat(io->h0, io->h0 == io->h_last ? 0 : bh)};
    const Rows out[] = {y, flat(io->h_last, bh)};
    if (any_overlap(in, out)) return SSM_ERR_ALIAS;
  }
  const int rc = check_handle(handle);
  if (rc != SSM_OK || empty) return rc;
  GatedStepParams p;
  p.x = io->x, p.ag = io->a_gate, p.xg = io->x_gate, p.A_log = io->A_log, p.slots = io->slots, p.h0 = io->h0;
  p.h_last = io->h_last, p.y = io->y, p.x_rs = io->x_row_stride, p.ag_rs = io->a_gate_row_stride;
  p.xg_rs = io->x_gate_row_stride, p.y_rs = io->y_row_stride, p.n_slots = rows;
  p.nb = static_cast<int32_t>(nb), p.nd = static_cast<int32_t>(nd);
  constexpr int V = 4;
  const dim3 grid(static_cast<unsigned>((nd + 256 * V - 1) / (256 * V)), static_cast<unsigned>(nb));
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dims->io_dtype == SSM_IO_BF16)
    hipLaunchKernelGGL((gated_step_kernel<uint16_t, V>), grid, dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((gated_step_kernel<float, V>), grid, dim3(256), 0, s, p);
  return launched();
}

}  // extern "C"
