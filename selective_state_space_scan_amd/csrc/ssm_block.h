// Internals shared by the operators around the scan (short convolution,
// single-token steps, norms): vector access at any alignment, activations,
// wave reductions, and the host's argument checks.
//
// Times in these sources are GPU times of a call, both passes where there are
// two: events around 30 queued calls, three input sets in turn.  What is a
// kernel's own duration in a trace, or a whole call with its CPU time, says so.
#pragma once

#include "ssm_internal.h"
#include "ssm_scan.h"

namespace {

// ---- vector access -------------------------------------------------------
//
// A lane moves V consecutive elements (16 bytes) of a row at once.  Rows start
// wherever strides and odd widths put them, so the vector types carry only
// their element's alignment; gfx950 code objects run in unaligned access mode
// and the compiler emits one 16-byte instruction for them all the same.  A
// row's last n < V elements are moved one by one.

template <typename IO>
struct VecIO;

template <>
struct VecIO<float> {
  static constexpr int kWide = 4;
  typedef float vec4 __attribute__((ext_vector_type(4), aligned(4)));
  typedef float vec2 __attribute__((ext_vector_type(2), aligned(4)));
  template <int V>
  static __device__ __forceinline__ void load(const float* p, float (&o)[V]) {
    constexpr int kWhole = V / 4 * 4;
#pragma unroll
    for (int i = 0; i < kWhole; i += 4) {
      const vec4 v = *reinterpret_cast<const vec4*>(p + i);
      o[i] = v.x, o[i + 1] = v.y, o[i + 2] = v.z, o[i + 3] = v.w;
    }
    if constexpr (V % 4 >= 2) {
      const vec2 v = *reinterpret_cast<const vec2*>(p + kWhole);
      o[kWhole] = v.x, o[kWhole + 1] = v.y;
    }
    if constexpr (V % 2 == 1) o[V - 1] = p[V - 1];
  }
  template <int V>
  static __device__ __forceinline__ void store(float* p, const float (&o)[V]) {
    static_assert(V <= 2 || V % 4 == 0, "whole 16-byte pieces, one or two elements");
    if constexpr (V == 1) {
      *p = o[0];
    } else if constexpr (V == 2) {
      vec2 v;
      v.x = o[0], v.y = o[1];
      *reinterpret_cast<vec2*>(p) = v;
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        vec4 v;
        v.x = o[i], v.y = o[i + 1], v.z = o[i + 2], v.w = o[i + 3];
        *reinterpret_cast<vec4*>(p + i) = v;
      }
    }
  }
  // a store past the caches, for what is not read again soon
  static __device__ __forceinline__ void stream(float* p, const float (&o)[4]) {
    vec4 v;
    v.x = o[0], v.y = o[1], v.z = o[2], v.w = o[3];
    __builtin_nontemporal_store(v, reinterpret_cast<vec4*>(p));
  }
  static __device__ __forceinline__ void stream(float* p, const float (&o)[1]) { *p = o[0]; }
  static __device__ __forceinline__ float get(const float* p) { return *p; }
  static __device__ __forceinline__ void put(float* p, float v) { *p = v; }
};

// bf16 is carried as its 16-bit pattern; widening to fp32 is exact, narrowing
// rounds to nearest even.
template <>
struct VecIO<uint16_t> {
  static constexpr int kWide = 8;
  typedef uint32_t vec4 __attribute__((ext_vector_type(4), aligned(2)));
  typedef uint32_t vec2 __attribute__((ext_vector_type(2), aligned(2)));
  typedef uint32_t vec1 __attribute__((aligned(2)));
  static __device__ __forceinline__ float lo(uint32_t u) { return __builtin_bit_cast(float, u << 16); }
  static __device__ __forceinline__ float hi(uint32_t u) { return __builtin_bit_cast(float, u & 0xffff0000u); }
  static __device__ __forceinline__ uint16_t narrow(float v) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {  // v_cvt_pk_bf16_f32
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    f32x2 v;
    v.x = a, v.y = b;
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
  }
  template <int V>
  static __device__ __forceinline__ void load(const uint16_t* p, float (&o)[V]) {
    static_assert(V % 8 == 0 || V == 4 || V == 2 || V == 1, "whole 16-, 8- or 4-byte pieces, or one element");
    if constexpr (V == 1) {
      o[0] = get(p);
    } else if constexpr (V == 2) {
      const vec1 v = *reinterpret_cast<const vec1*>(p);
      o[0] = lo(v), o[1] = hi(v);
    } else if constexpr (V == 4) {
      const vec2 v = *reinterpret_cast<const vec2*>(p);
      o[0] = lo(v.x), o[1] = hi(v.x), o[2] = lo(v.y), o[3] = hi(v.y);
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 8) {
        const vec4 v = *reinterpret_cast<const vec4*>(p + i);
        o[i] = lo(v.x), o[i + 1] = hi(v.x), o[i + 2] = lo(v.y), o[i + 3] = hi(v.y);
        o[i + 4] = lo(v.z), o[i + 5] = hi(v.z), o[i + 6] = lo(v.w), o[i + 7] = hi(v.w);
      }
    }
  }
  template <int V>
  static __device__ __forceinline__ void store(uint16_t* p, const float (&o)[V]) {
    if constexpr (V == 1) {
      put(p, o[0]);
    } else if constexpr (V == 2) {
      *reinterpret_cast<vec1*>(p) = pack(o[0], o[1]);
    } else if constexpr (V == 4) {
      vec2 v;
      v.x = pack(o[0], o[1]), v.y = pack(o[2], o[3]);
      *reinterpret_cast<vec2*>(p) = v;
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 8) {
        vec4 v;
        v.x = pack(o[i], o[i + 1]), v.y = pack(o[i + 2], o[i + 3]);
        v.z = pack(o[i + 4], o[i + 5]), v.w = pack(o[i + 6], o[i + 7]);
        *reinterpret_cast<vec4*>(p + i) = v;
      }
    }
  }
  static __device__ __forceinline__ void stream(uint16_t* p, const float (&o)[4]) {
    vec2 v;
    v.x = pack(o[0], o[1]), v.y = pack(o[2], o[3]);
    __builtin_nontemporal_store(v, reinterpret_cast<vec2*>(p));
  }
  static __device__ __forceinline__ void stream(uint16_t* p, const float (&o)[1]) { put(p, o[0]); }
  static __device__ __forceinline__ float get(const uint16_t* p) {
    return __builtin_bit_cast(float, static_cast<uint32_t>(*p) << 16);
  }
  static __device__ __forceinline__ void put(uint16_t* p, float v) { *p = narrow(v); }
};

// V elements as they stand in memory: what a lane keeps of a load in flight,
// unpacked when it is used.  load_once: past the caches, for what is not read again.
template <typename IO, int V>
struct RawVec;

template <int V>
struct RawVec<float, V> {
  float v[V];
  __device__ __forceinline__ void load(const float* p) { VecIO<float>::load(p, v); }
  __device__ __forceinline__ void load_once(const float* p) {
    if constexpr (V == 4) {
      const auto w = __builtin_nontemporal_load(reinterpret_cast<const VecIO<float>::vec4*>(p));
      v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = __builtin_nontemporal_load(p + i);
    }
  }
  __device__ __forceinline__ void unpack(float (&o)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = v[i];
  }
};

template <int V>
struct RawVec<uint16_t, V> {
  typedef uint32_t vec __attribute__((ext_vector_type(V / 2), aligned(2)));
  vec v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const vec*>(p); }
  __device__ __forceinline__ void load_once(const uint16_t* p) {
    v = __builtin_nontemporal_load(reinterpret_cast<const vec*>(p));
  }
  __device__ __forceinline__ void unpack(float (&o)[V]) const {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) o[2 * i] = VecIO<uint16_t>::lo(v[i]), o[2 * i + 1] = VecIO<uint16_t>::hi(v[i]);
  }
};

template <>
struct RawVec<uint16_t, 2> {
  uint32_t v;
  __device__ __forceinline__ void load(const uint16_t* p) {
    v = *reinterpret_cast<const VecIO<uint16_t>::vec1*>(p);
  }
  __device__ __forceinline__ void load_once(const uint16_t* p) {
    v = __builtin_nontemporal_load(reinterpret_cast<const VecIO<uint16_t>::vec1*>(p));
  }
  __device__ __forceinline__ void unpack(float (&o)[2]) const {
    o[0] = VecIO<uint16_t>::lo(v), o[1] = VecIO<uint16_t>::hi(v);
  }
};

template <>
struct RawVec<uint16_t, 1> {
  uint16_t v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *p; }
  __device__ __forceinline__ void load_once(const uint16_t* p) { v = __builtin_nontemporal_load(p); }
  __device__ __forceinline__ void unpack(float (&o)[1]) const { o[0] = VecIO<uint16_t>::lo(v); }
};

// The first n (0 <= n <= V) of V elements; the others read as `rest` and are not
// written.
template <typename IO, int V>
__device__ __forceinline__ void load_n(const IO* p, int n, float (&o)[V], float rest = 0.0f) {
  if (n == V) {
    VecIO<IO>::load(p, o);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = i < n ? VecIO<IO>::get(p + i) : rest;
  }
}
template <typename IO, int V>
__device__ __forceinline__ void store_n(IO* p, int n, const float (&o)[V]) {
  if (n == V) {
    VecIO<IO>::store(p, o);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) VecIO<IO>::put(p + i, o[i]);
  }
}

// ---- workgroups ------------------------------------------------------------

// Workgroups are dealt to the 8 XCDs in turn, each with an L2 of its own.
// Renumbered like this, an XCD gets runs of kRun consecutive pieces of work, so
// that what neighbours share (rows in front of a chunk, the other part of a
// line) is found in its L2, while the runs stay short enough that rows of
// different lengths spread over all XCDs.  What is left over behind the last
// whole round of runs keeps its numbers.
constexpr uint32_t kRun = 8;

__device__ __forceinline__ uint32_t xcd_run(uint32_t block, uint32_t blocks) {
  if (block >= blocks / (8 * kRun) * (8 * kRun)) return block;
  const uint32_t x = block % 8, i = block / 8;
  return (i / kRun * 8 + x) * kRun + i % kRun;
}

// ---- activations ---------------------------------------------------------

// sigmoid(v) = 1 / (1 + e^-v).  v_exp_f32 is 2^x: the rounding error of
// v * log2(e), which would grow with |v| in the result, is recovered by an FMA
// with the constant's low part and put back as a first-order factor.  |v| is
// cut at 110, where e^-v has long left fp32's range (2^158.7 is infinite, and
// the result 0), so that infinities stay out of the correction.
__device__ __forceinline__ float sigmoid_exact(float v) {
  constexpr float kLog2eLow = 1.925962991e-8f;  // log2(e) - kLog2e
  const float c = __builtin_amdgcn_fmed3f(v, -110.0f, 110.0f);
  const float t = -c * kLog2e;
  const float r = __builtin_fmaf(-c, kLog2eLow, __builtin_fmaf(-c, kLog2e, -t));
  const float e = fast_exp2(t);
  return __builtin_amdgcn_rcpf(__builtin_fmaf(e, __builtin_fmaf(r, kLn2, 1.0f), 1.0f));
}

// The same for bf16 inputs: the exponent's rounding error (|v| 2^-24 relative)
// is far below bf16's step wherever the result is not 0 or 1 to it, and the
// short form has half the instructions.  The convolution's backward also sums
// fp32 weight gradients of bf16 inputs from it: there the error stays in, at
// most 16 * 2^-24 (1 + |v|) of dy a term, where dy came rounded to 2^-8.
__device__ __forceinline__ float sigmoid_short(float v) {
  return __builtin_amdgcn_rcpf(1.0f + fast_exp2(-v * kLog2e));
}

template <typename IO>
__device__ __forceinline__ float sigmoid_for(float v) {
  if constexpr (sizeof(IO) == 2)
    return sigmoid_short(v);
  else
    return sigmoid_exact(v);
}

// ---- wave reductions -----------------------------------------------------

template <int CTRL>
__device__ __forceinline__ float dpp_move(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

// Sum over aligned groups of LANES (4, 8 or 16) consecutive lanes; every lane
// of the group gets the total.  quad_perm [1,0,3,2] and [2,3,0,1], then
// row_half_mirror (the other quad of eight lanes) and row_mirror (the other
// eight of a row).
template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
  static_assert(LANES == 4 || LANES == 8 || LANES == 16, "within a row of 16 lanes");
  v += dpp_move<0xB1>(v);
  v += dpp_move<0x4E>(v);
  if constexpr (LANES >= 8) v += dpp_move<0x141>(v);
  if constexpr (LANES >= 16) v += dpp_move<0x140>(v);
  return v;
}

// Sum over the 64 lanes of a wave; every lane gets the total.
__device__ __forceinline__ float wave_sum(float v) {
  v = group_sum<16>(v);
  float a, b;
  rows_swap16(v, a, b);
  v = a + b;
  rows_swap32(v, a, b);
  return a + b;
}

// ---- steps on a cache ------------------------------------------------------

// Which of the batch rows b .. b + R - 1 of a single-token step run on their
// cache rows `slot`: not one whose slot lies outside the cache (rows that pad
// the batch carry -1), nor one whose cache row an earlier batch row names, whose
// update then stands alone (two rows updating one would race).  Every wave
// looks through the earlier rows for itself, four a lane and load.
template <int R>
__device__ __forceinline__ void step_rows_active(const int32_t* slots, int32_t b, int32_t nb, const int32_t (&slot)[R],
                                                 int64_t n_slots, bool (&active)[R]) {
  bool taken[R] = {};
  if (slots != nullptr) {
    typedef int32_t vec4 __attribute__((ext_vector_type(4), aligned(4)));
    for (int32_t i = static_cast<int32_t>(threadIdx.x % 64) * 4; i < b; i += 256) {
      if (i + 4 <= b) {
        const vec4 v = *reinterpret_cast<const vec4*>(slots + i);
#pragma unroll
        for (int r = 0; r < R; ++r) taken[r] |= v.x == slot[r] || v.y == slot[r] || v.z == slot[r] || v.w == slot[r];
      } else {
        for (int32_t k = i; k < b; ++k) {
#pragma unroll
          for (int r = 0; r < R; ++r) taken[r] |= slots[k] == slot[r];
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    bool free = !__any(taken[r]);
#pragma unroll
    for (int q = 0; q < r; ++q) free = free && slot[q] != slot[r];
    active[r] = b + r < nb && slot[r] >= 0 && slot[r] < n_slots && free;
  }
}

// ---- host checks ---------------------------------------------------------

// HIP counts a launch's work-items per dimension in 32 bits.
inline bool grid_fits(int64_t blocks, int threads) { return blocks > 0 && blocks <= 0xffffffffLL / threads; }

constexpr int64_t kMaxSize = 0x7fffffffLL;

// Bytes from a strided [n0, n1, dim] tensor's first element to behind its last
// (dim fastest, strides in elements); -1 if a stride is negative or the span
// leaves 62 bits.
inline int64_t span_bytes(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t dim, int64_t e) {
  if (s0 < 0 || s1 < 0) return -1;
  if (n0 == 0 || n1 == 0 || dim == 0) return 0;
  const __int128 n = static_cast<__int128>(n0 - 1) * s0 + static_cast<__int128>(n1 - 1) * s1 + dim;
  return n * e < (static_cast<__int128>(1) << 62) ? static_cast<int64_t>(n * e) : -1;
}

// Whether no two elements of a strided [n0, n1, dim] tensor share an address:
// the outer dimension with the smaller stride steps over whole rows, the other
// over all of those.
inline bool rows_disjoint(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t dim) {
  if (n0 <= 1 && n1 <= 1) return true;
  if (n0 <= 1) return s1 >= dim;
  if (n1 <= 1) return s0 >= dim;
  const int64_t ns = s0 < s1 ? n0 : n1, ss = s0 < s1 ? s0 : s1, sl = s0 < s1 ? s1 : s0;
  return ss >= dim && static_cast<__int128>(sl) >= static_cast<__int128>(ns - 1) * ss + dim;
}

// A byte range a call reads or writes.
struct Range {
  const void* p;
  int64_t n;
};

// Whether an output overlaps an input or another output.
template <int NI, int NO>
inline bool any_overlap(const Range (&in)[NI], const Range (&out)[NO]) {
  for (int o = 0; o < NO; ++o) {
    for (int i = 0; i < NI; ++i)
      if (overlaps(out[o].p, static_cast<size_t>(out[o].n), in[i].p, static_cast<size_t>(in[i].n))) return true;
    for (int k = 0; k < o; ++k)
      if (overlaps(out[o].p, static_cast<size_t>(out[o].n), out[k].p, static_cast<size_t>(out[k].n))) return true;
  }
  return false;
}

// A strided [n0, n1, dim] tensor that a call reads or writes (dim fastest,
// strides in elements of e bytes), or none of one.
struct Rows {
  const void* p;
  int64_t n0, s0, n1, s1, dim, e;
  int64_t bytes() const { return span_bytes(n0, s0, n1, s1, dim, e); }
  bool disjoint() const { return rows_disjoint(n0, s0, n1, s1, dim); }
};

// n bytes in one piece.
inline Rows flat(const void* p, int64_t n) { return Rows{p, 1, 0, 1, 0, n, 1}; }

// Whether two tensors overlap, as the ranges from their first byte to their
// last; but the columns of one buffer do not: with strides that are all
// multiples of one, m, in both, a row's elements keep their places modulo m.
inline bool rows_overlap(const Rows& a, const Rows& b) {
  if (!overlaps(a.p, static_cast<size_t>(a.bytes()), b.p, static_cast<size_t>(b.bytes()))) return false;
  int64_t m = 0;
  for (const Rows* r : {&a, &b}) {
    if (r->n0 > 1 && (m == 0 || r->s0 * r->e < m)) m = r->s0 * r->e;
    if (r->n1 > 1 && (m == 0 || r->s1 * r->e < m)) m = r->s1 * r->e;
  }
  if (m == 0) return true;
  for (const Rows* r : {&a, &b})
    if ((r->n0 > 1 && r->s0 * r->e % m != 0) || (r->n1 > 1 && r->s1 * r->e % m != 0)) return true;
  const int64_t wide = reinterpret_cast<intptr_t>(b.p) - reinterpret_cast<intptr_t>(a.p);
  const int64_t off = (wide % m + m) % m;
  return off < a.dim * a.e || off + b.dim * b.e > m;
}

template <int NI, int NO>
inline bool any_overlap(const Rows (&in)[NI], const Rows (&out)[NO]) {
  for (int o = 0; o < NO; ++o) {
    for (int i = 0; i < NI; ++i)
      if (rows_overlap(out[o], in[i])) return true;
    for (int k = 0; k < o; ++k)
      if (rows_overlap(out[o], out[k])) return true;
  }
  return false;
}

// The handle, and that the calling thread's current device is the handle's.
inline int check_handle(ssm_scan_t handle) {
  if (handle == nullptr) return SSM_ERR_INVALID_ARG;
  int cur = -1;
  if (hipGetDevice(&cur) != hipSuccess) {
    (void)hipGetLastError();
    return SSM_ERR_HIP;
  }
  return cur == handle->device ? SSM_OK : SSM_ERR_DEVICE_MISMATCH;
}

inline int launched() { return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP; }

// ---- partial sums --------------------------------------------------------

// out(c) = sum over p of ws[p * cols + c]: the second pass of a weight
// gradient, whose first pass left one row of sums per workgroup.  A workgroup
// of 1024 takes 16 columns (64 bytes of a row) and 64 row lanes; each lane
// adds every 64th row, eight loads in flight, and the lanes join in a fixed
// order (a wave's four by row exchanges, the 16 waves through LDS once), so the
// result does not depend on timing.  Bound by latency: 160 rows of 5120 columns
// take 4.7 us in the kernel trace, beside the 46 of the convolution that left
// them.
constexpr int kReduceCols = 16, kReduceLanes = 64;

template <typename Out>
__global__ __launch_bounds__(kReduceCols * kReduceLanes) void reduce_partials_kernel(const float* ws, int64_t parts,
                                                                                    int64_t cols, Out out) {
  constexpr int kWaves = kReduceCols * kReduceLanes / 64, kAhead = 8;
  __shared__ float lds[kWaves][kReduceCols];
  const int c = threadIdx.x % kReduceCols, r = threadIdx.x / kReduceCols;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * kReduceCols + c;
  const float* at = ws + (col < cols ? col : cols - 1);
  float sum = 0.0f, a, b;
  for (int64_t p = r; p < parts; p += kAhead * kReduceLanes) {
    float v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t q = p + i * kReduceLanes;  // rows past the last repeat it and count nothing
      v[i] = at[(q < parts ? q : parts - 1) * cols];
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) sum += p + i * kReduceLanes < parts ? v[i] : 0.0f;
  }
  rows_swap16(sum, a, b);
  sum = a + b;
  rows_swap32(sum, a, b);
  sum = a + b;
  if (threadIdx.x % 64 < kReduceCols) lds[threadIdx.x / 64][c] = sum;
  __syncthreads();
  if (threadIdx.x < 64) {
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kWaves / 4; ++i) sum += lds[threadIdx.x / 16 * (kWaves / 4) + i][c];
    rows_swap16(sum, a, b);
    sum = a + b;
    rows_swap32(sum, a, b);
    sum = a + b;
    if (threadIdx.x < kReduceCols && col < cols) out(col, sum);
  }
}

// Whether that pass's grid takes so many columns.
inline bool reduce_fits(int64_t cols) {
  return grid_fits((cols + kReduceCols - 1) / kReduceCols, kReduceCols * kReduceLanes);
}

template <typename Out>
inline void launch_reduce(const float* ws, int64_t parts, int64_t cols, const Out& out, hipStream_t s) {
  hipLaunchKernelGGL(reduce_partials_kernel<Out>, dim3(static_cast<unsigned>((cols + kReduceCols - 1) / kReduceCols)),
                     dim3(kReduceCols * kReduceLanes), 0, s, ws, parts, cols, out);
}

}  // namespace
