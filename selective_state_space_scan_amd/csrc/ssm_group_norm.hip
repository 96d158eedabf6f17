// Group norm of every step's channels, with its activation or gate, for MI355X
// (gfx950): forward and backward.
//
// For each row of dim = groups * n channels and each group of n adjacent ones, with
// act(u) = u sigmoid(u) (silu) or u:
//
//     v = x (gate in front: x act(z)),  m = mean(v) (0 for RMS),  r = (mean((v - m)^2) + eps)^(-1/2)
//     p = (v - m) r w + b,  y = act(p) without a gate, p act(z) with one behind, p with one in front
//
// Backward, with xh = (v - m) r:
//
//     dp = dy act'(p), dy act(z) or dy;  k = dp w;  dv = r (k - mean(k) - xh mean(k xh))  (no mean(k) for RMS)
//     dx = dv (gate in front: dv act(z));  dz = dy p act'(z) or dv x act'(z)
//     dw = sum over rows of dp xh,  db = sum over rows of dp
//
// 10 to 30 operations an element on 4 to 20 bytes: bound by memory.  A group is
// held in registers between its one read and its one write, by as few lanes as
// hold it at 16 bytes a lane (1 to 64 of a wave, several groups side by side), then
// at 16 elements a lane, by up to 512 lanes.  A lane keeps its channels from row
// to row, so weights are read once and dw, db stay in registers, and it asks for
// its next row before it works on the one it has (us, 32768 x 1024 bf16 with a gate:
// forward 38 to 45, 52 without that; backward 61 to 65, with the sums' pass of 5; the
// bytes of a copy's rate 40 and 66).

#include <hip/hip_runtime.h>

#include <cstdint>

#include "ssm_block.h"

namespace {

constexpr int64_t kMaxGroup = 8192, kMaxGroupedDim = 1 << 29;

struct Strides {
  int64_t batch, time;
};

struct GroupParams {
  const void* x;
  const void* z;
  const float* w;
  const float* bias;
  const int32_t* valid_len;
  void* y;
  float* mean;
  float* rstd;
  Strides xs, zs, ys;
  uint32_t rows, L;  // L: steps of a row of the strides, and of valid_len
  int32_t n, groups, gpb, rpb;
  int32_t rms, silu;
  float eps, inv_n;
};

struct GroupBwdParams {
  const void* dy;
  const void* x;
  const void* z;
  const float* w;
  const float* bias;
  const float* mean;
  const float* rstd;
  const int32_t* valid_len;
  void* dx;
  void* dz;
  float* ws;
  Strides dys, xs, zs, dxs, dzs;
  uint32_t rows, L;
  int32_t n, groups, gpb, rpb;
  int32_t rms, silu, with_bias;
  float inv_n;
};

// Sums of K values over a group's TPL lanes; every lane gets them.  A group
// wider than a wave joins its waves in LDS (called by the whole workgroup then,
// which holds one group).
template <int TPL, int K>
__device__ __forceinline__ void lane_sums(float (&v)[K], float* lds) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float a, b;
    if constexpr (TPL == 2) v[k] += dpp_move<0xB1>(v[k]);
    if constexpr (TPL >= 4) v[k] = group_sum<(TPL < 16 ? TPL : 16)>(v[k]);
    if constexpr (TPL >= 32) {
      rows_swap16(v[k], a, b);
      v[k] = a + b;
    }
    if constexpr (TPL >= 64) {
      rows_swap32(v[k], a, b);
      v[k] = a + b;
    }
  }
  if constexpr (TPL > 64) {
    const int wave = threadIdx.x / 64;
    __syncthreads();  // the values of the last sums have been read
    if (threadIdx.x % 64 == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) lds[wave * K + k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = 0.0f;
#pragma unroll
      for (int w = 0; w < TPL / 64; ++w) v[k] += lds[w * K + k];
    }
  }
}

// act(u) and act'(u).
template <typename IO>
__device__ __forceinline__ float act_of(float u, bool silu) {
  return silu ? u * sigmoid_for<IO>(u) : u;
}
template <typename IO>
__device__ __forceinline__ void act_slope(float u, bool silu, float& act, float& slope) {
  if (silu) {
    const float s = sigmoid_for<IO>(u);
    act = u * s;
    slope = __builtin_fmaf(act, 1.0f - s, s);
  } else {
    act = u;
    slope = 1.0f;
  }
}

// A lane's rows, one after another at equal distances, as steps of rows of L.
struct Walk {
  uint32_t row, b, t, by, by_b, by_t, L;
  __device__ __forceinline__ Walk(uint32_t first, uint32_t step, uint32_t len)
      : row(first), b(first / len), t(first - first / len * len), by(step), by_b(step / len),
        by_t(step - step / len * len), L(len) {}
  // Whether the step passed one end of a row more than by_b.
  __device__ __forceinline__ bool next() {
    row += by, b += by_b, t += by_t;
    const bool over = t >= L;
    t -= over ? L : 0;
    b += over ? 1 : 0;
    return over;
  }
};
// A strided tensor along them.
template <typename IO>
struct Along {
  IO* p;
  int64_t by, over;
  __device__ __forceinline__ Along(const void* base, const Strides& s, const Walk& w, int64_t c0)
      : p(static_cast<IO*>(const_cast<void*>(base)) + w.b * s.batch + w.t * s.time + c0),
        by(w.by_b * s.batch + w.by_t * s.time), over(s.batch - w.L * s.time) {}
  __device__ __forceinline__ void next(bool o) { p += by + (o ? over : 0); }
};

// Where a lane works: its group (of the row), its place in it, and the first of
// its rows; workgroups take gpb groups of rpb rows at once.
struct Place {
  int lane, rs, g;
  bool active;
};
template <int TPL>
__device__ __forceinline__ Place place(int32_t gpb, int32_t rpb, int32_t groups) {
  Place p;
  const int sub = threadIdx.x / TPL;
  p.lane = threadIdx.x % TPL;
  p.rs = sub / gpb;
  p.g = static_cast<int>(blockIdx.x) * gpb + sub % gpb;
  p.active = p.rs < rpb && p.g < groups;
  return p;
}

template <int TPL>
constexpr int block_of = TPL > 256 ? TPL : (TPL > 64 ? TPL : 256);

// A lane's pieces: piece k of it is the group's piece k * TPL + lane, moved back to
// the last V elements where it would reach past the group's end.  Its first `skip`
// elements are another's then: both compute and write the same for them, and they
// count in one's sums.  A piece behind the end (skip = V) writes nothing.
template <int V, int TPL, int NV>
struct Pieces {
  int32_t d[NV], skip[NV];
  __device__ __forceinline__ Pieces(int lane, int32_t n) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int32_t first = (k * TPL + lane) * V;
      d[k] = first < n - V ? first : n - V;
      skip[k] = first - d[k] < V ? first - d[k] : V;
    }
  }
};

// Whether the row at w, whose length has been read, is not padding.
__device__ __forceinline__ int32_t length_at(const int32_t* valid_len, const Walk& w, bool have) {
  return valid_len == nullptr ? INT32_MAX : (have ? valid_len[w.b] : 0);
}

template <typename IO, int V, int TPL, int NV, int GATE>
__global__ __launch_bounds__(block_of<TPL>) void group_fwd_kernel(const GroupParams prm) {
  constexpr int BLOCK = block_of<TPL>;
  __shared__ float lds[BLOCK / 64 * 2];
  const Place at = place<TPL>(prm.gpb, prm.rpb, prm.groups);
  const int64_t c0 = static_cast<int64_t>(at.g) * prm.n;
  const Pieces<V, TPL, NV> pc(at.lane, prm.n);
  const uint32_t step = gridDim.y * prm.rpb;
  Walk walk(blockIdx.y * prm.rpb + at.rs, step, prm.L), far = walk;
  Along<const IO> x(prm.x, prm.xs, walk, c0), z(prm.z, prm.zs, walk, c0);
  Along<IO> y(prm.y, prm.ys, walk, c0);
  // the row to work on has been asked for, and the next one's length
  RawVec<IO, V> rx[NV], rz[NV];
  const auto ask = [&](bool valid) __attribute__((always_inline)) {
    if (!valid || prm.n == 0) return;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      rx[k].load(x.p + pc.d[k]);
      if constexpr (GATE != SSM_GATE_NONE) rz[k].load(z.p + pc.d[k]);
    }
  };
  bool have = at.active && walk.row < prm.rows;
  bool valid = have && static_cast<int32_t>(walk.t) < length_at(prm.valid_len, walk, have);
  ask(valid);
  far.next();
  int32_t len = length_at(prm.valid_len, far, at.active && far.row < prm.rows);
  float w[NV][V], bias[NV][V] = {};
  if (at.active && prm.n > 0) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      VecIO<float>::load(prm.w + c0 + pc.d[k], w[k]);
      if (prm.bias != nullptr) VecIO<float>::load(prm.bias + c0 + pc.d[k], bias[k]);
    }
  }
  const bool silu = prm.silu != 0;
  // every lane of a workgroup makes the same number of turns
  for (uint32_t base = blockIdx.y * prm.rpb; base < prm.rows; base += step) {
    float v[NV][V], zv[NV][V];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      rx[k].unpack(v[k]);
      if constexpr (GATE != SSM_GATE_NONE) rz[k].unpack(zv[k]);
    }
    const uint32_t row = walk.row;
    const bool had = have, was = valid, over = walk.next();
    x.next(over), z.next(over);
    have = at.active && walk.row < prm.rows;
    valid = have && static_cast<int32_t>(walk.t) < len;
    ask(valid);
    far.next();
    len = length_at(prm.valid_len, far, at.active && far.row < prm.rows);
    if constexpr (GATE != SSM_GATE_NONE) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          zv[k][i] = act_of<IO>(zv[k][i], silu);
          if constexpr (GATE == SSM_GATE_BEFORE) v[k][i] *= zv[k][i];
        }
    }
    float mean = 0.0f;
    if (!prm.rms) {
      float s[1] = {0.0f};
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) s[0] += i >= pc.skip[k] ? v[k][i] : 0.0f;
      lane_sums<TPL>(s, lds);
      mean = s[0] * prm.inv_n;
    }
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[k][i] -= mean;
        const float c = i >= pc.skip[k] ? v[k][i] : 0.0f;
        s[0] += c;
        s[1] = __builtin_fmaf(c, c, s[1]);
      }
    lane_sums<TPL>(s, lds);
    // the small sum of the differences corrects mean and variance, so groups
    // whose mean is far from zero lose nothing
    const float off = prm.rms ? 0.0f : s[0] * prm.inv_n;
    float var = __builtin_fmaf(-off, off, s[1] * prm.inv_n);
    var = var < 0.0f ? 0.0f : var;
    const float rstd = 1.0f / __builtin_sqrtf(var + prm.eps);
    if (had) {
      if (at.lane == 0) {
        const int64_t st = static_cast<int64_t>(row) * prm.groups + at.g;
        if (prm.mean != nullptr) prm.mean[st] = was ? mean + off : 0.0f;
        if (prm.rstd != nullptr) prm.rstd[st] = was ? rstd : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float p = __builtin_fmaf((v[k][i] - off) * rstd, w[k][i], bias[k][i]);
          if constexpr (GATE == SSM_GATE_NONE) p = act_of<IO>(p, silu);
          if constexpr (GATE == SSM_GATE_AFTER) p *= zv[k][i];
          o[i] = was ? p : 0.0f;
        }
        if (pc.skip[k] < V) VecIO<IO>::store(y.p + pc.d[k], o);
      }
    }
    y.next(over);
  }
}

// Each workgroup leaves one row of [dw | db] for its groups, the second pass
// adds them.
template <typename IO, int V, int TPL, int NV, int GATE>
__global__ __launch_bounds__(block_of<TPL>) void group_bwd_kernel(const GroupBwdParams prm) {
  constexpr int BLOCK = block_of<TPL>;
  __shared__ float lds[BLOCK / 64 * 2];
  __shared__ float join[TPL < BLOCK ? BLOCK * V : 1];
  const Place at = place<TPL>(prm.gpb, prm.rpb, prm.groups);
  const int64_t c0 = static_cast<int64_t>(at.g) * prm.n, nd = static_cast<int64_t>(prm.groups) * prm.n;
  const Pieces<V, TPL, NV> pc(at.lane, prm.n);
  const uint32_t step = gridDim.y * prm.rpb;
  Walk walk(blockIdx.y * prm.rpb + at.rs, step, prm.L), far = walk;
  Along<const IO> x(prm.x, prm.xs, walk, c0), z(prm.z, prm.zs, walk, c0), dy(prm.dy, prm.dys, walk, c0);
  Along<IO> dx(prm.dx, prm.dxs, walk, c0), dz(prm.dz, prm.dzs, walk, c0);
  RawVec<IO, V> rx[NV], rz[NV], rg[NV];
  float rm = 0.0f, rr = 0.0f;
  const auto ask = [&](bool valid) __attribute__((always_inline)) {
    rm = rr = 0.0f;
    if (!valid) return;
    const int64_t st = static_cast<int64_t>(walk.row) * prm.groups + at.g;
    if (!prm.rms) rm = prm.mean[st];
    rr = prm.rstd[st];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      rx[k].load_once(x.p + pc.d[k]);
      if constexpr (GATE != SSM_GATE_NONE) rz[k].load_once(z.p + pc.d[k]);
      rg[k].load_once(dy.p + pc.d[k]);
    }
  };
  bool have = at.active && walk.row < prm.rows;
  bool valid = have && static_cast<int32_t>(walk.t) < length_at(prm.valid_len, walk, have);
  ask(valid);
  far.next();
  int32_t len = length_at(prm.valid_len, far, at.active && far.row < prm.rows);
  float w[NV][V], bias[NV][V] = {}, dw[NV][V] = {}, db[NV][V] = {};
  if (at.active) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      VecIO<float>::load(prm.w + c0 + pc.d[k], w[k]);
      if constexpr (GATE != SSM_GATE_BEFORE)  // p is not wanted there
        if (prm.bias != nullptr) VecIO<float>::load(prm.bias + c0 + pc.d[k], bias[k]);
    }
  }
  const bool silu = prm.silu != 0;
  for (uint32_t base = blockIdx.y * prm.rpb; base < prm.rows; base += step) {
    float xv[NV][V], zv[NV][V], g[NV][V], h[NV][V];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      rx[k].unpack(xv[k]);
      if constexpr (GATE != SSM_GATE_NONE) rz[k].unpack(zv[k]);
      rg[k].unpack(g[k]);
    }
    const float mean = rm, rstd = rr;
    const bool had = have, was = valid, over = walk.next();
    x.next(over), z.next(over), dy.next(over);
    have = at.active && walk.row < prm.rows;
    valid = have && static_cast<int32_t>(walk.t) < len;
    ask(valid);
    far.next();
    len = length_at(prm.valid_len, far, at.active && far.row < prm.rows);
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float v = xv[k][i];
        if constexpr (GATE == SSM_GATE_BEFORE) v *= act_of<IO>(zv[k][i], silu);
        // what a row of padding finds in the registers counts as nothing
        const float xh = was ? (v - mean) * rstd : 0.0f;
        h[k][i] = xh;
        float dp = g[k][i];
        if constexpr (GATE != SSM_GATE_BEFORE) {
          const float p = __builtin_fmaf(xh, w[k][i], bias[k][i]);
          float act, slope;
          if constexpr (GATE == SSM_GATE_NONE) {
            act_slope<IO>(p, silu, act, slope);
            dp *= slope;
          } else {
            act_slope<IO>(zv[k][i], silu, act, slope);
            zv[k][i] = dp * p * slope;  // dz
            dp *= act;
          }
        }
        dp = was ? dp : 0.0f;
        dw[k][i] = __builtin_fmaf(dp, xh, dw[k][i]);
        db[k][i] += dp;
        g[k][i] = dp * w[k][i];
        const float k1 = i >= pc.skip[k] ? g[k][i] : 0.0f;
        s[0] = __builtin_fmaf(k1, xh, s[0]);
        s[1] += k1;
      }
    lane_sums<TPL>(s, lds);
    if (had) {
      const float along = s[0] * prm.inv_n, off = prm.rms ? 0.0f : s[1] * prm.inv_n;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float o[V], oz[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float dv = (g[k][i] - off - h[k][i] * along) * rstd;
          if constexpr (GATE == SSM_GATE_AFTER) oz[i] = was ? zv[k][i] : 0.0f;
          if constexpr (GATE == SSM_GATE_BEFORE) {
            float act, slope;
            act_slope<IO>(zv[k][i], silu, act, slope);
            oz[i] = was ? dv * xv[k][i] * slope : 0.0f;
            dv *= act;
          }
          o[i] = was ? dv : 0.0f;
        }
        if (pc.skip[k] < V) {
          VecIO<IO>::store(dx.p + pc.d[k], o);
          if constexpr (GATE != SSM_GATE_NONE) VecIO<IO>::store(dz.p + pc.d[k], oz);
        }
      }
    }
    dx.next(over), dz.next(over);
  }
  // One row of sums a workgroup: [dw | db].
  float* out = prm.ws + static_cast<int64_t>(blockIdx.y) * (prm.with_bias ? 2 : 1) * nd + c0;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    if (q == 1 && !prm.with_bias) break;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float sum[V];
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] = q == 0 ? dw[k][i] : db[k][i];
      if constexpr (TPL < BLOCK) {
        if (prm.rpb > 1) {
          __syncthreads();
#pragma unroll
          for (int i = 0; i < V; ++i) join[i * BLOCK + threadIdx.x] = sum[i];
          __syncthreads();
          if (at.rs == 0) {
#pragma unroll
            for (int i = 0; i < V; ++i)
              for (int r = 1; r < prm.rpb; ++r) sum[i] += join[i * BLOCK + r * prm.gpb * TPL + threadIdx.x];
          }
        }
      }
      if (at.active && at.rs == 0 && pc.skip[k] < V) VecIO<float>::store(out + q * nd + pc.d[k], sum);
    }
  }
}

struct GroupGrads {
  float* dw;
  float* db;
  int64_t nd;
  __device__ __forceinline__ void operator()(int64_t col, float v) const {
    if (col < nd)
      dw[col] = v;
    else
      db[col - nd] = v;
  }
};

__global__ void group_fill_kernel(float* p, int64_t n, float v) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) p[i] = v;
}

// ---- host ------------------------------------------------------------------

int check_group_dims(const ssm_group_norm_dims* dims) {
  if (dims == nullptr || dims->batch < 0 || dims->seqlen < 0 || dims->dim < 0) return SSM_ERR_INVALID_ARG;
  if (dims->groups < 1 || dims->dim % dims->groups != 0) return SSM_ERR_INVALID_ARG;
  if (dims->io_dtype != SSM_IO_F32 && dims->io_dtype != SSM_IO_BF16) return SSM_ERR_INVALID_ARG;
  if (dims->rms != 0 && dims->rms != 1) return SSM_ERR_INVALID_ARG;
  if (dims->silu != 0 && dims->silu != 1) return SSM_ERR_INVALID_ARG;
  if (dims->gate != SSM_GATE_NONE && dims->gate != SSM_GATE_AFTER && dims->gate != SSM_GATE_BEFORE)
    return SSM_ERR_INVALID_ARG;
  if (!(dims->eps > 0.0f && dims->eps < __builtin_inff())) return SSM_ERR_INVALID_ARG;
  if (dims->dim / dims->groups > kMaxGroup || dims->dim >= kMaxGroupedDim || dims->batch > kMaxSize ||
      dims->seqlen > kMaxSize || dims->batch * dims->seqlen > kMaxSize || dims->groups > kMaxSize)
    return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

// Calls f.template operator()<IO, V, TPL, NV>(): the fewest lanes that hold a group at
// one piece (16 bytes, or as much of it as a group has) a lane, up to a wave, and from
// there at 16 elements.
template <typename IO, typename F>
void for_lanes(int64_t n, const F& f) {
  constexpr int V = VecIO<IO>::kWide, E = 16;
  if (n == 1)
    f.template operator()<IO, 1, 1, 1>();
  else if (n < 4)
    f.template operator()<IO, 2, 2, 1>();
  else if (n < V)
    f.template operator()<IO, 4, 2, 1>();
  else if (n == V)
    f.template operator()<IO, V, 1, 1>();
  else if (n <= 2 * V)
    f.template operator()<IO, V, 2, 1>();
  else if (n <= 4 * V)
    f.template operator()<IO, V, 4, 1>();
  else if (n <= 8 * V)
    f.template operator()<IO, V, 8, 1>();
  else if (n <= 16 * V)
    f.template operator()<IO, V, 16, 1>();
  else if (n <= 32 * V)
    f.template operator()<IO, V, 32, 1>();
  else if (n <= 64 * V)
    f.template operator()<IO, V, 64, 1>();
  else if (n <= 128 * V)
    f.template operator()<IO, V, 64, 2>();
  else if (n <= 64 * E)
    f.template operator()<IO, V, 64, E / V>();
  else if (n <= 128 * E)
    f.template operator()<IO, V, 128, E / V>();
  else if (n <= 256 * E)
    f.template operator()<IO, V, 256, E / V>();
  else
    f.template operator()<IO, V, 512, E / V>();
}

template <typename F>
void for_group(const ssm_group_norm_dims* dims, const F& f) {
  const int64_t n = dims->dim / dims->groups;
  const auto gated = [&]<typename IO, int V, int TPL, int NV>() {
    if (dims->gate == SSM_GATE_NONE)
      f.template operator()<IO, V, TPL, NV, SSM_GATE_NONE>();
    else if (dims->gate == SSM_GATE_AFTER)
      f.template operator()<IO, V, TPL, NV, SSM_GATE_AFTER>();
    else
      f.template operator()<IO, V, TPL, NV, SSM_GATE_BEFORE>();
  };
  if (dims->io_dtype == SSM_IO_BF16)
    for_lanes<uint16_t>(n, gated);
  else
    for_lanes<float>(n, gated);
}

// How a workgroup of `units` group places covers rows of `groups` groups: whole
// rows, or where they have more groups than it has places, an even share of one.
struct Cover {
  int64_t gpb, rpb, columns, stripes;
};
Cover cover(int64_t units, int64_t groups, int64_t rows, int64_t most) {
  Cover c;
  c.columns = (groups + units - 1) / units;
  c.gpb = (groups + c.columns - 1) / c.columns;
  c.rpb = units / c.gpb;
  const int64_t all = (rows + c.rpb - 1) / c.rpb;
  int64_t s = (most + c.columns - 1) / c.columns;
  if (s > 65535) s = 65535;
  c.stripes = all < s ? all : s;
  return c;
}

// Waves, each lane with its row in flight: 24 a CU forward, 8 backward (us, 32768 x 1024
// bf16 with a gate behind: 38 forward at 24, 40 at 12; backward 63 at 8, 67 at 12, 85
// with 16 and loads through the caches, which hold what nothing reads again: 73 at 8;
// 8192 channels a group 65 and 80).  Groups of up to four channels are bound by their
// loads' latency rather: 65536 x 128 groups of 4 takes 103 at 16, 131 at 8.
constexpr int64_t kFwdWaves = 256 * 24, kBwdWaves = 256 * 8, kSmallBwdWaves = 256 * 16;

template <int TPL>
Cover fwd_cover(const ssm_group_norm_dims* dims) {
  return cover(block_of<TPL> / TPL, dims->groups, dims->batch * dims->seqlen, kFwdWaves * 64 / block_of<TPL>);
}
template <int V, int TPL, int NV>
Cover bwd_cover(const ssm_group_norm_dims* dims) {
  return cover(block_of<TPL> / TPL, dims->groups, dims->batch * dims->seqlen, (V * NV <= 4 && TPL <= 2 ? kSmallBwdWaves : kBwdWaves) * 64 / block_of<TPL>);
}

}  // namespace

extern "C" {

int ssm_group_norm_fwd(ssm_scan_t handle, const ssm_group_norm_dims* dims, const ssm_group_norm_fwd_io* io,
                       void* stream) {
  const int bad = check_group_dims(dims);
  if (bad != SSM_OK) return bad;
  if (io == nullptr) return SSM_ERR_INVALID_ARG;
  const int64_t nb = dims->batch, L = dims->seqlen, nd = dims->dim, rows = nb * L;
  const int64_t e = dims->io_dtype == SSM_IO_BF16 ? 2 : 4;
  const bool gated = dims->gate != SSM_GATE_NONE;
  if (gated != (io->z != nullptr) && rows > 0 && nd > 0) return SSM_ERR_INVALID_ARG;
  // rows of no elements still have statistics
  const bool empty = rows == 0 || (nd == 0 && io->mean == nullptr && io->rstd == nullptr);
  if (!empty) {
    if (nd > 0 && (io->x == nullptr || io->weight == nullptr || io->y == nullptr)) return SSM_ERR_INVALID_ARG;
    const Rows x{io->x, nb, io->x_batch_stride, L, io->x_time_stride, nd, e};
    const Rows z{io->z, nb, io->z_batch_stride, L, io->z_time_stride, nd, e};
    const Rows y{io->y, nb, io->y_batch_stride, L, io->y_time_stride, nd, e};
    if (x.bytes() < 0 || (gated && z.bytes() < 0) || y.bytes() < 0 || (nd > 0 && !y.disjoint()))
      return SSM_ERR_INVALID_ARG;
    if (!aligned(io->x, e) || !aligned(io->z, e) || !aligned(io->y, e) || !aligned(io->weight, 4) ||
        !aligned(io->bias, 4) || !aligned(io->valid_len, 4) || !aligned(io->mean, 4) || !aligned(io->rstd, 4))
      return SSM_ERR_UNSUPPORTED;
    const int64_t stats = rows * dims->groups * 4;
    const Rows in[] = {x, gated ? z : flat(nullptr, 0), flat(io->weight, nd * 4), flat(io->bias, nd * 4),
                       flat(io->valid_len, nb * 4)};
    const Rows out[] = {y, flat(io->mean, stats), flat(io->rstd, stats)};
    if (any_overlap(in, out)) return SSM_ERR_ALIAS;
  }
  const int rc = check_handle(handle);
  if (rc != SSM_OK || empty) return rc;

  GroupParams p;
  p.x = io->x, p.z = io->z, p.w = io->weight, p.bias = io->bias, p.valid_len = io->valid_len, p.y = io->y;
  p.mean = io->mean, p.rstd = io->rstd;
  p.xs = {io->x_batch_stride, io->x_time_stride}, p.zs = {io->z_batch_stride, io->z_time_stride};
  p.ys = {io->y_batch_stride, io->y_time_stride};
  p.rows = static_cast<uint32_t>(rows), p.L = static_cast<uint32_t>(L);
  p.n = static_cast<int32_t>(nd / dims->groups), p.groups = static_cast<int32_t>(dims->groups);
  p.rms = dims->rms, p.silu = dims->silu, p.eps = dims->eps, p.inv_n = nd > 0 ? 1.0f / static_cast<float>(p.n) : 0.0f;
  for_group(dims, [&]<typename IO, int V, int TPL, int NV, int GATE>() {
    const Cover c = fwd_cover<TPL>(dims);
    p.gpb = static_cast<int32_t>(c.gpb), p.rpb = static_cast<int32_t>(c.rpb);
    hipLaunchKernelGGL((group_fwd_kernel<IO, V, TPL, NV, GATE>),
                       dim3(static_cast<unsigned>(c.columns), static_cast<unsigned>(c.stripes)), dim3(block_of<TPL>), 0,
                       static_cast<hipStream_t>(stream), p);
  });
  return launched();
}

int64_t ssm_group_norm_bwd_workspace_bytes(const ssm_group_norm_dims* dims) {
  if (check_group_dims(dims) != SSM_OK) return -1;
  int64_t bytes = 0;
  for_group(dims, [&]<typename IO, int V, int TPL, int NV, int GATE>() {
    bytes = bwd_cover<V, TPL, NV>(dims).stripes * 2 * dims->dim * 4;
  });
  return bytes;
}

int ssm_group_norm_bwd(ssm_scan_t handle, const ssm_group_norm_dims* dims, const ssm_group_norm_bwd_io* io,
                       void* stream) {
  const int bad = check_group_dims(dims);
  if (bad != SSM_OK) return bad;
  if (io == nullptr || io->workspace_bytes < 0) return SSM_ERR_INVALID_ARG;
  const int64_t nb = dims->batch, L = dims->seqlen, nd = dims->dim, rows = nb * L;
  const int64_t e = dims->io_dtype == SSM_IO_BF16 ? 2 : 4;
  const int64_t need = ssm_group_norm_bwd_workspace_bytes(dims);
  const bool gated = dims->gate != SSM_GATE_NONE;
  if (rows > 0 && nd > 0 && !reduce_fits((io->dbias != nullptr ? 2 : 1) * nd)) return SSM_ERR_UNSUPPORTED;
  if (nd > 0) {
    if (io->weight == nullptr || io->dweight == nullptr) return SSM_ERR_INVALID_ARG;
    if (rows > 0 && (gated != (io->z != nullptr) || gated != (io->dz != nullptr))) return SSM_ERR_INVALID_ARG;
    if (rows > 0 && (io->dy == nullptr || io->x == nullptr || io->rstd == nullptr || io->dx == nullptr ||
                     (!dims->rms && io->mean == nullptr) || io->workspace == nullptr || io->workspace_bytes < need))
      return SSM_ERR_INVALID_ARG;
    const Rows dy{io->dy, nb, io->dy_batch_stride, L, io->dy_time_stride, nd, e};
    const Rows x{io->x, nb, io->x_batch_stride, L, io->x_time_stride, nd, e};
    const Rows z = gated ? Rows{io->z, nb, io->z_batch_stride, L, io->z_time_stride, nd, e} : flat(nullptr, 0);
    const Rows dx{io->dx, nb, io->dx_batch_stride, L, io->dx_time_stride, nd, e};
    const Rows dz = gated ? Rows{io->dz, nb, io->dz_batch_stride, L, io->dz_time_stride, nd, e} : flat(nullptr, 0);
    for (const Rows* r : {&dy, &x, &z, &dx, &dz})
      if (r->bytes() < 0) return SSM_ERR_INVALID_ARG;
    if (!dx.disjoint() || !dz.disjoint()) return SSM_ERR_INVALID_ARG;
    for (const Rows* r : {&dy, &x, &z, &dx, &dz})
      if (!aligned(r->p, e)) return SSM_ERR_UNSUPPORTED;
    if (!aligned(io->weight, 4) || !aligned(io->bias, 4) || !aligned(io->mean, 4) || !aligned(io->rstd, 4) ||
        !aligned(io->valid_len, 4) || !aligned(io->dweight, 4) || !aligned(io->dbias, 4) || !aligned(io->workspace, 4))
      return SSM_ERR_UNSUPPORTED;
    const int64_t stats = rows * dims->groups * 4;
    const Rows in[] = {dy, x, z, flat(io->weight, nd * 4), flat(io->bias, nd * 4), flat(io->mean, stats),
                       flat(io->rstd, stats), flat(io->valid_len, nb * 4)};
    const Rows out[] = {dx, dz, flat(io->dweight, nd * 4), flat(io->dbias, nd * 4),
                        flat(io->workspace, io->workspace_bytes)};
    if (any_overlap(in, out)) return SSM_ERR_ALIAS;
  }
  const int rc = check_handle(handle);
  if (rc != SSM_OK || nd == 0) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (rows == 0) {  // sums over nothing
    const dim3 grid(static_cast<unsigned>((nd + 255) / 256));
    hipLaunchKernelGGL(group_fill_kernel, grid, dim3(256), 0, s, io->dweight, nd, 0.0f);
    if (io->dbias != nullptr) hipLaunchKernelGGL(group_fill_kernel, grid, dim3(256), 0, s, io->dbias, nd, 0.0f);
    return launched();
  }
  GroupBwdParams p;
  p.dy = io->dy, p.x = io->x, p.z = io->z, p.w = io->weight, p.bias = io->bias, p.mean = io->mean, p.rstd = io->rstd;
  p.valid_len = io->valid_len, p.dx = io->dx, p.dz = io->dz, p.ws = static_cast<float*>(io->workspace);
  p.dys = {io->dy_batch_stride, io->dy_time_stride}, p.xs = {io->x_batch_stride, io->x_time_stride};
  p.zs = {io->z_batch_stride, io->z_time_stride}, p.dxs = {io->dx_batch_stride, io->dx_time_stride};
  p.dzs = {io->dz_batch_stride, io->dz_time_stride};
  p.rows = static_cast<uint32_t>(rows), p.L = static_cast<uint32_t>(L);
  p.n = static_cast<int32_t>(nd / dims->groups), p.groups = static_cast<int32_t>(dims->groups);
  p.rms = dims->rms, p.silu = dims->silu, p.with_bias = io->dbias != nullptr, p.inv_n = 1.0f / static_cast<float>(p.n);
  int64_t stripes = 0;
  for_group(dims, [&]<typename IO, int V, int TPL, int NV, int GATE>() {
    const Cover c = bwd_cover<V, TPL, NV>(dims);
    stripes = c.stripes;
    p.gpb = static_cast<int32_t>(c.gpb), p.rpb = static_cast<int32_t>(c.rpb);
    hipLaunchKernelGGL((group_bwd_kernel<IO, V, TPL, NV, GATE>),
                       dim3(static_cast<unsigned>(c.columns), static_cast<unsigned>(c.stripes)), dim3(block_of<TPL>), 0,
                       s, p);
  });
  if (launched() != SSM_OK) return SSM_ERR_HIP;
  launch_reduce(p.ws, stripes, (p.with_bias ? 2 : 1) * nd, GroupGrads{io->dweight, io->dbias, nd}, s);
  return launched();
}

}  // extern "C"
