// The short causal convolution in front of the scan, for MI355X (gfx950):
// forward, backward, and one step on a cache.
//
// For every batch row b, channel d and step t < valid_len[b], with W taps:
//
//     p[t] = bias[d] + sum_k w[d,k] * xs[t - (W-1) + k],   y[t] = p or p * sigmoid(p)
//
// xs is the row's input behind the W-1 inputs carried from before it (or
// zeros).  Each channel is its own convolution, so there is nothing for the
// matrix units: 2W operations on 2 elements moved, bound by memory.
//
// Backward, with g[t] = dy[t] * (dy/dp)(p[t]) and g = 0 outside [0, valid_len):
//
//     dxs[t] = sum_k w[k] * g[t + (W-1) - k],  dw[k] = sum_{b,t} g[t] * xs[t - (W-1) + k],  dbias = sum_{b,t} g[t]
//
// Layout: dim is fastest, so a lane owns a few adjacent channels and a chunk of
// steps, the last W-1 inputs in registers as it goes; lanes of a wave take
// adjacent channels.  Chunks are short and all their inputs are in flight at
// once, so workgroups advance through memory side by side, and what neighbours
// share (the W-1 inputs around a chunk) is in L2 when it is read again.  Long
// chunks with a few loads ahead were slower: 53 us forward and 57 backward for
// the sizes below, the backward fetching 16 % over its inputs (now 4 %).
//
// Measured (copy of 1 GiB: 5.3 TB/s): forward of 16 rows of up to 8192 steps x
// 512 channels, bf16, lengths uniform: 29.7 us, 6.8 TB/s of what it has to move
// (the inputs partly from the 256 MiB cache).  Backward of 8 x 4096 x 1024 bf16,
// W = 4, silu: 49.6 us, 4.1 TB/s (in a kernel trace 46.1 and 4.7 for the second
// pass): the vector units are busy two thirds of it (26 operations a step and
// channel, 16/13 of the g's), and 16 rows of lengths uniform up to 4096 take
// 70.5; fp32 of half the elements moves 4.6 TB/s.  2 x 256 x 64 fp32: 3.8 us
// forward; 3 x 1021 x 200: 8.8 us backward.  One token of 256 of 512 slots x
// 2048: 4.1 us into another cache, 4.6 in place with eight caches in turn; of
// one row 2.6.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "ssm_block.h"

namespace {

// Channels of a lane: 16 bytes of fp32, 8 of bf16 (16 there cost twice the
// registers and lost 10 %); one where dim is smaller than that.
constexpr int kVec = 4;

// The first channel of a lane.  Where dim is no multiple of V the last lane
// starts early and shares channels with its neighbour: both compute and store
// the same values, and no lane is partly filled.  Not for a cache in place,
// where a value must be written once.
template <int V>
__device__ __forceinline__ int64_t first_channel(int64_t vec, int64_t nd) {
  const int64_t d = vec * V, last = nd - V;
  return d < last ? d : last;
}

// The carried inputs of a row, (W-1) * dim, are counted in 32 bits.
constexpr int64_t kMaxConvDim = 1 << 29;

struct ConvParams {
  const void* x;
  const float* w;
  const float* bias;
  const int32_t* valid_len;
  const void* conv0;
  void* y;
  void* conv_last;
  int64_t x_bs, x_ts, y_bs, y_ts;
  int64_t L;
  uint32_t n_chunks, items, n_vec;
  int32_t nd;
};

struct ConvBwdParams {
  const void* x;
  const float* w;
  const float* bias;
  const int32_t* valid_len;
  const void* conv0;
  const void* dy;
  const void* dconv_last;
  void* dx;
  void* dconv0;
  float* ws;
  int64_t x_bs, x_ts, dy_bs, dy_ts, dx_bs, dx_ts;
  int64_t L;
  uint32_t n_groups, n_tiles;
  int32_t nd, n_vec, M, log2_cx;
};

struct ConvStepParams {
  const void* x;
  const float* w;
  const float* bias;
  const int32_t* slots;
  const void* conv0;
  void* conv_last;
  void* y;
  int64_t x_rs, y_rs, n_slots;
  int32_t nd, n_vec;
};

__device__ __forceinline__ int64_t row_len(const int32_t* valid_len, int64_t b, int64_t L) {
  if (valid_len == nullptr) return L;
  const int64_t n = valid_len[b];
  return n < 0 ? 0 : (n > L ? L : n);
}

template <int W, int V>
struct Taps {
  float w[W][V];
  float bias[V];
  // n < V: the channels from the n-th on are zero
  __device__ __forceinline__ void load(const float* wp, const float* bp, int64_t d, int n = V) {
    // V channels' taps are adjacent
    float f[V * W];
    load_n<float, V * W>(wp + d * W, n * W, f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int k = 0; k < W; ++k) w[k][i] = f[i * W + k];
    }
    if (bp != nullptr) {
      load_n<float, V>(bp + d, n, bias);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) bias[i] = 0.0f;
    }
  }
  // p from the W inputs that end with this step's
  __device__ __forceinline__ void apply(const float (&xs)[W][V], float (&p)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] = bias[i];
#pragma unroll
      for (int k = 0; k < W; ++k) p[i] = __builtin_fmaf(w[k][i], xs[k][i], p[i]);
    }
  }
};

template <int W, int V>
__device__ __forceinline__ void shift(float (&xs)[W][V]) {
#pragma unroll
  for (int k = 0; k + 1 < W; ++k) {
#pragma unroll
    for (int i = 0; i < V; ++i) xs[k][i] = xs[k + 1][i];
  }
}

// The input of step t (t >= -(W-1)) of a row; zeros where nothing is carried.
template <typename IO, int W, int V>
__device__ __forceinline__ void input_at(const IO* x, const IO* conv0, int64_t t, int64_t x_ts, int64_t nd,
                                         float (&o)[V]) {
  if (t >= 0) {
    VecIO<IO>::load(x + t * x_ts, o);
  } else if (conv0 != nullptr) {
    VecIO<IO>::load(conv0 + (W - 1 + t) * nd, o);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = 0.0f;
  }
}

// ---- forward ---------------------------------------------------------------

// One lane: T steps of V channels.  Chunks, not channels, run over the grid's
// slow index, so that a workgroup's lanes cover whole rows where dim allows.
// y is stored past the caches, which leaves them to the inputs: 36.4 -> 29.7 us
// for 16 x 8192 x 512 ragged bf16, and with the copy that writes x and the
// operator that reads y around it 205 -> 195 us (full rows; 8 x 4096 x 1024: 99.4
// -> 97.2).  The same in the backward and the norms was no gain, or a loss with
// what reads their outputs (norm and reader at 32768 x 2048: 192 -> 206 us).
template <typename IO, int V, int W, bool SILU, int T>
__global__ __launch_bounds__(256) void conv_fwd_kernel(const ConvParams prm) {
  // a launch has fewer than 2^32 work-items
  const uint32_t item = xcd_run(blockIdx.x, gridDim.x) * 256 + threadIdx.x;
  if (item >= prm.items) return;
  const uint32_t row = item / prm.n_vec;
  const int64_t d = first_channel<V>(item - row * prm.n_vec, prm.nd);
  const uint32_t batch = row / prm.n_chunks;
  const int64_t b = batch, c0 = static_cast<int64_t>(row - batch * prm.n_chunks) * T;
  const int64_t len = row_len(prm.valid_len, b, prm.L);
  const IO* x = static_cast<const IO*>(prm.x) + b * prm.x_bs + d;
  const IO* conv0 = prm.conv0 == nullptr ? nullptr : static_cast<const IO*>(prm.conv0) + b * (W - 1) * prm.nd + d;
  IO* y = static_cast<IO*>(prm.y) + b * prm.y_bs + d;

  const int64_t c1 = c0 + T < prm.L ? c0 + T : prm.L;
  const int64_t v1 = c1 < len ? c1 : len;
  if (v1 > c0) {
    // The chunk's inputs are all in flight at once; those past its valid
    // steps repeat its last.
    RawVec<IO, V> in[T];
    const IO* xp = x + c0 * prm.x_ts;
    const int valid = static_cast<int>(v1 - c0);
#pragma unroll
    for (int u = 0; u < T; ++u) in[u].load(xp + (u < valid ? u : valid - 1) * prm.x_ts);
    Taps<W, V> taps;
    taps.load(prm.w, prm.bias, d);
    float xs[W][V];
#pragma unroll
    for (int k = 0; k + 1 < W; ++k) input_at<IO, W, V>(x, conv0, c0 - (W - 1) + k, prm.x_ts, prm.nd, xs[k]);
    IO* yp = y + c0 * prm.y_ts;
    const auto step = [&](int u) {
      in[u].unpack(xs[W - 1]);
      float p[V];
      taps.apply(xs, p);
      if constexpr (SILU) {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] *= sigmoid_for<IO>(p[i]);
      }
      VecIO<IO>::stream(yp + u * prm.y_ts, p);
      shift<W, V>(xs);
    };
    if (valid == T) {
#pragma unroll
      for (int u = 0; u < T; ++u) step(u);
    } else {
#pragma unroll
      for (int u = 0; u < T; ++u)
        if (u < valid) step(u);
    }
  }
  const float zero[V] = {};
  for (int64_t t = v1 > c0 ? v1 : c0; t < c1; ++t) VecIO<IO>::stream(y + t * prm.y_ts, zero);

  // The row's last W-1 inputs, by the lanes of its first chunk.
  if (c0 == 0 && prm.conv_last != nullptr) {
    IO* last = static_cast<IO*>(prm.conv_last) + b * (W - 1) * prm.nd + d;
#pragma unroll
    for (int k = 0; k + 1 < W; ++k) {
      float v[V];
      input_at<IO, W, V>(x, conv0, len - (W - 1) + k, prm.x_ts, prm.nd, v);
      VecIO<IO>::store(last + k * prm.nd, v);
    }
  }
}

// ---- backward --------------------------------------------------------------

// One lane: chunks of T steps of V channels, all in flight at once, and the
// gradients g of the W-1 steps behind each, which its last dxs need (computed
// twice, once by either chunk).  A workgroup's ty chunks are adjacent, and it
// takes M such runs one after the other, so what chunks share is read at about
// the same time.  The weights' sums join in LDS at the end; each workgroup
// leaves W+1 rows of sums.
//
// 13 steps, us for 8 x 4096 x 1024 bf16 / 16 ragged rows of them / 3 x 1021 x 200
// fp32: 49.9 / 70.7 / 8.6; 9 steps 51.3 / 66.2 / 7.8, 16 steps 52.4 / 66.1 / 9.2, 21
// steps 53.0 / 70.6 / 10.1.  Two channels a lane: with four, 71.8 / 87.6 / 9.6.
constexpr int kBwdChunk = 13;
constexpr int kBwdVec = 2;

template <typename IO, int V, int W, bool SILU>
__global__ __launch_bounds__(256) void conv_bwd_kernel(const ConvBwdParams prm) {
  constexpr int T = kBwdChunk, H = W - 1;
  const int shift_x = prm.log2_cx, cx = 1 << shift_x, ty = 256 >> shift_x;
  const int lane = threadIdx.x & (cx - 1), sub = threadIdx.x >> shift_x;
  const uint32_t block = xcd_run(blockIdx.x, gridDim.x);
  const uint32_t part = block / prm.n_tiles, tile = block - part * prm.n_tiles;
  const int64_t vec = static_cast<int64_t>(tile) * cx + lane;
  const uint32_t batch = part / prm.n_groups, group = part - batch * prm.n_groups;
  const int64_t b = batch;
  const int64_t d = first_channel<V>(vec, prm.nd);
  const int64_t len = row_len(prm.valid_len, b, prm.L);
  float dw[W + 1][V] = {};

  if (vec < prm.n_vec) {
    const IO* x = static_cast<const IO*>(prm.x) + b * prm.x_bs + d;
    const IO* dy = static_cast<const IO*>(prm.dy) + b * prm.dy_bs + d;
    IO* dx = static_cast<IO*>(prm.dx) + b * prm.dx_bs + d;
    const int64_t edge = b * H * prm.nd + d;
    const IO* conv0 = prm.conv0 == nullptr ? nullptr : static_cast<const IO*>(prm.conv0) + edge;
    const IO* dlast = prm.dconv_last == nullptr ? nullptr : static_cast<const IO*>(prm.dconv_last) + edge;
    IO* d0 = prm.dconv0 == nullptr ? nullptr : static_cast<IO*>(prm.dconv0) + edge;
    Taps<W, V> taps;
    taps.load(prm.w, prm.bias, d);

    // EDGE: the row's first chunk, or one that reaches past its valid steps.
    const auto chunk = [&]<bool EDGE>(int64_t c0) {
      RawVec<IO, V> xr[T + 2 * H], gr[T + H];
      const IO* xp = x + (c0 - H) * prm.x_ts;
      const IO* gp = dy + c0 * prm.dy_ts;
      IO* op = dx + c0 * prm.dx_ts;
#pragma unroll
      for (int u = 0; u < T + 2 * H; ++u) {
        if constexpr (EDGE) {
          const int64_t t = c0 - H + u;
          xr[u] = {};
          if (t < 0) {
            if (conv0 != nullptr) xr[u].load(conv0 + (H + t) * prm.nd);
          } else if (t < len) {
            xr[u].load(xp + u * prm.x_ts);
          }
        } else {
          xr[u].load(xp + u * prm.x_ts);
        }
      }
#pragma unroll
      for (int u = 0; u < T + H; ++u) {
        if constexpr (EDGE) {
          gr[u] = {};
          if (c0 + u < len) gr[u].load(gp + u * prm.dy_ts);
        } else {
          gr[u].load(gp + u * prm.dy_ts);
        }
      }
      float xs[W][V], g[W][V] = {};
#pragma unroll
      for (int k = 0; k < H; ++k) xr[k].unpack(xs[k]);
#pragma unroll
      for (int j = 0; j < T + H; ++j) {
        // step t = c0 + j gives g[t] (0 past the row's end), and with it dxs
        // of step t - (W-1)
        xr[j + H].unpack(xs[H]);
        gr[j].unpack(g[H]);
        if constexpr (SILU) {
          float p[V];
          taps.apply(xs, p);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float s = sigmoid_for<IO>(p[i]);
            g[H][i] *= s * __builtin_fmaf(p[i], 1.0f - s, 1.0f);
          }
          if (EDGE && c0 + j >= len) {
#pragma unroll
            for (int i = 0; i < V; ++i) g[H][i] = 0.0f;
          }
        }
        if (j < T) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int k = 0; k < W; ++k) {
              // past the row's end g = 0, but xs may still hold an infinity or NaN (a
              // select: with a branch around the sums the registers fall to four
              // waves' and whole calls, CPU time included, of full rows take 55.2 us
              // for 53.3, of ragged ones 65 for 69)
              const float in = EDGE && c0 + j >= len ? 0.0f : xs[k][i];
              dw[k][i] = __builtin_fmaf(g[H][i], in, dw[k][i]);
            }
            dw[W][i] += g[H][i];
          }
        }
        if (j >= H || (EDGE && c0 == 0)) {
          float v[V];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            v[i] = 0.0f;  // the sum of products with g = 0 is +0 whatever their signs
#pragma unroll
            for (int k = 0; k < W; ++k) v[i] = __builtin_fmaf(taps.w[k][i], g[H - k][i], v[i]);
          }
          if constexpr (EDGE) {
            const int64_t o = c0 + j - H;
            if (dlast != nullptr && o < len && o >= len - H) {
              float e[V];
              VecIO<IO>::load(dlast + (o - len + H) * prm.nd, e);
#pragma unroll
              for (int i = 0; i < V; ++i) v[i] += e[i];
            }
            if (o < 0) {
              if (d0 != nullptr) VecIO<IO>::store(d0 + (o + H) * prm.nd, v);
            } else if (o < len) {
              VecIO<IO>::store(op + (j - H) * prm.dx_ts, v);
            }
          } else {
            VecIO<IO>::store(op + (j - H) * prm.dx_ts, v);
          }
        }
        shift<W, V>(xs);
        shift<W, V>(g);
      }
    };
    for (int m = 0; m < prm.M; ++m) {
      const int64_t c0 = ((static_cast<int64_t>(group) * prm.M + m) * ty + sub) * T;
      if (c0 > 0 && c0 + T + H <= len) {
        chunk.template operator()<false>(c0);
      } else {
        if (c0 == 0 || c0 < len) chunk.template operator()<true>(c0);
        // +0 past the row's end (a sum of taps times g = 0 would be NaN for an infinite one)
        const float zero[V] = {};
        const int64_t c1 = c0 + T < prm.L ? c0 + T : prm.L;
        for (int64_t t = c0 < len ? len : c0; t < c1; ++t) VecIO<IO>::store(dx + t * prm.dx_ts, zero);
      }
    }
  }

  // Join the workgroup's ty chunks.
  __shared__ float lds[(W + 1) * V * 256];
#pragma unroll
  for (int k = 0; k <= W; ++k) {
#pragma unroll
    for (int i = 0; i < V; ++i) lds[(k * V + i) * 256 + threadIdx.x] = dw[k][i];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < (W + 1) * cx * V; e += 256) {
    const int k = e / V >> shift_x, c = e - (k * V << shift_x);
    const int64_t v = static_cast<int64_t>(tile) * cx + c / V, ch = v * V + c % V;
    if (ch >= prm.nd) continue;
    const int i = static_cast<int>(ch - first_channel<V>(v, prm.nd));  // of lane c / V
    float sum = 0.0f;
    for (int r = 0; r < ty; ++r) sum += lds[(k * V + i) * 256 + r * cx + c / V];
    prm.ws[(static_cast<int64_t>(part) * (W + 1) + k) * prm.nd + ch] = sum;
  }
}

// Columns of the partial sums, [W+1][dim], to dweight [dim][W] and dbias.
struct ConvGrads {
  float* dw;
  float* db;
  int64_t nd;
  int32_t W;
  __device__ __forceinline__ void operator()(int64_t col, float v) const {
    const int64_t k = col / nd, d = col - k * nd;
    if (k < W)
      dw[d * W + k] = v;
    else if (db != nullptr)
      db[d] = v;
  }
};

__global__ void conv_zero_kernel(float* p, int64_t n) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) p[i] = 0.0f;
}

// ---- one step --------------------------------------------------------------

// One workgroup: 256 lanes' channels of one batch row.
template <typename IO, int W, bool SILU>
__global__ __launch_bounds__(256) void conv_step_kernel(const ConvStepParams prm) {
  constexpr int V = kVec;
  const int32_t b = blockIdx.y;
  const int64_t vec = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t d = vec * V;
  const int n = vec >= prm.n_vec ? 0 : (prm.nd - d < V ? static_cast<int>(prm.nd - d) : V);
  const int32_t slot[1] = {prm.slots == nullptr ? b : prm.slots[b]};
  bool active[1];
  step_rows_active<1>(prm.slots, b, b + 1, slot, prm.n_slots, active);
  if (n == 0) return;
  IO* y = static_cast<IO*>(prm.y) + b * prm.y_rs + d;
  float p[V] = {};
  if (active[0]) {
    const int64_t at = static_cast<int64_t>(slot[0]) * (W - 1) * prm.nd + d;
    const IO* from = static_cast<const IO*>(prm.conv0) + at;
    IO* to = static_cast<IO*>(prm.conv_last) + at;
    float xs[W][V];
#pragma unroll
    for (int k = 0; k + 1 < W; ++k) load_n<IO, V>(from + k * prm.nd, n, xs[k]);
    load_n<IO, V>(static_cast<const IO*>(prm.x) + b * prm.x_rs + d, n, xs[W - 1]);
    Taps<W, V> taps;
    taps.load(prm.w, prm.bias, d, n);
    taps.apply(xs, p);
    if constexpr (SILU) {
#pragma unroll
      for (int i = 0; i < V; ++i) p[i] *= sigmoid_for<IO>(p[i]);
    }
#pragma unroll
    for (int k = 0; k + 1 < W; ++k) store_n<IO, V>(to + k * prm.nd, n, xs[k + 1]);
  }
  store_n<IO, V>(y, n, p);
}

// ---- host ------------------------------------------------------------------

// Calls f.template operator()<IO, W, SILU>() for these dims.
template <typename F>
void for_conv(const ssm_conv_dims* dims, const F& f) {
  const auto width = [&]<typename IO, bool SILU>() {
    switch (dims->width) {
      case 2:
        f.template operator()<IO, 2, SILU>();
        break;
      case 3:
        f.template operator()<IO, 3, SILU>();
        break;
      default:
        f.template operator()<IO, 4, SILU>();
    }
  };
  if (dims->io_dtype == SSM_IO_BF16) {
    if (dims->silu)
      width.template operator()<uint16_t, true>();
    else
      width.template operator()<uint16_t, false>();
  } else {
    if (dims->silu)
      width.template operator()<float, true>();
    else
      width.template operator()<float, false>();
  }
}

// Channels of a lane of the sequence kernels.
int64_t vec_of(int64_t nd) { return nd < kVec ? 1 : kVec; }

int check_conv_dims(const ssm_conv_dims* dims) {
  if (dims == nullptr) return SSM_ERR_INVALID_ARG;
  if (dims->batch < 0 || dims->seqlen < 0 || dims->dim < 0) return SSM_ERR_INVALID_ARG;
  if (dims->io_dtype != SSM_IO_F32 && dims->io_dtype != SSM_IO_BF16) return SSM_ERR_INVALID_ARG;
  if (dims->silu != 0 && dims->silu != 1) return SSM_ERR_INVALID_ARG;
  if (dims->width < 2 || dims->width > 4) return SSM_ERR_UNSUPPORTED;
  if (dims->batch > kMaxSize || dims->seqlen > kMaxSize || dims->dim >= kMaxConvDim) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

// Steps a lane of the forward walks: long chunks read fewer of the inputs in
// front of them twice, short ones fill the GPU sooner and answer sooner.  us at
// 4 / 12 steps: fp32 2 x 256 steps x 64 channels 3.3 / 5.0, bf16 2 x 1000 x 512 3.7 /
// 4.5, 2 x 2000 x 1024 6.4 / 6.4, 4 x 2000 x 1024 10.1 / 8.7, 8 x 4096 x 1024 30.7 /
// 23.9.
constexpr int kShortChunk = 4, kLongChunk = 12;
constexpr int64_t kShortWork = 3 << 19;  // (step, lane) pairs

// The backward's tiling: 2^log2_cx lanes over the channels and ty = 256 /
// 2^log2_cx chunks a workgroup, M times.
struct BwdTiling {
  int64_t V, n_vec, ty, n_tiles, n_groups, parts;
  int log2_cx, M;
};

constexpr int64_t kBwdBlocks = 1200;

BwdTiling bwd_tiling(const ssm_conv_dims* dims) {
  BwdTiling t;
  t.V = dims->dim < kBwdVec ? 1 : kBwdVec;
  t.n_vec = (dims->dim + t.V - 1) / t.V;
  t.log2_cx = 6;
  while (t.log2_cx > 0 && (1 << (t.log2_cx - 1)) >= t.n_vec) --t.log2_cx;
  const int64_t cx = 1 << t.log2_cx;
  t.ty = 256 / cx;
  t.n_tiles = (t.n_vec + cx - 1) / cx;
  const int64_t run = kBwdChunk * t.ty, runs = dims->seqlen > 0 ? (dims->seqlen + run - 1) / run : 1;
  // Fewer, longer workgroups leave fewer sums; at least kBwdBlocks of them
  // fill the GPU.  us at M = 1 / 2 / 4 / 8: bf16 8 x 4096 x 1024 - / 51.6 / 49.9 /
  // 55.6, fp32 8 x 2048 x 1024 44.4 / 44.3 / 46.7 / -, and against the rule bf16 16
  // ragged rows of 4096 x 1024 - / - / 65.5 / 70.7.  A workgroup stays within one
  // batch row, so there is one set of sums a row at least, however short the
  // rows are, and M ends at a row's runs.
  const __int128 all = static_cast<__int128>(dims->batch) * runs * t.n_tiles;
  t.M = 1;
  while (t.M < 8 && t.M < runs && all >= (t.M + 1) * kBwdBlocks) ++t.M;
  t.n_groups = (runs + t.M - 1) / t.M;
  t.parts = dims->batch * t.n_groups;
  return t;
}

}  // namespace

extern "C" {

int ssm_causal_conv_fwd(ssm_scan_t handle, const ssm_conv_dims* dims, const ssm_conv_fwd_io* io, void* stream) {
  const int bad = check_conv_dims(dims);
  if (bad != SSM_OK) return bad;
  if (io == nullptr) return SSM_ERR_INVALID_ARG;
  const int64_t nb = dims->batch, L = dims->seqlen, nd = dims->dim, W = dims->width;
  const int64_t e = dims->io_dtype == SSM_IO_BF16 ? 2 : 4;
  const bool empty = nb == 0 || nd == 0;
  if (!empty) {
    if (io->weight == nullptr) return SSM_ERR_INVALID_ARG;
    if (L > 0 && (io->x == nullptr || io->y == nullptr)) return SSM_ERR_INVALID_ARG;
    const int64_t bx = span_bytes(nb, io->x_batch_stride, L, io->x_time_stride, nd, e);
    const int64_t by = span_bytes(nb, io->y_batch_stride, L, io->y_time_stride, nd, e);
    if (bx < 0 || by < 0 || !rows_disjoint(nb, io->y_batch_stride, L, io->y_time_stride, nd))
      return SSM_ERR_INVALID_ARG;
    if (!aligned(io->x, e) || !aligned(io->y, e) || !aligned(io->conv0, e) || !aligned(io->conv_last, e) ||
        !aligned(io->weight, 4) || !aligned(io->bias, 4) || !aligned(io->valid_len, 4))
      return SSM_ERR_UNSUPPORTED;
    const int64_t bc = nb * (W - 1) * nd * e;
    const Range in[] = {{io->x, bx},       {io->weight, nd * W * 4}, {io->bias, nd * 4},
                        {io->valid_len, nb * 4}, {io->conv0, bc}};
    const Range out[] = {{io->y, by}, {io->conv_last, bc}};
    if (any_overlap(in, out)) return SSM_ERR_ALIAS;
  }
  const int rc = check_handle(handle);
  if (rc != SSM_OK || empty) return rc;
  if (L == 0 && io->conv_last == nullptr) return SSM_OK;

  ConvParams p;
  p.x = io->x, p.w = io->weight, p.bias = io->bias, p.valid_len = io->valid_len, p.conv0 = io->conv0;
  p.y = io->y, p.conv_last = io->conv_last;
  p.x_bs = io->x_batch_stride, p.x_ts = io->x_time_stride, p.y_bs = io->y_batch_stride, p.y_ts = io->y_time_stride;
  const int64_t V = vec_of(nd);
  p.L = L, p.nd = static_cast<int32_t>(nd);
  const int64_t n_vec = (nd + V - 1) / V;
  const bool brief = V == 1 || static_cast<__int128>(nb) * L * n_vec <= kShortWork;
  const int64_t T = brief ? kShortChunk : kLongChunk, n_chunks = L > 0 ? (L + T - 1) / T : 1;
  const __int128 items = static_cast<__int128>(nb) * n_chunks * n_vec;
  if (items > 0xffffff00) return SSM_ERR_UNSUPPORTED;
  p.n_vec = static_cast<uint32_t>(n_vec), p.n_chunks = static_cast<uint32_t>(n_chunks);
  p.items = static_cast<uint32_t>(items);
  const int64_t blocks = (static_cast<int64_t>(items) + 255) / 256;
  for_conv(dims, [&]<typename IO, int TAPS, bool SILU>() {
    const auto kernel = V == 1  ? conv_fwd_kernel<IO, 1, TAPS, SILU, kShortChunk>
                        : brief ? conv_fwd_kernel<IO, kVec, TAPS, SILU, kShortChunk>
                                : conv_fwd_kernel<IO, kVec, TAPS, SILU, kLongChunk>;
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, static_cast<hipStream_t>(stream), p);
  });
  return launched();
}

int64_t ssm_causal_conv_bwd_workspace_bytes(const ssm_conv_dims* dims) {
  if (check_conv_dims(dims) != SSM_OK) return -1;
  const __int128 n = static_cast<__int128>(bwd_tiling(dims).parts) * (dims->width + 1) * dims->dim * 4;
  return n < (static_cast<__int128>(1) << 62) ? static_cast<int64_t>(n) : -1;
}

int ssm_causal_conv_bwd(ssm_scan_t handle, const ssm_conv_dims* dims, const ssm_conv_bwd_io* io, void* stream) {
  const int bad = check_conv_dims(dims);
  if (bad != SSM_OK) return bad;
  if (io == nullptr) return SSM_ERR_INVALID_ARG;
  const int64_t nb = dims->batch, L = dims->seqlen, nd = dims->dim, W = dims->width;
  const int64_t e = dims->io_dtype == SSM_IO_BF16 ? 2 : 4;
  const int64_t need = ssm_causal_conv_bwd_workspace_bytes(dims);
  if (need < 0) return SSM_ERR_UNSUPPORTED;
  if (io->workspace_bytes < 0) return SSM_ERR_INVALID_ARG;
  if (nd > 0) {
    if (io->weight == nullptr || io->dweight == nullptr) return SSM_ERR_INVALID_ARG;
    if (nb > 0 && L > 0 && (io->x == nullptr || io->dy == nullptr || io->dx == nullptr)) return SSM_ERR_INVALID_ARG;
    if (nb > 0 && (io->workspace == nullptr || io->workspace_bytes < need)) return SSM_ERR_INVALID_ARG;
    const int64_t bx = span_bytes(nb, io->x_batch_stride, L, io->x_time_stride, nd, e);
    const int64_t bdy = span_bytes(nb, io->dy_batch_stride, L, io->dy_time_stride, nd, e);
    const int64_t bdx = span_bytes(nb, io->dx_batch_stride, L, io->dx_time_stride, nd, e);
    if (bx < 0 || bdy < 0 || bdx < 0 || !rows_disjoint(nb, io->dx_batch_stride, L, io->dx_time_stride, nd))
      return SSM_ERR_INVALID_ARG;
    if (!aligned(io->x, e) || !aligned(io->dy, e) || !aligned(io->dx, e) || !aligned(io->conv0, e) ||
        !aligned(io->dconv_last, e) || !aligned(io->dconv0, e) || !aligned(io->weight, 4) || !aligned(io->bias, 4) ||
        !aligned(io->valid_len, 4) || !aligned(io->dweight, 4) || !aligned(io->dbias, 4) || !aligned(io->workspace, 4))
      return SSM_ERR_UNSUPPORTED;
    const int64_t bc = nb * (W - 1) * nd * e;
    const Range in[] = {{io->x, bx},       {io->dy, bdy},    {io->weight, nd * W * 4}, {io->bias, nd * 4},
                        {io->valid_len, nb * 4}, {io->conv0, bc}, {io->dconv_last, bc}};
    const Range out[] = {{io->dx, bdx},     {io->dweight, nd * W * 4}, {io->dbias, nd * 4},
                         {io->dconv0, bc}, {io->workspace, io->workspace_bytes}};
    if (any_overlap(in, out)) return SSM_ERR_ALIAS;
  }
  const int rc = check_handle(handle);
  if (rc != SSM_OK || nd == 0) return rc;

  hipStream_t s = static_cast<hipStream_t>(stream);
  if (nb == 0) {  // sums over nothing
    if (!grid_fits((nd * W + 255) / 256, 256)) return SSM_ERR_UNSUPPORTED;
    hipLaunchKernelGGL(conv_zero_kernel, dim3(static_cast<unsigned>((nd * W + 255) / 256)), dim3(256), 0, s,
                       io->dweight, nd * W);
    if (io->dbias != nullptr)
      hipLaunchKernelGGL(conv_zero_kernel, dim3(static_cast<unsigned>((nd + 255) / 256)), dim3(256), 0, s, io->dbias,
                         nd);
    return launched();
  }
  const BwdTiling t = bwd_tiling(dims);
  ConvBwdParams p;
  p.x = io->x, p.w = io->weight, p.bias = io->bias, p.valid_len = io->valid_len, p.conv0 = io->conv0;
  p.dy = io->dy, p.dconv_last = io->dconv_last, p.dx = io->dx, p.dconv0 = io->dconv0;
  p.ws = static_cast<float*>(io->workspace);
  p.x_bs = io->x_batch_stride, p.x_ts = io->x_time_stride;
  p.dy_bs = io->dy_batch_stride, p.dy_ts = io->dy_time_stride;
  p.dx_bs = io->dx_batch_stride, p.dx_ts = io->dx_time_stride;
  p.L = L, p.n_groups = static_cast<uint32_t>(t.n_groups), p.n_tiles = static_cast<uint32_t>(t.n_tiles);
  p.nd = static_cast<int32_t>(nd), p.n_vec = static_cast<int32_t>(t.n_vec), p.M = t.M;
  p.log2_cx = t.log2_cx;
  const __int128 all = static_cast<__int128>(t.parts) * t.n_tiles;
  if (all > kMaxSize) return SSM_ERR_UNSUPPORTED;
  const int64_t blocks = static_cast<int64_t>(all);
  const int64_t cols = (W + 1) * nd;
  if (!grid_fits(blocks, 256) || !reduce_fits(cols)) return SSM_ERR_UNSUPPORTED;
  for_conv(dims, [&]<typename IO, int TAPS, bool SILU>() {
    const auto kernel = t.V == 1 ? conv_bwd_kernel<IO, 1, TAPS, SILU> : conv_bwd_kernel<IO, kBwdVec, TAPS, SILU>;
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, p);
  });
  if (launched() != SSM_OK) return SSM_ERR_HIP;
  launch_reduce(p.ws, t.parts, cols, ConvGrads{io->dweight, io->dbias, nd, static_cast<int32_t>(W)}, s);
  return launched();
}

int ssm_causal_conv_step(ssm_scan_t handle, const ssm_conv_dims* dims, const ssm_conv_step_io* io, void* stream) {
  const int bad = check_conv_dims(dims);
  if (bad != SSM_OK) return bad;
  if (io == nullptr || dims->seqlen != 1 || io->n_slots < 0) return SSM_ERR_INVALID_ARG;
  const int64_t nb = dims->batch, nd = dims->dim, W = dims->width;
  const int64_t e = dims->io_dtype == SSM_IO_BF16 ? 2 : 4;
  const int64_t rows = io->slots == nullptr ? nb : io->n_slots;
  if (nb > 65535 || rows > kMaxSize) return SSM_ERR_UNSUPPORTED;
  const bool empty = nb == 0 || nd == 0;
  if (!empty) {
    if (io->x == nullptr || io->y == nullptr || io->weight == nullptr ||
        (rows > 0 && (io->conv0 == nullptr || io->conv_last == nullptr)))
      return SSM_ERR_INVALID_ARG;
    const int64_t bx = span_bytes(nb, io->x_row_stride, 1, 0, nd, e);
    const int64_t by = span_bytes(nb, io->y_row_stride, 1, 0, nd, e);
    const int64_t bc = span_bytes(rows, (W - 1) * nd, 1, 0, (W - 1) * nd, e);
    if (bx < 0 || by < 0 || !rows_disjoint(nb, io->y_row_stride, 1, 0, nd)) return SSM_ERR_INVALID_ARG;
    if (bc < 0) return SSM_ERR_UNSUPPORTED;
    if (!aligned(io->x, e) || !aligned(io->y, e) || !aligned(io->conv0, e) || !aligned(io->conv_last, e) ||
        !aligned(io->weight, 4) || !aligned(io->bias, 4) || !aligned(io->slots, 4))
      return SSM_ERR_UNSUPPORTED;
    // the cache in place is one range: conv0 is then left out of the inputs
    const Range in[] = {{io->x, bx},       {io->weight, nd * W * 4}, {io->bias, nd * 4},
                        {io->slots, nb * 4}, {io->conv0, io->conv0 == io->conv_last ? 0 : bc}};
    const Range out[] = {{io->y, by}, {io->conv_last, bc}};
    if (any_overlap(in, out)) return SSM_ERR_ALIAS;
  }
  const int rc = check_handle(handle);
  if (rc != SSM_OK || empty) return rc;

  ConvStepParams p;
  p.x = io->x, p.w = io->weight, p.bias = io->bias, p.slots = io->slots, p.conv0 = io->conv0;
  p.conv_last = io->conv_last, p.y = io->y, p.x_rs = io->x_row_stride, p.y_rs = io->y_row_stride, p.n_slots = rows;
  const int64_t V = kVec;
  p.nd = static_cast<int32_t>(nd), p.n_vec = static_cast<int32_t>((nd + V - 1) / V);
  const int64_t tiles = (p.n_vec + 255) / 256;
  if (!grid_fits(tiles, 256)) return SSM_ERR_UNSUPPORTED;
  for_conv(dims, [&]<typename IO, int TAPS, bool SILU>() {
    hipLaunchKernelGGL((conv_step_kernel<IO, TAPS, SILU>), dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(nb)),
                       dim3(256), 0, static_cast<hipStream_t>(stream), p);
  });
  return launched();
}

}  // extern "C"
