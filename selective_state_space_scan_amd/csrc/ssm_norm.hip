// Layer norm and RMS norm of the rows in front of a block, with the residual
// add, for MI355X (gfx950): forward and backward.
//
// Forward, for each row of n = dim values:
//
//     v = x + residual,  m = mean(v) (0 for RMS),  r = (mean((v - m)^2) + eps)^(-1/2),  y = (v - m) r w + b
//
// Backward, with xh = (v - m) r and g = dy w:
//
//     dv = r (g - mean(g) - xh mean(g xh)) + dresidual_out      (mean(g) is left out for RMS)
//     dw = sum over rows of dy xh,  db = sum over rows of dy
//
// About ten operations an element on 4 to 16 bytes: bound by memory.  A row is
// held in registers between its one read and its one write: eight elements a
// lane (16 beyond dim 8192, and forward for rows of bf16 without a residual
// stream), 64 to 1024 lanes a row (dim <= 16384).  The mean is subtracted before
// squares are summed, and the small sum of the differences corrects both it and
// the variance, so rows whose mean is far from zero lose nothing.
//
// Measured, 32768 rows x 1024 in bf16 with the residual stream in fp32 (a copy of
// 1 GiB: 5.3 TB/s): forward 74.7 us, 5.4 TB/s; backward 100.1 us, 5.4 TB/s (in a
// kernel trace 95.6 and 4.6 for the second pass).  24 rows x 1000 fp32 forward
// 2.8 us, 1021 x 600 backward 8.4 us (two dependent launches).
//
// Further from the bytes: narrow rows, which leave most of a wave's lanes idle
// (524288 x 64 bf16 forward, stream in bf16: 248 us, 1.1 TB/s); rows that end
// within a lane's elements, moved one by one there (32768 x 1001 bf16 forward 27.8
// us, x 1024 23.5); and the backward beyond dim 8192, whose 16 elements a lane
// spill 36 to 92 bytes of scratch a lane (2048 x 12288 bf16 66.4 us, 3.0 TB/s).

#include <hip/hip_runtime.h>

#include <cstdint>

#include "ssm_block.h"

namespace {

constexpr int64_t kMaxNormDim = 16384;
constexpr int kLaneElems = 16;

struct NormParams {
  const void* x;
  const void* residual;
  const float* w;
  const float* bias;
  const int32_t* valid_len;
  void* y;
  void* residual_out;
  float* mean;
  float* rstd;
  int64_t rows, L;
  int32_t nd, rms;
  float eps, inv_n;
};

struct NormBwdParams {
  const void* dy;
  const void* v;
  const float* w;
  const float* mean;
  const float* rstd;
  const int32_t* valid_len;
  const void* dresidual_out;
  void* dx;
  void* dresidual;
  float* ws;
  int64_t rows, L;
  int32_t nd, rms, with_bias;
  float inv_n;
};

// Sums of K values over a row's TPR lanes; every lane gets them.  A row wider
// than a wave joins its waves in LDS (called by the whole workgroup then).
template <int TPR, int K>
__device__ __forceinline__ void row_sums(float (&v)[K], float* lds) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = wave_sum(v[k]);
  if constexpr (TPR > 64) {
    constexpr int WPR = TPR / 64;
    const int wave = threadIdx.x / 64;
    __syncthreads();  // the values of the last sums have been read
    if (threadIdx.x % 64 == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) lds[wave * K + k] = v[k];
    }
    __syncthreads();
    const int first = wave / WPR * WPR;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = 0.0f;
      for (int w = 0; w < WPR; ++w) v[k] += lds[(first + w) * K + k];
    }
  }
}

__device__ __forceinline__ bool row_valid(const int32_t* valid_len, int64_t row, int64_t rows, int64_t L) {
  if (row >= rows) return false;
  if (valid_len == nullptr) return true;
  const int64_t b = row / L;
  return row - b * L < valid_len[b];
}

// One row: TPR lanes with NV pieces of V elements each; piece k of lane l is
// the row's piece k * TPR + l.
template <typename IO, typename RT, int TPR, int NV>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void norm_fwd_kernel(const NormParams prm) {
  constexpr int V = VecIO<IO>::kWide, BLOCK = TPR > 256 ? TPR : 256, RPB = BLOCK / TPR;
  __shared__ float lds[BLOCK / 64 * 2];
  const int lane = threadIdx.x % TPR;
  const int64_t row = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * RPB + threadIdx.x / TPR;
  const bool valid = row_valid(prm.valid_len, row, prm.rows, prm.L);
  const int64_t at = row * prm.nd;
  float v[NV][V];
  int n[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int d = (k * TPR + lane) * V;
    n[k] = d >= prm.nd ? 0 : (prm.nd - d < V ? prm.nd - d : V);
    const int m = valid ? n[k] : 0;
    load_n<IO, V>(static_cast<const IO*>(prm.x) + at + d, m, v[k]);
    if (prm.residual != nullptr) {
      float r[V];
      load_n<RT, V>(static_cast<const RT*>(prm.residual) + at + d, m, r);
#pragma unroll
      for (int i = 0; i < V; ++i) v[k][i] += r[i];
    }
    if (prm.residual_out != nullptr && row < prm.rows)
      store_n<RT, V>(static_cast<RT*>(prm.residual_out) + at + d, n[k], v[k]);
  }
  float mean = 0.0f;
  if (!prm.rms) {
    float s[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) s[0] += v[k][i];
    row_sums<TPR>(s, lds);
    mean = s[0] * prm.inv_n;
  }
  float s[2] = {0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      // elements past the row's end stay zero
      const float c = i < n[k] ? v[k][i] - mean : 0.0f;
      v[k][i] = c;
      s[0] += c;
      s[1] = __builtin_fmaf(c, c, s[1]);
    }
  row_sums<TPR>(s, lds);
  const float off = prm.rms ? 0.0f : s[0] * prm.inv_n;
  // far from zero a constant row's two terms agree but for their rounding
  float var = __builtin_fmaf(-off, off, s[1] * prm.inv_n);
  var = var < 0.0f ? 0.0f : var;
  const float rstd = 1.0f / __builtin_sqrtf(var + prm.eps);
  if (row >= prm.rows) return;
  if (lane == 0) {
    if (prm.mean != nullptr) prm.mean[row] = valid ? mean + off : 0.0f;
    if (prm.rstd != nullptr) prm.rstd[row] = valid ? rstd : 0.0f;
  }
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int d = (k * TPR + lane) * V;
    float w[V], o[V] = {};
    load_n<float, V>(prm.w + d, n[k], w);
    if (prm.bias != nullptr) load_n<float, V>(prm.bias + d, n[k], o);
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = valid ? __builtin_fmaf((v[k][i] - off) * rstd, w[i], o[i]) : 0.0f;
    store_n<IO, V>(static_cast<IO*>(prm.y) + at + d, n[k], o);
  }
}

// Workgroups walk the rows with a stride and keep their sums of dw and db in
// registers; each leaves one row of both for the second pass.
template <typename IO, typename RT, int TPR, int NV, bool BIAS>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void norm_bwd_kernel(const NormBwdParams prm) {
  constexpr int V = VecIO<IO>::kWide, BLOCK = TPR > 256 ? TPR : 256, RPB = BLOCK / TPR;
  __shared__ float lds[BLOCK / 64 * 2];
  __shared__ float join[RPB > 1 ? BLOCK * V : 1];
  const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  float w[NV][V], dw[NV][V] = {}, db[NV][V] = {};
  int n[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int d = (k * TPR + lane) * V;
    n[k] = d >= prm.nd ? 0 : (prm.nd - d < V ? prm.nd - d : V);
    load_n<float, V>(prm.w + d, n[k], w[k]);
  }
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * RPB; base < prm.rows;
       base += static_cast<int64_t>(gridDim.x) * RPB) {
    const int64_t row = base + sub;
    const bool valid = row_valid(prm.valid_len, row, prm.rows, prm.L);
    const int64_t at = row * prm.nd;
    const float mean = valid && !prm.rms ? prm.mean[row] : 0.0f;
    const float rstd = valid ? prm.rstd[row] : 0.0f;
    float xh[NV][V], g[NV][V];
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int d = (k * TPR + lane) * V;
      const int m = valid ? n[k] : 0;
      // past the row's end v = mean, so that h there is 0: from 0 it would be
      // -mean * rstd, which may leave fp32's range, and g h is then no number
      load_n<RT, V>(static_cast<const RT*>(prm.v) + at + d, m, xh[k], mean);
      load_n<IO, V>(static_cast<const IO*>(prm.dy) + at + d, m, g[k]);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        // an element past the row's end has g = 0 and h = 0, and a row that is
        // not valid has rstd = 0 on zeros: both add nothing
        const float h = (xh[k][i] - mean) * rstd;
        xh[k][i] = h;
        dw[k][i] = __builtin_fmaf(g[k][i], h, dw[k][i]);
        if constexpr (BIAS) db[k][i] += g[k][i];
        g[k][i] *= w[k][i];
        s[0] = __builtin_fmaf(g[k][i], h, s[0]);
        s[1] += g[k][i];
      }
    row_sums<TPR>(s, lds);
    const float along = s[0] * prm.inv_n, off = prm.rms ? 0.0f : s[1] * prm.inv_n;
    if (row < prm.rows) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int d = (k * TPR + lane) * V;
        float o[V] = {};
        if (prm.dresidual_out != nullptr)
          load_n<RT, V>(static_cast<const RT*>(prm.dresidual_out) + at + d, valid ? n[k] : 0, o);
#pragma unroll
        for (int i = 0; i < V; ++i)
          // a padded row is +0 whatever the weight (its g is 0 w: NaN for an infinite one)
          o[i] = valid ? __builtin_fmaf(g[k][i] - off - xh[k][i] * along, rstd, o[i]) : 0.0f;
        store_n<IO, V>(static_cast<IO*>(prm.dx) + at + d, n[k], o);
        if (prm.dresidual != nullptr) store_n<RT, V>(static_cast<RT*>(prm.dresidual) + at + d, n[k], o);
      }
    }
  }
  // One row of sums a workgroup: [dw | db].
  const int64_t cols = static_cast<int64_t>(BIAS ? 2 : 1) * prm.nd;
  float* out = prm.ws + blockIdx.x * cols;
#pragma unroll
  for (int q = 0; q < (BIAS ? 2 : 1); ++q) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int d = (k * TPR + lane) * V;
      float sum[V];
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] = q == 0 ? dw[k][i] : db[k][i];
      if constexpr (RPB > 1) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) join[i * BLOCK + threadIdx.x] = sum[i];
        __syncthreads();
        if (sub == 0) {
#pragma unroll
          for (int i = 0; i < V; ++i)
            for (int r = 1; r < RPB; ++r) sum[i] += join[i * BLOCK + r * TPR + lane];
        }
      }
      if (sub == 0) store_n<float, V>(out + q * prm.nd + d, n[k], sum);
    }
  }
}

struct NormGrads {
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

// ---- host ------------------------------------------------------------------

int check_norm_dims(const ssm_norm_dims* dims) {
  if (dims == nullptr || dims->batch < 0 || dims->seqlen < 0 || dims->dim < 0) return SSM_ERR_INVALID_ARG;
  if (dims->io_dtype != SSM_IO_F32 && dims->io_dtype != SSM_IO_BF16) return SSM_ERR_INVALID_ARG;
  if (dims->residual_dtype != SSM_IO_F32 && dims->residual_dtype != dims->io_dtype) return SSM_ERR_INVALID_ARG;
  if (dims->rms != 0 && dims->rms != 1) return SSM_ERR_INVALID_ARG;
  if (!(dims->eps > 0.0f && dims->eps < __builtin_inff())) return SSM_ERR_INVALID_ARG;
  if (dims->dim > kMaxNormDim || dims->batch > kMaxSize || dims->seqlen > kMaxSize) return SSM_ERR_UNSUPPORTED;
  // rows are counted in 64 bits; their elements stay within them
  if (static_cast<__int128>(dims->batch) * dims->seqlen * kMaxNormDim * 4 >= (static_cast<__int128>(1) << 62))
    return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

// Calls f.template operator()<IO, RT, TPR, NV>(): the fewest lanes a row that
// hold it at E elements each (16 where 1024 lanes would not), one piece a lane
// where a wave holds it so.
template <int E, typename IO, typename RT, typename F>
void for_row(int64_t nd, const F& f) {
  constexpr int V = VecIO<IO>::kWide;
  if (nd <= 64 * V)
    f.template operator()<IO, RT, 64, 1>();
  else if (nd <= 64 * 8)
    f.template operator()<IO, RT, 64, 8 / V>();
  else if (nd <= 64 * E)
    f.template operator()<IO, RT, 64, E / V>();
  else if (nd <= 128 * E)
    f.template operator()<IO, RT, 128, E / V>();
  else if (nd <= 256 * E)
    f.template operator()<IO, RT, 256, E / V>();
  else if (nd <= 512 * E)
    f.template operator()<IO, RT, 512, E / V>();
  else if (nd <= 1024 * E)
    f.template operator()<IO, RT, 1024, E / V>();
  else
    f.template operator()<IO, RT, 1024, kLaneElems / V>();
}

// Eight elements a lane: more waves of fewer registers than with sixteen (us
// forward / backward, 32768 x 1024 bf16 with an fp32 stream 74.4 / 100.0 against
// 79.8 / 102.2; 16384 x 2048 fp32 97.6 against 103.0 forward; 24 x 1000 3.1 against
// 3.7).  Rows of bf16 alone, 4 bytes an element, want the sixteen forward (32768
// x 1024: 23.5 against 26.5 us).
constexpr int kShortElems = 8;

template <typename F>
void for_norm_fwd(const ssm_norm_dims* dims, bool residual, const F& f) {
  if (dims->io_dtype == SSM_IO_F32)
    for_row<kShortElems, float, float>(dims->dim, f);
  else if (dims->residual_dtype == SSM_IO_F32)
    for_row<kShortElems, uint16_t, float>(dims->dim, f);
  else if (residual)
    for_row<kShortElems, uint16_t, uint16_t>(dims->dim, f);
  else
    for_row<kLaneElems, uint16_t, uint16_t>(dims->dim, f);
}

template <typename F>
void for_norm_bwd(const ssm_norm_dims* dims, const F& f) {
  if (dims->io_dtype == SSM_IO_F32)
    for_row<kShortElems, float, float>(dims->dim, f);
  else if (dims->residual_dtype == SSM_IO_F32)
    for_row<kShortElems, uint16_t, float>(dims->dim, f);
  else
    for_row<kShortElems, uint16_t, uint16_t>(dims->dim, f);
}

template <int TPR>
constexpr int block_of = TPR > 256 ? TPR : 256;

// Workgroups of the backward, each walking several rows, all on the GPU at
// once (256 CUs), so that none waits for another's end.  Three a CU keep the
// memory busy where a row has fp32 in it, five where all is bf16 (us at 3 / 4 / 5:
// 32768 x 1024 with an fp32 stream 100.0 / 102.3 / 105.5, in bf16 62.1 / 55.0 / 50.8;
// 16384 x 1024 fp32 51.5 / 50.7 / 51.4); one where a row takes more than 256 lanes
// (4096 x 8192, one / two: 101.3 / 105.5).
int64_t bwd_groups(const ssm_norm_dims* dims) {
  int64_t tpr = 64;
  while (tpr < 1024 && dims->dim > tpr * kShortElems) tpr *= 2;
  const int64_t rows = dims->batch * dims->seqlen, rpb = tpr > 256 ? 1 : 256 / tpr;
  const bool short_rows = dims->io_dtype == SSM_IO_BF16 && dims->residual_dtype == SSM_IO_BF16;
  const int64_t all = (rows + rpb - 1) / rpb, most = 256 * (tpr > 256 ? 1 : short_rows ? 5 : 3);
  return all < most ? all : most;
}

__global__ void norm_zero_kernel(float* p, int64_t n) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) p[i] = 0.0f;
}

}  // namespace

extern "C" {

int ssm_layer_norm_fwd(ssm_scan_t handle, const ssm_norm_dims* dims, const ssm_norm_fwd_io* io, void* stream) {
  const int bad = check_norm_dims(dims);
  if (bad != SSM_OK) return bad;
  if (io == nullptr) return SSM_ERR_INVALID_ARG;
  const int64_t rows = dims->batch * dims->seqlen, nd = dims->dim;
  const int64_t e = dims->io_dtype == SSM_IO_BF16 ? 2 : 4, r = dims->residual_dtype == SSM_IO_BF16 ? 2 : 4;
  // rows of no elements still have statistics
  const bool empty = rows == 0 || (nd == 0 && io->mean == nullptr && io->rstd == nullptr);
  if (!empty) {
    if (nd > 0 && (io->x == nullptr || io->weight == nullptr || io->y == nullptr)) return SSM_ERR_INVALID_ARG;
    if (!aligned(io->x, e) || !aligned(io->y, e) || !aligned(io->residual, r) || !aligned(io->residual_out, r) ||
        !aligned(io->weight, 4) || !aligned(io->bias, 4) || !aligned(io->valid_len, 4) || !aligned(io->mean, 4) ||
        !aligned(io->rstd, 4))
      return SSM_ERR_UNSUPPORTED;
    // the residual stream may be updated in place: a lane reads its elements before it writes them
    const bool in_place = io->residual != nullptr && io->residual == io->residual_out;
    const Range in[] = {{io->x, rows * nd * e}, {io->residual, in_place ? 0 : rows * nd * r}, {io->weight, nd * 4},
                        {io->bias, nd * 4},     {io->valid_len, dims->batch * 4}};
    const Range out[] = {{io->y, rows * nd * e}, {io->residual_out, rows * nd * r}, {io->mean, rows * 4},
                         {io->rstd, rows * 4}};
    if (any_overlap(in, out)) return SSM_ERR_ALIAS;
  }
  const int rc = check_handle(handle);
  if (rc != SSM_OK || empty) return rc;

  NormParams p;
  p.x = io->x, p.residual = io->residual, p.w = io->weight, p.bias = io->bias, p.valid_len = io->valid_len;
  p.y = io->y, p.residual_out = io->residual_out, p.mean = io->mean, p.rstd = io->rstd;
  p.rows = rows, p.L = dims->seqlen, p.nd = static_cast<int32_t>(nd), p.rms = dims->rms;
  p.eps = dims->eps, p.inv_n = nd > 0 ? 1.0f / static_cast<float>(nd) : 0.0f;
  bool fits = true;
  for_norm_fwd(dims, io->residual != nullptr, [&]<typename IO, typename RT, int TPR, int NV>() {
    constexpr int BLOCK = block_of<TPR>, RPB = BLOCK / TPR;
    // a grid's side holds fewer than 2^32 lanes: more rows take another side
    const int64_t blocks = (rows + RPB - 1) / RPB, wide = blocks < (1 << 21) ? blocks : 1 << 21;
    const int64_t high = (blocks + wide - 1) / wide;
    fits = high <= 65535;
    if (fits)
      hipLaunchKernelGGL((norm_fwd_kernel<IO, RT, TPR, NV>),
                         dim3(static_cast<unsigned>(wide), static_cast<unsigned>(high)), dim3(BLOCK), 0,
                         static_cast<hipStream_t>(stream), p);
  });
  return fits ? launched() : SSM_ERR_UNSUPPORTED;
}

int64_t ssm_layer_norm_bwd_workspace_bytes(const ssm_norm_dims* dims) {
  if (check_norm_dims(dims) != SSM_OK) return -1;
  return bwd_groups(dims) * 2 * dims->dim * 4;
}

int ssm_layer_norm_bwd(ssm_scan_t handle, const ssm_norm_dims* dims, const ssm_norm_bwd_io* io, void* stream) {
  const int bad = check_norm_dims(dims);
  if (bad != SSM_OK) return bad;
  if (io == nullptr || io->workspace_bytes < 0) return SSM_ERR_INVALID_ARG;
  const int64_t rows = dims->batch * dims->seqlen, nd = dims->dim;
  const int64_t e = dims->io_dtype == SSM_IO_BF16 ? 2 : 4, r = dims->residual_dtype == SSM_IO_BF16 ? 2 : 4;
  const int64_t need = ssm_layer_norm_bwd_workspace_bytes(dims);
  if (nd > 0) {
    if (io->weight == nullptr || io->dweight == nullptr) return SSM_ERR_INVALID_ARG;
    if (rows > 0 && (io->dy == nullptr || io->v == nullptr || io->rstd == nullptr || io->dx == nullptr ||
                     (!dims->rms && io->mean == nullptr) || io->workspace == nullptr || io->workspace_bytes < need))
      return SSM_ERR_INVALID_ARG;
    if (!aligned(io->dy, e) || !aligned(io->dx, e) || !aligned(io->v, r) || !aligned(io->dresidual_out, r) ||
        !aligned(io->dresidual, r) || !aligned(io->weight, 4) || !aligned(io->mean, 4) || !aligned(io->rstd, 4) ||
        !aligned(io->valid_len, 4) || !aligned(io->dweight, 4) || !aligned(io->dbias, 4) || !aligned(io->workspace, 4))
      return SSM_ERR_UNSUPPORTED;
    const Range in[] = {{io->dy, rows * nd * e}, {io->v, rows * nd * r},
                        {io->dresidual_out, rows * nd * r}, {io->weight, nd * 4}, {io->mean, rows * 4},
                        {io->rstd, rows * 4}, {io->valid_len, dims->batch * 4}};
    const Range out[] = {{io->dx, rows * nd * e}, {io->dresidual, rows * nd * r}, {io->dweight, nd * 4},
                         {io->dbias, nd * 4}, {io->workspace, io->workspace_bytes}};
    if (any_overlap(in, out)) return SSM_ERR_ALIAS;
  }
  const int rc = check_handle(handle);
  if (rc != SSM_OK || nd == 0) return rc;

  hipStream_t s = static_cast<hipStream_t>(stream);
  if (rows == 0) {  // sums over nothing
    const dim3 grid(static_cast<unsigned>((nd + 255) / 256));
    hipLaunchKernelGGL(norm_zero_kernel, grid, dim3(256), 0, s, io->dweight, nd);
    if (io->dbias != nullptr) hipLaunchKernelGGL(norm_zero_kernel, grid, dim3(256), 0, s, io->dbias, nd);
    return launched();
  }
  NormBwdParams p;
  p.dy = io->dy, p.v = io->v, p.w = io->weight, p.mean = io->mean, p.rstd = io->rstd, p.valid_len = io->valid_len;
  p.dresidual_out = io->dresidual_out, p.dx = io->dx, p.dresidual = io->dresidual;
  p.ws = static_cast<float*>(io->workspace);
  p.rows = rows, p.L = dims->seqlen, p.nd = static_cast<int32_t>(nd), p.rms = dims->rms;
  p.with_bias = io->dbias != nullptr, p.inv_n = 1.0f / static_cast<float>(nd);
  const int64_t groups = bwd_groups(dims);
  for_norm_bwd(dims, [&]<typename IO, typename RT, int TPR, int NV>() {
    const auto kernel = p.with_bias ? norm_bwd_kernel<IO, RT, TPR, NV, true> : norm_bwd_kernel<IO, RT, TPR, NV, false>;
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(groups)), dim3(block_of<TPR>), 0, s, p);
  });
  if (launched() != SSM_OK) return SSM_ERR_HIP;
  launch_reduce(p.ws, groups, (p.with_bias ? 2 : 1) * nd, NormGrads{io->dweight, io->dbias, nd}, s);
  return launched();
}

}  // extern "C"
