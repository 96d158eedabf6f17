// The selective scan for one token of every sequence, for MI355X (gfx950):
// the step a server takes on its cache of states.
//
// For batch row b, channel d and state n, with A = -exp(A_log[d,n]):
//
//     delta = clip(softplus(raw[b,d] + bias[d]))
//     h'[n] = exp(delta * A) h[n] + delta * B[b,n] * x[b,d]
//     y[b,d] = (sum_n C[b,n] h'[n] + D[d] x[b,d]) (* silu(z[b,d]))
//
// that is, one step of the scan's recurrence with the scan's formulas.  The
// states, 4 bytes a (channel, state) read and written, are nearly all that
// moves: bound by memory for a full batch, by latency for one row.
//
// Layout: a lane owns four adjacent states of one channel (16 bytes), so a
// wave reads 1 KB of one cache row; a channel's dstate / 4 lanes are adjacent
// and add their parts of C.h' by DPP within a row of 16 lanes.
//
// Measured: 256 rows x 2048 channels x 16 states in bf16, 71 MB: 15.2 us from 256
// of 512 slots into another cache (4.7 TB/s; a copy of 1 GiB runs at 5.3, and the
// states of three input sets stay in the 256 MiB cache in part); in place, eight
// such caches in turn, 19.4 us a step (3.7 TB/s), and 19.5 without slots.  One
// row: 2.6 us, the latency of two dependent reads.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "ssm_block.h"

namespace {

struct StepParams {
  const void* x;
  const void* delta;
  const float* A_log;
  const void* B;
  const void* C;
  const float* D;
  const float* delta_bias;
  const void* z;
  const int32_t* slots;
  const float* h0;
  float* h_last;
  void* y;
  int64_t x_rs, delta_rs, B_rs, C_rs, z_rs, y_rs, n_slots;
  float dmin, dmax;
  int32_t nb, nd, softplus, clamp;
};

// One workgroup: 1024 / N channels of R batch rows, the states of all of them
// in flight at once; what depends on the channel alone is read once.
template <typename IO, int N, int R>
__global__ __launch_bounds__(256) void scan_step_kernel(const StepParams prm) {
  constexpr int LPC = N / 4, CH = 256 / LPC;
  const int32_t b = blockIdx.y * R;
  const int64_t d = static_cast<int64_t>(blockIdx.x) * CH + threadIdx.x / LPC;
  const int n0 = (threadIdx.x % LPC) * 4;
  const bool mine = d < prm.nd;  // a channel's lanes agree
  int32_t slot[R];
#pragma unroll
  for (int r = 0; r < R; ++r)
    slot[r] = b + r >= prm.nb ? -1 : (prm.slots == nullptr ? b + r : prm.slots[b + r]);
  float h[R][4], al[4] = {}, Bv[R][4], Cv[R][4], x[R], dt[R], z[R], skip = 0.0f, bias = 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t row = b + r;
    // rows that turn out idle are read all the same, inside their bounds
    if (mine && slot[r] >= 0 && slot[r] < prm.n_slots) {
      VecIO<float>::load(prm.h0 + (slot[r] * static_cast<int64_t>(prm.nd) + d) * N + n0, h[r]);
      x[r] = VecIO<IO>::get(static_cast<const IO*>(prm.x) + row * prm.x_rs + d);
      dt[r] = VecIO<IO>::get(static_cast<const IO*>(prm.delta) + row * prm.delta_rs + d);
      z[r] = prm.z == nullptr ? 0.0f : VecIO<IO>::get(static_cast<const IO*>(prm.z) + row * prm.z_rs + d);
      VecIO<IO>::load(static_cast<const IO*>(prm.B) + row * prm.B_rs + n0, Bv[r]);
      VecIO<IO>::load(static_cast<const IO*>(prm.C) + row * prm.C_rs + n0, Cv[r]);
    }
  }
  if (mine) {
    VecIO<float>::load(prm.A_log + d * N + n0, al);
    if (prm.delta_bias != nullptr) bias = prm.delta_bias[d];
    if (prm.D != nullptr) skip = prm.D[d];
  }
  bool active[R];
  step_rows_active<R>(prm.slots, b, prm.nb, slot, prm.n_slots, active);
  if (!mine) return;
  float a[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = -fast_exp2(al[i] * kLog2e) * kLog2e;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (b + r >= prm.nb) return;
    IO* y = static_cast<IO*>(prm.y) + (b + r) * prm.y_rs + d;
    if (!active[r]) {
      if (n0 == 0) VecIO<IO>::put(y, 0.0f);
      continue;
    }
    float delta = dt[r] + bias;
    if (prm.softplus) delta = softplus_f32(delta);
    if (prm.clamp) delta = __builtin_fminf(__builtin_fmaxf(delta, prm.dmin), prm.dmax);
    const float u = delta * x[r];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[r][i] = __builtin_fmaf(fast_exp2(delta * a[i]), h[r][i], u * Bv[r][i]);
      sum = __builtin_fmaf(Cv[r][i], h[r][i], sum);
    }
    // past the caches: next read a token and all other layers' states later
    // (into another cache 17.7 -> 15.4 us; in place no difference)
    VecIO<float>::stream(prm.h_last + (slot[r] * static_cast<int64_t>(prm.nd) + d) * N + n0, h[r]);
    sum = group_sum<LPC>(sum);
    if (n0 == 0) {
      if (prm.D != nullptr) sum = __builtin_fmaf(skip, x[r], sum);
      if (prm.z != nullptr) sum *= z[r] * sigmoid_exact(z[r]);
      VecIO<IO>::put(y, sum);
    }
  }
}

// Rows of a workgroup where there are slots and kSeveral workgroups of one row:
// they share the look through the slots and its latency.  us at 1 / 2 / 4 rows,
// 2048 channels, dstate 16, in place with eight caches in turn: 128 rows 10.9 /
// 10.1 / 10.5, 256 rows 21.6 / 19.5 / 21.7, 1024 rows x 1024 channels 45.5 / 40.4 /
// 42.5; at 1 / 2, 64 rows into another cache 5.4 / 5.5 (in place 6.8 both).
// Without slots one row is the faster (256 rows 15.3 / 15.9).
constexpr int kStepRows = 2;
constexpr int64_t kSeveral = 4096;

template <typename IO, int N>
void launch_step_n(bool several, dim3 grid, const StepParams& p, hipStream_t s) {
  const auto kernel = several ? scan_step_kernel<IO, N, kStepRows> : scan_step_kernel<IO, N, 1>;
  hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, p);
}

template <typename IO>
void launch_step(int64_t N, bool several, dim3 grid, const StepParams& p, hipStream_t s) {
  switch (N) {
    case 16:
      return launch_step_n<IO, 16>(several, grid, p, s);
    case 32:
      return launch_step_n<IO, 32>(several, grid, p, s);
    default:
      return launch_step_n<IO, 64>(several, grid, p, s);
  }
}

}  // namespace

extern "C" {

int ssm_selective_scan_step(ssm_scan_t handle, const ssm_scan_dims* dims, const ssm_scan_step_io* io, void* stream) {
  if (dims == nullptr || io == nullptr) return SSM_ERR_INVALID_ARG;
  const int64_t nb = dims->batch, nd = dims->dim, N = dims->dstate;
  if (nb < 0 || nd < 0 || N < 0 || dims->seqlen != 1 || io->n_slots < 0) return SSM_ERR_INVALID_ARG;
  if (dims->io_dtype != SSM_IO_F32 && dims->io_dtype != SSM_IO_BF16) return SSM_ERR_INVALID_ARG;
  if (dims->delta_softplus != 0 && dims->delta_softplus != 1) return SSM_ERR_INVALID_ARG;
  if (dims->delta_clamp != 0 && dims->delta_clamp != 1) return SSM_ERR_INVALID_ARG;
  if (dims->delta_clamp == 1 && !(dims->delta_min >= 0.0f && dims->delta_min <= dims->delta_max &&
                                  dims->delta_max < __builtin_inff()))
    return SSM_ERR_INVALID_ARG;
  if (N != 16 && N != 32 && N != 64) return SSM_ERR_UNSUPPORTED;
  const int64_t rows = io->slots == nullptr ? nb : io->n_slots;
  if (nb > 65535 || nd > kMaxSize || rows > kMaxSize) return SSM_ERR_UNSUPPORTED;
  const int64_t e = dims->io_dtype == SSM_IO_BF16 ? 2 : 4;
  const bool empty = nb == 0 || nd == 0;
  if (!empty) {
    if (io->x == nullptr || io->delta == nullptr || io->A_log == nullptr || io->B == nullptr || io->C == nullptr ||
        io->y == nullptr || (rows > 0 && (io->h0 == nullptr || io->h_last == nullptr)))
      return SSM_ERR_INVALID_ARG;
    const int64_t bx = span_bytes(nb, io->x_row_stride, 1, 0, nd, e);
    const int64_t bd = span_bytes(nb, io->delta_row_stride, 1, 0, nd, e);
    const int64_t bB = span_bytes(nb, io->B_row_stride, 1, 0, N, e);
    const int64_t bC = span_bytes(nb, io->C_row_stride, 1, 0, N, e);
    const int64_t bz = io->z == nullptr ? 0 : span_bytes(nb, io->z_row_stride, 1, 0, nd, e);
    const int64_t by = span_bytes(nb, io->y_row_stride, 1, 0, nd, e);
    const int64_t bh = span_bytes(rows, nd * N, 1, 0, nd * N, 4);
    if (bx < 0 || bd < 0 || bB < 0 || bC < 0 || bz < 0 || by < 0 || !rows_disjoint(nb, io->y_row_stride, 1, 0, nd))
      return SSM_ERR_INVALID_ARG;
    if (bh < 0) return SSM_ERR_UNSUPPORTED;
    if (!aligned(io->x, e) || !aligned(io->delta, e) || !aligned(io->B, e) || !aligned(io->C, e) ||
        !aligned(io->z, e) || !aligned(io->y, e) || !aligned(io->A_log, 4) || !aligned(io->D, 4) ||
        !aligned(io->delta_bias, 4) || !aligned(io->slots, 4) || !aligned(io->h0, 4) || !aligned(io->h_last, 4))
      return SSM_ERR_UNSUPPORTED;
    // the states in place are one range: h0 is then left out of the inputs
    const Range in[] = {{io->x, bx}, {io->delta, bd}, {io->B, bB}, {io->C, bC}, {io->z, bz},
                        {io->A_log, nd * N * 4}, {io->D, nd * 4}, {io->delta_bias, nd * 4},
                        {io->slots, nb * 4}, {io->h0, io->h0 == io->h_last ? 0 : bh}};
    const Range out[] = {{io->y, by}, {io->h_last, bh}};
    if (any_overlap(in, out)) return SSM_ERR_ALIAS;
  }
  const int rc = check_handle(handle);
  if (rc != SSM_OK || empty) return rc;

  StepParams p;
  p.x = io->x, p.delta = io->delta, p.A_log = io->A_log, p.B = io->B, p.C = io->C, p.D = io->D;
  p.delta_bias = io->delta_bias, p.z = io->z, p.slots = io->slots, p.h0 = io->h0, p.h_last = io->h_last, p.y = io->y;
  p.x_rs = io->x_row_stride, p.delta_rs = io->delta_row_stride, p.B_rs = io->B_row_stride;
  p.C_rs = io->C_row_stride, p.z_rs = io->z_row_stride, p.y_rs = io->y_row_stride, p.n_slots = rows;
  p.dmin = dims->delta_min, p.dmax = dims->delta_max, p.nb = static_cast<int32_t>(nb), p.nd = static_cast<int32_t>(nd);
  p.softplus = dims->delta_softplus, p.clamp = dims->delta_clamp;
  const int64_t ch = 1024 / N, tiles = (nd + ch - 1) / ch;
  if (!grid_fits(tiles, 256)) return SSM_ERR_UNSUPPORTED;
  const bool several = io->slots != nullptr && nb * tiles >= kSeveral;
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(several ? (nb + kStepRows - 1) / kStepRows : nb));
  if (dims->io_dtype == SSM_IO_BF16)
    launch_step<uint16_t>(N, several, grid, p, static_cast<hipStream_t>(stream));
  else
    launch_step<float>(N, several, grid, p, static_cast<hipStream_t>(stream));
  return launched();
}

}  // extern "C"
