// ccv_gnorm.hip -- group norm of each row's channels, with an activation or a gate.
//
//   n = (x - mean) rstd over each group of a row,  y = n w + b,
//   out = act(y), or with a gate z: out = y act(z).
//
// Bound by memory: x (and z) in, out out.  A group of a row is read once into the registers of
// `LANES` threads (4 to 256), the variance summed from the deviations there, in fp32.  Threads
// keep their group and walk the rows at a stride, so its weights are loaded once, with the next row's loads under
// way while a row's sums are made.  Widths that are no multiple of a vector end with a vector that starts earlier
// (ccv_norm_device.hpp).
// 65536 rows of 20 groups of 128 in fp16 with a gate (1.0 GB): 208 us, 4.8 TB/s; 256 x 4096 in bf16: 4.4 us, a launch's and a row's latency.
#include "ccv_gnorm_device.hpp"

namespace ccv {
namespace {

template <int DT, int LANES, int NV, bool FULL, bool GATE>
__global__ __launch_bounds__(256) void fwd_kernel(const GroupNormArgs a) {
  constexpr int V = Vec<DT>::n;
  __shared__ float red[2][2][8];
  int turn = 0;
  const Walker me = walker_at<LANES>(a);
  if (me.idle) return;                                     // whole rows of lanes; no barrier joins them with others
  const Columns<DT, LANES, NV, FULL> cols(a.width);
  const int64_t first = (int64_t)me.group * a.width;
  const int ws = a.w_dtype == CCV_DT_F32 ? 4 : 2;
  float w[NV][V], b[NV][V];
  cols.weights(w, a.w ? static_cast<const char*>(a.w) + first * ws : nullptr, a.w_dtype, 1.0f);
  cols.weights(b, a.b ? static_cast<const char*>(a.b) + first * ws : nullptr, a.w_dtype, 0.0f);
  const float inv = 1.0f / (float)a.width;
  u32x4 raw[NV], rz[NV];
  const auto load = [&](int64_t r) {
    cols.load(raw, at<DT>(a.x, r * a.x_s + first));
    if constexpr (GATE) cols.load(rz, at<DT>(a.z, r * a.z_s + first));
  };
  load(me.row);
  for (int64_t row = me.row; row < a.rows; row += a.walkers) {
    float x[NV][V], z[NV][V], s = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      cols.unpack(raw[i], x[i]);
      if constexpr (GATE) cols.unpack(rz[i], z[i]);
#pragma unroll
      for (int e = 0; e < V; ++e) s += cols.mine(i, e) ? x[i][e] : 0.0f;
    }
    if (row + a.walkers < a.rows) load(row + a.walkers);
    const float mean = row_sums<LANES, 1>(f32x2{s, 0}, red, turn)[0] * inv;
    float q = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        x[i][e] -= mean;
        const float d = cols.mine(i, e) ? x[i][e] : 0.0f;
        q = __builtin_fmaf(d, d, q);
      }
    const float rstd = 1.0f / __builtin_sqrtf(row_sums<LANES, 1>(f32x2{q, 0}, red, turn)[0] * inv + a.eps);
    if (threadIdx.x % LANES == 0) {
      if (a.mean) a.mean[row * a.groups + me.group] = mean;
      if (a.rstd) a.rstd[row * a.groups + me.group] = rstd;
    }
    char* op = at<DT>(a.out, row * a.o_s + first);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float y[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        y[e] = __builtin_fmaf(x[i][e] * rstd, w[i][e], b[i][e]);
        if constexpr (GATE) y[e] *= act_value(z[i][e], a.silu);
        else y[e] = act_value(y[e], a.silu);
      }
      cols.store(op, i, y);
    }
  }
}

// Element by element: groups narrower than a vector (THREADS 1) or wider than 256 threads hold.  Far from the copy's rate, for accesses of
// an element and a second and third walk of wide ones: calls with a gate of 65536 rows of 4 groups of 5 in fp16 take 10 us, 262144 of 32 of 6 in
// bf16 218 (their bytes need 58), 4096 of one of 16384 in bf16 403 (77).
template <int DT, int THREADS>
__global__ __launch_bounds__(THREADS == 1 ? 256 : THREADS) void any_fwd_kernel(const GroupNormArgs a) {
  __shared__ float red[16];
  const int64_t step = THREADS == 1 ? (int64_t)gridDim.x * 256 : gridDim.x, items = a.rows * a.groups;
  const int t = THREADS == 1 ? 0 : threadIdx.x;
  for (int64_t item = THREADS == 1 ? (int64_t)blockIdx.x * 256 + threadIdx.x : blockIdx.x; item < items; item += step) {
    const int64_t row = item / a.groups, group = item - row * a.groups, first = group * a.width;
    const char* xp = at<DT>(a.x, row * a.x_s + first);
    float s = 0, q = 0;
    for (int i = t; i < a.width; i += THREADS) s += load1<DT>(at<DT>((const void*)xp, i));
    const float mean = any_sum<THREADS>(s, red) / (float)a.width;
    for (int i = t; i < a.width; i += THREADS) {
      const float d = load1<DT>(at<DT>((const void*)xp, i)) - mean;
      q = __builtin_fmaf(d, d, q);
    }
    const float rstd = 1.0f / __builtin_sqrtf(any_sum<THREADS>(q, red) / (float)a.width + a.eps);
    if (t == 0) {
      if (a.mean) a.mean[item] = mean;
      if (a.rstd) a.rstd[item] = rstd;
    }
    for (int i = t; i < a.width; i += THREADS) {
      const float n = (load1<DT>(at<DT>((const void*)xp, i)) - mean) * rstd;
      const float y = __builtin_fmaf(n, a.w ? load_param(a.w, a.w_dtype, first + i) : 1.0f, a.b ? load_param(a.b, a.w_dtype, first + i) : 0.0f);
      const float o = a.z ? y * act_value(load1<DT>(at<DT>(a.z, row * a.z_s + first + i)), a.silu) : act_value(y, a.silu);
      store1<DT>(at<DT>(a.out, row * a.o_s + first + i), o);
    }
  }
}

}  // namespace

int launch_group_norm_fwd(const GroupNormArgs& a, void* stream) {
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const NormShape s = group_norm_shape(a.width, a.x_dtype == CCV_DT_F32 ? 4 : 2);
  if (!s.lanes) {
    const int64_t items = a.rows * a.groups;
    by_type(a, [&](auto dt) {
      constexpr int DT = decltype(dt)::value;
      if (a.width < 8) any_fwd_kernel<DT, 1><<<(uint32_t)(items < 2048 * 256 ? (items + 255) / 256 : 2048), 256, 0, st>>>(a);
      else any_fwd_kernel<DT, 1024><<<(uint32_t)(items < 4096 ? items : 4096), 1024, 0, st>>>(a);
    });
    return (int)hipGetLastError();
  }
  const uint32_t grid = (uint32_t)(((int64_t)a.walkers * a.groups + 256 / s.lanes - 1) / (256 / s.lanes));
  by_shape(a, [&](auto dt, auto lanes, auto nv, auto full, auto gated) {
    fwd_kernel<decltype(dt)::value, decltype(lanes)::value, decltype(nv)::value, decltype(full)::value, decltype(gated)::value>
        <<<grid, 256, 0, st>>>(a);
  });
  return (int)hipGetLastError();
}

}  // namespace ccv
