// ccv_gnorm_bwd.hip -- gradients of group norm with an activation or a gate.
//
//   without a gate: dy = dout act'(y);  with one: dy = dout act(z), dz = dout y act'(z);
//   e = dy w,  dx = rstd (e - mean(e) - n mean(e n)) over each group,  dw = sum over rows of dy n,  db = sum of dy.
//
// Bound by memory: x, dout (and z) in, dx (and dz) out, each once; n, y and the activation are made
// again from x, the statistics and the weights in registers.  Threads keep their group, so their sums of dw and db
// stay in registers too; each walker leaves a partial row, and a second kernel adds them in a fixed order.
// 65536 rows of 20 groups of 128 in fp16 with a gate (1.7 GB): 337 us, 5.0 TB/s, and 7 us for the sums.  Where a row has few channels there are
// many walkers, and few workgroups to add their partial rows: 65536 rows of 32 channels in bf16 take 45 us, 15 without dw and db, of 128 57 and 16.
#include "ccv_gnorm_device.hpp"

namespace ccv {
namespace {

template <int DT, int LANES, int NV, bool FULL, bool GATE>
__global__ __launch_bounds__(256) void bwd_kernel(const GroupNormArgs a) {
  constexpr int V = Vec<DT>::n;
  __shared__ float red[2][2][8];
  int turn = 0;
  const Walker me = walker_at<LANES>(a);
  if (me.idle) return;
  const Columns<DT, LANES, NV, FULL> cols(a.width);
  const int64_t first = (int64_t)me.group * a.width;
  const int ws = a.w_dtype == CCV_DT_F32 ? 4 : 2;
  float w[NV][V], b[NV][V], dw[NV][V], db[NV][V];
  cols.weights(w, a.w ? static_cast<const char*>(a.w) + first * ws : nullptr, a.w_dtype, 1.0f);
  cols.weights(b, a.b ? static_cast<const char*>(a.b) + first * ws : nullptr, a.w_dtype, 0.0f);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) dw[i][e] = db[i][e] = 0.0f;
  const float inv = 1.0f / (float)a.width;
  u32x4 xr[NV], dr[NV], zr[NV];
  float mean, rstd;
  const auto load = [&](int64_t r) {
    cols.load(xr, at<DT>(a.x, r * a.x_s + first));
    cols.load(dr, at<DT>(a.dout, r * a.do_s + first));
    if constexpr (GATE) cols.load(zr, at<DT>(a.z, r * a.z_s + first));
    mean = a.mean[r * a.groups + me.group];
    rstd = a.rstd[r * a.groups + me.group];
  };
  load(me.row);
  for (int64_t row = me.row; row < a.rows; row += a.walkers) {
    const float mu = mean, rs = rstd;
    float x[NV][V], d[NV][V], s1 = 0, s2 = 0;
    char* zp = GATE && a.dz ? at<DT>(a.dz, row * a.dz_s + first) : nullptr;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float z[V];
      cols.unpack(xr[i], x[i]);
      cols.unpack(dr[i], d[i]);
      if constexpr (GATE) cols.unpack(zr[i], z);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        x[i][e] = (x[i][e] - mu) * rs;
        const float y = __builtin_fmaf(x[i][e], w[i][e], b[i][e]);
        float value, slope;
        act_both(GATE ? z[e] : y, a.silu, value, slope);
        if constexpr (GATE) {
          z[e] = d[i][e] * y * slope;
          d[i][e] *= value;
        } else {
          d[i][e] *= slope;
        }
        const float dy = cols.mine(i, e) ? d[i][e] : 0.0f;
        dw[i][e] = __builtin_fmaf(dy, x[i][e], dw[i][e]);
        db[i][e] += dy;
        d[i][e] *= w[i][e];
        const float ee = cols.mine(i, e) ? d[i][e] : 0.0f;
        s1 += ee;
        s2 = __builtin_fmaf(ee, x[i][e], s2);
      }
      if constexpr (GATE)
        if (zp) cols.store(zp, i, z);
    }
    if (row + a.walkers < a.rows) load(row + a.walkers);
    const f32x2 m = row_sums<LANES, 2>(f32x2{s1, s2}, red, turn) * inv;
    if (!a.dx) continue;
    char* op = at<DT>(a.dx, row * a.dx_s + first);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float y[V];
#pragma unroll
      for (int e = 0; e < V; ++e) y[e] = rs * (d[i][e] - m[0] - x[i][e] * m[1]);
      cols.store(op, i, y);
    }
  }
  if (!a.part) return;
  const int64_t C = (int64_t)a.groups * a.width;
  float* part = a.part + (int64_t)me.row * 2 * C + first;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (cols.mine(i, e)) {
        part[cols.col[i] + e] = dw[i][e];
        part[C + cols.col[i] + e] = db[i][e];
      }
}

__global__ __launch_bounds__(1024) void reduce_kernel(const GroupNormArgs a) {
  sum_partials(a.part, a.walkers, a.groups * a.width, a.dw, a.db, a.w_dtype);
}

// Element by element, as the forward's.  What dy, n and y are of an element:
template <int DT>
struct Element {
  float n, dy, dz;
  __device__ inline Element(const GroupNormArgs& a, int64_t row, int64_t c, float mean, float rstd) {
    n = (load1<DT>(at<DT>(a.x, row * a.x_s + c)) - mean) * rstd;
    const float y = __builtin_fmaf(n, a.w ? load_param(a.w, a.w_dtype, c) : 1.0f, a.b ? load_param(a.b, a.w_dtype, c) : 0.0f);
    const float d = load1<DT>(at<DT>(a.dout, row * a.do_s + c));
    float value, slope;
    act_both(a.z ? load1<DT>(at<DT>(a.z, row * a.z_s + c)) : y, a.silu, value, slope);
    dy = d * (a.z ? value : slope);
    dz = d * y * slope;
  }
};

template <int DT, int THREADS>
__global__ __launch_bounds__(THREADS == 1 ? 256 : THREADS) void any_dx_kernel(const GroupNormArgs a) {
  __shared__ float red[16];
  const int64_t step = THREADS == 1 ? (int64_t)gridDim.x * 256 : gridDim.x, items = a.rows * a.groups;
  const int t = THREADS == 1 ? 0 : threadIdx.x;
  for (int64_t item = THREADS == 1 ? (int64_t)blockIdx.x * 256 + threadIdx.x : blockIdx.x; item < items; item += step) {
    const int64_t row = item / a.groups, group = item - row * a.groups, first = group * a.width;
    const float mean = a.mean[item], rstd = a.rstd[item];
    float s1 = 0, s2 = 0;
    for (int i = t; i < a.width; i += THREADS) {
      const Element<DT> el(a, row, first + i, mean, rstd);
      const float e = el.dy * (a.w ? load_param(a.w, a.w_dtype, first + i) : 1.0f);
      s1 += e;
      s2 = __builtin_fmaf(e, el.n, s2);
      if (a.dz) store1<DT>(at<DT>(a.dz, row * a.dz_s + first + i), el.dz);
    }
    const float m1 = any_sum<THREADS>(s1, red) / (float)a.width, m2 = any_sum<THREADS>(s2, red) / (float)a.width;
    if (!a.dx) continue;
    for (int i = t; i < a.width; i += THREADS) {
      const Element<DT> el(a, row, first + i, mean, rstd);
      const float e = el.dy * (a.w ? load_param(a.w, a.w_dtype, first + i) : 1.0f);
      store1<DT>(at<DT>(a.dx, row * a.dx_s + first + i), rstd * (e - m1 - el.n * m2));
    }
  }
}

// Partial sums of dw and db: a thread has one column, blockIdx.y its rows.  Its rows come one after the other, so many rows of few channels take
// long: of the gradients of 65536 rows of 4 groups of 5 in fp16 (603 us; 15 without dw and db) and of 1048576 rows of 4 channels in bf16 (9.5 ms and
// 38 us) this is nearly all, of 4096 rows of 16384 in bf16 a fifth (748 and 593).
template <int DT>
__global__ __launch_bounds__(256) void any_sums_kernel(const GroupNormArgs a) {
  const int64_t C = (int64_t)a.groups * a.width, c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= C) return;
  const int64_t group = c / a.width;
  float dws = 0, dbs = 0;
  for (int64_t row = blockIdx.y; row < a.rows;) {
    const int64_t run = (int64_t)kNormRun * a.walkers, end = a.rows - row > run ? row + run : a.rows;
    float dw = 0, db = 0;
    for (; row < end; row += a.walkers) {
      const Element<DT> el(a, row, c, a.mean[row * a.groups + group], a.rstd[row * a.groups + group]);
      dw = __builtin_fmaf(el.dy, el.n, dw);
      db += el.dy;
    }
    dws += dw;
    dbs += db;
  }
  a.part[(int64_t)blockIdx.y * 2 * C + c] = dws;
  a.part[((int64_t)blockIdx.y * 2 + 1) * C + c] = dbs;
}

}  // namespace

int launch_group_norm_bwd(const GroupNormArgs& a, void* stream) {
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const NormShape s = group_norm_shape(a.width, a.x_dtype == CCV_DT_F32 ? 4 : 2);
  const int64_t C = (int64_t)a.groups * a.width;
  int e = 0;
  if (a.rows > 0 && !s.lanes) {
    const int64_t items = a.rows * a.groups;
    by_type(a, [&](auto dt) {
      constexpr int DT = decltype(dt)::value;
      if (a.dx || a.dz) {
        if (a.width < 8) any_dx_kernel<DT, 1><<<(uint32_t)(items < 2048 * 256 ? (items + 255) / 256 : 2048), 256, 0, st>>>(a);
        else any_dx_kernel<DT, 1024><<<(uint32_t)(items < 4096 ? items : 4096), 1024, 0, st>>>(a);
      }
      if (a.part) any_sums_kernel<DT><<<dim3((uint32_t)((C + 255) / 256), a.walkers), 256, 0, st>>>(a);
    });
    e = (int)hipGetLastError();
  } else if (a.rows > 0) {
    const uint32_t grid = (uint32_t)(((int64_t)a.walkers * a.groups + 256 / s.lanes - 1) / (256 / s.lanes));
    by_shape(a, [&](auto dt, auto lanes, auto nv, auto full, auto gated) {
      bwd_kernel<decltype(dt)::value, decltype(lanes)::value, decltype(nv)::value, decltype(full)::value, decltype(gated)::value>
          <<<grid, 256, 0, st>>>(a);
    });
    e = (int)hipGetLastError();
  }
  if (e || (!a.dw && !a.db)) return e;
  reduce_kernel<<<dim3((uint32_t)((C + 31) / 32), 2), 1024, 0, st>>>(a);      // no rows: zeros
  return (int)hipGetLastError();
}

}  // namespace ccv
