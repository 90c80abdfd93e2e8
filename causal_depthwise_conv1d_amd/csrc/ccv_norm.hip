// ccv_norm.hip -- layer norm over the last dimension and its gradients.
//
//   n = (x - mean) rstd,  out = n w + b;     a = dout w,
//   dx = rstd (a - mean(a) - n mean(a n)),   dw = sum over rows of dout n,   db = sum of dout.
// Bound by memory: x in, out out; in the backward x and dout in, dx out.  A row is read
// once into registers, `LANES` threads a row (16 for a head's width, up to 512), and the
// variance is summed from the deviations there, in fp32.  Workgroups walk rows at a
// stride, with the next row's loads under way while a row's sums pass through LDS; a thread
// always has the same columns, so the weights stay in registers, and in the backward so do
// the thread's sums of dw and db.  Each workgroup leaves one partial row, and a second
// kernel adds the partial rows in a fixed order.
// 32768 rows of 4096 in bf16: forward 99 us, 0.54 GB at 5.4 TB/s; backward 170 us, 0.81 GB at 4.7, and
// 8.5 us for the 1024 partial rows (2048 of them cost more than the shorter walks gain: 182 and 164 us
// for 65536 x 2048).  65536 x 20 rows of 128 in fp16: 131, 211 and 5 us.
// Every access is 16 bytes at any alignment.  Where the width is no multiple of that, a
// row's last vector starts where it ends with the row; the elements that it shares with
// the vector before it are left out of sums and written twice, with the same value.
#include "ccv_delta_device.hpp"
#include "ccv_norm_launch.hpp"

namespace ccv {
namespace {

template <int DT> struct Vec { static constexpr int n = DT == CCV_DT_F32 ? 4 : 8; };

// Sums over the `LANES` threads of a row of N values; every one of them gets them.  Rows of more
// than a wave: through `red`, two pieces of it in turn, so that one barrier suffices.
template <int LANES, int N>
__device__ inline f32x2 row_sums(f32x2 v, float (*red)[2][8], int& turn) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    float s = sum16(v[n]);
    if constexpr (LANES >= 64) s = sum4rows(s);
    v[n] = s;
  }
  if constexpr (LANES > 64) {
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int n = 0; n < N; ++n) red[turn][n][w] = v[n];
    lds_barrier();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float s = 0;
#pragma unroll
      for (int i = 0; i < LANES / 64; ++i) s += red[turn][n][i];
      v[n] = s;
    }
    turn ^= 1;
  }
  return v;
}

// Row r of a view; rows that follow each other at one stride need no division (n1 is then 0).
__device__ inline int64_t row_at(const int64_t* s, int64_t r, uint32_t n1) {
  if (n1 == 0) return r * s[1];
  const uint32_t i = (uint32_t)r / n1;
  return i * s[0] + ((uint32_t)r - i * n1) * s[1];
}
template <int DT>
__device__ inline const char* norm_row(const void* p, const int64_t* s, int64_t r, uint32_t n1) {
  return static_cast<const char*>(p) + row_at(s, r, n1) * (DT == CCV_DT_F32 ? 4 : 2);
}
template <int DT>
__device__ inline char* norm_row(void* p, const int64_t* s, int64_t r, uint32_t n1) {
  return static_cast<char*>(p) + row_at(s, r, n1) * (DT == CCV_DT_F32 ? 4 : 2);
}

template <int LANES> constexpr int kThreads = LANES > 256 ? LANES : 256;

// A thread's vectors of a row.
template <int DT, int LANES, int NV, bool FULL>
struct Columns {
  static constexpr int V = Vec<DT>::n, ES = DT == CCV_DT_F32 ? 4 : 2;
  int col[NV], skip[NV];                 // first element; elements that belong to another thread (V: all)
  __device__ inline Columns(int width) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * LANES + (int)(threadIdx.x % LANES)) * V;
      col[i] = FULL || c + V <= width ? c : width - V;
      skip[i] = FULL ? 0 : c >= width ? V : c - col[i];
    }
  }
  __device__ inline bool mine(int i, int e) const { return FULL || e >= skip[i]; }
  __device__ inline void load(u32x4 (&raw)[NV], const char* row) const {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      raw[i] = gload<u32x4>(pick(FULL || skip[i] < V, reinterpret_cast<uintptr_t>(row) + (uint32_t)col[i] * ES,
                                 reinterpret_cast<uintptr_t>(kZeroSrc)));
  }
  __device__ static inline void unpack(u32x4 raw, float* x) {
    if constexpr (DT == CCV_DT_F32) F32::unpack(raw, x);
    else if constexpr (DT == CCV_DT_BF16) BF16::unpack(raw, x);
    else F16::unpack(raw, x);
  }
  __device__ inline void store(char* row, int i, const float* y) const {
    if (!FULL && skip[i] >= V) return;
    char* p = row + (uint32_t)col[i] * ES;
    if constexpr (DT == CCV_DT_F32) store16(p, F32::pack(y));
    else if constexpr (DT == CCV_DT_BF16) store16(p, BF16::pack(y));
    else store16(p, F16::pack(y));
  }
  __device__ inline void weights(float (&w)[NV][V], const void* p, int dtype, float other) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!p || (!FULL && skip[i] >= V)) {
#pragma unroll
        for (int e = 0; e < V; ++e) w[i][e] = other;
      } else if (dtype == CCV_DT_F32) {
#pragma unroll
        for (int e = 0; e < V; e += 4) F32::unpack(load16(static_cast<const float*>(p) + col[i] + e), w[i] + e);
      } else {
        const uint16_t* q = static_cast<const uint16_t*>(p) + col[i];
#pragma unroll
        for (int e = 0; e < V; e += 4) {
          const u32x2 d = gload<u32x2>(reinterpret_cast<uintptr_t>(q + e));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t two = d[j / 2];
            const uint16_t h = (uint16_t)(two >> (16 * (j % 2)));
            w[i][e + j] = dtype == CCV_DT_BF16 ? BF16::to_f(h) : F16::to_f(h);
          }
        }
      }
    }
  }
};

template <int DT, int LANES, int NV, bool FULL>
__global__ __launch_bounds__(kThreads<LANES>) void fwd_kernel(NormArgs a) {
  constexpr int V = Vec<DT>::n, RW = kThreads<LANES> / LANES;
  __shared__ float red[2][2][8];
  int turn = 0;
  const Columns<DT, LANES, NV, FULL> cols(a.width);
  float w[NV][V], b[NV][V];
  cols.weights(w, a.w, a.w_dtype, 1.0f);
  cols.weights(b, a.b, a.w_dtype, 0.0f);
  const float inv = 1.0f / (float)a.width;
  const int64_t step = (int64_t)gridDim.x * RW;
  int64_t row = (int64_t)blockIdx.x * RW + threadIdx.x / LANES;
  u32x4 raw[NV];
  cols.load(raw, norm_row<DT>(a.x, a.x_s, row < a.rows ? row : a.rows - 1, a.n1));
  // the trip count is the same for all threads of a workgroup; rows past the last are read as it
  for (int64_t base = (int64_t)blockIdx.x * RW; base < a.rows; base += step, row += step) {
    float x[NV][V], s = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      cols.unpack(raw[i], x[i]);
#pragma unroll
      for (int e = 0; e < V; ++e) s += cols.mine(i, e) ? x[i][e] : 0.0f;
    }
    if (base + step < a.rows) cols.load(raw, norm_row<DT>(a.x, a.x_s, row + step < a.rows ? row + step : a.rows - 1, a.n1));
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
    if (row >= a.rows) continue;
    if (threadIdx.x % LANES == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    char* op = norm_row<DT>(a.out, a.o_s, row, a.n1);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float y[V];
#pragma unroll
      for (int e = 0; e < V; ++e) y[e] = __builtin_fmaf(x[i][e] * rstd, w[i][e], b[i][e]);
      cols.store(op, i, y);
    }
  }
}

template <int DT, int LANES, int NV, bool FULL>
__global__ __launch_bounds__(kThreads<LANES>) void bwd_kernel(NormArgs a) {
  constexpr int V = Vec<DT>::n, TH = kThreads<LANES>, RW = TH / LANES;
  __shared__ float red[2][2][8];
  __shared__ float sums[RW > 1 ? TH * V : 1];
  int turn = 0;
  const Columns<DT, LANES, NV, FULL> cols(a.width);
  float w[NV][V], dw[NV][V], db[NV][V];
  cols.weights(w, a.w, a.w_dtype, 1.0f);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) dw[i][e] = db[i][e] = 0.0f;
  const float inv = 1.0f / (float)a.width;
  const int64_t step = (int64_t)gridDim.x * RW;
  int64_t row = (int64_t)blockIdx.x * RW + threadIdx.x / LANES;
  u32x4 xr[NV], dr[NV];
  float mean, rstd;
  const auto load = [&](int64_t r) {
    r = r < a.rows ? r : a.rows - 1;
    cols.load(xr, norm_row<DT>(a.x, a.x_s, r, a.n1));
    cols.load(dr, norm_row<DT>(a.dout, a.do_s, r, a.n1));
    mean = a.mean[r];
    rstd = a.rstd[r];
  };
  load(row);
  for (int64_t base = (int64_t)blockIdx.x * RW; base < a.rows; base += step, row += step) {
    const bool live = row < a.rows;
    const float mu = mean, rs = rstd;
    float x[NV][V], d[NV][V];
    float s1 = 0, s2 = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      cols.unpack(xr[i], x[i]);
      cols.unpack(dr[i], d[i]);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        x[i][e] = (x[i][e] - mu) * rs;
        const float dd = cols.mine(i, e) && live ? d[i][e] : 0.0f;
        dw[i][e] = __builtin_fmaf(dd, x[i][e], dw[i][e]);
        db[i][e] += dd;
        d[i][e] *= w[i][e];
        const float aa = FULL ? d[i][e] : cols.mine(i, e) ? d[i][e] : 0.0f;
        s1 += aa;
        s2 = __builtin_fmaf(aa, x[i][e], s2);
      }
    }
    if (base + step < a.rows) load(row + step);
    const f32x2 m = row_sums<LANES, 2>(f32x2{s1, s2}, red, turn) * inv;
    if (!live || !a.dx) continue;
    char* op = norm_row<DT>(a.dx, a.dx_s, row, a.n1);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float y[V];
#pragma unroll
      for (int e = 0; e < V; ++e) y[e] = rs * (d[i][e] - m[0] - x[i][e] * m[1]);
      cols.store(op, i, y);
    }
  }
  if (!a.part) return;
  // the workgroup's partial row: its RW threads of a column in their order
  float* part = a.part + (int64_t)blockIdx.x * 2 * a.width;
#pragma unroll
  for (int side = 0; side < 2; ++side)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float* src = side ? db[i] : dw[i];
      if constexpr (RW > 1) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < V; ++e) sums[threadIdx.x * V + e] = src[e];
        __syncthreads();
        for (int o = threadIdx.x; o < LANES * V; o += TH) {
          const int c = (i * LANES + o / V) * V, col = FULL || c + V <= a.width ? c : a.width - V, e = o % V;
          float s = 0;
#pragma unroll
          for (int r = 0; r < RW; ++r) s += sums[r * LANES * V + o];
          if (FULL || (c < a.width && e >= c - col)) part[side * (int64_t)a.width + col + e] = s;
        }
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (cols.mine(i, e)) part[side * (int64_t)a.width + cols.col[i] + e] = src[e];
      }
    }
}

// Column sums of the partial rows: a workgroup has 32 columns of one side, 32 threads a
// column, joined through LDS.
__global__ __launch_bounds__(1024) void reduce_kernel(NormArgs a) {
  __shared__ float t[32][33];
  const int side = blockIdx.y, c = threadIdx.x & 31, g = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
  void* out = side ? a.db : a.dw;
  if (!out) return;
  float all = 0;
  for (int r = g; col < a.width && r < a.groups;) {
    const int end = min(a.groups, r + 32 * kNormRun);
    float s = 0;
#pragma unroll 8
    for (; r < end; r += 32) s += a.part[((int64_t)r * 2 + side) * a.width + col];
    all += s;
  }
  t[g][c] = all;
  __syncthreads();
  for (int h = 16; h; h >>= 1) {
    if (g < h) t[g][c] += t[g + h][c];
    __syncthreads();
  }
  if (g == 0 && col < a.width) store_gate(out, a.w_dtype, col, t[0][c]);
}

// ---- rows wider than 512 threads hold (walked again for each sum; they stay in L2), or narrower than a vector ----
// 6700 rows of 20000 in bf16: forward 190 to 205 us, 2.7 TB/s of the row in and out; backward 405 to 419 us.

__device__ inline float block_sum(float v, float* red) {
  v = sum4rows(sum16(v));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0;
  for (int i = 0; i < 16; ++i) v += red[i];
  return v;
}

// A vector of such a row: the last one ends with the row; what it shares with the one before is not its own.
// Rows narrower than a vector are one vector, element by element.
template <int DT>
struct Piece16 {
  static constexpr int V = Vec<DT>::n, ES = DT == CCV_DT_F32 ? 4 : 2;
  int col, skip, n;
  __device__ inline Piece16(int i, int width)
      : col(i + V <= width ? i : width < V ? 0 : width - V), skip(i - col), n(width < V ? width : V) {}
  __device__ inline bool mine(int e) const { return e >= skip && e < n; }
  __device__ inline void load(const char* row, float* x) const {
    if (n == V) Columns<DT, 16, 1, false>::unpack(gload<u32x4>(reinterpret_cast<uintptr_t>(row) + (uint32_t)col * ES), x);
    else
      for (int e = 0; e < V; ++e) x[e] = e < n ? load1<DT>(row + e * ES) : 0.0f;
  }
  __device__ inline void store(char* row, const float* y) const {
    char* p = row + (uint32_t)col * ES;
    if (n < V) {
      for (int e = 0; e < n; ++e) store1<DT>(p + e * ES, y[e]);
    } else if constexpr (DT == CCV_DT_F32) {
      store16(p, F32::pack(y));
    } else if constexpr (DT == CCV_DT_BF16) {
      store16(p, BF16::pack(y));
    } else {
      store16(p, F16::pack(y));
    }
  }
  __device__ inline void weights(const void* p, int dtype, float other, float* w) const {
    if (p && n == V && dtype == CCV_DT_F32) {
#pragma unroll
      for (int e = 0; e < V; e += 4) F32::unpack(gload<u32x4>(reinterpret_cast<uintptr_t>(p) + ((uint32_t)col + e) * 4), w + e);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) w[e] = p && e < n ? load_param(p, dtype, col + e) : other;
    }
  }
};

template <int DT>
__global__ __launch_bounds__(1024) void wide_fwd_kernel(NormArgs a) {
  constexpr int V = Vec<DT>::n;
  __shared__ float red[16];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const char* xp = norm_row<DT>(a.x, a.x_s, row, a.n1);
    char* op = norm_row<DT>(a.out, a.o_s, row, a.n1);
    float s = 0, q = 0, x[V], w[V], b[V];
    for (int i = threadIdx.x * V; i < a.width; i += 1024 * V) {
      const Piece16<DT> p(i, a.width);
      p.load(xp, x);
#pragma unroll
      for (int e = 0; e < V; ++e) s += p.mine(e) ? x[e] : 0.0f;
    }
    const float mean = block_sum(s, red) / (float)a.width;
    for (int i = threadIdx.x * V; i < a.width; i += 1024 * V) {
      const Piece16<DT> p(i, a.width);
      p.load(xp, x);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = p.mine(e) ? x[e] - mean : 0.0f;
        q = __builtin_fmaf(d, d, q);
      }
    }
    const float rstd = 1.0f / __builtin_sqrtf(block_sum(q, red) / (float)a.width + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    for (int i = threadIdx.x * V; i < a.width; i += 1024 * V) {
      const Piece16<DT> p(i, a.width);
      p.load(xp, x);
      p.weights(a.w, a.w_dtype, 1.0f, w);
      p.weights(a.b, a.w_dtype, 0.0f, b);
#pragma unroll
      for (int e = 0; e < V; ++e) x[e] = __builtin_fmaf((x[e] - mean) * rstd, w[e], b[e]);
      p.store(op, x);
    }
  }
}

template <int DT>
__global__ __launch_bounds__(1024) void wide_dx_kernel(NormArgs a) {
  constexpr int V = Vec<DT>::n;
  __shared__ float red[16];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const char* xp = norm_row<DT>(a.x, a.x_s, row, a.n1);
    const char* dp = norm_row<DT>(a.dout, a.do_s, row, a.n1);
    char* op = norm_row<DT>(a.dx, a.dx_s, row, a.n1);
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s1 = 0, s2 = 0, x[V], d[V], w[V];
    for (int i = threadIdx.x * V; i < a.width; i += 1024 * V) {
      const Piece16<DT> p(i, a.width);
      p.load(xp, x);
      p.load(dp, d);
      p.weights(a.w, a.w_dtype, 1.0f, w);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float y = p.mine(e) ? d[e] * w[e] : 0.0f;
        s1 += y;
        s2 += p.mine(e) ? y * ((x[e] - mean) * rstd) : 0.0f;
      }
    }
    const float m1 = block_sum(s1, red) / (float)a.width, m2 = block_sum(s2, red) / (float)a.width;
    for (int i = threadIdx.x * V; i < a.width; i += 1024 * V) {
      const Piece16<DT> p(i, a.width);
      p.load(xp, x);
      p.load(dp, d);
      p.weights(a.w, a.w_dtype, 1.0f, w);
#pragma unroll
      for (int e = 0; e < V; ++e) x[e] = rstd * (d[e] * w[e] - m1 - (x[e] - mean) * rstd * m2);
      p.store(op, x);
    }
  }
}

// Partial sums of dw and db: a thread has one vector of columns, blockIdx.y its rows.
template <int DT>
__global__ __launch_bounds__(256) void wide_sums_kernel(NormArgs a) {
  constexpr int V = Vec<DT>::n;
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V;
  if (i >= a.width) return;
  const Piece16<DT> p((int)i, a.width);
  float dws[V] = {}, dbs[V] = {}, x[V], d[V];
  for (int64_t row = blockIdx.y; row < a.rows;) {
    const int64_t run = (int64_t)kNormRun * gridDim.y, end = a.rows - row > run ? row + run : a.rows;
    float dw[V] = {}, db[V] = {};
#pragma unroll 4
    for (; row < end; row += gridDim.y) {
      p.load(norm_row<DT>(a.dout, a.do_s, row, a.n1), d);
      p.load(norm_row<DT>(a.x, a.x_s, row, a.n1), x);
      const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        dw[e] = __builtin_fmaf(d[e], (x[e] - mean) * rstd, dw[e]);
        db[e] += d[e];
      }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      dws[e] += dw[e];
      dbs[e] += db[e];
    }
  }
#pragma unroll
  for (int e = 0; e < V; ++e)
    if (p.mine(e)) {
      a.part[((int64_t)blockIdx.y * 2) * a.width + p.col + e] = dws[e];
      a.part[((int64_t)blockIdx.y * 2 + 1) * a.width + p.col + e] = dbs[e];
    }
}

int64_t min64(int64_t x, int64_t y) { return x < y ? x : y; }

template <int DT, int LANES, int NV>
void go(const NormArgs& a, bool bwd, int grid, hipStream_t st) {
  constexpr int T = kThreads<LANES>;
  const bool full = a.width == LANES * NV * Vec<DT>::n;
  if (bwd && full) bwd_kernel<DT, LANES, NV, true><<<grid, T, 0, st>>>(a);
  else if (bwd) bwd_kernel<DT, LANES, NV, false><<<grid, T, 0, st>>>(a);
  else if (full) fwd_kernel<DT, LANES, NV, true><<<grid, T, 0, st>>>(a);
  else fwd_kernel<DT, LANES, NV, false><<<grid, T, 0, st>>>(a);
}
template <int DT, int LANES>
void go(const NormArgs& a, bool bwd, int nv, int grid, hipStream_t st) {
  if (nv == 1) return go<DT, LANES, 1>(a, bwd, grid, st);
  if constexpr (LANES == 16) return go<DT, LANES, 2>(a, bwd, grid, st);
  else return nv == 2 ? go<DT, LANES, 2>(a, bwd, grid, st) : go<DT, LANES, 4>(a, bwd, grid, st);
}
template <int DT>
void go(const NormArgs& a, bool bwd, int cus, hipStream_t st) {
  const NormShape s = norm_shape(a.width, DT == CCV_DT_F32 ? 4 : 2);
  if (!s.lanes) {
    const int grid = (int)min64(a.rows, 4096);
    if (!bwd) {
      wide_fwd_kernel<DT><<<grid, 1024, 0, st>>>(a);
    } else {
      if (a.dx) wide_dx_kernel<DT><<<grid, 1024, 0, st>>>(a);
      if (a.part) wide_sums_kernel<DT><<<dim3((a.width + 256 * Vec<DT>::n - 1) / (256 * Vec<DT>::n), a.groups), 256, 0, st>>>(a);
    }
    return;
  }
  const int rows_per = (s.lanes > 256 ? s.lanes : 256) / s.lanes;
  const int64_t need = (a.rows + rows_per - 1) / rows_per;
  const int grid = bwd ? a.groups : (int)min64(need, (int64_t)cus * (s.lanes > 256 ? 2 : 8));
  if (s.lanes == 16) go<DT, 16>(a, bwd, s.nv, grid, st);
  else if (s.lanes == 64) go<DT, 64>(a, bwd, s.nv, grid, st);
  else if (s.lanes == 256) go<DT, 256>(a, bwd, s.nv, grid, st);
  else go<DT, 512>(a, bwd, s.nv, grid, st);
}

void any(const NormArgs& a, bool bwd, int cus, hipStream_t st) {
  if (a.x_dtype == CCV_DT_F32) go<CCV_DT_F32>(a, bwd, cus, st);
  else if (a.x_dtype == CCV_DT_F16) go<CCV_DT_F16>(a, bwd, cus, st);
  else go<CCV_DT_BF16>(a, bwd, cus, st);
}

}  // namespace

int launch_norm_fwd(const NormArgs& a, int cus, void* stream) {
  any(a, false, cus, static_cast<hipStream_t>(stream));
  return (int)hipGetLastError();
}

int launch_norm_bwd(const NormArgs& a, void* stream) {
  const hipStream_t st = static_cast<hipStream_t>(stream);
  int e = 0;
  if (a.rows > 0) {
    any(a, true, 0, st);
    e = (int)hipGetLastError();
  }
  if (e || (!a.dw && !a.db)) return e;
  reduce_kernel<<<dim3((a.width + 31) / 32, 2), 1024, 0, st>>>(a);      // no rows: zeros
  return (int)hipGetLastError();
}

}  // namespace ccv
