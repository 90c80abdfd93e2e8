// ccv_norm_device.hpp -- parts shared by the kernels of layer norm and of group norm: a row's vectors in
// its threads' registers, sums over a row, sums of partial rows.
#pragma once

#include "ccv_delta_device.hpp"
#include "ccv_norm_launch.hpp"

namespace ccv {

template <int DT> struct Vec { static constexpr int n = DT == CCV_DT_F32 ? 4 : 8; };

// Sum over the 4 lanes of a quad; every one of them gets it.
__device__ inline float sum4(float v) {
  v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0xb1, 0xf, 0xf, true));   // lanes 1 0 3 2
  v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x4e, 0xf, 0xf, true));   // lanes 2 3 0 1
  return v;
}

// Sums over the `LANES` threads of a row of N values; every one of them gets them.  Rows of more
// than a wave: through `red`, two pieces of it in turn, so that one barrier suffices.
template <int LANES, int N>
__device__ inline f32x2 row_sums(f32x2 v, float (*red)[2][8], int& turn) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    float s = LANES == 4 ? sum4(v[n]) : sum16(v[n]);
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

// Column sums of `groups` partial rows [2][width] of dw and db: a workgroup of 1024 has 32 columns of one side
// (blockIdx.y), 32 threads a column, joined through LDS.
__device__ inline void sum_partials(const float* part, int groups, int width, void* dw, void* db, int w_dtype) {
  __shared__ float t[32][33];
  const int side = blockIdx.y, c = threadIdx.x & 31, g = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
  void* out = side ? db : dw;
  if (!out) return;
  float all = 0;
  for (int r = g; col < width && r < groups;) {
    const int end = min(groups, r + 32 * kNormRun);
    float s = 0;
#pragma unroll 8
    for (; r < end; r += 32) s += part[((int64_t)r * 2 + side) * width + col];
    all += s;
  }
  t[g][c] = all;
  __syncthreads();
  for (int h = 16; h; h >>= 1) {
    if (g < h) t[g][c] += t[g + h][c];
    __syncthreads();
  }
  if (g == 0 && col < width) store_gate(out, w_dtype, col, t[0][c]);
}

}  // namespace ccv
