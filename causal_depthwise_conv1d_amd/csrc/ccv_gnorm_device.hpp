// ccv_gnorm_device.hpp -- what group norm's forward and backward kernels share: a thread's place and the
// activation.
#pragma once

#include <type_traits>

#include "ccv_norm_device.hpp"

namespace ccv {

// act(v) and act'(v).
__device__ inline float act_value(float v, int silu_on) { return silu_on ? silu(v) : v; }
__device__ inline void act_both(float v, int silu_on, float& value, float& slope) {
  if (silu_on) {
    const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -kLog2e));
    value = v * s;
    slope = __builtin_fmaf(value, 1.0f - s, s);
  } else {
    value = v;
    slope = 1.0f;
  }
}

// Threads of `lanes` that walk the rows of one group: `group` and first row.  The same group for every row, so that
// its weights and their gradients' sums stay in registers.
struct Walker { uint32_t group, row; bool idle; };
template <int LANES>
__device__ inline Walker walker_at(const GroupNormArgs& a) {
  const uint32_t slot = blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  Walker w;
  w.row = slot / (uint32_t)a.groups;
  w.group = slot - w.row * (uint32_t)a.groups;
  w.idle = w.row >= (uint32_t)a.walkers;
  return w;
}

// f(type, lanes, vectors, full, gated) with constants, for the shapes that group_norm_shape gives.
template <class F>
inline void by_shape(const GroupNormArgs& a, F f) {
  const auto on_dt = [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    const NormShape s = group_norm_shape(a.width, DT == CCV_DT_F32 ? 4 : 2);
    const bool full = a.width == s.lanes * s.nv * Vec<DT>::n;
    const auto on_gate = [&](auto lanes, auto nv, auto whole) {
      if (a.z) f(dt, lanes, nv, whole, std::true_type{});
      else f(dt, lanes, nv, whole, std::false_type{});
    };
    const auto on_full = [&](auto lanes, auto nv) {
      if (full) on_gate(lanes, nv, std::true_type{});
      else on_gate(lanes, nv, std::false_type{});
    };
    const auto on_nv = [&](auto lanes) {
      if (s.nv == 1) return on_full(lanes, std::integral_constant<int, 1>{});
      if constexpr (decltype(lanes)::value == 256)
        if (s.nv == 4) return on_full(lanes, std::integral_constant<int, 4>{});
      on_full(lanes, std::integral_constant<int, 2>{});
    };
    if (s.lanes == 4) on_nv(std::integral_constant<int, 4>{});
    else if (s.lanes == 16) on_nv(std::integral_constant<int, 16>{});
    else if (s.lanes == 64) on_nv(std::integral_constant<int, 64>{});
    else on_nv(std::integral_constant<int, 256>{});
  };
  if (a.x_dtype == CCV_DT_F32) on_dt(std::integral_constant<int, CCV_DT_F32>{});
  else if (a.x_dtype == CCV_DT_F16) on_dt(std::integral_constant<int, CCV_DT_F16>{});
  else on_dt(std::integral_constant<int, CCV_DT_BF16>{});
}

template <class F>
inline void by_type(const GroupNormArgs& a, F f) {
  if (a.x_dtype == CCV_DT_F32) f(std::integral_constant<int, CCV_DT_F32>{});
  else if (a.x_dtype == CCV_DT_F16) f(std::integral_constant<int, CCV_DT_F16>{});
  else f(std::integral_constant<int, CCV_DT_BF16>{});
}

// Groups that no vector kernel takes: by one thread each, or one workgroup each.
template <int THREADS>
__device__ inline float any_sum(float v, float* red) {
  if constexpr (THREADS == 1) return v;
  v = sum4rows(sum16(v));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0;
  for (int i = 0; i < THREADS / 64; ++i) v += red[i];
  return v;
}
template <int DT>
__device__ inline const char* at(const void* p, int64_t i) { return static_cast<const char*>(p) + i * (DT == CCV_DT_F32 ? 4 : 2); }
template <int DT>
__device__ inline char* at(void* p, int64_t i) { return static_cast<char*>(p) + i * (DT == CCV_DT_F32 ? 4 : 2); }

}  // namespace ccv
