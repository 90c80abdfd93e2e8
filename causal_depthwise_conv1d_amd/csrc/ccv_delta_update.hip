// ccv_delta_update.hip -- gated delta rule: a few new steps against states in a cache,
// advanced in place (decoding).
//
//   S <- e^g S;  u = beta (v - S^T k);  S <- S + k u^T;  o = scale S^T q,
// the last as scale ((e^g S)^T q + (k.q) u), so that both products with S come from one look
// at it.  A step reads and writes its fp32 state once and little else: bound by memory.
// One wave takes 32 values of a head (a 128-byte line of each of the state's rows): lane l
// holds values 4 (l % 8) .. + 3 of RPT consecutive rows, RPT = 8 or 16 for up to 64 or 128
// keys, the sums over rows finish across the wave's eight row groups, and no LDS or
// barrier is needed.  The state stays in registers over the call's steps.  Bound by the state's way in
// and out: 256 rows of 32 heads of 128 x 128, 1.08 GB, 204 us, 5.3 TB/s; 5 rows of 20 heads are two round
// trips to memory, the slot's number before the state, and the launch: 7.2 us (8.6 with a branch around each load).
#include "ccv_delta_device.hpp"

namespace ccv {
namespace {

// Sum over lanes l, l + 8, ..., l + 56.
__device__ inline float sum8rows(float v) {
  v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x128, 0xf, 0xf, true));
  return sum4rows(v);
}

// A gate as stored, of either size, and its value: both loads stand, so that no branch waits for one.
struct Gate { uint16_t h; uint32_t w; };
__device__ inline Gate gate_at(const void* p, int dtype, int64_t i) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p) + i * (dtype == CCV_DT_F32 ? 4 : 2), none = reinterpret_cast<uintptr_t>(kZeroSrc);
  return {gload<uint16_t>(at), gload<uint32_t>(pick(dtype == CCV_DT_F32, at, none))};
}
__device__ inline float gate_value(Gate g, int dtype) {
  return dtype == CCV_DT_F32 ? __builtin_bit_cast(float, g.w) : dtype == CCV_DT_BF16 ? BF16::to_f(g.h) : F16::to_f(g.h);
}

// Four consecutive elements where the lane has them, else zeros.  VEC: whole vectors, without a branch.
template <int DT, bool VEC>
__device__ inline Raw4<DT> take4(const void* p, int left) {
  if constexpr (VEC) {
    const uintptr_t at = pick(left > 0, reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(kZeroSrc));
    if constexpr (DT == CCV_DT_F32) return {gload<u32x4>(at)};
    const u32x2 d = gload<u32x2>(at);
    return {u32x4{d[0], d[1], 0, 0}};
  } else {
    Raw4<DT> r{};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= left) continue;
      if constexpr (DT == CCV_DT_F32) r.d[i] = static_cast<const uint32_t*>(p)[i];
      else r.d[i / 2] |= (uint32_t) static_cast<const uint16_t*>(p)[i] << (16 * (i % 2));
    }
    return r;
  }
}

template <int DT, int RPT, bool VEC>
__global__ __launch_bounds__(256) void step_kernel(DeltaStepArgs a, int32_t nslice, int64_t items) {
  constexpr int ES = DT == CCV_DT_F32 ? 4 : 2;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (item >= items) return;
  const int slice = (int)(item % nslice);
  const int64_t bh = item / nslice;
  const int b = (int)(bh / a.Hv), h = (int)(bh - (int64_t)b * a.Hv), hk = h / (a.Hv / a.Hk);
  const int l = threadIdx.x & 63, rg = l >> 3, dv = 32 * slice + 4 * (l & 7), left = a.Dv - dv;
  // a step's inputs, under way before the slot's number is known
  Raw4<DT> rk[RPT / 4], rq[RPT / 4], rv;
  Gate gd, gb;
  const auto load = [&](int t) {
    const char* kp = row_ptr<DT>(a.k, a.k_s, b, t, hk) + RPT * rg * ES;
    const char* qp = row_ptr<DT>(a.q, a.q_s, b, t, hk) + RPT * rg * ES;
#pragma unroll
    for (int i = 0; i < RPT; i += 4) {
      rk[i / 4] = take4<DT, VEC>(kp + i * ES, a.Dk - RPT * rg - i);
      rq[i / 4] = take4<DT, VEC>(qp + i * ES, a.Dk - RPT * rg - i);
    }
    rv = take4<DT, VEC>(row_ptr<DT>(a.v, a.v_s, b, t, h) + dv * ES, left);
    gd = gate_at(a.g, a.g_dtype, b * a.g_s[0] + t * a.g_s[1] + h * a.g_s[2]);
    gb = gate_at(a.beta, a.b_dtype, b * a.b_s[0] + t * a.b_s[1] + h * a.b_s[2]);
  };
  load(0);
  const int64_t slot = a.slots ? a.slots[b] : b;
  if (slot < 0 || slot >= a.nslots) {               // an idle row: its state is nobody's
    if (rg == 0)
      for (int t = 0; t < a.T; ++t)
        store4<DT>(row_ptr<DT>(a.out, a.o_s, b, t, h) + dv * ES, f32x4{0, 0, 0, 0}, left, VEC);
    return;
  }
  float* st = a.state + slot * a.st_s[0] + h * a.st_s[1] + dv;
  f32x4 S[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int dk = RPT * rg + i;
    S[i] = widen4<CCV_DT_F32>(take4<CCV_DT_F32, VEC>(st + dk * a.st_s[2], dk < a.Dk ? left : 0));
  }
  for (int t = 0; t < a.T; ++t) {
    float k[RPT], q[RPT];
#pragma unroll
    for (int i = 0; i < RPT; i += 4) {
      const f32x4 k4 = widen4<DT>(rk[i / 4]), q4 = widen4<DT>(rq[i / 4]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        k[i + e] = k4[e];
        q[i + e] = q4[e];
      }
    }
    const f32x4 v = widen4<DT>(rv);
    const float alpha = __builtin_amdgcn_exp2f(gate_value(gd, a.g_dtype) * kLog2e), beta = gate_value(gb, a.b_dtype);
    if (t + 1 < a.T) load(t + 1);
    f32x4 sk = {0, 0, 0, 0}, sq = {0, 0, 0, 0};
    float kq = 0;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        S[i][e] *= alpha;
        sk[e] = __builtin_fmaf(S[i][e], k[i], sk[e]);
        sq[e] = __builtin_fmaf(S[i][e], q[i], sq[e]);
      }
      kq = __builtin_fmaf(k[i], q[i], kq);
    }
    kq = sum8rows(kq);
    f32x4 u, o;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      u[e] = beta * (v[e] - sum8rows(sk[e]));
      o[e] = a.scale * __builtin_fmaf(kq, u[e], sum8rows(sq[e]));
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[i][e] = __builtin_fmaf(k[i], u[e], S[i][e]);
    if (rg == 0) store4<DT>(row_ptr<DT>(a.out, a.o_s, b, t, h) + dv * ES, o, left, VEC);
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int dk = RPT * rg + i;
    if (dk < a.Dk) store4<CCV_DT_F32>(st + dk * a.st_s[2], S[i], left, VEC);
  }
}

template <int DT>
void launch(const DeltaStepArgs& a, hipStream_t st) {
  const int32_t nslice = (a.Dv + 31) / 32;
  const int64_t items = (int64_t)a.B * a.Hv * nslice;
  const dim3 grid((uint32_t)((items + 3) / 4));
  if (a.Dk <= 64) {
    if (a.vec) step_kernel<DT, 8, true><<<grid, 256, 0, st>>>(a, nslice, items);
    else step_kernel<DT, 8, false><<<grid, 256, 0, st>>>(a, nslice, items);
  } else {
    if (a.vec) step_kernel<DT, 16, true><<<grid, 256, 0, st>>>(a, nslice, items);
    else step_kernel<DT, 16, false><<<grid, 256, 0, st>>>(a, nslice, items);
  }
}

}  // namespace

int launch_delta_step(const DeltaStepArgs& a, void* stream) {
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (a.x_dtype == CCV_DT_F32) launch<CCV_DT_F32>(a, st);
  else if (a.x_dtype == CCV_DT_F16) launch<CCV_DT_F16>(a, st);
  else launch<CCV_DT_BF16>(a, st);
  return (int)hipGetLastError();
}

}  // namespace ccv
