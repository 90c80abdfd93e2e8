// ccv_linrec_bwd.hip -- gradients of the gated linear recurrence.
//
//   D[t] = dout[t] + E[t+1],  E[t] = e^g[t] D[t]      (E past a sequence's last step: dfinal_state)
//   dx[t] = s[t] D[t],  dg[t] = h[t-1] E[t] - (e^2g[t] / s[t]) x[t] D[t]  (the second part where x is normalised),
//   dinitial_state = E at a sequence's first step.
//
// E runs as the forward's h does, from the last step to the first: the same tiles, chain and
// maps, E <- A E + E' with A the product of the steps' decays, tiles taken last first.  h[t-1] is made again
// inside a tile from the state before it, which the forward left (or makes now).
//
// 2 x 4096 x 4096 in bf16, normalised: 83 us, 4.0 TB/s (the forward before it 50), with the vector units issuing for 63 % of that.
// Two workgroups a compute unit, in 128 registers (three, in 80: 235 us for the two calls against 152).  Normalised 16-bit data are 9 to 15
// registers more than that (40 to 64 bytes a lane through memory), fp32 x and dout 102 when normalised, else 43 (62 and 13 with 16-bit
// decays): fp32 calls of at most kFewTiles take one a compute unit, and spill none (normalised: 34 us for 1 x 16384 x 128 with two, 19 with
// one; 95 and 83 for 2 x 4096 x 2048, 2048 tiles; 167 and 174 for 2 x 4096 x 4096.  bf16: 36 and 41 for 2 x 4096 x 1024).
#include "ccv_linrec_device.hpp"

namespace ccv {
namespace {

// -(ds/dg) x / e^g = x e^g / s; 0 where s is.
__device__ inline float turned(float x, float a, float s) { return s > 0.0f ? x * (a * __builtin_amdgcn_rcpf(s)) : 0.0f; }

struct BwdShared {
  alignas(16) Map fmaps[kLrWaves][kLrChannels], rmaps[kLrWaves][kLrChannels];
  Heard heard;
};

template <int DT, int GT, bool NORM, bool MARKS>
__device__ __forceinline__ void bwd_tile(const LinrecArgs& a, const Place& at, int wave, Pair<DT> (&xr)[kLrSteps], Pair<DT> (&dr)[kLrSteps],
                                         const Pair<GT> (&gr)[kLrSteps], BwdShared& shared) {
  constexpr int S = kLrSteps;
  const int lane = threadIdx.x & 63, half = lane >> 5, slot = 2 * (lane & 31);
  float h[2], E[2] = {0.0f, 0.0f};
#pragma unroll
  for (int e = 0; e < 2; ++e) h[e] = a.carries[((int64_t)at.b * a.tiles + at.tile) * a.C + (at.c + e < a.C ? at.c + e : a.C - 1)];
  Marks marks{};
  if constexpr (MARKS) marks = marks_of(a, at);

  float A[S][2], W[S][2];                                  // decays and weights
  if (all_slow<GT>(gr)) {
#pragma unroll
    for (int j = 0; j < S; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float y;
        slow_decay(pair_value<GT>(gr[j], e), A[j][e], y);
        W[j][e] = NORM ? slow_weight(y) : 1.0f;
      }
  } else {
#pragma unroll
    for (int j = 0; j < S; ++j) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float y;
        decay(pair_value<GT>(gr[j], e), A[j][e], y);
        W[j][e] = NORM ? input_weight(y) : 1.0f;
      }
      __builtin_amdgcn_sched_barrier(0);                   // a step after the other, in few registers
    }
  }
  const auto in = [&](int j, int e) { return NORM ? W[j][e] * pair_value<DT>(xr[j], e) : pair_value<DT>(xr[j], e); };
  Map fwd[2] = {{1.0f, 0.0f}, {1.0f, 0.0f}}, rev[2] = {{1.0f, 0.0f}, {1.0f, 0.0f}};
#pragma unroll
  for (int j = 0; j < S; ++j) {
    [[maybe_unused]] const bool starts = marks.start >> j & 1;
    [[maybe_unused]] const int64_t seq = MARKS ? __shfl(marks.id, S * half + j) : 0;
    if constexpr (MARKS)
      if (marks.dead >> j & 1) {                           // a step that does nothing
        xr[j] = dr[j] = Pair<DT>{};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          A[j][e] = 1.0f;
          W[j][e] = 0.0f;
        }
      }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if constexpr (MARKS) {
        const float h0 = starts && a.init && (at.own >> e & 1) ? a.init[seq * a.init_s + at.c + e] : 0.0f;
        fwd[e] = then(fwd[e], starts ? Map{kCut, __builtin_fmaf(A[j][e], h0, in(j, e))} : Map{A[j][e], in(j, e)});
      } else {
        fwd[e].H = __builtin_fmaf(A[j][e], fwd[e].H, in(j, e));
        fwd[e].A *= A[j][e];
      }
    }
  }
#pragma unroll
  for (int j = S - 1; j >= 0; --j) {
    [[maybe_unused]] const bool ends = marks.end >> j & 1;
    [[maybe_unused]] const int64_t seq = MARKS ? __shfl(marks.id, S * half + j) : 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if constexpr (MARKS) {
        const float late = ends && a.dfinal && (at.own >> e & 1) ? a.dfinal[seq * a.df_s + at.c + e] : 0.0f;
        rev[e] = then(rev[e], Map{ends ? kCut : A[j][e], A[j][e] * (pair_value<DT>(dr[j], e) + late)});
      } else {
        rev[e].H = A[j][e] * (pair_value<DT>(dr[j], e) + rev[e].H);
      }
    }
  }
  if constexpr (!MARKS)
#pragma unroll
    for (int e = 0; e < 2; ++e) rev[e].A = fwd[e].A;
  Map early[2], late[2];                                   // of the other half: before this one's steps, behind them
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    early[e] = other_half(fwd[e]);
    late[e] = other_half(rev[e]);
    if (half) shared.fmaps[wave][slot + e] = then(early[e], fwd[e]);
    else shared.rmaps[wave][slot + e] = then(late[e], rev[e]);
  }
  lds_barrier();
  if (a.tiles > 1) {
    exchange(a, at, wave, shared.heard, [&]() {
      Map m = shared.rmaps[kLrWaves - 1][lane];
#pragma unroll
      for (int w = kLrWaves - 2; w >= 0; --w) m = then(m, shared.rmaps[w][lane]);
      return m;
    });
    state_before(a, at, shared.heard, slot, E);
  }
  apply_parts<false>(shared.fmaps, wave, slot, h);
  apply_parts<true>(shared.rmaps, wave + 1, slot, E);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (half) h[e] = apply(early[e], h[e]);
    else E[e] = apply(late[e], E[e]);
  }

  // For each step h[t-1], less what its weight adds: dg is that times E.  Then the steps from the last to the first.  What
  // was made of x and dout before is made again, not kept in registers.
  hide_steps(xr);
  hide_steps(dr);
  float G[S][2];
#pragma unroll
  for (int j = 0; j < S; ++j) {
    [[maybe_unused]] const bool starts = marks.start >> j & 1;
    [[maybe_unused]] const int64_t seq = MARKS ? __shfl(marks.id, S * half + j) : 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if constexpr (MARKS)
        if (starts) h[e] = a.init && (at.own >> e & 1) ? a.init[seq * a.init_s + at.c + e] : 0.0f;
      G[j][e] = NORM ? h[e] - turned(pair_value<DT>(xr[j], e), A[j][e], W[j][e]) : h[e];
      h[e] = __builtin_fmaf(A[j][e], h[e], in(j, e));
    }
  }
#pragma unroll
  for (int j = S - 1; j >= 0; --j) {
    [[maybe_unused]] const bool starts = marks.start >> j & 1, ends = marks.end >> j & 1, none = marks.dead >> j & 1;
    [[maybe_unused]] const int64_t seq = MARKS ? __shfl(marks.id, S * half + j) : 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if constexpr (MARKS)
        if (ends) E[e] = a.dfinal && (at.own >> e & 1) ? a.dfinal[seq * a.df_s + at.c + e] : 0.0f;
      const float d = pair_value<DT>(dr[j], e) + E[e];
      E[e] = A[j][e] * d;
      if constexpr (MARKS)
        if (starts && a.dinit && (at.own >> e & 1)) a.dinit[seq * a.di_s + at.c + e] = E[e];
      G[j][e] = MARKS && none ? 0.0f : G[j][e] * E[e];
      W[j][e] = MARKS && none ? 0.0f : NORM ? W[j][e] * d : d;
    }
  }
  store_steps<DT>(a.dx, a.dx_s, at, a.L, W);
  store_steps<GT>(a.dg, a.dg_s, at, a.L, G);
}

constexpr uint32_t kFewTiles = 2048;

template <int DT, int GT, bool NORM, int GROUPS>
__global__ __launch_bounds__(64 * kLrWaves, 2 * GROUPS) void bwd_kernel(const LinrecArgs a) {
  __shared__ BwdShared shared;
  __shared__ uint32_t ticket[2];
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const Place at = place_of<true>(a, take_ticket(a, ticket), wave);
  Pair<DT> xr[kLrSteps], dr[kLrSteps];
  Pair<GT> gr[kLrSteps];
  load_steps<false>(gr, a.g, a.g_s, at, a.L, a.C);
  load_steps<false>(xr, a.x, a.x_s, at, a.L, a.C);
  load_steps<false>(dr, a.dout, a.do_s, at, a.L, a.C);
  if (has_marks(a, at)) bwd_tile<DT, GT, NORM, true>(a, at, wave, xr, dr, gr, shared);
  else bwd_tile<DT, GT, NORM, false>(a, at, wave, xr, dr, gr, shared);
}

}  // namespace

int launch_linrec_bwd(const LinrecArgs& a, void* stream) {
  by_types(a.x_dtype, a.g_dtype, [&](auto dt, auto gt) {
    constexpr int DT = decltype(dt)::value, GT = decltype(gt)::value;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const uint32_t grid = a.tiles * a.chains;
    if constexpr (DT == CCV_DT_F32)
      if (grid <= kFewTiles) {
        if (a.normalize) bwd_kernel<DT, GT, true, 1><<<grid, 64 * kLrWaves, 0, st>>>(a);
        else bwd_kernel<DT, GT, false, 1><<<grid, 64 * kLrWaves, 0, st>>>(a);
        return;
      }
    if (a.normalize) bwd_kernel<DT, GT, true, 2><<<grid, 64 * kLrWaves, 0, st>>>(a);
    else bwd_kernel<DT, GT, false, 2><<<grid, 64 * kLrWaves, 0, st>>>(a);
  });
  return (int)hipGetLastError();
}

}  // namespace ccv
