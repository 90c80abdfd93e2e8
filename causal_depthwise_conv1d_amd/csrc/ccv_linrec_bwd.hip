// ccv_linrec_bwd.hip -- gradients of the gated linear recurrence.
//
//   D[t] = dout[t] + E[t+1],  E[t] = e^g[t] D[t]      (E past a sequence's last step: dfinal_state)
//   dx[t] = s[t] D[t],  dg[t] = h[t-1] E[t] - (e^2g[t] / s[t]) x[t] D[t]  (the second part where x is normalised),
//   dinitial_state = E at a sequence's first step.
//
// E runs as the forward's h does, from the last step to the first: the same tiles, chain and
// maps, E <- A E + E' with A the product of the steps' decays, tiles taken last first.  h[t-1] is made again
// inside a tile from the state before it, which the forward left (or makes now).
#include "ccv_linrec_device.hpp"

namespace ccv {
namespace {

template <int DT, int GT, bool NORM>
__global__ __launch_bounds__(512, 4) void bwd_kernel(const LinrecArgs a) {
  constexpr int S = kLrSteps;
  __shared__ f32x4 fmaps[kLrRows][32], rmaps[kLrRows][32];     // (A, H) and (A, E) of two channels
  __shared__ LrWait wait;
  __shared__ uint32_t ticket;
  const uint32_t item = take_ticket(a, &ticket);
  const uint32_t turn = item / a.chains, chain = item - turn * a.chains, tile = a.tiles - 1 - turn;
  const uint32_t b = chain / a.cblocks, cb = chain - b * a.cblocks;
  const LrLane me(cb, a.C);
  const bool one = a.C < 2;
  const int64_t T = (int64_t)tile * kLrTile + 2 * S * me.wave;
  const bool tail = T + 2 * S > a.L;

  Pair<DT> xr[S], dr[S];
  Pair<GT> gr[S];
  const char* xb = static_cast<const char*>(a.x) + (b * a.x_s[0] + T * a.x_s[1]) * kBytes<DT>;
  const char* db = static_cast<const char*>(a.dout) + (b * a.do_s[0] + T * a.do_s[1]) * kBytes<DT>;
  const char* gb = static_cast<const char*>(a.g) + (b * a.g_s[0] + T * a.g_s[1]) * kBytes<GT>;
  if (!tail) {
    const uint32_t xo = (uint32_t)((me.half * S * a.x_s[1] + me.c) * kBytes<DT>);
    const uint32_t od = (uint32_t)((me.half * S * a.do_s[1] + me.c) * kBytes<DT>);
    const uint32_t go = (uint32_t)((me.half * S * a.g_s[1] + me.c) * kBytes<GT>);
#pragma unroll
    for (int j = 0; j < S; ++j) {
      gr[j] = load_pair<GT>(gb + j * a.g_s[1] * kBytes<GT>, go, one);
      xr[j] = load_pair<DT>(xb + j * a.x_s[1] * kBytes<DT>, xo, one);
      dr[j] = load_pair<DT>(db + j * a.do_s[1] * kBytes<DT>, od, one);
    }
  } else {                                                 // steps past the last are read as it
#pragma unroll
    for (int j = 0; j < S; ++j) {
      const int64_t t = T + S * me.half + j, d = (t < a.L ? t : a.L - 1) - T;
      gr[j] = load_pair<GT>(gb + d * a.g_s[1] * kBytes<GT>, me.c * kBytes<GT>, one);
      xr[j] = load_pair<DT>(xb + d * a.x_s[1] * kBytes<DT>, me.c * kBytes<DT>, one);
      dr[j] = load_pair<DT>(db + d * a.do_s[1] * kBytes<DT>, me.c * kBytes<DT>, one);
    }
  }
  float h[2], E[2] = {0.0f, 0.0f};
#pragma unroll
  for (int e = 0; e < 2; ++e) h[e] = a.carries[((int64_t)b * a.tiles + tile) * a.C + me.c + (one ? 0 : e)];
  const Marks marks = marks_at(a, b, T);
  const uint32_t start = marks.start >> (S * me.half), end = marks.end >> (S * me.half), dead = marks.dead >> (S * me.half);

  float A[S][2], W[S][2], D[S][2];                         // decays, weights, dout and what joins it
  Map fwd[2] = {{1.0f, 0.0f}, {1.0f, 0.0f}}, rev[2] = {{1.0f, 0.0f}, {1.0f, 0.0f}};
  float h0[S][2];                                          // of sequences that start here, 0 elsewhere
#pragma unroll
  for (int j = 0; j < S; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float y;
      decay(pair_value<GT>(gr[j], e), A[j][e], y);
      W[j][e] = NORM ? input_weight(y) : 1.0f;
      D[j][e] = pair_value<DT>(dr[j], e);
      h0[j][e] = 0.0f;
    }
  if (!marks.any) {
#pragma unroll
    for (int j = 0; j < S; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        fwd[e].H = __builtin_fmaf(A[j][e], fwd[e].H, NORM ? W[j][e] * pair_value<DT>(xr[j], e) : pair_value<DT>(xr[j], e));
        fwd[e].A *= A[j][e];
        rev[e].H = A[S - 1 - j][e] * (D[S - 1 - j][e] + rev[e].H);
      }
#pragma unroll
    for (int e = 0; e < 2; ++e) rev[e].A = fwd[e].A;
  } else {
#pragma unroll
    for (int j = 0; j < S; ++j) {
      const bool starts = start >> j & 1, ends = end >> j & 1, none = dead >> j & 1;
      const int64_t seq = __shfl(marks.id, S * me.half + j);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (none) {                                        // a step that does nothing
          A[j][e] = 1.0f;
          W[j][e] = D[j][e] = 0.0f;
        }
        const bool mine = e + me.own >= 2;
        if (ends && a.dfinal && mine) D[j][e] += a.dfinal[seq * a.df_s + me.c + (one ? 0 : e)];
        if (starts && a.init && mine) h0[j][e] = a.init[seq * a.init_s + me.c + (one ? 0 : e)];
        const float x = none ? 0.0f : pair_value<DT>(xr[j], e), in = NORM ? W[j][e] * x : x;
        fwd[e] = then(fwd[e], starts ? Map{kCut, __builtin_fmaf(A[j][e], h0[j][e], in)} : Map{A[j][e], in});
      }
    }
#pragma unroll
    for (int j = S - 1; j >= 0; --j) {
      const bool ends = end >> j & 1;
#pragma unroll
      for (int e = 0; e < 2; ++e) rev[e] = then(rev[e], Map{ends ? kCut : A[j][e], A[j][e] * D[j][e]});
    }
  }
  fmaps[me.row][threadIdx.x & 31] = f32x4{fwd[0].A, fwd[0].H, fwd[1].A, fwd[1].H};
  rmaps[me.row][threadIdx.x & 31] = f32x4{rev[0].A, rev[0].H, rev[1].A, rev[1].H};
  lds_barrier();
  Map after[2] = {{1.0f, 0.0f}, {1.0f, 0.0f}};             // of the tile's steps behind the lane's
#pragma unroll 4
  for (int r = kLrRows - 1; r > me.row; --r) {
    const f32x4 m = rmaps[r][threadIdx.x & 31];
#pragma unroll
    for (int e = 0; e < 2; ++e) after[e] = then(after[e], Map{m[2 * e], m[2 * e + 1]});
  }
  if (a.tiles > 1) {
    const bool last = me.row == 0 && tile > 0;
    Map all[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      all[e] = then(after[e], rev[e]);
      if (last) put(map_word(a, chain, turn, me.slot + e), all[e]);
    }
    if (turn > 0) wait_state(a, me, chain, turn, wait, E);
    if (last && turn % kLrGroup == kLrGroup - 1)
#pragma unroll
      for (int e = 0; e < 2; ++e) put(state_word(a, chain, turn / kLrGroup, me.slot + e), Map{0.0f, apply(all[e], E[e])});
  }
#pragma unroll 4
  for (int r = 0; r < me.row; ++r) {
    const f32x4 m = fmaps[r][threadIdx.x & 31];
#pragma unroll
    for (int e = 0; e < 2; ++e) h[e] = apply(Map{m[2 * e], m[2 * e + 1]}, h[e]);
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) E[e] = apply(after[e], E[e]);

  // h before each step, then the steps from the last to the first
  float hp[S][2];
  char* xo = static_cast<char*>(a.dx) + (b * a.dx_s[0] + T * a.dx_s[1] - one) * kBytes<DT>;
  char* go = static_cast<char*>(a.dg) + (b * a.dg_s[0] + T * a.dg_s[1] - one) * kBytes<GT>;
  const uint32_t xoff = (uint32_t)((me.half * S * a.dx_s[1] + me.c) * kBytes<DT>), goff = (uint32_t)((me.half * S * a.dg_s[1] + me.c) * kBytes<GT>);
#pragma unroll
  for (int j = 0; j < S; ++j) {
    const bool starts = marks.any && (start >> j & 1), none = marks.any && (dead >> j & 1);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      hp[j][e] = starts ? h0[j][e] : h[e];
      const float x = none ? 0.0f : pair_value<DT>(xr[j], e);
      h[e] = __builtin_fmaf(A[j][e], hp[j][e], NORM ? W[j][e] * x : x);
    }
  }
#pragma unroll
  for (int j = S - 1; j >= 0; --j) {
    const bool starts = start >> j & 1, ends = end >> j & 1, none = dead >> j & 1;
    const int64_t seq = __shfl(marks.id, S * me.half + j);
    float dx[2], dg[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float d = marks.any && ends ? D[j][e] : D[j][e] + E[e];
      E[e] = A[j][e] * d;
      dx[e] = NORM ? W[j][e] * d : d;
      dg[e] = hp[j][e] * E[e];
      if (NORM) {
        const float turned = W[j][e] > 0.0f ? A[j][e] * __builtin_amdgcn_rcpf(W[j][e]) : 0.0f;      // -ds/dg / e^g
        dg[e] = __builtin_fmaf(-pair_value<DT>(xr[j], e) * turned, E[e], dg[e]);
      }
      if (marks.any) {
        if (starts && a.dinit && e + me.own >= 2) a.dinit[seq * a.di_s + me.c + (one ? 0 : e)] = E[e];
        if (none) dx[e] = dg[e] = 0.0f;
      }
    }
    if (!tail || T + S * me.half + j < a.L) {
      store_pair<DT>(xo + j * a.dx_s[1] * kBytes<DT>, xoff, dx[0], dx[1], me.own);
      store_pair<GT>(go + j * a.dg_s[1] * kBytes<GT>, goff, dg[0], dg[1], me.own);
    }
  }
}

}  // namespace

int launch_linrec_bwd(const LinrecArgs& a, void* stream) {
  by_types(a.x_dtype, a.g_dtype, [&](auto dt, auto gt) {
    constexpr int DT = decltype(dt)::value, GT = decltype(gt)::value;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (a.normalize) bwd_kernel<DT, GT, true><<<a.tiles * a.chains, 512, 0, st>>>(a);
    else bwd_kernel<DT, GT, false><<<a.tiles * a.chains, 512, 0, st>>>(a);
  });
  return (int)hipGetLastError();
}

}  // namespace ccv
