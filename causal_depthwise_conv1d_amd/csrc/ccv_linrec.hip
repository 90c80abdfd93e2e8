// ccv_linrec.hip -- gated linear recurrence: one state a channel, over whole sequences and step by
// step.
//
//   h <- e^g[t] h + s[t] x[t],  out[t] = h;   s = 1, or sqrt(1 - e^2g) where x is normalised.
//
// One pass over the data.  A workgroup takes a tile of 128 steps and 64 channels into registers: pairs of
// channels a lane, 32 lanes a row, 8 consecutive steps a lane, so that loads are whole 128-byte
// lines and a lane walks its steps with one fused multiply-add each.  Each lane makes the map
// (A, H) of its 8 steps, folds those of the lanes before it out of LDS, and the tiles of a
// sequence pass their maps on through memory (ccv_linrec_device.hpp), so x and g are read once.
// With the state before its steps a lane walks them again from registers and stores.
#include "ccv_linrec_device.hpp"

#include <algorithm>

namespace ccv {
namespace {

template <int DT, int GT, bool NORM>
__global__ __launch_bounds__(512, 4) void fwd_kernel(const LinrecArgs a) {
  constexpr int S = kLrSteps;
  __shared__ f32x4 maps[kLrRows][32];                      // (A, H) of two channels
  __shared__ LrWait wait;
  __shared__ uint32_t ticket;
  const uint32_t item = take_ticket(a, &ticket);
  const uint32_t tile = item / a.chains, chain = item - tile * a.chains;
  const uint32_t b = chain / a.cblocks, cb = chain - b * a.cblocks;
  const LrLane me(cb, a.C);
  const bool one = a.C < 2;
  const int64_t T = (int64_t)tile * kLrTile + 2 * S * me.wave;       // the wave's first step
  const bool tail = T + 2 * S > a.L;

  Pair<DT> xr[S];
  Pair<GT> gr[S];
  const char* xb = static_cast<const char*>(a.x) + (b * a.x_s[0] + T * a.x_s[1]) * kBytes<DT>;
  const char* gb = static_cast<const char*>(a.g) + (b * a.g_s[0] + T * a.g_s[1]) * kBytes<GT>;
  if (!tail) {
    const uint32_t xo = (uint32_t)((me.half * S * a.x_s[1] + me.c) * kBytes<DT>);
    const uint32_t go = (uint32_t)((me.half * S * a.g_s[1] + me.c) * kBytes<GT>);
#pragma unroll
    for (int j = 0; j < S; ++j) {
      gr[j] = load_pair<GT>(gb + j * a.g_s[1] * kBytes<GT>, go, one);
      xr[j] = load_pair<DT>(xb + j * a.x_s[1] * kBytes<DT>, xo, one);
    }
  } else {                                                 // steps past the last are read as it
#pragma unroll
    for (int j = 0; j < S; ++j) {
      const int64_t t = T + S * me.half + j, d = (t < a.L ? t : a.L - 1) - T;
      gr[j] = load_pair<GT>(gb + d * a.g_s[1] * kBytes<GT>, me.c * kBytes<GT>, one);
      xr[j] = load_pair<DT>(xb + d * a.x_s[1] * kBytes<DT>, me.c * kBytes<DT>, one);
    }
  }
  const Marks marks = marks_at(a, b, T);
  const uint32_t start = marks.start >> (S * me.half), end = marks.end >> (S * me.half), dead = marks.dead >> (S * me.half);

  float A[S][2], H[S][2];
  Map own[2] = {{1.0f, 0.0f}, {1.0f, 0.0f}};
#pragma unroll
  for (int j = 0; j < S; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float y;
      decay(pair_value<GT>(gr[j], e), A[j][e], y);
      const float x = pair_value<DT>(xr[j], e);
      H[j][e] = NORM ? input_weight(y) * x : x;
    }
  if (!marks.any) {
#pragma unroll
    for (int j = 0; j < S; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        own[e].H = __builtin_fmaf(A[j][e], own[e].H, H[j][e]);
        own[e].A *= A[j][e];
      }
  } else {
#pragma unroll
    for (int j = 0; j < S; ++j) {
      const bool starts = start >> j & 1, none = dead >> j & 1;
      const int64_t seq = __shfl(marks.id, S * me.half + j);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (starts) {
          if (a.init && e + me.own >= 2) H[j][e] = __builtin_fmaf(A[j][e], a.init[seq * a.init_s + me.c + (one ? 0 : e)], H[j][e]);
          A[j][e] = kCut;
        }
        if (none) {
          A[j][e] = 1.0f;
          H[j][e] = 0.0f;
        }
        own[e] = then(own[e], Map{A[j][e], H[j][e]});
      }
    }
  }
  maps[me.row][threadIdx.x & 31] = f32x4{own[0].A, own[0].H, own[1].A, own[1].H};
  lds_barrier();
  Map pre[2] = {{1.0f, 0.0f}, {1.0f, 0.0f}};               // of the tile's steps before the lane's
#pragma unroll 4
  for (int r = 0; r < me.row; ++r) {
    const f32x4 m = maps[r][threadIdx.x & 31];
#pragma unroll
    for (int e = 0; e < 2; ++e) pre[e] = then(pre[e], Map{m[2 * e], m[2 * e + 1]});
  }
  float h[2] = {0.0f, 0.0f};
  if (a.tiles > 1) {
    const bool last = me.row == kLrRows - 1 && tile + 1 < a.tiles;
    Map all[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      all[e] = then(pre[e], own[e]);
      if (last) put(map_word(a, chain, tile, me.slot + e), all[e]);
    }
    if (tile > 0) wait_state(a, me, chain, tile, wait, h);
    if (last && tile % kLrGroup == kLrGroup - 1)
#pragma unroll
      for (int e = 0; e < 2; ++e) put(state_word(a, chain, tile / kLrGroup, me.slot + e), Map{0.0f, apply(all[e], h[e])});
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) h[e] = apply(pre[e], h[e]);
  if (a.carries && me.row == 0)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (e + me.own >= 2) a.carries[((int64_t)b * a.tiles + tile) * a.C + me.c + (one ? 0 : e)] = h[e];
  if (!a.out) return;
  char* ob = static_cast<char*>(a.out) + (b * a.o_s[0] + T * a.o_s[1] - one) * kBytes<DT>;
  const uint32_t oo = (uint32_t)((me.half * S * a.o_s[1] + me.c) * kBytes<DT>);
  if (!marks.any) {
#pragma unroll
    for (int j = 0; j < S; ++j) {
#pragma unroll
      for (int e = 0; e < 2; ++e) h[e] = __builtin_fmaf(A[j][e], h[e], H[j][e]);
      store_pair<DT>(ob + j * a.o_s[1] * kBytes<DT>, oo, h[0], h[1], me.own);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < S; ++j) {
    const bool none = dead >> j & 1, ends = end >> j & 1;
    const int64_t seq = __shfl(marks.id, S * me.half + j);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      h[e] = apply(Map{A[j][e], H[j][e]}, h[e]);
      if (ends && a.final && e + me.own >= 2) a.final[seq * a.final_s + me.c + (one ? 0 : e)] = h[e];
    }
    if (T + S * me.half + j < a.L) store_pair<DT>(ob + j * a.o_s[1] * kBytes<DT>, oo, none ? 0.0f : h[0], none ? 0.0f : h[1], me.own);
  }
}

// ---- before the tiles ---------------------------------------------------------------------------
//
// Clears the words and the tickets; of a packed row also makes each step's sequence, and passes the
// states of empty sequences on (from -> to).  Offsets count as their running maximum, clamped to [0, L], the first as 0.

constexpr int kPiece = 4096, kSpan = 4096;

__device__ inline uint32_t wave_max(uint32_t x) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t y = __shfl_up(x, d);
    if ((int)(threadIdx.x & 63) >= d) x = max(x, y);
  }
  return x;
}

__device__ inline void pass_on(const float* from, int64_t from_s, float* to, int64_t to_s, int64_t s, int64_t C) {
  for (int64_t c = threadIdx.x; c < C; c += 1024) to[s * to_s + c] = from ? from[s * from_s + c] : 0.0f;
}

__global__ __launch_bounds__(1024) void prepare_kernel(const LinrecArgs a, const float* from, int64_t from_s, float* to, int64_t to_s) {
  __shared__ uint32_t wave[16];
  __shared__ uint32_t start[kPiece + 1];
  for (int64_t i = (int64_t)blockIdx.x * 1024 + threadIdx.x; i < a.clear_count; i += (int64_t)gridDim.x * 1024) a.clear[i] = kEmpty;
  if (!a.cu) {
    if (a.L == 0 && to)
      for (int64_t s = blockIdx.x; s < a.B; s += gridDim.x) pass_on(from, from_s, to, to_s, s, a.C);
    return;
  }
  const int tid = threadIdx.x, l = tid & 63, w = tid >> 6;
  const uint32_t most = (uint32_t)a.L;
  uint32_t carry = 0;
  for (int64_t base = 0; base < a.nseq; base += kPiece) {
    uint32_t x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t i = base + 4 * tid + j;
      const int32_t v = i < a.nseq ? a.cu[i + 1] : 0;
      x[j] = v < 0 ? 0 : min((uint32_t)v, most);
    }
#pragma unroll
    for (int j = 1; j < 4; ++j) x[j] = max(x[j], x[j - 1]);
    const uint32_t top = wave_max(x[3]);
    if (l == 63) wave[w] = top;
    uint32_t prior = __shfl_up(top, 1);
    if (l == 0) prior = 0;
    __syncthreads();
    uint32_t all = carry;
    for (int k = 0; k < 16; ++k) {
      if (k == w) prior = max(prior, all);
      all = max(all, wave[k]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) start[4 * tid + j + 1] = max(x[j], prior);
    if (tid == 0) start[0] = carry;
    __syncthreads();
    const int n = (int)min((int64_t)kPiece, a.nseq - base);
    // the steps of this piece's sequences, in spans dealt to the workgroups
    for (int64_t span = blockIdx.x; span * kSpan < (int64_t)all; span += gridDim.x) {
      if ((span + 1) * kSpan <= (int64_t)carry) continue;
#pragma unroll
      for (int i = 0; i < kSpan / 1024; ++i) {
        const uint32_t t = (uint32_t)(span * kSpan) + i * 1024 + tid;
        if (t < carry || t >= all) continue;
        int s0 = 0;                                     // the last sequence that starts at or before the step: not empty
#pragma unroll
        for (int d = kPiece / 2; d; d >>= 1) s0 += start[s0 + d] <= t ? d : 0;
        a.sid[t] = (int)base + s0;
      }
    }
    if (to)
      for (int i = blockIdx.x; i < n; i += gridDim.x)
        if (start[i] == start[i + 1]) pass_on(from, from_s, to, to_s, base + i, a.C);
    carry = all;
    __syncthreads();
  }
  for (int64_t t = carry + (int64_t)blockIdx.x * 1024 + tid; t < a.L; t += (int64_t)gridDim.x * 1024) a.sid[t] = -1;
}

// ---- decoding -------------------------------------------------------------------------------------
//
// A lane has a pair of channels of a row: its state's way in and out is the work.

template <int DT, int GT, bool NORM>
__global__ __launch_bounds__(256) void step_kernel(const LinrecStepArgs a, uint32_t pairs, int64_t items) {
  const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (item >= items) return;
  const uint32_t b = (uint32_t)(item / pairs), p = (uint32_t)(item - (int64_t)b * pairs);
  const bool one = a.C < 2;
  const int64_t at = 2 * (int64_t)p;
  const int own = at + 2 <= a.C ? 2 : 1;
  const uint32_t c = (uint32_t)(one ? 0 : own == 2 ? at : a.C - 2);
  const char* xp = static_cast<const char*>(a.x) + (b * a.x_s[0] + c) * kBytes<DT>;
  const char* gp = static_cast<const char*>(a.g) + (b * a.g_s[0] + c) * kBytes<GT>;
  char* op = static_cast<char*>(a.out) + (b * a.o_s[0] + (int64_t)c - one) * kBytes<DT>;
  Pair<DT> x = load_pair<DT>(xp, 0, one);
  Pair<GT> g = load_pair<GT>(gp, 0, one);
  const int64_t slot = a.slots ? a.slots[b] : b;
  if (slot < 0 || slot >= a.nslots) {                   // an idle row
    for (int64_t t = 0; t < a.T; ++t) store_pair<DT>(op + t * a.o_s[1] * kBytes<DT>, 0, 0.0f, 0.0f, own);
    return;
  }
  char* st = reinterpret_cast<char*>(a.state + slot * a.st_s + c);
  const Pair<CCV_DT_F32> s = load_pair<CCV_DT_F32>(st, 0, one);
  float h[2] = {pair_value<CCV_DT_F32>(s, 0), pair_value<CCV_DT_F32>(s, 1)};
  for (int64_t t = 0; t < a.T; ++t) {
    const Pair<DT> xt = x;
    const Pair<GT> gt = g;
    if (t + 1 < a.T) {
      x = load_pair<DT>(xp + (t + 1) * a.x_s[1] * kBytes<DT>, 0, one);
      g = load_pair<GT>(gp + (t + 1) * a.g_s[1] * kBytes<GT>, 0, one);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float d, y;
      decay(pair_value<GT>(gt, e), d, y);
      const float v = pair_value<DT>(xt, e);
      h[e] = __builtin_fmaf(d, h[e], NORM ? input_weight(y) * v : v);
    }
    store_pair<DT>(op + t * a.o_s[1] * kBytes<DT>, 0, h[0], h[1], own);
  }
  store_pair<CCV_DT_F32>(st - 4 * one, 0, h[0], h[1], own);
}

template <int DT, int GT>
void fwd(const LinrecArgs& a, hipStream_t st) {
  const uint32_t grid = a.tiles * a.chains;
  if (a.normalize) fwd_kernel<DT, GT, true><<<grid, 512, 0, st>>>(a);
  else fwd_kernel<DT, GT, false><<<grid, 512, 0, st>>>(a);
}
template <int DT, int GT>
void step(const LinrecStepArgs& a, hipStream_t st) {
  const uint32_t pairs = (uint32_t)((a.C + 1) / 2);
  const int64_t items = a.B * pairs;
  const uint32_t grid = (uint32_t)((items + 255) / 256);
  if (a.normalize) step_kernel<DT, GT, true><<<grid, 256, 0, st>>>(a, pairs, items);
  else step_kernel<DT, GT, false><<<grid, 256, 0, st>>>(a, pairs, items);
}
}  // namespace

int launch_linrec_prepare(const LinrecArgs& a, const float* from, int64_t from_s, float* to, int64_t to_s, void* stream) {
  int64_t need = a.cu ? (a.L + kSpan - 1) / kSpan : 1;
  need = std::max(need, (a.clear_count + 8191) / 8192);
  prepare_kernel<<<(uint32_t)std::min<int64_t>(std::max<int64_t>(need, 1), 512), 1024, 0, static_cast<hipStream_t>(stream)>>>(a, from, from_s, to, to_s);
  return (int)hipGetLastError();
}

int launch_linrec_fwd(const LinrecArgs& a, void* stream) {
  by_types(a.x_dtype, a.g_dtype, [&](auto dt, auto gt) { fwd<decltype(dt)::value, decltype(gt)::value>(a, static_cast<hipStream_t>(stream)); });
  return (int)hipGetLastError();
}

int launch_linrec_step(const LinrecStepArgs& a, void* stream) {
  by_types(a.x_dtype, a.g_dtype, [&](auto dt, auto gt) { step<decltype(dt)::value, decltype(gt)::value>(a, static_cast<hipStream_t>(stream)); });
  return (int)hipGetLastError();
}

}  // namespace ccv
