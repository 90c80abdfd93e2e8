// ccv_linrec.hip -- gated linear recurrence: one state a channel, over whole sequences and step by
// step.
//
//   h <- e^g[t] h + s[t] x[t],  out[t] = h;   s = 1, or sqrt(1 - e^2g) where x is normalised.
//
// One pass over the data.  A workgroup takes tiles of 128 steps and 64 channels into registers: pairs of
// channels a lane, 32 lanes a row, 8 consecutive steps a lane, so that loads are whole 128-byte
// lines and a lane walks its steps with one fused multiply-add each.  Each lane makes the map (A, H) of
// its 8 steps, a wave joins its two, the workgroup's eight meet in LDS, and the tiles of a sequence pass their
// maps on through memory (ccv_linrec_device.hpp), so x and g are read once.  With the state before its
// steps a lane walks them again from registers and stores.
//
// Calls of 4 x 4096 x 2048 in bf16, normalised, take 56 to 58 us, 3.5 TB/s; 65536 x 2560 in fp16 with fp32 decays, 64 sequences,
// normalised: 359 to 364 us, 3.7; 2 x 1048576 x 128 in fp32: 680 us, 4.7.  Without the exchange of maps they would take 52, 287 and
// 536 us, without the decays' arithmetic too 46, 262 and 534.  The two longer ones wait in order, for the slowest of the
// tiles under way before one's own.  The first, whose bytes alone need 39 us, is bound by no one thing: its loads and stores
// with what comes before the tiles take 7 more, the decays 6, the exchange and its waits 4 to 6.
#include "ccv_linrec_device.hpp"

#include <algorithm>

namespace ccv {
namespace {

struct FwdShared {
  alignas(16) Map maps[kLrWaves][kLrChannels];
  Heard heard;
};

template <int DT, int GT, bool NORM, bool MARKS>
__device__ __forceinline__ void fwd_tile(const LinrecArgs& a, const Place& at, int wave, const Pair<DT> (&xr)[kLrSteps], const Pair<GT> (&gr)[kLrSteps],
                                         FwdShared& shared) {
  constexpr int S = kLrSteps;
  const int lane = threadIdx.x & 63, half = lane >> 5, slot = 2 * (lane & 31);
  Marks marks{};
  if constexpr (MARKS) marks = marks_of(a, at);
  // decays and weighted inputs of the lane's steps, and their map
  float A[S][2], H[S][2];
  if (all_slow<GT>(gr)) {
#pragma unroll
    for (int j = 0; j < S; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float y;
        slow_decay(pair_value<GT>(gr[j], e), A[j][e], y);
        const float x = pair_value<DT>(xr[j], e);
        H[j][e] = NORM ? slow_weight(y) * x : x;
      }
  } else {
#pragma unroll
    for (int j = 0; j < S; ++j) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float y;
        decay(pair_value<GT>(gr[j], e), A[j][e], y);
        const float x = pair_value<DT>(xr[j], e);
        H[j][e] = NORM ? input_weight(y) * x : x;
      }
      __builtin_amdgcn_sched_barrier(0);                   // a step after the other, in few registers
    }
  }
  Map own[2] = {{1.0f, 0.0f}, {1.0f, 0.0f}};
#pragma unroll
  for (int j = 0; j < S; ++j) {
    [[maybe_unused]] const bool starts = marks.start >> j & 1, none = marks.dead >> j & 1;
    [[maybe_unused]] const int64_t seq = MARKS ? __shfl(marks.id, S * half + j) : 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if constexpr (MARKS) {
        if (starts) {
          if (a.init && (at.own >> e & 1)) H[j][e] = __builtin_fmaf(A[j][e], a.init[seq * a.init_s + at.c + e], H[j][e]);
          A[j][e] = kCut;
        }
        if (none) {
          A[j][e] = 1.0f;
          H[j][e] = 0.0f;
        }
        own[e] = then(own[e], Map{A[j][e], H[j][e]});
      } else {
        own[e].H = __builtin_fmaf(A[j][e], own[e].H, H[j][e]);
        own[e].A *= A[j][e];
      }
    }
  }
  Map early[2];                                            // of the half before this one
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    early[e] = other_half(own[e]);
    if (half) shared.maps[wave][slot + e] = then(early[e], own[e]);
  }
  lds_barrier();
  float h[2] = {0.0f, 0.0f};
  if (a.tiles > 1) {
    exchange(a, at, wave, shared.heard, [&]() {
      Map m = shared.maps[0][lane];
#pragma unroll
      for (int w = 1; w < kLrWaves; ++w) m = then(m, shared.maps[w][lane]);
      return m;
    });
    state_before(a, at, shared.heard, slot, h);
  }
  if (a.carries && wave == 0 && half == 0)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (at.own >> e & 1) a.carries[((int64_t)at.b * a.tiles + at.tile) * a.C + at.c + e] = h[e];
  if (!a.out) return;
  apply_parts<false>(shared.maps, wave, slot, h);
#pragma unroll
  for (int e = 0; e < 2; ++e)
    if (half) h[e] = apply(early[e], h[e]);
#pragma unroll
  for (int j = 0; j < S; ++j) {
    [[maybe_unused]] const bool none = marks.dead >> j & 1, ends = marks.end >> j & 1;
    [[maybe_unused]] const int64_t seq = MARKS ? __shfl(marks.id, S * half + j) : 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if constexpr (MARKS) {
        h[e] = apply(Map{A[j][e], H[j][e]}, h[e]);
        if (ends && a.final && (at.own >> e & 1)) a.final[seq * a.final_s + at.c + e] = h[e];
        H[j][e] = none ? 0.0f : h[e];
      } else {
        H[j][e] = h[e] = __builtin_fmaf(A[j][e], h[e], H[j][e]);
      }
    }
  }
  store_steps<DT>(a.out, a.o_s, at, a.L, H);
}

// Three workgroups a compute unit, in 80 registers, for 32-bit data that are not normalised and have kManyTiles and more: 680 us for
// 2 x 1048576 x 128, 722 with two; 557 and 613 for 2 x 32768 x 4096.  Else two, in 128.  The 58 registers that 80 are short of cost a small
// call more: 17.4 us for 1 x 16384 x 128, 13.5 with two; 101 and 96 for 1 x 65536 x 512 (4096 tiles).  They cross between 6144 tiles (three and
// two: 142 and 142 us in rows of 128 channels, 139 and 137 of 512, 121 and 113 of 4096) and 10240 (225 and 230, 221 and 222, 188 and 188); at 12288
// three are the faster in all (266 and 274, 262 and 265, 221 and 228).  With more to compute, or halves to
// convert, three are slower at any size (2 x 1048576 x 128 normalised: 835 us, 731 with two).
constexpr uint32_t kManyTiles = 12288;

template <int DT, int GT, bool NORM, int GROUPS>
__global__ __launch_bounds__(64 * kLrWaves, 2 * GROUPS) void fwd_kernel(const LinrecArgs a) {
  __shared__ FwdShared shared;
  __shared__ uint32_t ticket[2];
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const Place at = place_of<false>(a, take_ticket(a, ticket), wave);
  Pair<DT> xr[kLrSteps];
  Pair<GT> gr[kLrSteps];
  load_steps<true>(gr, a.g, a.g_s, at, a.L, a.C);
  load_steps<true>(xr, a.x, a.x_s, at, a.L, a.C);
  if (has_marks(a, at)) fwd_tile<DT, GT, NORM, true>(a, at, wave, xr, gr, shared);
  else fwd_tile<DT, GT, NORM, false>(a, at, wave, xr, gr, shared);
}

// ---- before the tiles ---------------------------------------------------------------------------
//
// Clears the words and the tickets; of a packed row also makes each step's sequence, and passes the
// states of empty sequences on (from -> to).  Offsets count as their running maximum, clamped to [0, L], the first as 0.
// A kernel's launch and the stores: 3 us for 2 x 4096 x 4096, 10 for 1 x 65536 x 2560 with 64 sequences (12 MB of words).

constexpr int kPiece = 4096, kSpan = 1024;

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
  // two words a store: their number is even
  for (int64_t i = (int64_t)blockIdx.x * 1024 + threadIdx.x; 2 * i < a.clear_count; i += (int64_t)gridDim.x * 1024)
    store16(reinterpret_cast<char*>(a.clear + 2 * i), u32x4{~0u, ~0u, ~0u, ~0u});
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
      const uint32_t t = (uint32_t)(span * kSpan) + tid;
      if (t < carry || t >= all) continue;
      int s0 = 0;                                       // the last sequence that starts at or before the step: not empty
#pragma unroll
      for (int d = kPiece / 2; d; d >>= 1) s0 += start[s0 + d] <= t ? d : 0;
      a.sid[t] = (int)base + s0;
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
// A lane has a pair of channels of a row: its state's way in and out is the work (256 x 4096 in bf16, 14.7 MB: 4.6 us, of which a
// launch that finds its data in the caches is about 3).

template <int DT, int GT, bool NORM>
__global__ __launch_bounds__(256) void step_kernel(const LinrecStepArgs a, uint32_t pairs, int64_t items) {
  const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (item >= items) return;
  const uint32_t b = (uint32_t)(item / pairs), c = 2 * (uint32_t)(item - (int64_t)b * pairs);
  const bool both = c + 1 < a.C;                        // else the last of an odd number, by itself
  const uint32_t next = both ? 1 : 0;
  const char* xp = static_cast<const char*>(a.x) + (b * a.x_s[0] + c) * kBytes<DT>;
  const char* gp = static_cast<const char*>(a.g) + (b * a.g_s[0] + c) * kBytes<GT>;
  char* op = static_cast<char*>(a.out) + (b * a.o_s[0] + c) * kBytes<DT>;
  const auto load = [&](Pair<DT>& x, Pair<GT>& g, int64_t t) {
    x = both ? load_pair<DT>(xp + t * a.x_s[1] * kBytes<DT>, 0) : load_one<DT>(xp + t * a.x_s[1] * kBytes<DT>, 0);
    g = both ? load_pair<GT>(gp + t * a.g_s[1] * kBytes<GT>, 0) : load_one<GT>(gp + t * a.g_s[1] * kBytes<GT>, 0);
  };
  const auto store = [&](int64_t t, float y0, float y1) {
    if (both) store_pair<DT>(op + t * a.o_s[1] * kBytes<DT>, 0, y0, y1);
    else store1<DT>(op + t * a.o_s[1] * kBytes<DT>, y0);
  };
  Pair<DT> x;
  Pair<GT> g;
  load(x, g, 0);
  const int64_t slot = a.slots ? a.slots[b] : b;
  if (slot < 0 || slot >= a.nslots) {                   // an idle row
    for (int64_t t = 0; t < a.T; ++t) store(t, 0.0f, 0.0f);
    return;
  }
  float* st = a.state + slot * a.st_s + c;
  float h[2] = {st[0], st[next]};
  for (int64_t t = 0; t < a.T; ++t) {
    const Pair<DT> xt = x;
    const Pair<GT> gt = g;
    if (t + 1 < a.T) load(x, g, t + 1);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float d, y;
      decay(pair_value<GT>(gt, e), d, y);
      const float v = pair_value<DT>(xt, e);
      h[e] = __builtin_fmaf(d, h[e], NORM ? input_weight(y) * v : v);
    }
    store(t, h[0], h[1]);
  }
  st[0] = h[0];
  if (both) st[1] = h[1];
}

template <int DT, int GT>
void fwd(const LinrecArgs& a, hipStream_t st) {
  const uint32_t grid = a.tiles * a.chains;
  if constexpr (DT == CCV_DT_F32 && GT == CCV_DT_F32)
    if (!a.normalize && grid >= kManyTiles) {
      fwd_kernel<DT, GT, false, 3><<<grid, 64 * kLrWaves, 0, st>>>(a);
      return;
    }
  if (a.normalize) fwd_kernel<DT, GT, true, 2><<<grid, 64 * kLrWaves, 0, st>>>(a);
  else fwd_kernel<DT, GT, false, 2><<<grid, 64 * kLrWaves, 0, st>>>(a);
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
  need = std::max(need, (a.clear_count + 4095) / 4096);
  prepare_kernel<<<(uint32_t)std::min<int64_t>(std::max<int64_t>(need, 1), 1024), 1024, 0, static_cast<hipStream_t>(stream)>>>(a, from, from_s, to, to_s);
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
