// ccv_linrec_device.hpp -- parts shared by the gated linear recurrence's kernels: the decay of a
// step, pairs of channels in memory, affine maps and the chain of tiles.
#pragma once

#include <type_traits>

#include "ccv_delta_device.hpp"
#include "ccv_linrec_launch.hpp"

namespace ccv {

// a = e^g and y = 1 - e^g, each to about a unit of its last place.  g = k ln 2 + r with |r| <= ln 2 / 2 and
// e^r - 1 = r (1 + r q(r)), q of degree 4 fitted to it (off by at most 1.4e-8 of e^r - 1).  The
// hardware's exponential does not serve: next to 1 its results lie 0.11 units of the last place too
// low on average (measured), which over a memory of a thousand steps and more adds up to 1e-5 of a state.
__device__ inline void decay(float g, float& a, float& y) {
  g = g < -150.0f ? -150.0f : g;                       // also -inf; NaN stays
  const float k = __builtin_rintf(g * 1.44269504088896341f);
  float r = __builtin_fmaf(k, -0.693145751953125f, g);   // ln 2 in two parts, the first exact in products with k
  r = __builtin_fmaf(k, -1.42860676e-06f, r);
  float q = __builtin_fmaf(r, 0.001394649618305266f, 0.00836661085486412f);
  q = __builtin_fmaf(r, q, 0.04166628047823906f);
  q = __builtin_fmaf(r, q, 0.1666654348373413f);
  q = __builtin_fmaf(r, q, 0.5f);
  const float m = r * __builtin_fmaf(r, q, 1.0f);
  a = __builtin_ldexpf(1.0f + m, (int)k);
  y = k == 0.0f ? -m : 1.0f - a;
}

// What x is weighted with: sqrt(1 - a^2) = sqrt(y (2 - y)); 0 where a > 1.
__device__ inline float input_weight(float y) {
  const float v = y * (2.0f - y);
  return __builtin_amdgcn_sqrtf(v < 0.0f ? 0.0f : v);
}

// Two neighbouring channels as stored.
template <int DT> struct Pair { uint32_t d[DT == CCV_DT_F32 ? 2 : 1]; };
template <int DT> constexpr int kBytes = DT == CCV_DT_F32 ? 4 : 2;

typedef const char __attribute__((address_space(1)))* gcptr;
typedef char __attribute__((address_space(1)))* gptr;

// From a uniform address and a lane's offset.  one: there is only one channel, at the address.
template <int DT>
__device__ inline Pair<DT> load_pair(const char* base, uint32_t off, bool one) {
  const gcptr p = (gcptr)base + off;
  Pair<DT> r;
  if constexpr (DT == CCV_DT_F32) {
    if (one) {
      r.d[0] = r.d[1] = *(const uint32_t __attribute__((address_space(1)))*)p;
    } else {
      const u32x2 v = *(const u32x2 __attribute__((address_space(1)))*)p;
      r.d[0] = v[0];
      r.d[1] = v[1];
    }
  } else {
    if (one) r.d[0] = *(const uint16_t __attribute__((address_space(1)))*)p * 0x10001u;
    else r.d[0] = *(const uint32_t __attribute__((address_space(1)))*)p;
  }
  return r;
}
template <int DT>
__device__ inline float pair_value(const Pair<DT>& r, int e) {
  if constexpr (DT == CCV_DT_F32) return __builtin_bit_cast(float, r.d[e]);
  else if constexpr (DT == CCV_DT_BF16) return __builtin_bit_cast(float, e ? r.d[0] & 0xffff0000u : r.d[0] << 16);
  else return F16::to_f((uint16_t)(r.d[0] >> (16 * e)));
}
// own: which of the two are stored (2: both, 1: the second alone, 0: none).
template <int DT>
__device__ inline void store_pair(char* base, uint32_t off, float y0, float y1, int own) {
  const gptr p = (gptr)base + off;
  if (own == 2) {
    if constexpr (DT == CCV_DT_F32) {
      *(u32x2 __attribute__((address_space(1)))*)p = u32x2{__builtin_bit_cast(uint32_t, y0), __builtin_bit_cast(uint32_t, y1)};
    } else {
      const f32x2 y = {as_f32(y0), as_f32(y1)};
      uint32_t d;
      if constexpr (DT == CCV_DT_BF16) d = __builtin_bit_cast(uint32_t, __builtin_convertvector(y, bf16x2));
      else d = __builtin_bit_cast(uint32_t, __builtin_convertvector(y, f16x2));
      *(uint32_t __attribute__((address_space(1)))*)p = d;
    }
  } else if (own == 1) {
    if constexpr (DT == CCV_DT_F32) *(float __attribute__((address_space(1)))*)(p + 4) = y1;
    else if constexpr (DT == CCV_DT_BF16) *(uint16_t __attribute__((address_space(1)))*)(p + 2) = BF16::from_f(y1);
    else *(uint16_t __attribute__((address_space(1)))*)(p + 2) = F16::from_f(y1);
  }
}

// The map h -> A h + H of a run of steps.  A sequence that starts within the run cuts off what was
// before it: then A is -0 and h is not looked at, so that no infinity or NaN of one
// sequence reaches another.
struct Map { float A, H; };
constexpr float kCut = -0.0f;          // decays are never negative, and so no product of them is
__device__ inline bool is_cut(float A) { return __builtin_bit_cast(uint32_t, A) == 0x80000000u; }
__device__ inline float apply(Map m, float h) { return is_cut(m.A) ? m.H : __builtin_fmaf(m.A, h, m.H); }
// First `before`, then m.
__device__ inline Map then(Map before, Map m) {
  return {is_cut(m.A) ? kCut : is_cut(before.A) ? kCut : m.A * before.A, apply(m, before.H)};
}

// A lane's place: the tile's row of lanes it belongs to, its two channels from `c`, of which it owns `own`
// (the last of an odd number of channels is the second of a pair), `slot` its first place of 64.
struct LrLane {
  int wave, half, row, slot, own;
  uint32_t c;
  __device__ inline LrLane(uint32_t cb, int64_t C) {
    const int l = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    half = l >> 5;
    row = 2 * wave + half;
    slot = 2 * (l & 31);
    const int64_t at = (int64_t)cb * kLrChannels + slot;
    own = at + 2 <= C ? 2 : at < C ? 1 : 0;
    c = (uint32_t)(C < 2 ? 0 : at + 2 <= C ? at : C - 2);
  }
};

// The 16 steps from T of a wave, 8 a half: bit i of the masks belongs to step T + i.
struct Marks {
  uint32_t start, end, dead;           // first and last steps of sequences; steps of none
  int id;                              // the sequence of step T + lane % 16
  bool any;                            // whether there are such steps at all; the same in every lane
};
__device__ inline Marks marks_at(const LinrecArgs& a, int64_t b, int64_t T) {
  Marks m;
  const int l = threadIdx.x & 15;
  const int64_t t = T + l;
  bool start, end, dead = t >= a.L;
  if (a.sid) {
    const int64_t in = dead ? a.L - 1 : t;
    m.id = a.sid[in];
    const int before = t > 0 && !dead ? a.sid[t - 1] : -2, after = t + 1 < a.L ? a.sid[t + 1] : -2;
    dead = dead || m.id < 0;
    start = !dead && m.id != before;
    end = !dead && m.id != after;
  } else {
    m.id = (int)b;
    start = t == 0;
    end = t == a.L - 1;
  }
  m.start = (uint32_t)(__builtin_amdgcn_ballot_w64(start) & 0xffff);
  m.end = (uint32_t)(__builtin_amdgcn_ballot_w64(end) & 0xffff);
  m.dead = (uint32_t)(__builtin_amdgcn_ballot_w64(dead) & 0xffff);
  m.any = (m.start | m.end | m.dead) != 0;
  return m;
}

// ---- the chain of tiles -----------------------------------------------------------------------
//
// A tile's map reaches the later tiles of its sequence's chain through one 64-bit word a channel,
// (A, H), written once a call by an atomic store: the word is the message and its own flag, so no
// fence is needed.  ~0 is an empty word (A is then no NaN that a tile could write: put() makes
// NaNs positive).  Tiles are grouped by 32: a tile takes the state behind the group before
// its own (one word, written by that group's last tile) through the maps of the tiles before it in the group, in their
// order, so results do not depend on which word came first.  Every wait ends: a tile waits only for tiles with
// lower tickets, whose workgroups run already and wait only for lower ones again; those of ticket 0 wait for nothing.
constexpr uint64_t kEmpty = ~0ull;

__device__ inline void put(uint64_t* w, Map m) {
  uint32_t A = __builtin_bit_cast(uint32_t, m.A);
  if (m.A != m.A) A = 0x7fc00000u;
  __hip_atomic_store(w, ((uint64_t)__builtin_bit_cast(uint32_t, m.H) << 32) | A, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline uint64_t peek(const uint64_t* w) { return __hip_atomic_load(w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ inline Map map_of(uint64_t w) {
  return {__builtin_bit_cast(float, (uint32_t)w), __builtin_bit_cast(float, (uint32_t)(w >> 32))};
}

// The state before tile `i` of a chain (in the order of the walk), for the slots me.slot and + 1; the whole workgroup calls it.
// Each wave takes four of the tiles before it in the group, slot by lane, and folds their maps in order.
struct LrWait { Map part[kLrRows / 2][kLrChannels]; float state[kLrChannels]; };

__device__ inline void wait_state(const LinrecArgs& a, const LrLane& me, uint32_t chain, uint32_t i, LrWait& shared, float (&h)[2]) {
  constexpr int each = kLrGroup / (kLrRows / 2);
  const int lane = threadIdx.x & 63;
  const uint32_t group = i / kLrGroup, first = group * kLrGroup, n = i - first, j0 = me.wave * each;
  if (j0 < n || me.wave == 0) {
    const uint64_t* maps = a.words + ((int64_t)chain * a.tiles + first + j0) * kLrChannels + lane;
    const uint64_t* state = a.words + ((int64_t)a.chains * a.tiles + (int64_t)chain * a.groups + group - 1) * kLrChannels + lane;
    const bool behind = me.wave == 0 && group > 0;
    uint64_t w[each], s = kEmpty;
#pragma unroll
    for (int j = 0; j < each; ++j) w[j] = kEmpty;
    for (;;) {
      bool ok = true;
      if (behind) {
        if (s == kEmpty) s = peek(state);
        ok = s != kEmpty;
      }
#pragma unroll
      for (int j = 0; j < each; ++j)
        if (j0 + j < n && w[j] == kEmpty) w[j] = peek(maps + j * kLrChannels);
#pragma unroll
      for (int j = 0; j < each; ++j) ok = ok && (j0 + j >= n || w[j] != kEmpty);
      if (__builtin_amdgcn_ballot_w64(!ok) == 0) break;
      __builtin_amdgcn_s_sleep(1);
    }
    Map m = {1.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < each; ++j)
      if (j0 + j < n) m = then(m, map_of(w[j]));
    shared.part[me.wave][lane] = m;
    if (me.wave == 0) shared.state[lane] = behind ? map_of(s).H : 0.0f;
  }
  lds_barrier();
#pragma unroll
  for (int e = 0; e < 2; ++e) h[e] = shared.state[me.slot + e];
  for (uint32_t k = 0; k * each < n; ++k)
#pragma unroll
    for (int e = 0; e < 2; ++e) h[e] = apply(shared.part[k][me.slot + e], h[e]);
}

__device__ inline uint64_t* map_word(const LinrecArgs& a, uint32_t chain, uint32_t i, int slot) {
  return a.words + ((int64_t)chain * a.tiles + i) * kLrChannels + slot;
}
__device__ inline uint64_t* state_word(const LinrecArgs& a, uint32_t chain, uint32_t group, int slot) {
  return a.words + ((int64_t)a.chains * a.tiles + (int64_t)chain * a.groups + group) * kLrChannels + slot;
}

// This workgroup's place in the order of tiles: all chains' first ones, then their second ones ...
__device__ inline uint32_t take_ticket(const LinrecArgs& a, uint32_t* shared) {
  if (a.tiles == 1) return blockIdx.x;
  if (threadIdx.x == 0)        // from a cleared word, all bits set
    *shared = 1u + __hip_atomic_fetch_add(reinterpret_cast<uint32_t*>(a.ticket), 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(*shared);
}

// The types' numbers as constants: f(x's, g's).
template <class F>
inline void by_types(int x, int g, F f) {
  const auto on_g = [&](auto dt) {
    if (g == CCV_DT_F32) f(dt, std::integral_constant<int, CCV_DT_F32>{});
    else if (g == CCV_DT_F16) f(dt, std::integral_constant<int, CCV_DT_F16>{});
    else f(dt, std::integral_constant<int, CCV_DT_BF16>{});
  };
  if (x == CCV_DT_F32) on_g(std::integral_constant<int, CCV_DT_F32>{});
  else if (x == CCV_DT_F16) on_g(std::integral_constant<int, CCV_DT_F16>{});
  else on_g(std::integral_constant<int, CCV_DT_BF16>{});
}


}  // namespace ccv
