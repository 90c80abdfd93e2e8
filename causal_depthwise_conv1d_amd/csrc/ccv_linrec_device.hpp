// ccv_linrec_device.hpp -- parts shared by the gated linear recurrence's kernels: the decay of a
// step, pairs of channels in memory, affine maps and the chain of tiles.
#pragma once

#include <type_traits>

#include "ccv_delta_device.hpp"
#include "ccv_linrec_launch.hpp"

namespace ccv {

// a = e^g and y = 1 - e^g, each to about a unit of its last place.  g = k ln 2 + r with |r| <= ln 2 / 2 and
// e^r - 1 = r (1 + r q(r)), q of degree 4 fitted to it (off by at most 1.9e-8 of e^r - 1).  The
// hardware's exponential does not serve: next to 1 its results lie 0.11 units of the last place too
// low on average (measured), which over a memory of a thousand steps and more adds up to 1e-5 of a state.
__device__ inline float expm1_near(float r) {
  float q = __builtin_fmaf(r, 0.001394649618305266f, 0.00836661085486412f);
  q = __builtin_fmaf(r, q, 0.04166628047823906f);
  q = __builtin_fmaf(r, q, 0.1666654348373413f);
  q = __builtin_fmaf(r, q, 0.5f);
  return r * __builtin_fmaf(r, q, 1.0f);
}
__device__ inline void decay(float g, float& a, float& y) {
  g = g < -150.0f ? -150.0f : g;                       // also -inf; NaN stays
  const float k = __builtin_rintf(g * 1.44269504088896341f);
  float r = __builtin_fmaf(k, -0.693145751953125f, g);   // ln 2 in two parts, the first exact in products with k
  r = __builtin_fmaf(k, -1.42860676e-06f, r);
  const float m = expm1_near(r);
  a = __builtin_ldexpf(1.0f + m, (int)k);
  y = k == 0.0f ? -m : 1.0f - a;
}
// The same for kSlow <= g <= 0, where k is 0: the same bits.
constexpr float kSlow = -0.34f;
__device__ inline void slow_decay(float g, float& a, float& y) {
  const float m = expm1_near(g);
  a = 1.0f + m;
  y = -m;
}

// What x is weighted with: sqrt(1 - a^2) = sqrt(y (2 - y)); 0 where a > 1.
__device__ inline float input_weight(float y) {
  const float v = y * (2.0f - y);
  return __builtin_amdgcn_sqrtf(v < 0.0f ? 0.0f : v);
}
__device__ inline float slow_weight(float y) { return __builtin_amdgcn_sqrtf(y * (2.0f - y)); }

// Two neighbouring channels as stored.
template <int DT> struct Pair { uint32_t d[DT == CCV_DT_F32 ? 2 : 1]; };
template <int DT> constexpr int kBytes = DT == CCV_DT_F32 ? 4 : 2;

typedef const char __attribute__((address_space(1)))* gcptr;
typedef char __attribute__((address_space(1)))* gptr;

// From a uniform address and a lane's offset; STREAM: not to be kept in the caches (2 x 1048576 x 128 in fp32: 685 us so, 721 otherwise).
template <int DT, bool STREAM = false>
__device__ inline Pair<DT> load_pair(const char* base, uint32_t off) {
  const gcptr p = (gcptr)base + off;
  Pair<DT> r;
  if constexpr (DT == CCV_DT_F32) {
    const auto q = (const u32x2 __attribute__((address_space(1)))*)p;
    const u32x2 v = STREAM ? __builtin_nontemporal_load(q) : *q;
    r.d[0] = v[0];
    r.d[1] = v[1];
  } else {
    const auto q = (const uint32_t __attribute__((address_space(1)))*)p;
    r.d[0] = STREAM ? __builtin_nontemporal_load(q) : *q;
  }
  return r;
}
// One element, and 0.
template <int DT>
__device__ inline Pair<DT> load_one(const char* base, uint32_t off) {
  const gcptr p = (gcptr)base + off;
  Pair<DT> r;
  if constexpr (DT == CCV_DT_F32) {
    r.d[0] = *(const uint32_t __attribute__((address_space(1)))*)p;
    r.d[1] = 0;
  } else {
    r.d[0] = *(const uint16_t __attribute__((address_space(1)))*)p;
  }
  return r;
}
template <int DT>
__device__ inline float pair_value(const Pair<DT>& r, int e) {
  if constexpr (DT == CCV_DT_F32) return __builtin_bit_cast(float, r.d[e]);
  else if constexpr (DT == CCV_DT_BF16) return __builtin_bit_cast(float, e ? r.d[0] & 0xffff0000u : r.d[0] << 16);
  else return F16::to_f((uint16_t)(r.d[0] >> (16 * e)));
}
// The same registers, of which the compiler no longer knows what was made of them before.
template <int DT, int N>
__device__ inline void hide_steps(Pair<DT> (&r)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int i = 0; i < (DT == CCV_DT_F32 ? 2 : 1); ++i) asm("" : "+v"(r[j].d[i]));
}
// A streaming store: results are not read again here (a training step of 2 x 4096 x 4096 in bf16 takes 144 us so, 152 otherwise).
template <int DT>
__device__ inline void store_pair(char* base, uint32_t off, float y0, float y1) {
  const gptr p = (gptr)base + off;
  if constexpr (DT == CCV_DT_F32) {
    __builtin_nontemporal_store(u32x2{__builtin_bit_cast(uint32_t, y0), __builtin_bit_cast(uint32_t, y1)}, (u32x2 __attribute__((address_space(1)))*)p);
  } else {
    const f32x2 y = {as_f32(y0), as_f32(y1)};
    uint32_t d;
    if constexpr (DT == CCV_DT_BF16) d = __builtin_bit_cast(uint32_t, __builtin_convertvector(y, bf16x2));
    else d = __builtin_bit_cast(uint32_t, __builtin_convertvector(y, f16x2));
    __builtin_nontemporal_store(d, (uint32_t __attribute__((address_space(1)))*)p);
  }
}

// Whether all of a wave's decays are slow ones.
template <int GT>
__device__ inline bool all_slow(const Pair<GT> (&g)[kLrSteps]) {
  float least = 0.0f, most = kSlow;                // of a NaN either way makes a NaN
#pragma unroll
  for (int j = 0; j < kLrSteps; ++j) {
    const float g0 = pair_value<GT>(g[j], 0), g1 = pair_value<GT>(g[j], 1);
    least = __builtin_fminf(least, __builtin_fminf(g0, g1));
    most = __builtin_fmaxf(most, __builtin_fmaxf(g0, g1));
  }
  return __builtin_amdgcn_ballot_w64(!(least >= kSlow && most <= 0.0f)) == 0;
}

// The map h -> A h + H of a run of steps.  A sequence that starts within the run cuts off what was
// before it: then A is -0 and h is not looked at, so that no infinity or NaN of one
// sequence reaches another.
struct alignas(8) Map { float A, H; };
constexpr float kCut = -0.0f;          // decays are never negative, and so no product of them is
__device__ inline bool is_cut(float A) { return __builtin_bit_cast(uint32_t, A) == 0x80000000u; }
__device__ inline float apply(Map m, float h) { return __builtin_fmaf(m.A, is_cut(m.A) ? 0.0f : h, m.H); }
// First `before`, then m.
__device__ inline Map then(Map before, Map m) {
  return {is_cut(m.A) ? kCut : is_cut(before.A) ? kCut : m.A * before.A, apply(m, before.H)};
}

// n / d for a divisor whose magic the host has made, in scalar instructions.
__device__ inline uint32_t divide(uint32_t n, const LrDivisor& d) {
  const uint32_t t = (uint32_t)(((uint64_t)n * d.magic) >> 32);
  return (t + ((n - t) >> d.first)) >> d.second;
}

// The i-th pair of the channels from `first`: its first channel, and which of the two are its own (bit 0, bit 1): of
// an odd number of channels the last is the second of a pair, a single one the first; pairs past the last have none.
struct Channels { uint32_t c, own; };
__device__ inline Channels channels_of(uint32_t first, uint32_t i, int64_t C) {
  const uint32_t at = first + 2 * i;
  if (at + 2 <= C) return {at, 3u};
  return C < 2 ? Channels{0u, at < C ? 1u : 0u} : Channels{(uint32_t)C - 2, at < C ? 2u : 0u};
}

// A workgroup's tile: its queue, and its number there.
struct Ticket { uint32_t queue, number; };

// A tile's place, the same in every lane of a wave but for c and own, the lane's channels; T: the wave's first step.
struct Place {
  uint32_t order, chain, tile, b, first, c, own;       // order: of the tile in its chain's walk; first: its first channel
  int64_t T;
  bool edge;                               // the wave has steps past the last, or the tile channels past the last
};
template <bool REVERSE>
__device__ inline Place place_of(const LinrecArgs& a, const Ticket& t, int wave) {
  Place p;
  p.order = a.tiles == 1 ? 0 : divide(t.number, t.queue < a.longer ? a.by_more : a.by_fewer);
  p.chain = a.tiles == 1 ? t.number : t.number - p.order * a.chains_of(t.queue) + a.first_chain(t.queue);
  p.tile = REVERSE ? a.tiles - 1 - p.order : p.order;
  p.b = divide(p.chain, a.by_cblocks);
  const uint32_t cb = p.chain - p.b * a.cblocks;
  p.first = cb * kLrChannels;
  const Channels ch = channels_of(p.first, threadIdx.x & 31, a.C);
  p.c = ch.c;
  p.own = ch.own;
  p.T = (int64_t)p.tile * kLrTile + 2 * kLrSteps * wave;
  p.edge = p.T + 2 * kLrSteps > a.L || (int64_t)(cb + 1) * kLrChannels > a.C;
  return p;
}

// A lane's eight steps of an array, at a uniform address for each step and a lane's offset; at an edge, steps past the last
// are read as it.
template <bool STREAM, int DT>
__device__ inline void load_steps(Pair<DT> (&r)[kLrSteps], const void* p, const int64_t (&s)[2], const Place& at, int64_t L, int64_t C) {
  const int half = (threadIdx.x >> 5) & 1;
  const char* base = static_cast<const char*>(p) + (at.b * s[0] + at.T * s[1]) * kBytes<DT>;
  int64_t step = s[1] * kBytes<DT>;
  if (!at.edge) {
    const uint32_t off = (uint32_t)(half * kLrSteps * (int)step) + at.c * kBytes<DT>;
    asm("" : "+s"(step));                  // not a multiple of it kept for each step
#pragma unroll
    for (int j = 0; j < kLrSteps; ++j, base += step) r[j] = load_pair<DT, STREAM>(base, off);
  } else {
    const int most = (int)(L - 1 - at.T < 2 * kLrSteps ? L - 1 - at.T : 2 * kLrSteps);    // of the wave's steps; < 0: all lie past the last
    base += (most < 0 ? most : 0) * step;
    const int top = most < 0 ? 0 : most;
    const auto off = [&](int j) { return (uint32_t)(min(kLrSteps * half + j, top) * (int)step) + at.c * kBytes<DT>; };
    if (C < 2) {
#pragma unroll
      for (int j = 0; j < kLrSteps; ++j) r[j] = load_one<DT>(base, off(j));
    } else {
#pragma unroll
      for (int j = 0; j < kLrSteps; ++j) r[j] = load_pair<DT, STREAM>(base, off(j));
    }
  }
}
template <int DT>
__device__ inline void store_steps(void* p, const int64_t (&s)[2], const Place& at, int64_t L, const float (&y)[kLrSteps][2]) {
  const int half = (threadIdx.x >> 5) & 1;
  char* base = static_cast<char*>(p) + (at.b * s[0] + at.T * s[1]) * kBytes<DT>;
  int64_t step = s[1] * kBytes<DT>;
  const uint32_t off = (uint32_t)(half * kLrSteps * (int)step) + at.c * kBytes<DT>;
  if (!at.edge) {
    asm("" : "+s"(step));
#pragma unroll
    for (int j = 0; j < kLrSteps; ++j, base += step) store_pair<DT>(base, off, y[j][0], y[j][1]);
  } else {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (at.own >> e & 1)
#pragma unroll
        for (int j = 0; j < kLrSteps; ++j)
          if (at.T + kLrSteps * half + j < L) store1<DT>(base + j * step + off + e * kBytes<DT>, y[j][e]);
  }
}

// Whether a tile has steps at which a sequence starts or ends, or steps of none; the same in the whole workgroup.  With such
// steps it takes a code path of its own, through which the other one's values need not be kept in registers.
__device__ inline bool has_marks(const LinrecArgs& a, const Place& at) {
  const int64_t t0 = (int64_t)at.tile * kLrTile, t1 = t0 + kLrTile;
  if (t0 == 0 || t1 >= a.L) return true;
  if (!a.sid) return false;
  const int id = a.sid[t0];                        // of a row's steps the sequences' numbers ascend, and then come steps of none
  return id < 0 || a.sid[t0 - 1] != id || a.sid[t1] != id;
}
// Bit j of the masks belongs to the lane's step j.
struct Marks {
  uint32_t start, end, dead;           // first and last steps of sequences; steps of none
  int id;                              // the sequence of step T + lane % 16 of the wave's 16 from T
};
__device__ inline Marks marks_of(const LinrecArgs& a, const Place& at) {
  const int64_t t = at.T + (threadIdx.x & 15);
  bool start = t == 0, end = t == a.L - 1, dead = t >= a.L;
  int id = (int)at.b;
  if (a.sid) {
    const int64_t in = t < a.L ? t : a.L - 1;
    id = a.sid[in];
    dead = dead || id < 0;
    start = !dead && (start || id != a.sid[in > 0 ? in - 1 : 0]);
    end = !dead && (end || id != a.sid[in + 1 < a.L ? in + 1 : in]);
  }
  const uint32_t s = (uint32_t)__builtin_amdgcn_ballot_w64(start) & 0xffff, e = (uint32_t)__builtin_amdgcn_ballot_w64(end) & 0xffff,
                 d = (uint32_t)__builtin_amdgcn_ballot_w64(dead) & 0xffff;
  const int shift = threadIdx.x & 32 ? kLrSteps : 0;
  return {s >> shift, e >> shift, d >> shift, id};
}

// The map of the other 32 lanes' steps of the same channels.
__device__ inline Map other_half(Map m) { return {__shfl_xor(m.A, 32), __shfl_xor(m.H, 32)}; }

// ---- the chain of tiles -----------------------------------------------------------------------
//
// A tile's map reaches the later tiles of its chain through one 64-bit word a channel, (A, H), written
// once a call by an atomic store: the word is the message and its own flag, so no fence is needed.  ~0 is an empty
// word (A is then no NaN that a tile could write: put() makes NaNs positive).  8 tiles are a group, and 8 groups a
// stretch.  A group's last tile joins its maps into the group's, as soon as they are there; a stretch's last tile gives
// the state behind it.  A tile applies to the state behind the stretch before its own the maps of the groups and then
// of the tiles between, in their order: results do not depend on which word came first, and what
// has to wait for each other is one tile in 64.  Each wave asks for one tile's word and one group's: groups of 4 or 16 tiles, and
// stretches of 16 or of one group, take the same time to 1 %.
// Tiles are taken in the order of their chains' walks, by tickets; a queue of tickets has the chains of one of the eight dies,
// whose L2 then passes their words on, and its own counter: one counter for all gives a ticket in 12 ns, which is
// a third of the time that a tile's data take.  A workgroup whose die's queue is empty takes from another's.  Every wait
// ends: a tile waits only for tiles with lower tickets of its own queue, whose workgroups run already, and the lowest unfinished
// one waits for nothing.  How many workgroups run at a time, of this call or of others, does not matter.
constexpr uint64_t kEmpty = ~0ull;

// Words of a chain's tile i, group i, stretch i, for slot 0.
__device__ inline uint64_t* tile_words(const LinrecArgs& a, const Place& at, uint32_t i) {
  return a.words + ((int64_t)at.chain * a.tiles + i) * kLrChannels;
}
__device__ inline uint64_t* group_words(const LinrecArgs& a, const Place& at, uint32_t i) {
  return a.words + ((int64_t)a.chains * a.tiles + (int64_t)at.chain * a.groups + i) * kLrChannels;
}
__device__ inline uint64_t* stretch_words(const LinrecArgs& a, const Place& at, uint32_t i) {
  return a.words + ((int64_t)a.chains * (a.tiles + a.groups) + (int64_t)at.chain * a.stretches + i) * kLrChannels;
}
// The word of this lane's slot, from that of slot 0.
__device__ inline void put(uint64_t* w, Map m) {
  uint32_t A = __builtin_bit_cast(uint32_t, m.A);
  if (m.A != m.A) A = 0x7fc00000u;
  auto p = (uint64_t __attribute__((address_space(1)))*)((gptr)(char*)w + 8 * (threadIdx.x & 63));
  __hip_atomic_store(p, ((uint64_t)__builtin_bit_cast(uint32_t, m.H) << 32) | A, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline uint64_t peek(const uint64_t* w) {
  auto p = (const uint64_t __attribute__((address_space(1)))*)((gcptr)(const char*)w + 8 * (threadIdx.x & 63));
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline Map map_of(uint64_t w) {
  return {__builtin_bit_cast(float, (uint32_t)w), __builtin_bit_cast(float, (uint32_t)(w >> 32))};
}

// Counters start from cleared words, all bits set.  There is a workgroup for each tile, so one that finds
// all queues empty would have found every tile taken by another.  Calls of one tile a chain wait for nothing: there the
// tickets are the workgroups' numbers.
__device__ inline Ticket take_ticket(const LinrecArgs& a, uint32_t* shared) {
  if (a.tiles == 1) return {0, blockIdx.x};
  if (threadIdx.x == 0) {
    constexpr int kXccId = 20 | (31 << 11);                // the hardware register XCC_ID, all bits
    uint32_t q = ((uint32_t)__builtin_amdgcn_s_getreg(kXccId) & 7u) % a.queues, t;
    while ((t = 1u + __hip_atomic_fetch_add(reinterpret_cast<uint32_t*>(a.ticket + kLrTicketWords * q), 1u, __ATOMIC_RELAXED,
                                            __HIP_MEMORY_SCOPE_AGENT)) >= a.chains_of(q) * a.tiles)
      q = q + 1 < a.queues ? q + 1 : 0;
    shared[0] = q;
    shared[1] = t;
  }
  __syncthreads();
  return {(uint32_t)__builtin_amdgcn_readfirstlane(shared[0]), (uint32_t)__builtin_amdgcn_readfirstlane(shared[1])};
}

// What a tile hears of those before it, by slot: the maps of the group's tiles and of the stretch's groups, a wave each, and a state.
struct Heard {
  alignas(16) Map tiles[kLrWaves][kLrChannels], groups[kLrWaves][kLrChannels];
  float state[kLrChannels];
};
// Waits for a wave's word, w as it was found first.  While it is missing one lane alone asks: words come a wave's store at a time.
__device__ inline Map wait_word(const uint64_t* at, uint64_t w) {
  while (__builtin_amdgcn_ballot_w64(w == kEmpty) != 0) {
    for (bool there = false; __builtin_amdgcn_ballot_w64(there) == 0;) {
      __builtin_amdgcn_s_sleep(1);
      if ((threadIdx.x & 63) == 0) there = peek(at) != kEmpty;
    }
    w = peek(at);
  }
  return map_of(w);
}

// The tile's own map is given to the others, and theirs are waited for; the whole workgroup calls this, `all()` gives the
// tile's map by slot (lane) to one wave.  Afterwards heard holds what state_before() needs, but for a chain's first tile.
template <class F>
__device__ inline void exchange(const LinrecArgs& a, const Place& at, int wave, Heard& heard, F all) {
  const int lane = threadIdx.x & 63;
  const uint32_t in_group = at.order % kLrGroup, group = at.order / kLrGroup;
  const uint32_t in_stretch = group % kLrStretch, stretch = group / kLrStretch;
  const bool talks = wave == kLrWaves - 1, follows = at.order + 1 < a.tiles, closes = in_group == kLrGroup - 1 && follows;
  Map mine = {1.0f, 0.0f};
  if (talks && follows) {
    mine = all();
    put(tile_words(a, at, at.order), mine);
  }
  if (at.order == 0) return;
  const bool of_tile = (uint32_t)wave < in_group, of_group = (uint32_t)wave < in_stretch;
  const uint64_t *tw = tile_words(a, at, at.order - in_group + wave), *gw = group_words(a, at, group - in_stretch + wave);
  uint64_t wt = 0, wg = 0;
  if (of_group) wg = peek(gw);
  if (of_tile) wt = peek(tw);
  if (of_tile) heard.tiles[wave][lane] = wait_word(tw, wt);
  if (closes) {                                            // the same for the whole workgroup
    lds_barrier();
    if (talks) {
      Map m = heard.tiles[0][lane];
#pragma unroll 1                                           // in few registers: else fp32 loads are spilled, at twice the time
      for (uint32_t k = 1; k < kLrGroup - 1; ++k) m = then(m, heard.tiles[k][lane]);
      mine = then(m, mine);
      if (in_stretch < kLrStretch - 1) put(group_words(a, at, group), mine);
    }
  }
  if (of_group) heard.groups[wave][lane] = wait_word(gw, wg);
  if (talks) {
    float h = 0.0f;                                        // a chain begins with a sequence: nothing looks at the 0
    if (stretch > 0) {
      const uint64_t* ss = stretch_words(a, at, stretch - 1);
      uint64_t s;
      while (__builtin_amdgcn_ballot_w64((s = peek(ss)) == kEmpty) != 0) __builtin_amdgcn_s_sleep(1);
      h = map_of(s).H;
    }
    heard.state[lane] = h;
  }
  lds_barrier();
  if (talks && closes && in_stretch == kLrStretch - 1) {
    float h = heard.state[lane];
    for (uint32_t k = 0; k < in_stretch; ++k) h = apply(heard.groups[k][lane], h);
    put(stretch_words(a, at, stretch), Map{0.0f, apply(mine, h)});
  }
}
// Two slots' maps, by wave in LDS, applied from the first to the n-th, or from the last to the n-th; four are read at a time.
template <bool BACK>
__device__ inline void apply_parts(const Map (&parts)[kLrWaves][kLrChannels], uint32_t n, int slot, float (&h)[2]) {
#pragma unroll
  for (int k0 = 0; k0 < kLrWaves; k0 += 4) {
    f32x4 m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = *reinterpret_cast<const f32x4*>(&parts[BACK ? kLrWaves - 1 - k0 - i : k0 + i][slot]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (BACK ? (uint32_t)(kLrWaves - 1 - k0 - i) >= n : (uint32_t)(k0 + i) < n)
#pragma unroll
        for (int e = 0; e < 2; ++e) h[e] = apply(Map{m[i][2 * e], m[i][2 * e + 1]}, h[e]);
    __builtin_amdgcn_sched_barrier(0);
  }
}
// The state before the tile, for two slots.
__device__ inline void state_before(const LinrecArgs& a, const Place& at, const Heard& heard, int slot, float (&h)[2]) {
  if (at.order == 0) return;
  h[0] = heard.state[slot];
  h[1] = heard.state[slot + 1];
  apply_parts<false>(heard.groups, at.order / kLrGroup % kLrStretch, slot, h);
  apply_parts<false>(heard.tiles, at.order % kLrGroup, slot, h);
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
