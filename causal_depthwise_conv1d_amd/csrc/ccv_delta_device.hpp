// ccv_delta_device.hpp -- matrix fragments of the gated delta rule's kernels.
//
// Every product runs on the bf16 matrix instruction 16x16x32.  An fp32 value is held as a
// sum of bf16 planes, hi + mid + lo (8 significant bits each, 24 together), and a product
// of two such values is the sum of the six plane products whose indexes add up to at most
// 2, which keeps about 2^-23 of the result: 6 instructions where the fp32 matrix
// instruction takes the time of 16.  Results that are rounded to 16 bits are computed so
// too: with two planes, 16 bits, of S, N and P in place of 24, three times as many of them come
// out on the other side of a rounding as of 32-bit sums (in the 2-norm, 1.2e-4 from the rounded
// 64-bit result in bf16).  bf16 inputs are one plane, exactly; fp16 inputs are two, exactly.
#pragma once

#include "ccv_device.hpp"
#include "ccv_delta_launch.hpp"

namespace ccv {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896341f;

// planes of an input element
template <int DT> struct InPlanes { static constexpr int n = DT == CCV_DT_BF16 ? 1 : DT == CCV_DT_F16 ? 2 : 3; };
constexpr int kOrder = 2;      // of the plane products that are kept

template <int P> struct Frag { bf16x8 p[P]; };

// Two values rounded to bf16 in one dword, and taken off: x, y keep the remainders.
__device__ inline uint32_t take2(float& x, float& y) {
  const uint32_t h = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x, y}, bf16x2));
  x -= __builtin_bit_cast(float, h << 16);
  y -= __builtin_bit_cast(float, h & 0xffff0000u);
  return h;
}

template <int P>
__device__ inline Frag<P> split8(f32x8 x) {
  Frag<P> f;
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = x[j];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    u32x4 d;
#pragma unroll
    for (int j = 0; j < 4; ++j) d[j] = take2(v[2 * j], v[2 * j + 1]);
    f.p[i] = __builtin_bit_cast(bf16x8, d);
  }
  return f;
}

// acc += a b over 32 steps of the contraction; the small terms first.
template <int PA, int PB>
__device__ inline f32x4 mma(const Frag<PA>& a, const Frag<PB>& b, f32x4 acc) {
#pragma unroll
  for (int s = kOrder; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < PA; ++i)
      if (s - i >= 0 && s - i < PB) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[i], b.p[s - i], acc, 0, 0, 0);
  return acc;
}

// The same with a sum for each size of term: chains of dependent instructions a third as long.
struct Sums {
  f32x4 s[kOrder + 1];
  __device__ inline Sums() {
#pragma unroll
    for (int i = 0; i <= kOrder; ++i) s[i] = f32x4{0, 0, 0, 0};
  }
  template <int PA, int PB>
  __device__ inline void add(const Frag<PA>& a, const Frag<PB>& b) {
#pragma unroll
    for (int i = 0; i < PA; ++i)
#pragma unroll
      for (int j = 0; j < PB; ++j)
        if (i + j <= kOrder) s[i + j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[i], b.p[j], s[i + j], 0, 0, 0);
  }
  __device__ inline f32x4 total() const {
    f32x4 t = s[kOrder];
#pragma unroll
    for (int i = kOrder - 1; i >= 0; --i) t += s[i];
    return t;
  }
};

// Eight consecutive elements of a row, as stored.
template <int DT> struct Raw8 { u32x4 d[DT == CCV_DT_F32 ? 2 : 1]; };

// Loads of a chunk's rows go through buffer descriptors: a uniform base in scalar registers,
// one 32-bit byte offset a lane that stays the same from chunk to chunk, and the
// descriptor's bound, past which a load gives zeros without a branch (a branch around a
// load makes the compiler wait for it where the paths join).  The bound ends the rows of
// a short last chunk; a lane whose columns lie past the row's width has kNowhere.
constexpr uint32_t kNowhere = 0x80000000u;

__device__ inline __amdgpu_buffer_rsrc_t buffer(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00027000);
}
__device__ inline u32x4 buf16(__amdgpu_buffer_rsrc_t b, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, off, 0, 0));
}
__device__ inline f32x4 buf_f4(__amdgpu_buffer_rsrc_t b, uint32_t off) { return __builtin_bit_cast(f32x4, buf16(b, off)); }

template <int P>
__device__ inline Frag<P> buf_planes(__amdgpu_buffer_rsrc_t b, uint32_t off, uint32_t plane) {
  Frag<P> f;
#pragma unroll
  for (int i = 0; i < P; ++i) f.p[i] = __builtin_bit_cast(bf16x8, buf16(b, off + i * plane));
  return f;
}
template <int DT>
__device__ inline Raw8<DT> buf8(__amdgpu_buffer_rsrc_t b, uint32_t off) {
  Raw8<DT> r;
#pragma unroll
  for (int i = 0; i < (DT == CCV_DT_F32 ? 2 : 1); ++i) r.d[i] = buf16(b, off + 16 * i);
  return r;
}
// One element as stored, and its value: the conversion stands where the value is used, so that
// the load may still be under way until then.
template <int DT> struct Stored { using type = uint16_t; };
template <> struct Stored<CCV_DT_F32> { using type = uint32_t; };

template <int DT>
__device__ inline typename Stored<DT>::type buf_raw(__amdgpu_buffer_rsrc_t b, uint32_t off) {
  if constexpr (DT == CCV_DT_F32) return __builtin_amdgcn_raw_buffer_load_b32(b, off, 0, 0);
  else return __builtin_amdgcn_raw_buffer_load_b16(b, off, 0, 0);
}
template <int DT>
__device__ inline float widen(typename Stored<DT>::type r) {
  if constexpr (DT == CCV_DT_F32) return __builtin_bit_cast(float, r);
  else return DT == CCV_DT_BF16 ? BF16::to_f(r) : F16::to_f(r);
}
template <int DT> struct Raw4 { u32x4 d; };      // four elements; 16-bit ones in the first two dwords
template <int DT>
__device__ inline Raw4<DT> buf_raw4(__amdgpu_buffer_rsrc_t b, uint32_t off) {
  if constexpr (DT == CCV_DT_F32) return {buf16(b, off)};
  const u32x2 d = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(b, off, 0, 0));
  return {u32x4{d[0], d[1], 0, 0}};
}
template <int DT>
__device__ inline f32x4 widen4(const Raw4<DT>& r) {
  if constexpr (DT == CCV_DT_F32) return __builtin_bit_cast(f32x4, r.d);
  f32x4 x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t two = r.d[i / 2];
    const uint16_t h = (uint16_t)(two >> (16 * (i % 2)));
    x[i] = DT == CCV_DT_BF16 ? BF16::to_f(h) : F16::to_f(h);
  }
  return x;
}
template <int DT>
__device__ inline float buf1(__amdgpu_buffer_rsrc_t b, uint32_t off) {
  if constexpr (DT == CCV_DT_F32) return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(b, off, 0, 0));
  const uint16_t h = __builtin_amdgcn_raw_buffer_load_b16(b, off, 0, 0);
  return DT == CCV_DT_BF16 ? BF16::to_f(h) : F16::to_f(h);
}
template <int DT>
__device__ inline Frag<InPlanes<DT>::n> planes(const Raw8<DT>& r) {
  Frag<InPlanes<DT>::n> f;
  if constexpr (DT == CCV_DT_BF16) {
    f.p[0] = __builtin_bit_cast(bf16x8, r.d[0]);
  } else if constexpr (DT == CCV_DT_F16) {
    f = split8<2>(__builtin_convertvector(__builtin_bit_cast(f16x8, r.d[0]), f32x8));
  } else {
    f32x8 x;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __builtin_bit_cast(float, dword(r.d[i / 4], i % 4));
    f = split8<3>(x);
  }
  return f;
}

template <int DT>
__device__ inline float load1(const void* p) {
  if constexpr (DT == CCV_DT_F32) return *static_cast<const float*>(p);
  else if constexpr (DT == CCV_DT_BF16) return BF16::to_f(*static_cast<const uint16_t*>(p));
  else return F16::to_f(*static_cast<const uint16_t*>(p));
}
template <int DT>
__device__ inline void store1(void* p, float x) {
  if constexpr (DT == CCV_DT_F32) *static_cast<float*>(p) = x;
  else if constexpr (DT == CCV_DT_BF16) *static_cast<uint16_t*>(p) = BF16::from_f(x);
  else *static_cast<uint16_t*>(p) = F16::from_f(x);
}
__device__ inline void store_gate(void* p, int dtype, int64_t i, float x) {
  if (dtype == CCV_DT_F32) static_cast<float*>(p)[i] = x;
  else static_cast<uint16_t*>(p)[i] = dtype == CCV_DT_BF16 ? BF16::from_f(x) : F16::from_f(x);
}

// The first `left` of 4 consecutive elements at p, from fp32.
template <int DT>
__device__ inline void store4(void* p, f32x4 x, int left, bool vec) {
  if (vec && left >= 4) {
    if constexpr (DT == CCV_DT_F32) {
      *static_cast<f32x4*>(p) = x;
    } else {
      u32x2 d;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f32x2 y = {as_f32(x[2 * i]), as_f32(x[2 * i + 1])};
        if constexpr (DT == CCV_DT_BF16) d[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(y, bf16x2));
        else d[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(y, f16x2));
      }
      *static_cast<u32x2*>(p) = d;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < left) store1<DT>(static_cast<char*>(p) + i * (DT == CCV_DT_F32 ? 4 : 2), x[i]);
}

// Four fp32 values into P planes of an LDS array whose planes are `plane` elements apart.
template <int P>
__device__ inline void put4(__bf16* at, int plane, f32x4 x) {
  float v[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
  for (int i = 0; i < P; ++i) {
    u32x2 d;
#pragma unroll
    for (int j = 0; j < 2; ++j) d[j] = take2(v[2 * j], v[2 * j + 1]);
    *reinterpret_cast<u32x2*>(at + i * plane) = d;
  }
}
template <int P>
__device__ inline Frag<P> get8(const __bf16* at, int plane) {
  Frag<P> f;
#pragma unroll
  for (int i = 0; i < P; ++i) f.p[i] = *reinterpret_cast<const bf16x8*>(at + i * plane);
  return f;
}

// The transposed fragment: lane l of a wave gets column l % 16 of rows 8 (l / 16) .. + 7 of the
// 32 x 16 block at `block` (row stride ld).  The transposing LDS read hands lane r of a group of 16 the
// r-th of the group's 4 x 4 elements of each row, rows coming from lanes 4 i .. 4 i + 3.
template <int P>
__device__ inline Frag<P> get8t(const __bf16* block, int ld, int plane, int lane) {
  const int r = lane & 15;
  const __bf16* at = block + (8 * (lane >> 4) + (r >> 2)) * ld + 4 * (r & 3);
  Frag<P> f;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    typedef __attribute__((address_space(3))) s16x4* lds4;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(at + i * plane));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(at + i * plane + 4 * ld));
    f.p[i] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
  return f;
}

// Sum over the 16 lanes of a row of a wave; every lane of the row gets it.
__device__ inline float sum16(float v) {
  v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x128, 0xf, 0xf, true));
  v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x124, 0xf, 0xf, true));
  v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x122, 0xf, 0xf, true));
  v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x121, 0xf, 0xf, true));
  return v;
}
// Sum over the four rows of 16 lanes.
__device__ inline float sum4rows(float v) {
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  return v;
}

// A workgroup barrier for data in LDS: every wave's LDS accesses before it are done, while its
// global loads and stores stay in flight (__syncthreads would wait for them too, which costs
// a prefetch its point).
__device__ inline void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// The workgroup's item of `items` (a sequence's, a part's or a chunk's value head) and its slice of the values.
// Workgroups go to the eight dies in turn, each with an L2 of its own: the slices of a head lie
// on one, whose L2 then holds the chunk's K, Q, W and P once for all of them, and where there are key
// heads enough to fill the chip so do the value heads that share K and Q (65536 packed steps, 10 / 20 heads in
// fp16: the matrices' kernel reads 0.42 GB instead of 0.76, the pass 1.57 instead of 1.92).
__device__ inline bool place(uint32_t share, uint32_t items, uint32_t slices, uint32_t* item, uint32_t* slice) {
  const uint32_t each = slices * share, b = blockIdx.x, r = b / 8 % each, g = r / slices;
  *item = (b / (8 * each) * 8 + b % 8) * share + g;
  *slice = r - g * slices;
  return *item < items;
}
inline uint32_t places(uint32_t share, int64_t items, uint32_t slices) {      // the grid for it
  return (uint32_t)((items / share + 7) / 8 * 8) * share * slices;
}

// Where a chunk lies; the same in every lane.
struct Chunk { int seq, row, t0, n; };

__device__ inline Chunk chunk_at(const DeltaArgs& a, int c) {
  Chunk k;
  if (a.packed) {
    k.seq = __builtin_amdgcn_readfirstlane(a.table[4 * c]);
    k.t0 = __builtin_amdgcn_readfirstlane(a.table[4 * c + 1]);
    k.n = __builtin_amdgcn_readfirstlane(a.table[4 * c + 2]);
    k.row = 0;
  } else {
    k.seq = c / a.chunks_per_row;
    k.t0 = (c - k.seq * a.chunks_per_row) * kDeltaChunk;
    const int64_t left = a.L - k.t0;
    k.n = left < kDeltaChunk ? (int)left : kDeltaChunk;
    k.row = k.seq;
  }
  return k;
}

// A sequence: its chunks are first .. end - 1, its steps t0 .. t0 + len - 1 of `row`.  A pass
// over its chunks needs no further look at the tables.
struct Sequence {
  int first, end, row, t0;
  int64_t len;
};

__device__ inline Sequence sequence_at(const DeltaArgs& a, int s) {
  Sequence q;
  if (a.packed) {
    const int32_t* begin = a.cstart + (a.nseq + 2);
    q.first = __builtin_amdgcn_readfirstlane(a.cstart[s]);
    q.end = __builtin_amdgcn_readfirstlane(a.cstart[s + 1]);
    q.t0 = __builtin_amdgcn_readfirstlane(begin[s]);
    q.len = __builtin_amdgcn_readfirstlane(begin[s + 1]) - q.t0;
    q.row = 0;
  } else {
    q.first = s * a.chunks_per_row;
    q.end = q.first + a.chunks_per_row;
    q.row = s;
    q.t0 = 0;
    q.len = a.L;
  }
  return q;
}

// The i-th sequence that a pass over the chunks takes.
__device__ inline int in_order(const DeltaArgs& a, int i) { return a.packed ? __builtin_amdgcn_readfirstlane(a.order[i]) : i; }

// What a workgroup of such a pass takes: a sequence, or a part of one.
struct Part {
  int seq, k, first;      // the sequence (nseq: the steps of none; above: nothing), which part of it, the number of its part 0
  int end;                // and of the part after its last
  bool last;
  Sequence sq;
};
__device__ inline Part part_at(const DeltaArgs& a, int s) {
  Part p{};
  if (!a.part_chunks) {
    p.seq = in_order(a, s);
    p.last = true;
    if (p.seq < a.nseq) p.sq = sequence_at(a, p.seq);
    return p;
  }
  if (a.packed) {
    p.seq = __builtin_amdgcn_readfirstlane(a.ptable[2 * s]);
    p.k = __builtin_amdgcn_readfirstlane(a.ptable[2 * s + 1]);
  } else {
    p.seq = s / a.parts_per_row;
    p.k = s - p.seq * a.parts_per_row;
  }
  p.first = s - p.k;
  if (p.seq >= a.nseq) return p;
  p.end = a.packed ? __builtin_amdgcn_readfirstlane(a.pstart[p.seq + 1]) : p.first + a.parts_per_row;
  p.sq = sequence_at(a, p.seq);
  const int64_t skip = (int64_t)p.k * a.part_chunks * kDeltaChunk, most = (int64_t)a.part_chunks * kDeltaChunk;
  p.sq.first += p.k * a.part_chunks;
  p.sq.t0 += (int)skip;
  p.last = p.sq.end <= p.sq.first + a.part_chunks;
  if (!p.last) p.sq.end = p.sq.first + a.part_chunks;
  p.sq.len = p.sq.len - skip < most ? p.sq.len - skip : most;
  return p;
}

// A part's map of the state in the workspace: T as right-to-left fragments (map_at), then B in 16 x 16 tiles as a
// wave's accumulators hold them, tiles of one 16 values together.
__device__ inline float* part_map(const DeltaArgs& a, int part, int h) {
  return a.carry + ((int64_t)part * a.Hv + h) * a.Dkp * (a.Dkp + a.Dvp);
}
template <int DKP>
__device__ inline int map_at(int row, int col) {       // element of T: a lane's 8 columns of a row lie together
  return (((row >> 4) * (DKP / 32) + (col >> 5)) * 64 + ((col >> 3) & 3) * 16 + (row & 15)) * 8 + (col & 7);
}
// The state that a part starts from, as the join left it in B's place: what the part next to it (step: -1 before, 1
// after) leaves.  The first of several parts, from the end the last, takes the sequence's own from the place of the
// part at the other end, which has no B: the caller may have the result written over the state that it came from, and
// the part that writes it may be done before the one that starts from it begins.  Null for a part that is a whole
// sequence: it reads what itself writes.
__device__ inline const f32x4* start_tiles(const DeltaArgs& a, const Part& p, int h, int step) {
  if (p.k == 0 && p.last) return nullptr;
  const int from = step < 0 ? (p.k == 0 ? p.end - 1 : p.first + p.k - 1) : p.last ? p.first : p.first + p.k + 1;
  return reinterpret_cast<const f32x4*>(part_map(a, from, h) + a.Dkp * a.Dkp);
}

template <int DT>
__device__ inline const char* row_ptr(const void* base, const int64_t* s, int row, int64_t t, int h) {
  return static_cast<const char*>(base) + (row * s[0] + t * s[1] + h * s[2]) * (DT == CCV_DT_F32 ? 4 : 2);
}
template <int DT>
__device__ inline char* row_ptr(void* base, const int64_t* s, int row, int64_t t, int h) {
  return static_cast<char*>(base) + (row * s[0] + t * s[1] + h * s[2]) * (DT == CCV_DT_F32 ? 4 : 2);
}

// A chunk's rows of a [B, L, H, D] array, `width` elements of each.
template <int DT>
__device__ inline __amdgpu_buffer_rsrc_t chunk_rows(const void* base, const int64_t* s, const Chunk& k, int h, int width) {
  constexpr int ES = DT == CCV_DT_F32 ? 4 : 2;
  const uint32_t bytes = (uint32_t)((k.n - 1) * (int32_t)(s[1] * ES) + width * ES);
  return buffer(row_ptr<DT>(base, s, k.row, k.t0, h), bytes);
}

// A sequence's chunks of such rows one after the other: the address moves by a constant.
template <int DT>
struct Rows {
  static constexpr int ES = DT == CCV_DT_F32 ? 4 : 2;
  const char* at;
  int64_t step;              // bytes from chunk to chunk
  uint32_t stride, width;    // bytes from step to step, and of a row
  __device__ inline Rows(const void* base, const int64_t* s, const Sequence& q, int h, int elements, int chunk)
      : at(row_ptr<DT>(base, s, q.row, q.t0 + (int64_t)(chunk - q.first) * kDeltaChunk, h)),
        step(s[1] * (kDeltaChunk * ES)), stride((uint32_t)(s[1] * ES)), width(elements * ES) {}
  // the chunk at hand, n steps of it (0: loads give zeros, stores do nothing)
  __device__ inline __amdgpu_buffer_rsrc_t rows(int n) const { return buffer(at, n > 0 ? (n - 1) * stride + width : 0); }
};

// The workspace's piece of a chunk, likewise.
template <class T>
struct Piece {
  const T* at;
  int64_t step;
  uint32_t bytes;
  __device__ inline Piece(const T* base, int64_t each, int hv, int64_t ch)
      : at(base + ch * each), step(each * hv), bytes((uint32_t)(each * sizeof(T))) {}
  __device__ inline __amdgpu_buffer_rsrc_t piece(bool there) const { return buffer(at, there ? bytes : 0); }
};

__device__ inline void buf_store_f4(__amdgpu_buffer_rsrc_t b, uint32_t off, f32x4 x) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), b, off, 0, 0);
}
template <int DT>
__device__ inline void buf_store1(__amdgpu_buffer_rsrc_t b, uint32_t off, float x) {
  if constexpr (DT == CCV_DT_F32) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, x), b, off, 0, 0);
  else __builtin_amdgcn_raw_buffer_store_b16(DT == CCV_DT_BF16 ? BF16::from_f(x) : F16::from_f(x), b, off, 0, 0);
}
// Four values, rounded; vec: the address takes them as one, and all four are in the row.
template <int DT>
__device__ inline void buf_store4(__amdgpu_buffer_rsrc_t b, uint32_t off, f32x4 x, int left, bool vec) {
  if (vec) {
    if constexpr (DT == CCV_DT_F32) {
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), b, off, 0, 0);
    } else {
      u32x2 d;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const f32x2 y = {as_f32(x[2 * i]), as_f32(x[2 * i + 1])};
        if constexpr (DT == CCV_DT_BF16) d[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(y, bf16x2));
        else d[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(y, f16x2));
      }
      __builtin_amdgcn_raw_buffer_store_b64(d, b, off, 0, 0);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) buf_store1<DT>(b, i < left ? off + i * (DT == CCV_DT_F32 ? 4 : 2) : kNowhere, x[i]);
}

// 16 rows of a chunk's 64, as a wave moves them: 16 bytes a lane with consecutive lanes on
// consecutive bytes, to LDS planes of row stride LD.  (Loading matrix fragments straight
// from rows puts 16 neighbouring lanes on 16 rows: 64 cache accesses an instruction where
// this takes 16.)
template <int DT, int DKP, int LD>
struct RowTile {
  static constexpr int ES = DT == CCV_DT_F32 ? 4 : 2, kLanes = DKP * ES / 16, kLoads = kLanes / 4, NA = InPlanes<DT>::n;
  u32x4 raw[kLoads];
  uint32_t off;          // byte offset of the first load; the others follow by 64 / kLanes rows
  uint32_t next;
  int at;                // element offset in a plane of LDS, likewise
  __device__ inline RowTile(int w, int l, uint32_t stride, int width) {
    const int row = 16 * w + l / kLanes, c = l % kLanes * (16 / ES);
    off = c < width ? row * stride + c * ES : kNowhere;
    next = c < width ? 64 / kLanes * stride : 0;
    at = row * LD + c;
  }
  __device__ inline void load(__amdgpu_buffer_rsrc_t b) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) raw[i] = buf16(b, off + i * next);
  }
  __device__ inline void store(__bf16* lds, int plane) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      __bf16* p = lds + at + i * (64 / kLanes) * LD;
      if constexpr (DT == CCV_DT_BF16) {
        *reinterpret_cast<u32x4*>(p) = raw[i];
      } else if constexpr (DT == CCV_DT_F16) {
        const Frag<2> f = split8<2>(__builtin_convertvector(__builtin_bit_cast(f16x8, raw[i]), f32x8));
        *reinterpret_cast<bf16x8*>(p) = f.p[0];
        *reinterpret_cast<bf16x8*>(p + plane) = f.p[1];
      } else {
        put4<3>(p, plane, __builtin_bit_cast(f32x4, raw[i]));
      }
    }
  }
};

// Where element (m, k .. k + 7) of a 64 x 64 matrix lies in a plane of the workspace: in the
// order in which a wave's lanes hold it as fragments, so that they load it in a row.
__device__ inline int fragment_at(int m, int k) {
  return (((m >> 4) * 2 + (k >> 5)) * 64 + ((k >> 3) & 3) * 16 + (m & 15)) * 8;
}

// ---- products that stay in a wave's registers ------------------------------------------------
//
// A wave that holds 16 columns of a product to the full height can use it as the next product's
// right-hand side without an exchange: the accumulator's lane (g4, r) holds rows 4 g4 + e of
// column r, the right-hand side's wants rows 8 g4 .. 8 g4 + 7 of 32.  So the left-hand side's rows
// are taken in another order: row 16 (2 s + o) + 4 q + e of the product is row 32 s + 8 q + 4 o + e of
// the matrix, and the tiles 2 s and 2 s + 1 joined are the right-hand side's fragment s.
__host__ __device__ constexpr int joined(int t) {      // matrix row t's place in that order
  return (t & 32) | ((t & 4) << 2) | ((t >> 1) & 12) | (t & 3);
}
__device__ inline f32x8 join(f32x4 a, f32x4 b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }

// A 16-bit input is one operand as it is stored; what it meets is fp32, in planes of the same type.
// In fp16 two planes keep 22 bits of an element, and 2^-39 of its column's largest: a column is scaled by a
// power of two that brings its largest value to 2^14 .. 2^15.
template <int DT> struct Cut { static constexpr int n = DT == CCV_DT_F16 ? 2 : 3; u32x4 p[n]; };

template <int DT>
__device__ inline f32x4 mfma16(u32x4 x, u32x4 y, f32x4 acc) {
  if constexpr (DT == CCV_DT_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), acc, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), acc, 0, 0, 0);
}
// The exponent that a column's values are taken relative to (0 in bf16, whose range is fp32's).
template <int DT, int N>
__device__ inline int column_exponent(const f32x4 (&x)[N]) {
  if constexpr (DT != CCV_DT_F16) return 0;
  float m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) m = __builtin_fmaxf(m, __builtin_fabsf(x[i][e]));
  m = __builtin_fmaxf(m, __shfl_xor(m, 16));
  m = __builtin_fmaxf(m, __shfl_xor(m, 32));
  return __builtin_amdgcn_frexp_expf(m) - 15;
}
template <int DT>
__device__ inline float scaled(float x, int exponent) { return DT == CCV_DT_F16 ? __builtin_ldexpf(x, exponent) : x; }
template <int DT>
__device__ inline f32x4 scaled(f32x4 x, int exponent) {
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = scaled<DT>(x[e], exponent);
  return x;
}
template <int DT>
__device__ inline Cut<DT> cut(f32x8 x, int exponent) {
  Cut<DT> c;
  if constexpr (DT == CCV_DT_F16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f32x2 y = {__builtin_ldexpf(x[2 * i], -exponent), __builtin_ldexpf(x[2 * i + 1], -exponent)};
      const f16x2 hi = __builtin_convertvector(y, f16x2);
      y = {y[0] - (float)hi[0], y[1] - (float)hi[1]};
      c.p[0][i] = __builtin_bit_cast(uint32_t, hi);
      c.p[1][i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(y, f16x2));
    }
  } else {
    const Frag<3> f = split8<3>(x);
#pragma unroll
    for (int i = 0; i < 3; ++i) c.p[i] = __builtin_bit_cast(u32x4, f.p[i]);
  }
  return c;
}

// The value, computed anew where it is used: kept out of the loop's registers.
__device__ inline uint32_t anew(uint32_t x) {
  asm volatile("" : "+v"(x));
  return x;
}

constexpr int kColumnWaves = 4;        // waves of a workgroup whose waves hold whole columns

// A chunk's 64 rows of 16-bit elements into LDS as they are, shared between NW waves; JOINED: in the
// order above.
template <int DKP, int LD, int NW, bool JOINED>
struct RowCopy {
  static constexpr int kLanes = DKP / 8, kEach = 64 / kLanes, kLoads = kLanes / NW;
  u32x4 raw[kLoads];
  uint32_t off, next;
  int at;
  __device__ inline RowCopy(int w, int l, uint32_t stride, int width) {
    const int row = w * (64 / NW) + l / kLanes, c = l % kLanes * 8;
    off = c < width ? row * stride + c * 2 : kNowhere;
    next = kEach * stride;       // the same in every lane: kNowhere and 63 steps stay above any bound and below 2^32
    at = (JOINED ? joined(row) : row) * LD + c;
  }
  __device__ inline void load(__amdgpu_buffer_rsrc_t b) {
    uint32_t o = anew(off);
#pragma unroll
    for (int i = 0; i < kLoads; ++i, o += next) raw[i] = buf16(b, o);
  }
  __device__ inline void store(uint16_t* lds) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)      // joined() moves bits, and these of the row lie apart from the lane's and the wave's
      *reinterpret_cast<u32x4*>(lds + at + (JOINED ? joined(i * kEach) : i * kEach) * LD) = raw[i];
  }
};

// Matrix instructions and memory accesses stay on their side of this line.  A wave alone on its SIMD has
// nothing to cover a load with but its own matrix instructions; left alone, the compiler moves a load down to
// where its value is used, which saves registers that such a wave has.
__device__ inline void keep_order() { __builtin_amdgcn_sched_barrier(0x0002 | 0x0004); }

// The transposed fragment of a joined LDS array: lane (g4, r) gets steps 32 s + 8 g4 .. + 7 of column
// 32 c + 8 (r / 4) + 4 o + r % 4 (columns in the joined order too).
template <int LD>
__device__ inline u32x4 get_joined_t(const uint16_t* lds, int s, int c, int o, int lane) {
  const int r = lane & 15;
  const uint16_t* at = lds + (32 * s + 4 * (lane >> 4) + (r >> 2)) * LD + 32 * c + 4 * o + 8 * (r & 3);
  typedef __attribute__((address_space(3))) s16x4* lds4;
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(at));
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(at + 16 * LD));
  return __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// ---- parts of sequences -----------------------------------------------------------------------
//
// The states at the parts' starts (BACK: the gradients at their ends), from the sequence's own and the parts'
// maps: S <- T S + B part by part, or S <- T^T S + B from the last on, each left where B was.  A workgroup
// takes 16 values of one sequence and head; a map is loaded while the one before it is applied.  About 1 us
// a part with 64 keys, 2.3 us with 128.
template <int DKP, bool BACK>
__global__ __launch_bounds__(256, 1) void join_kernel(DeltaArgs a) {
  constexpr int KS = DKP / 32, MT = DKP / 64, LDK = DKP + 16;
  __shared__ __bf16 Sp[3][16][LDK];
  const int seq = blockIdx.x / a.Hv, h = blockIdx.x - seq * a.Hv, dv0 = 16 * blockIdx.y;
  const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, r = l & 15, g4 = l >> 4;
  const int first = a.packed ? a.pstart[seq] : seq * a.parts_per_row, maps = (a.packed ? a.pstart[seq + 1] - first : a.parts_per_row) - 1;
  const int64_t each = (BACK ? -1 : 1) * (int64_t)a.Hv * DKP * (DKP + a.Dvp);
  float* map = part_map(a, first + (BACK ? maps : 0), h);
  f32x4* tiles = reinterpret_cast<f32x4*>(map + DKP * DKP) + (blockIdx.y * (DKP / 16) + MT * w) * 64 + l;
  struct Map {
    f32x8 T[MT][KS];
    f32x4 B[MT];
  } x, y;
  const auto load = [&](Map& t, int p) {
    if (p >= maps) return;
    const float* at = map + p * each;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int row = 16 * (MT * w + m) + r;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int k = 32 * s + 8 * g4;
        if constexpr (BACK) {
#pragma unroll
          for (int e = 0; e < 8; ++e) t.T[m][s][e] = at[map_at<DKP>(k + e, row)];
        } else {
          t.T[m][s] = *reinterpret_cast<const f32x8*>(at + map_at<DKP>(row, k));
        }
      }
      t.B[m] = tiles[p * each / 4 + m * 64];
    }
  };
  const float* own = BACK ? a.dht : a.h0;
  const int64_t* os = BACK ? a.dht_s : a.h0_s;
  f32x4 S[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int dk = 16 * (MT * w + m) + 4 * g4 + e, dv = dv0 + r;
      S[m][e] = own && dk < a.Dk && dv < a.Dv ? own[seq * os[0] + h * os[1] + dk * os[2] + dv] : 0.0f;
    }
  if (maps) {      // for the first part, or the last (start_tiles)
#pragma unroll
    for (int m = 0; m < MT; ++m) tiles[maps * each / 4 + m * 64] = S[m];
  }
  const auto apply = [&](Map& t, int p) {
#pragma unroll
    for (int m = 0; m < MT; ++m) put4<3>(&Sp[0][r][16 * (MT * w + m) + 4 * g4], 16 * LDK, S[m]);
    lds_barrier();
    Sums ts[MT];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const Frag<3> sf = get8<3>(&Sp[0][r][32 * s + 8 * g4], 16 * LDK);
#pragma unroll
      for (int m = 0; m < MT; ++m) ts[m].add(split8<3>(t.T[m][s]), sf);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) S[m] = ts[m].total() + t.B[m];
    load(t, p + 2);
#pragma unroll
    for (int m = 0; m < MT; ++m) tiles[p * each / 4 + m * 64] = S[m];
    lds_barrier();
  };
  load(x, 0);
  load(y, 1);
  for (int p = 0; p < maps; p += 2) {
    apply(x, p);
    if (p + 1 < maps) apply(y, p + 1);
  }
}

}  // namespace ccv
