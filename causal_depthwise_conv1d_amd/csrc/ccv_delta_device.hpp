// ccv_delta_device.hpp -- matrix fragments of the gated delta rule's kernels.
//
// Every product runs on the bf16 matrix instruction 16x16x32.  An fp32 value is held as a
// sum of bf16 planes, hi + mid + lo (8 significant bits each, 24 together), and a product
// of two such values is the sum of the plane products whose indexes add up to at most
// `ORDER`: order 2 keeps about 2^-23 of the result, which is what fp32 outputs (states,
// gate gradients) need; order 1 about 2^-16, enough for a 16-bit output.  An fp32 product
// through three planes takes 6 instructions where the fp32 matrix instruction takes the
// time of 16.  bf16 inputs are one plane, exactly; fp16 inputs are two, exactly.
#pragma once

#include "ccv_device.hpp"
#include "ccv_delta_launch.hpp"

namespace ccv {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896341f;

// planes of an input element
template <int DT> struct InPlanes { static constexpr int n = DT == CCV_DT_BF16 ? 1 : DT == CCV_DT_F16 ? 2 : 3; };
// order of products whose results are rounded to the input's type
template <int DT> struct OutOrder { static constexpr int n = DT == CCV_DT_F32 ? 2 : 1; };

template <int P> struct Frag { bf16x8 p[P]; };

template <int P>
__device__ inline Frag<P> split8(f32x8 x) {
  Frag<P> f;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    f.p[i] = __builtin_convertvector(x, bf16x8);
    if (i + 1 < P) x -= __builtin_convertvector(f.p[i], f32x8);
  }
  return f;
}

// acc += a b over 32 steps of the contraction; the small terms first.
template <int ORDER, int PA, int PB>
__device__ inline f32x4 mma(const Frag<PA>& a, const Frag<PB>& b, f32x4 acc) {
#pragma unroll
  for (int s = ORDER; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < PA; ++i)
      if (s - i >= 0 && s - i < PB) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[i], b.p[s - i], acc, 0, 0, 0);
  return acc;
}

// Eight consecutive elements of a row, as stored.
template <int DT> struct Raw8 { u32x4 d[DT == CCV_DT_F32 ? 2 : 1]; };

// The first `left` of 8 consecutive elements from p; zeros for the others.  vec: all or
// none of them are there and p is aligned for whole vectors.
template <int DT>
__device__ inline Raw8<DT> load8(const void* p, int left, bool vec) {
  Raw8<DT> r;
#pragma unroll
  for (int i = 0; i < (DT == CCV_DT_F32 ? 2 : 1); ++i) r.d[i] = u32x4{0, 0, 0, 0};
  if (left <= 0) return r;
  if (vec) {
    r.d[0] = load16(p);
    if constexpr (DT == CCV_DT_F32) r.d[1] = load16(static_cast<const char*>(p) + 16);
    return r;
  }
  if constexpr (DT == CCV_DT_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) r.d[i / 4][i % 4] = static_cast<const uint32_t*>(p)[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) r.d[0][i / 2] |= (uint32_t) static_cast<const uint16_t*>(p)[i] << (16 * (i % 2));
  }
  return r;
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

__device__ inline f32x8 load_f8(const float* p) {
  const f32x4 x = *reinterpret_cast<const f32x4*>(p), y = *reinterpret_cast<const f32x4*>(p + 4);
  return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
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

// The first `left` of 4 consecutive elements at p, widened.
template <int DT>
__device__ inline f32x4 load4(const void* p, int left, bool vec) {
  f32x4 x = {0, 0, 0, 0};
  if (vec && left >= 4) {
    if constexpr (DT == CCV_DT_F32) return *static_cast<const f32x4*>(p);
    const u32x2 d = *static_cast<const u32x2*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint16_t h = (uint16_t)(d[i / 2] >> (16 * (i % 2)));
      x[i] = DT == CCV_DT_BF16 ? BF16::to_f(h) : F16::to_f(h);
    }
    return x;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < left) x[i] = load1<DT>(static_cast<const char*>(p) + i * (DT == CCV_DT_F32 ? 4 : 2));
  return x;
}

// Four fp32 values into P planes of an LDS array whose planes are `plane` elements apart.
template <int P>
__device__ inline void put4(__bf16* at, int plane, f32x4 x) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const bf16x4 h = __builtin_convertvector(x, bf16x4);
    *reinterpret_cast<bf16x4*>(at + i * plane) = h;
    if (i + 1 < P) x -= __builtin_convertvector(h, f32x4);
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

// Where a chunk lies.
struct Chunk { int seq, row, t0, n; };

__device__ inline Chunk chunk_at(const DeltaArgs& a, int c) {
  Chunk k;
  if (a.packed) {
    k.seq = a.table[4 * c];
    k.t0 = a.table[4 * c + 1];
    k.n = a.table[4 * c + 2];
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

// Sequence s's chunks are first .. end - 1.
__device__ inline void chunks_of(const DeltaArgs& a, int s, int* first, int* end) {
  *first = a.packed ? a.cstart[s] : s * a.chunks_per_row;
  *end = a.packed ? a.cstart[s + 1] : (s + 1) * a.chunks_per_row;
}

template <int DT>
__device__ inline const char* row_ptr(const void* base, const int64_t* s, int row, int64_t t, int h) {
  return static_cast<const char*>(base) + (row * s[0] + t * s[1] + h * s[2]) * (DT == CCV_DT_F32 ? 4 : 2);
}
template <int DT>
__device__ inline char* row_ptr(void* base, const int64_t* s, int row, int64_t t, int h) {
  return static_cast<char*>(base) + (row * s[0] + t * s[1] + h * s[2]) * (DT == CCV_DT_F32 ? 4 : 2);
}

}  // namespace ccv
