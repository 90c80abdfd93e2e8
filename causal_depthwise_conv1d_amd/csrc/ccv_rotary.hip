// ccv_rotary.hip -- queries and keys turned by their positions.
//
//   (u, v) -> scale (u cos p f_i - v sin p f_i,  v cos p f_i + u sin p f_i)   for pair i of a head at position p,
// pairs of neighbours, or of elements half of the turned part apart.  Bound by memory: each array in and out
// once.  A workgroup makes the cosines and sines of a few tokens, once for all their heads, into LDS; then each
// thread has one place in a head (a vector of pairs, or one of what is only copied) and walks tokens and heads.
// 4 x 4096 tokens of 16 and 4 heads of 128 in bf16 (168 MB): 35 to 38 us, 4.4 to 4.8 TB/s; 512 or 2048 units a workgroup, and streaming
// loads or stores, take the same time.  256 tokens of 32 and 8 heads in fp16: 4.7 us, a launch and the angles' latency.
#include "ccv_delta_device.hpp"
#include "ccv_rotary_launch.hpp"

namespace ccv {
namespace {

// Cosine and sine of p f.  The angle in quarter turns is a product in 64 bits, so that far positions lose nothing; its
// whole part picks the quadrant, and the rest, at most half a quarter turn, goes into the two series:
// terms to x^9 and x^10, whose next ones are below 2^-28 at pi / 4.
__device__ inline void turn(int32_t p, double f, float& c, float& s) {
  const double q = (double)p * f * 0.63661977236758134308;
  const double whole = __builtin_rint(q);
  const int quadrant = (int)(4.0 * __builtin_amdgcn_fract(0.25 * whole));
  const float x = (float)((q - whole) * 1.57079632679489661923), x2 = x * x;
  float ps = __builtin_fmaf(x2, 2.7557319e-6f, -1.9841270e-4f);
  ps = __builtin_fmaf(x2, ps, 8.3333333e-3f);
  ps = __builtin_fmaf(x2, ps, -1.6666667e-1f);
  const float sn = __builtin_fmaf(x * x2, ps, x);
  float pc = __builtin_fmaf(x2, -2.7557319e-7f, 2.4801587e-5f);
  pc = __builtin_fmaf(x2, pc, -1.3888889e-3f);
  pc = __builtin_fmaf(x2, pc, 4.1666667e-2f);
  pc = __builtin_fmaf(x2, pc, -0.5f);
  const float cs = __builtin_fmaf(x2, pc, 1.0f);
  const float u = quadrant & 1 ? sn : cs, v = quadrant & 1 ? cs : sn;
  c = (quadrant + 1) & 2 ? -u : u;
  s = quadrant & 2 ? -v : v;
}

template <int DT> struct V16 { static constexpr int n = DT == CCV_DT_F32 ? 4 : 8, ES = DT == CCV_DT_F32 ? 4 : 2; };

template <int DT>
__device__ inline void unpack16(u32x4 raw, float* x) {
  if constexpr (DT == CCV_DT_F32) F32::unpack(raw, x);
  else if constexpr (DT == CCV_DT_BF16) BF16::unpack(raw, x);
  else F16::unpack(raw, x);
}
template <int DT>
__device__ inline u32x4 pack16(const float* x) {
  if constexpr (DT == CCV_DT_F32) return F32::pack(x);
  else if constexpr (DT == CCV_DT_BF16) return BF16::pack(x);
  else return F16::pack(x);
}

// The workgroup's cosines and sines, and where its tokens lie.
struct Tokens {
  float cos[kRotaryAngles], sin[kRotaryAngles];
  int32_t row[kRotaryAngles], step[kRotaryAngles];
};
__device__ inline void make_angles(const RotaryArgs& a, Tokens& t, int64_t first, int n) {
  for (int i = threadIdx.x; i < n; i += 256) {
    const uint32_t at = (uint32_t)(first + i), row = at / (uint32_t)a.L;
    t.row[i] = (int32_t)row;
    t.step[i] = (int32_t)(at - row * (uint32_t)a.L);
  }
  for (int i = threadIdx.x; i < n * a.half; i += 256) {
    const int tok = i / a.half, k = i - tok * a.half;
    const uint32_t at = (uint32_t)(first + tok), row = at / (uint32_t)a.L;
    float c, s;
    turn(a.pos[row * a.pos_s[0] + (at - row * (uint32_t)a.L) * a.pos_s[1]], a.freq[k], c, s);
    t.cos[i] = c * a.scale;
    t.sin[i] = s * a.scale * a.sign;
  }
}

template <int DT>
__device__ inline int64_t head_at(const RotaryArgs& a, const int64_t (&s)[2][3], const Tokens& t, int tok, int h, int which) {
  return t.row[tok] * s[which][0] + t.step[tok] * s[which][1] + h * s[which][2];
}

template <int DT, bool NEIGHBOURS>
__global__ __launch_bounds__(256) void vec_kernel(const RotaryArgs a) {
  constexpr int V = V16<DT>::n, ES = V16<DT>::ES;
  __shared__ Tokens t;
  const int64_t first = (int64_t)blockIdx.x * a.span;
  const int n = (int)(a.tokens - first < a.span ? a.tokens - first : a.span);
  make_angles(a, t, first, n);
  __syncthreads();
  const int per = 256 / a.units, place = threadIdx.x / a.units, unit = threadIdx.x - place * a.units;
  if (place >= per) return;
  const int all = a.heads[0] + a.heads[1];
  const bool turned = unit < a.turned_units;
  const int turned_width = NEIGHBOURS ? 2 * a.half : a.half;
  // the vector's first element in the head; the last of a part ends with it
  int at;
  if (turned) {
    at = unit * V;
    at = at + V <= turned_width ? at : turned_width - V;
  } else {
    at = 2 * a.half + (unit - a.turned_units) * V;
    at = at + V <= a.D ? at : a.D - V;
  }
  int tok = place / all, h = place - tok * all;
  const int step_tok = per / all, step_h = per - step_tok * all;
  while (tok < n) {
    const int which = h >= a.heads[0], head = h - (which ? a.heads[0] : 0);
    const char* ip = static_cast<const char*>(a.in[which]) + (head_at<DT>(a, a.in_s, t, tok, head, which) + at) * ES;
    char* op = static_cast<char*>(a.out[which]) + (head_at<DT>(a, a.out_s, t, tok, head, which) + at) * ES;
    if (!turned) {
      store16(op, load16(ip));
    } else if constexpr (NEIGHBOURS) {
      float x[V];
      unpack16<DT>(load16(ip), x);
      const float *c = t.cos + tok * a.half + at / 2, *s = t.sin + tok * a.half + at / 2;
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const float u = x[2 * i], v = x[2 * i + 1];
        x[2 * i] = __builtin_fmaf(u, c[i], -(v * s[i]));
        x[2 * i + 1] = __builtin_fmaf(v, c[i], u * s[i]);
      }
      store16(op, pack16<DT>(x));
    } else {
      float u[V], v[V];
      const u32x4 ru = load16(ip), rv = load16(ip + a.half * ES);
      unpack16<DT>(ru, u);
      unpack16<DT>(rv, v);
      const float *c = t.cos + tok * a.half + at, *s = t.sin + tok * a.half + at;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float x = u[i], y = v[i];
        u[i] = __builtin_fmaf(x, c[i], -(y * s[i]));
        v[i] = __builtin_fmaf(y, c[i], x * s[i]);
      }
      store16(op, pack16<DT>(u));
      store16(op + a.half * ES, pack16<DT>(v));
    }
    tok += step_tok;
    h += step_h;
    if (h >= all) {
      h -= all;
      ++tok;
    }
  }
}

// Element by element: each thread owns a pair, or an element that is only copied.
template <int DT>
__global__ __launch_bounds__(256) void any_kernel(const RotaryArgs a) {
  constexpr int ES = V16<DT>::ES;
  __shared__ Tokens t;
  const int64_t first = (int64_t)blockIdx.x * a.span;
  const int n = (int)(a.tokens - first < a.span ? a.tokens - first : a.span);
  make_angles(a, t, first, n);
  __syncthreads();
  const uint32_t units = (uint32_t)(a.half + (a.in_place ? 0 : a.D - 2 * a.half)), all = (uint32_t)(a.heads[0] + a.heads[1]);
  for (uint32_t i = threadIdx.x; i < units * all * n; i += 256) {
    const uint32_t th = i / units, unit = i - th * units, tok = th / all, h = th - tok * all;
    const int which = (int)h >= a.heads[0], head = (int)h - (which ? a.heads[0] : 0);
    const char* ip = static_cast<const char*>(a.in[which]) + head_at<DT>(a, a.in_s, t, (int)tok, head, which) * ES;
    char* op = static_cast<char*>(a.out[which]) + head_at<DT>(a, a.out_s, t, (int)tok, head, which) * ES;
    if ((int)unit >= a.half) {
      const uint32_t e = unit + a.half;
      store1<DT>(op + e * ES, load1<DT>(ip + e * ES));
      continue;
    }
    const uint32_t e0 = a.interleaved ? 2 * unit : unit, e1 = a.interleaved ? 2 * unit + 1 : unit + a.half;
    const float u = load1<DT>(ip + e0 * ES), v = load1<DT>(ip + e1 * ES), c = t.cos[tok * a.half + unit], s = t.sin[tok * a.half + unit];
    store1<DT>(op + e0 * ES, __builtin_fmaf(u, c, -(v * s)));
    store1<DT>(op + e1 * ES, __builtin_fmaf(v, c, u * s));
  }
}

template <int DT>
void launch(const RotaryArgs& a, hipStream_t st) {
  const uint32_t grid = (uint32_t)((a.tokens + a.span - 1) / a.span);
  if (!a.units) any_kernel<DT><<<grid, 256, 0, st>>>(a);
  else if (a.interleaved) vec_kernel<DT, true><<<grid, 256, 0, st>>>(a);
  else vec_kernel<DT, false><<<grid, 256, 0, st>>>(a);
}

}  // namespace

int launch_rotary(const RotaryArgs& a, void* stream) {
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (a.x_dtype == CCV_DT_F32) launch<CCV_DT_F32>(a, st);
  else if (a.x_dtype == CCV_DT_F16) launch<CCV_DT_F16>(a, st);
  else launch<CCV_DT_BF16>(a, st);
  return (int)hipGetLastError();
}

}  // namespace ccv
