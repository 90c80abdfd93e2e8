// ccv_delta_scan.hip -- gated delta rule: the pass over a sequence's chunks that carries
// the state, forward.
//
// With gam = e^G, del = e^(G63 - G), W and P of ccv_delta_prep.hip and S the state
// [Dk, Dv] at the chunk's start:
//   R = v - gam K S,  N = W (beta R),  o = scale (gam Q S + P N),  S <- gam63 S + K^T (del N).
// Columns of S (values) do not mix, so a workgroup takes CB = 16 NT of them for one
// sequence and head, and its four waves share the rows: 16 of a chunk's 64 steps and a
// quarter of the state's rows each, S staying in fp32 accumulators from the first chunk
// to the last.  What a wave needs of the others' rows (S, beta R, N as right-hand sides)
// passes through LDS as bf16 planes, three barriers a chunk.
#include "ccv_delta_device.hpp"

namespace ccv {
namespace {

constexpr int LDT = 72;      // row stride of an LDS array of 64 steps

// What a wave loads of a chunk before it computes on it.
template <int DT, int KS, int NT>
struct Loaded {
  Raw8<DT> k[KS], q[KS];
  f32x8 W[2], P[2];
  float v[NT][4];
  f32x4 gam, del, beta;
  float gam_row, last;
  int n, row, t0;
};

template <int DT, int DKP, int NT, bool BWD>
__global__ __launch_bounds__(256) void scan_kernel(DeltaArgs a, uint32_t heads, uint32_t heads_pad) {
  constexpr int NA = InPlanes<DT>::n, CB = 16 * NT, KS = DKP / 32, MT = DKP / 64, LDK = DKP + 8;
  constexpr int OO = OutOrder<DT>::n, ES = DT == CCV_DT_F32 ? 4 : 2;
  __shared__ __bf16 Sp[3][CB][LDK];        // S by columns
  __shared__ __bf16 Rp[3][CB][LDT];        // beta R by columns
  __shared__ __bf16 Np[OO + 1][CB][LDT];   // N
  __shared__ __bf16 Nd[3][CB][LDT];        // del N
  __shared__ __bf16 Kl[NA][64][LDK];
  const uint32_t hs = blockIdx.x % heads_pad, slice = blockIdx.x / heads_pad;
  if (hs >= heads) return;
  const int seq = hs / a.Hv, h = hs - seq * a.Hv, hk = h / (a.Hv / a.Hk), dv0 = slice * CB;
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, r = l & 15, g4 = l >> 4;

  if (seq >= a.nseq) {                     // the steps of a packed row that belong to no sequence
    if constexpr (!BWD) {
      const int32_t* begin = a.cstart + (a.nseq + 2);
      for (int64_t i = (int64_t)begin[a.nseq] * CB + tid; i < a.L * CB; i += 256) {
        const int64_t t = i / CB;
        const int d = dv0 + (int)(i - t * CB);
        if (d < a.Dv) store1<DT>(row_ptr<DT>(a.out, a.o_s, 0, t, h) + d * ES, 0.0f);
      }
    }
    return;
  }
  int c0, c1;
  chunks_of(a, seq, &c0, &c1);

  // the state: rows 16 (MT w + m) + 4 g4 + e, column 16 j + r
  f32x4 S[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int dk = 16 * (MT * w + m) + 4 * g4 + e, dv = dv0 + 16 * j + r;
        S[m][j][e] = a.h0 && dk < a.Dk && dv < a.Dv ? a.h0[seq * a.h0_s[0] + h * a.h0_s[1] + dk * a.h0_s[2] + dv] : 0.0f;
      }

  auto load = [&](int c) {
    Loaded<DT, KS, NT> x;
    const Chunk k = chunk_at(a, c);
    x.n = k.n;
    x.row = k.row;
    x.t0 = k.t0;
    const int64_t ch = (int64_t)c * a.Hv + h;
    const int i = 16 * w + r;
    const bool live = i < k.n;
    const char* kp = row_ptr<DT>(a.k, a.k_s, k.row, k.t0 + (live ? i : 0), hk);
    const char* qp = row_ptr<DT>(a.q, a.q_s, k.row, k.t0 + (live ? i : 0), hk);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int d = 32 * s + 8 * g4, left = live ? a.Dk - d : 0;
      x.k[s] = load8<DT>(kp + d * ES, left, a.vec_qk);
      x.q[s] = load8<DT>(qp + d * ES, left, a.vec_qk);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      x.W[s] = load_f8(a.W + ch * 4096 + i * 64 + 32 * s + 8 * g4);
      if constexpr (!BWD) x.P[s] = load_f8(a.P + ch * 4096 + i * 64 + 32 * s + 8 * g4);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = 16 * w + 4 * g4 + e;
      const char* vp = row_ptr<DT>(a.v, a.v_s, k.row, k.t0 + (t < k.n ? t : 0), h);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int dv = dv0 + 16 * j + r;
        x.v[j][e] = t < k.n && dv < a.Dv ? load1<DT>(vp + dv * ES) : 0.0f;
      }
    }
    const float* dec = a.dec + ch * kDeltaDec;
    x.gam = *reinterpret_cast<const f32x4*>(dec + 16 * w + 4 * g4);
    x.del = *reinterpret_cast<const f32x4*>(dec + 64 + 16 * w + 4 * g4);
    x.beta = *reinterpret_cast<const f32x4*>(dec + 128 + 16 * w + 4 * g4);
    x.gam_row = dec[i];
    x.last = dec[63];
    return x;
  };
  auto put_state = [&]() {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j) put4<3>(&Sp[0][16 * j + r][16 * (MT * w + m) + 4 * g4], CB * LDK, S[m][j]);
  };

  Loaded<DT, KS, NT> x;
  if (c0 < c1) x = load(c0);
  put_state();
  __syncthreads();
  for (int c = c0; c < c1; ++c) {
    const int64_t ch = (int64_t)c * a.Hv + h;
    const Loaded<DT, KS, NT> y = x;
    if (c + 1 < c1) x = load(c + 1);
    if constexpr (BWD) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            a.S[(ch * DKP + 16 * (MT * w + m) + 4 * g4 + e) * a.Dvp + dv0 + 16 * j + r] = S[m][j][e];
    }

    // K S (rows: steps) and S^T Q^T (columns: steps)
    f32x4 ks[NT], qs[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) ks[j] = qs[j] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const Frag<NA> kf = planes<DT>(y.k[s]), qf = planes<DT>(y.q[s]);
#pragma unroll
      for (int p = 0; p < NA; ++p) *reinterpret_cast<bf16x8*>(&Kl[p][16 * w + r][32 * s + 8 * g4]) = kf.p[p];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const Frag<3> sf = get8<3>(&Sp[0][16 * j + r][32 * s + 8 * g4], CB * LDK);
        ks[j] = mma<2>(kf, sf, ks[j]);
        qs[j] = mma<BWD ? 2 : OO>(sf, qf, qs[j]);
      }
    }
    // beta R
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      f32x4 R;
#pragma unroll
      for (int e = 0; e < 4; ++e) R[e] = __builtin_fmaf(-y.gam[e], ks[j][e], y.v[j][e]);
      if constexpr (BWD) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          a.R[(ch * 64 + 16 * w + 4 * g4 + e) * a.Dvp + dv0 + 16 * j + r] = R[e];
      }
      put4<3>(&Rp[0][16 * j + r][16 * w + 4 * g4], CB * LDT, R * y.beta);
    }
    __syncthreads();

    // N = W (beta R); W is lower triangular
    f32x4 N[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) N[j] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (2 * s > w) continue;
      const Frag<3> wf = split8<3>(y.W[s]);
#pragma unroll
      for (int j = 0; j < NT; ++j) N[j] = mma<2>(wf, get8<3>(&Rp[0][16 * j + r][32 * s + 8 * g4], CB * LDT), N[j]);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if constexpr (BWD) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          a.N[(ch * 64 + 16 * w + 4 * g4 + e) * a.Dvp + dv0 + 16 * j + r] = N[j][e];
      } else {
        put4<OO + 1>(&Np[0][16 * j + r][16 * w + 4 * g4], CB * LDT, N[j]);
      }
      put4<3>(&Nd[0][16 * j + r][16 * w + 4 * g4], CB * LDT, N[j] * y.del);
    }
    __syncthreads();

    // the state at the chunk's end
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j) S[m][j] *= y.last;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      Frag<3> nf[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) nf[j] = get8<3>(&Nd[0][16 * j + r][32 * s + 8 * g4], CB * LDT);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const Frag<NA> kt = get8t<NA>(&Kl[0][32 * s][16 * (MT * w + m)], LDK, 64 * LDK, l);
#pragma unroll
        for (int j = 0; j < NT; ++j) S[m][j] = mma<2>(kt, nf[j], S[m][j]);
      }
    }
    put_state();      // nobody has read the planes since the first barrier

    const int t = 16 * w + r;
    if constexpr (!BWD) {
      // o, four consecutive values of one step a lane
      Frag<OO + 1> pf[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) pf[s] = split8<OO + 1>(y.P[s]);
      char* op = row_ptr<DT>(a.out, a.o_s, y.row, (int64_t)y.t0 + t, h);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        f32x4 o = qs[j] * y.gam_row;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (2 * s > w) continue;
          o = mma<OO>(get8<OO + 1>(&Np[0][16 * j + r][32 * s + 8 * g4], CB * LDT), pf[s], o);
        }
        const int dv = dv0 + 16 * j + 4 * g4;
        if (t < y.n) store4<DT>(op + dv * ES, o * a.scale, a.Dv - dv, a.vec_o);
      }
    } else {
      // scale gam dO . (Q S): the part of dG that comes by the state
      const char* dp = row_ptr<DT>(a.dout, a.do_s, y.row, (int64_t)y.t0 + (t < y.n ? t : 0), h);
      float dot = 0;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int dv = dv0 + 16 * j + 4 * g4;
        const f32x4 d = load4<DT>(dp + dv * ES, t < y.n ? a.Dv - dv : 0, a.vec_do);
#pragma unroll
        for (int e = 0; e < 4; ++e) dot = __builtin_fmaf(d[e], qs[j][e], dot);
      }
      dot = sum4rows(dot) * y.gam_row * a.scale;
      if (g4 == 0) a.part[(ch * a.slices + slice) * kDeltaPart + t] = dot;
    }
    __syncthreads();
  }
  if (a.ht) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int dk = 16 * (MT * w + m) + 4 * g4 + e, dv = dv0 + 16 * j + r;
          if (dk < a.Dk && dv < a.Dv) a.ht[seq * a.ht_s[0] + h * a.ht_s[1] + dk * a.ht_s[2] + dv] = S[m][j][e];
        }
  }
}

template <int DT, int DKP, int NT>
void launch(const DeltaArgs& a, bool bwd, hipStream_t st) {
  const uint32_t heads = (uint32_t)(a.nseq + (a.packed ? 1 : 0)) * a.Hv;
  // slices of one head lie 8 k workgroups apart: on one XCD, whose L2 then holds the
  // chunk's K, Q, W and P once for all of them
  const uint32_t pad = (heads + 7) / 8 * 8;
  const dim3 grid(pad * ((a.Dvp + 16 * NT - 1) / (16 * NT)));
  if (bwd) scan_kernel<DT, DKP, NT, true><<<grid, 256, 0, st>>>(a, heads, pad);
  else scan_kernel<DT, DKP, NT, false><<<grid, 256, 0, st>>>(a, heads, pad);
}
template <int DT>
void launch(const DeltaArgs& a, bool bwd, int nt, hipStream_t st) {
  if (a.Dkp == 64) {
    if (nt == 1) launch<DT, 64, 1>(a, bwd, st);
    else launch<DT, 64, 2>(a, bwd, st);
  } else {
    if (nt == 1) launch<DT, 128, 1>(a, bwd, st);
    else launch<DT, 128, 2>(a, bwd, st);
  }
}

}  // namespace

int launch_delta_scan(const DeltaArgs& a, bool backward, int nt, void* stream) {
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (a.x_dtype == CCV_DT_F32) launch<CCV_DT_F32>(a, backward, nt, st);
  else if (a.x_dtype == CCV_DT_F16) launch<CCV_DT_F16>(a, backward, nt, st);
  else launch<CCV_DT_BF16>(a, backward, nt, st);
  return (int)hipGetLastError();
}

}  // namespace ccv
