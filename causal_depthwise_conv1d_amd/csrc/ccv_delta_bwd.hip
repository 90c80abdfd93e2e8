// ccv_delta_bwd.hip -- gated delta rule, backward: the pass over a sequence's chunks from
// its end, which carries the state's gradient, and the gradients that a chunk's steps
// have once the states at both of its ends are known.
//
// With the forward's gam, del, W, P, S, R, N (ccv_delta_scan.hip) and dS' the gradient of
// the state at the chunk's end:
//   dN = scale P^T dO + del (K dS'),   Y = W^T dN,   dv = dR = beta Y,
//   dS = gam63 dS' + Q^T (scale gam dO) - K^T (gam beta Y),
//   dA = -Y N^T,  E = beta e^(Gi - Gj) dA (i > j),   F = scale e^(Gi - Gj) dO N^T (i >= j),
//   dq = scale gam S dO + F K,
//   dk = -gam beta S Y + del dS' N + E K + F^T Q + E^T K,
//   dbeta_i = Y_i . R_i + sum_j e^(Gi - Gj) k_i.k_j dA_ij,
// and the gradient of G_i, with M = F o (Q K^T) + E o (K K^T) below the diagonal and
// c_j = del_j (K dS')_j . N_j:
//   dG_i = scale gam_i dO_i.(Q S)_i + dR_i.(R_i - v_i) + sum_j M_ij - sum_j M_ji - c_i,
//   dG_63 += sum_j c_j + gam63 <S, dS'>,          dg_t = sum of dG_i over i >= t.
// Terms whose two ends are the same step are left out of both sums, so gradients that are
// zero by the formula (a sequence of one step without a state) come out as zero.
#include "ccv_delta_device.hpp"

namespace ccv {
namespace {

constexpr int LDT = 72;

template <int DT, int KS, int NT>
struct LoadedBack {
  Raw8<DT> k[KS], q[KS];
  f32x8 WT[2], PT[2];
  float d[NT][4], v[NT][4], R[NT][4], N[NT][4];
  f32x4 gam, del, beta;
  float last;
  int n, row, t0;
};

template <int DT, int DKP, int NT>
__global__ __launch_bounds__(256) void reverse_kernel(DeltaArgs a, uint32_t heads, uint32_t heads_pad) {
  constexpr int NA = InPlanes<DT>::n, CB = 16 * NT, KS = DKP / 32, MT = DKP / 64, LDK = DKP + 8;
  constexpr int ES = DT == CCV_DT_F32 ? 4 : 2;
  __shared__ __bf16 Sp[3][CB][LDK];        // dS by columns
  __shared__ __bf16 Dp[NA][CB][LDT];       // dO
  __shared__ __bf16 Dd[3][CB][LDT];        // scale gam dO
  __shared__ __bf16 Rp[3][CB][LDT];        // dN
  __shared__ __bf16 Yp[3][CB][LDT];        // -gam beta Y
  __shared__ __bf16 Kl[NA][64][LDK], Ql[NA][64][LDK];
  const uint32_t hs = blockIdx.x % heads_pad, slice = blockIdx.x / heads_pad;
  if (hs >= heads) return;
  const int seq = hs / a.Hv, h = hs - seq * a.Hv, hk = h / (a.Hv / a.Hk), dv0 = slice * CB;
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, r = l & 15, g4 = l >> 4;

  if (seq >= a.nseq) {                     // steps of no sequence have no gradient
    const int32_t* begin = a.cstart + (a.nseq + 2);
    for (int64_t i = (int64_t)begin[a.nseq] * CB + tid; i < a.L * CB; i += 256) {
      const int64_t t = i / CB;
      const int d = dv0 + (int)(i - t * CB);
      if (d < a.Dv) store1<DT>(row_ptr<DT>(a.dv, a.dv_s, 0, t, h) + d * ES, 0.0f);
    }
    return;
  }
  int c0, c1;
  chunks_of(a, seq, &c0, &c1);

  f32x4 S[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int dk = 16 * (MT * w + m) + 4 * g4 + e, dv = dv0 + 16 * j + r;
        S[m][j][e] = a.dht && dk < a.Dk && dv < a.Dv ? a.dht[seq * a.dht_s[0] + h * a.dht_s[1] + dk * a.dht_s[2] + dv] : 0.0f;
      }

  auto load = [&](int c) {
    LoadedBack<DT, KS, NT> x;
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
      x.WT[s] = load_f8(a.WT + ch * 4096 + i * 64 + 32 * s + 8 * g4);
      x.PT[s] = load_f8(a.P + ch * 4096 + i * 64 + 32 * s + 8 * g4);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = 16 * w + 4 * g4 + e;
      const bool in = t < k.n;
      const char* vp = row_ptr<DT>(a.v, a.v_s, k.row, k.t0 + (in ? t : 0), h);
      const char* dp = row_ptr<DT>(a.dout, a.do_s, k.row, k.t0 + (in ? t : 0), h);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int dv = dv0 + 16 * j + r;
        x.v[j][e] = in && dv < a.Dv ? load1<DT>(vp + dv * ES) : 0.0f;
        x.d[j][e] = in && dv < a.Dv ? load1<DT>(dp + dv * ES) : 0.0f;
        x.R[j][e] = a.R[(ch * 64 + t) * a.Dvp + dv];
        x.N[j][e] = a.N[(ch * 64 + t) * a.Dvp + dv];
      }
    }
    const float* dec = a.dec + ch * kDeltaDec;
    x.gam = *reinterpret_cast<const f32x4*>(dec + 16 * w + 4 * g4);
    x.del = *reinterpret_cast<const f32x4*>(dec + 64 + 16 * w + 4 * g4);
    x.beta = *reinterpret_cast<const f32x4*>(dec + 128 + 16 * w + 4 * g4);
    x.last = dec[63];
    return x;
  };

  LoadedBack<DT, KS, NT> x;
  if (c0 < c1) x = load(c1 - 1);
  for (int c = c1 - 1; c >= c0; --c) {
    const int64_t ch = (int64_t)c * a.Hv + h;
    const LoadedBack<DT, KS, NT> y = x;
    if (c > c0) x = load(c - 1);
    float* part = a.part + (ch * a.slices + slice) * kDeltaPart;

    // the planes of this chunk
    Frag<NA> kf[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      kf[s] = planes<DT>(y.k[s]);
      const Frag<NA> qf = planes<DT>(y.q[s]);
#pragma unroll
      for (int p = 0; p < NA; ++p) {
        *reinterpret_cast<bf16x8*>(&Kl[p][16 * w + r][32 * s + 8 * g4]) = kf[s].p[p];
        *reinterpret_cast<bf16x8*>(&Ql[p][16 * w + r][32 * s + 8 * g4]) = qf.p[p];
      }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const f32x4 d = {y.d[j][0], y.d[j][1], y.d[j][2], y.d[j][3]};
      put4<NA>(&Dp[0][16 * j + r][16 * w + 4 * g4], CB * LDT, d);
      put4<3>(&Dd[0][16 * j + r][16 * w + 4 * g4], CB * LDT, d * y.gam * a.scale);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        put4<3>(&Sp[0][16 * j + r][16 * (MT * w + m) + 4 * g4], CB * LDK, S[m][j]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          a.dS[(ch * DKP + 16 * (MT * w + m) + 4 * g4 + e) * a.Dvp + dv0 + 16 * j + r] = S[m][j][e];
      }
    __syncthreads();

    // dN
    f32x4 kd[NT], pd[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) kd[j] = pd[j] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int j = 0; j < NT; ++j)
        kd[j] = mma<2>(kf[s], get8<3>(&Sp[0][16 * j + r][32 * s + 8 * g4], CB * LDK), kd[j]);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (2 * s + 1 < w) continue;           // P^T is upper triangular
      const Frag<3> pf = split8<3>(y.PT[s]);
#pragma unroll
      for (int j = 0; j < NT; ++j) pd[j] = mma<2>(pf, get8<NA>(&Dp[0][16 * j + r][32 * s + 8 * g4], CB * LDT), pd[j]);
    }
    f32x4 cs = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      kd[j] *= y.del;
#pragma unroll
      for (int e = 0; e < 4; ++e) cs[e] = __builtin_fmaf(kd[j][e], y.N[j][e], cs[e]);
      put4<3>(&Rp[0][16 * j + r][16 * w + 4 * g4], CB * LDT, pd[j] * a.scale + kd[j]);
    }
    __syncthreads();

    // Y, dv
    f32x4 Y[NT], bs = {0, 0, 0, 0}, gs = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < NT; ++j) Y[j] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (2 * s + 1 < w) continue;
      const Frag<3> wf = split8<3>(y.WT[s]);
#pragma unroll
      for (int j = 0; j < NT; ++j) Y[j] = mma<2>(wf, get8<3>(&Rp[0][16 * j + r][32 * s + 8 * g4], CB * LDT), Y[j]);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int dv = dv0 + 16 * j + r;
      const f32x4 dR = Y[j] * y.beta;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = 16 * w + 4 * g4 + e;
        bs[e] = __builtin_fmaf(Y[j][e], y.R[j][e], bs[e]);
        gs[e] = __builtin_fmaf(dR[e], y.R[j][e] - y.v[j][e], gs[e]);
        a.Y[(ch * 64 + t) * a.Dvp + dv] = Y[j][e];
        if (t < y.n && dv < a.Dv) store1<DT>(row_ptr<DT>(a.dv, a.dv_s, y.row, (int64_t)y.t0 + t, h) + dv * ES, dR[e]);
      }
      put4<3>(&Yp[0][16 * j + r][16 * w + 4 * g4], CB * LDT, dR * -y.gam);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float b = sum16(bs[e]), g = sum16(gs[e]), q = sum16(cs[e]);
      if (r == 0) {
        part[64 + 16 * w + 4 * g4 + e] = b;
        part[128 + 16 * w + 4 * g4 + e] = g;
        part[192 + 16 * w + 4 * g4 + e] = q;
      }
    }
    __syncthreads();

    // dS at the chunk's start
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j) S[m][j] *= y.last;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const Frag<NA> kt = get8t<NA>(&Kl[0][32 * s][16 * (MT * w + m)], LDK, 64 * LDK, l);
        const Frag<NA> qt = get8t<NA>(&Ql[0][32 * s][16 * (MT * w + m)], LDK, 64 * LDK, l);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          S[m][j] = mma<2>(qt, get8<3>(&Dd[0][16 * j + r][32 * s + 8 * g4], CB * LDT), S[m][j]);
          S[m][j] = mma<2>(kt, get8<3>(&Yp[0][16 * j + r][32 * s + 8 * g4], CB * LDT), S[m][j]);
        }
      }
    __syncthreads();
  }
  if (a.dh0) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int dk = 16 * (MT * w + m) + 4 * g4 + e, dv = dv0 + 16 * j + r;
          if (dk < a.Dk && dv < a.Dv) a.dh0[seq * a.dh0_s[0] + h * a.dh0_s[1] + dk * a.dh0_s[2] + dv] = S[m][j][e];
        }
  }
}

// ---- dq, dk, dg, dbeta of a chunk ------------------------------------------------------
//
// One workgroup a (chunk, key head): it adds up the key head's value heads in their order, so the
// gradients of shared heads need no atomics.  Eight waves: wave w has the steps of block
// w % 4; waves 0..3 the first half of the keys' columns and F, waves 4..7 the other half
// and E.  Contractions over the values go through LDS 32 values at a time.
template <int DT, int DKP>
__global__ __launch_bounds__(512) void grads_kernel(DeltaArgs a) {
  constexpr int NA = InPlanes<DT>::n, OO = OutOrder<DT>::n, OP = OO + 1, KS = DKP / 32, LDK = DKP + 8, LDV = 40;
  constexpr int ES = DT == CCV_DT_F32 ? 4 : 2, TK = DKP / 32;       // TK: a wave's 16-column tiles of the keys
  constexpr int kStage = (OP * DKP + 3 * 64) * LDV, kPair = 2 * OP * 64 * LDT;
  __shared__ __bf16 Kl[NA][64][LDK], Ql[NA][64][LDK];
  __shared__ __bf16 un[kStage > kPair ? kStage : kPair];
  __shared__ double G[64];
  __shared__ float rows[2][64], cols[8][64], bsum[64], dots[8];
  __bf16* St = un;                                  // [OP][DKP][LDV]
  __bf16* Ns = un + OP * DKP * LDV;                 // [3][64][LDV]
  __bf16* Ft = un;                                  // [OP][64][LDT], by columns j
  __bf16* Et = un + OP * 64 * LDT;
  const int c = blockIdx.x / a.Hk, hk = blockIdx.x - c * a.Hk, group = a.Hv / a.Hk;
  const Chunk k = chunk_at(a, c);
  if (k.n <= 0) return;
  const int tid = threadIdx.x, w8 = __builtin_amdgcn_readfirstlane(tid >> 6), w = w8 & 3, half = w8 >> 2, l = tid & 63, r = l & 15,
            g4 = l >> 4;
  const int t = 16 * w + r;
  const bool live = t < k.n;
  char* dqp = row_ptr<DT>(a.dq, a.dq_s, k.row, (int64_t)k.t0 + (live ? t : 0), hk);
  char* dkp = row_ptr<DT>(a.dk, a.dk_s, k.row, (int64_t)k.t0 + (live ? t : 0), hk);
  f32x4 dq[TK], dk[TK];
#pragma unroll
  for (int n = 0; n < TK; ++n) dq[n] = dk[n] = f32x4{0, 0, 0, 0};

  if (k.seq < a.nseq) {
    const char* kp = row_ptr<DT>(half ? a.k : a.q, half ? a.k_s : a.q_s, k.row, k.t0 + (live ? t : 0), hk);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int d = 32 * s + 8 * g4;
      const Frag<NA> f = planes<DT>(load8<DT>(kp + d * ES, live ? a.Dk - d : 0, a.vec_qk));
#pragma unroll
      for (int p = 0; p < NA; ++p) *reinterpret_cast<bf16x8*>(half ? &Kl[p][t][d] : &Ql[p][t][d]) = f.p[p];
    }
    for (int hg = 0; hg < group; ++hg) {
      const int h = hk * group + hg;
      const int64_t ch = (int64_t)c * a.Hv + h;
      const float* dec = a.dec + ch * kDeltaDec;
      const float* Sg = a.S + ch * DKP * a.Dvp;
      const float* Dg = a.dS + ch * DKP * a.Dvp;
      const float* Ng = a.N + ch * 64 * a.Dvp;
      const float* Yg = a.Y + (ch * 64 + t) * a.Dvp;
      const char* dop = row_ptr<DT>(a.dout, a.do_s, k.row, (int64_t)k.t0 + (live ? t : 0), h);
      if (tid < 64) G[tid] = reinterpret_cast<const double*>(dec + 192)[tid];
      f32x4 zq[TK], zy[TK], zn[TK], pr[4];
      float dot = 0;
#pragma unroll
      for (int n = 0; n < TK; ++n) zq[n] = zy[n] = zn[n] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int n = 0; n < 4; ++n) pr[n] = f32x4{0, 0, 0, 0};

      for (int v0 = 0; v0 < a.Dvp; v0 += 32) {
        // S and N; a thread moves 4 values of DKP / 64 rows
        constexpr int RS = DKP / 64;
        f32x4 s4[RS], d4[RS];
        const int sr = tid >> 3, sc = 4 * (tid & 7);
        const f32x4 n4 = *reinterpret_cast<const f32x4*>(Ng + sr * a.Dvp + v0 + sc);
#pragma unroll
        for (int i = 0; i < RS; ++i) {
          s4[i] = *reinterpret_cast<const f32x4*>(Sg + (64 * i + sr) * (int64_t)a.Dvp + v0 + sc);
          d4[i] = *reinterpret_cast<const f32x4*>(Dg + (64 * i + sr) * (int64_t)a.Dvp + v0 + sc);
#pragma unroll
          for (int e = 0; e < 4; ++e) dot = __builtin_fmaf(s4[i][e], d4[i][e], dot);
        }
        const int dv = v0 + 8 * g4;
        const Frag<NA> of = planes<DT>(load8<DT>(dop + dv * ES, live ? a.Dv - dv : 0, a.vec_do));
        const Frag<3> yf = split8<3>(load_f8(Yg + dv));
        __syncthreads();
        put4<3>(Ns + sr * LDV + sc, 64 * LDV, n4);
#pragma unroll
        for (int i = 0; i < RS; ++i) put4<OP>(St + (64 * i + sr) * LDV + sc, DKP * LDV, s4[i]);
        __syncthreads();
#pragma unroll
        for (int n = 0; n < TK; ++n) {
          const Frag<OP> sf = get8<OP>(St + (16 * (TK * half + n) + r) * LDV + 8 * g4, DKP * LDV);
          zq[n] = mma<OO>(sf, of, zq[n]);
          zy[n] = mma<OO>(sf, yf, zy[n]);
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          if (n > w) continue;
          const Frag<3> nf = get8<3>(Ns + (16 * n + r) * LDV + 8 * g4, 64 * LDV);
          pr[n] = half ? mma<2>(yf, nf, pr[n]) : mma<2>(of, nf, pr[n]);
        }
        const Frag<OP> nown = get8<OP>(Ns + t * LDV + 8 * g4, 64 * LDV);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < RS; ++i) put4<OP>(St + (64 * i + sr) * LDV + sc, DKP * LDV, d4[i]);
        __syncthreads();
#pragma unroll
        for (int n = 0; n < TK; ++n)
          zn[n] = mma<OO>(get8<OP>(St + (16 * (TK * half + n) + r) * LDV + 8 * g4, DKP * LDV), nown, zn[n]);
      }
      {
#pragma unroll
        for (int d = 32; d; d >>= 1) dot += __shfl_xor(dot, d);
        if (l == 0) dots[w8] = dot;
      }
      const float gam = dec[t], del = dec[64 + t], bet = dec[128 + t];
#pragma unroll
      for (int n = 0; n < TK; ++n) {
        dq[n] += zq[n] * (a.scale * gam);
        dk[n] += zn[n] * del - zy[n] * (gam * bet);
      }

      // F (waves 0..3) and E (4..7), their products with Q K^T and K K^T
      __syncthreads();
      f32x4 rs = {0, 0, 0, 0}, bs = {0, 0, 0, 0};
      double Gi[4];
      float bi[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        Gi[e] = G[16 * w + 4 * g4 + e];
        bi[e] = half ? dec[128 + 16 * w + 4 * g4 + e] : a.scale;
      }
      __bf16* Pt = half ? Et : Ft;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int j = 16 * n + r;
        f32x4 f = {0, 0, 0, 0};
        float cs = 0;
        if (n <= w) {
          f32x4 x = {0, 0, 0, 0};
#pragma unroll
          for (int s = 0; s < KS; ++s)
            x = mma<2>(half ? get8<NA>(&Kl[0][t][32 * s + 8 * g4], 64 * LDK) : get8<NA>(&Ql[0][t][32 * s + 8 * g4], 64 * LDK),
                       get8<NA>(&Kl[0][j][32 * s + 8 * g4], 64 * LDK), x);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = 16 * w + 4 * g4 + e;
            if (i < j || (half && i == j)) continue;
            const float d = __builtin_amdgcn_exp2f((float)(Gi[e] - G[j])) * (half ? -pr[n][e] : pr[n][e]);
            f[e] = d * bi[e];
            if (i > j) {
              rs[e] = __builtin_fmaf(f[e], x[e], rs[e]);
              bs[e] = __builtin_fmaf(d, x[e], bs[e]);
              cs = __builtin_fmaf(f[e], x[e], cs);
            }
          }
        }
        put4<OP>(Pt + j * LDT + 16 * w + 4 * g4, 64 * LDT, f);
        cs = sum4rows(cs);
        if (g4 == 0) cols[w8][j] = cs;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float rv = sum16(rs[e]), bv = sum16(bs[e]);
        if (r == 0) {
          rows[half][16 * w + 4 * g4 + e] = rv;
          if (half) bsum[16 * w + 4 * g4 + e] = bv;
        }
      }
      __syncthreads();
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const bool lo = 2 * s <= w, up = 2 * s + 1 >= w;      // rows i >= j; rows j <= i
        Frag<OP> fr, er, fc, ec;
        if (lo) {
          fr = get8t<OP>(Ft + 32 * s * LDT + 16 * w, LDT, 64 * LDT, l);
          er = get8t<OP>(Et + 32 * s * LDT + 16 * w, LDT, 64 * LDT, l);
        }
        if (up) {
          fc = get8<OP>(Ft + t * LDT + 32 * s + 8 * g4, 64 * LDT);
          ec = get8<OP>(Et + t * LDT + 32 * s + 8 * g4, 64 * LDT);
        }
#pragma unroll
        for (int n = 0; n < TK; ++n) {
          const Frag<NA> kt = get8t<NA>(&Kl[0][32 * s][16 * (TK * half + n)], LDK, 64 * LDK, l);
          const Frag<NA> qt = get8t<NA>(&Ql[0][32 * s][16 * (TK * half + n)], LDK, 64 * LDK, l);
          if (lo) {
            dq[n] = mma<OO>(kt, fr, dq[n]);
            dk[n] = mma<OO>(kt, er, dk[n]);
          }
          if (up) {
            dk[n] = mma<OO>(qt, fc, dk[n]);
            dk[n] = mma<OO>(kt, ec, dk[n]);
          }
        }
      }
      if (w8 == 0) {                                          // a step a lane
        float g = rows[0][l] + rows[1][l], b = bsum[l], cj = 0, cc = 0, sd = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          cc += cols[i][l];
          sd += dots[i];
        }
        g -= cc;
        const float* part = a.part + ch * a.slices * kDeltaPart;
        for (int i = 0; i < a.slices; ++i, part += kDeltaPart) {
          g += part[l] + part[128 + l];
          b += part[64 + l];
          cj += part[192 + l];
        }
        if (l >= k.n - 1) cj = 0;
        float tot = cj;
#pragma unroll
        for (int d = 32; d; d >>= 1) tot += __shfl_xor(tot, d);
        g -= cj;
        if (l == 63) g += tot + dec[63] * sd;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
          const float o = __shfl_down(g, d);
          if (l + d < 64) g += o;
        }
        if (l < k.n) {
          const int64_t s = (int64_t)k.t0 + l;
          store_gate(a.dg, a.g_dtype, k.row * a.dg_s[0] + s * a.dg_s[1] + h * a.dg_s[2], g);
          store_gate(a.dbeta, a.b_dtype, k.row * a.db_s[0] + s * a.db_s[1] + h * a.db_s[2], b);
        }
      }
      // the next head's first barrier comes before it writes any of this
      __syncthreads();
    }
  } else if (tid < 64 && tid < k.n) {
    for (int h = hk * group; h < (hk + 1) * group; ++h) {
      const int64_t s = (int64_t)k.t0 + tid;
      store_gate(a.dg, a.g_dtype, k.row * a.dg_s[0] + s * a.dg_s[1] + h * a.dg_s[2], 0.0f);
      store_gate(a.dbeta, a.b_dtype, k.row * a.db_s[0] + s * a.db_s[1] + h * a.db_s[2], 0.0f);
    }
  }
  if (live) {
#pragma unroll
    for (int n = 0; n < TK; ++n) {
      const int d = 16 * (TK * half + n) + 4 * g4;
      store4<DT>(dqp + d * ES, dq[n], a.Dk - d, a.vec_dqk);
      store4<DT>(dkp + d * ES, dk[n], a.Dk - d, a.vec_dqk);
    }
  }
}

template <int DT, int DKP, int NT>
void launch_rev(const DeltaArgs& a, hipStream_t st) {
  const uint32_t heads = (uint32_t)(a.nseq + (a.packed ? 1 : 0)) * a.Hv, pad = (heads + 7) / 8 * 8;
  const dim3 grid(pad * ((a.Dvp + 16 * NT - 1) / (16 * NT)));
  reverse_kernel<DT, DKP, NT><<<grid, 256, 0, st>>>(a, heads, pad);
}
template <int DT>
void launch_rev(const DeltaArgs& a, int nt, hipStream_t st) {
  if constexpr (DT == CCV_DT_F32) {
    if (a.Dkp == 64) launch_rev<DT, 64, 1>(a, st);
    else launch_rev<DT, 128, 1>(a, st);
  } else if (a.Dkp == 64) {
    if (nt == 1) launch_rev<DT, 64, 1>(a, st);
    else launch_rev<DT, 64, 2>(a, st);
  } else {
    if (nt == 1) launch_rev<DT, 128, 1>(a, st);
    else launch_rev<DT, 128, 2>(a, st);
  }
}
template <int DT>
void launch_grads(const DeltaArgs& a, hipStream_t st) {
  const dim3 grid((uint32_t)((int64_t)a.nchunks * a.Hk));
  if (a.Dkp == 64) grads_kernel<DT, 64><<<grid, 512, 0, st>>>(a);
  else grads_kernel<DT, 128><<<grid, 512, 0, st>>>(a);
}

}  // namespace

int launch_delta_reverse(const DeltaArgs& a, int nt, void* stream) {
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (a.x_dtype == CCV_DT_F32) launch_rev<CCV_DT_F32>(a, nt, st);
  else if (a.x_dtype == CCV_DT_F16) launch_rev<CCV_DT_F16>(a, nt, st);
  else launch_rev<CCV_DT_BF16>(a, nt, st);
  return (int)hipGetLastError();
}

int launch_delta_grads(const DeltaArgs& a, void* stream) {
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (a.x_dtype == CCV_DT_F32) launch_grads<CCV_DT_F32>(a, st);
  else if (a.x_dtype == CCV_DT_F16) launch_grads<CCV_DT_F16>(a, st);
  else launch_grads<CCV_DT_BF16>(a, st);
  return (int)hipGetLastError();
}

}  // namespace ccv
