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
  const Sequence sq = sequence_at(a, seq);
  const int c0 = sq.first, c1 = sq.end;

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

  // loaded a chunk ahead, each part when the one before it has been used
  const int i = 16 * w + r;
  Chunk k;
  Raw8<DT> xk[KS], xq[KS];
  Frag<3> xW[2], xP[2];
  typename Stored<DT>::type xd[NT][4], xv[NT][4];
  float xR[NT][4], xN[NT][4];
  struct Gates {
    f32x4 gam, del, beta;
    float last;
  } gt, gn;
  uint32_t ok[KS], oq[KS], ov[NT][4], odo[NT][4];      // byte offsets of this lane's parts
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    const int d = 32 * s + 8 * g4;
    ok[s] = d < a.Dk ? i * (uint32_t)(a.k_s[1] * ES) + d * ES : kNowhere;
    oq[s] = d < a.Dk ? i * (uint32_t)(a.q_s[1] * ES) + d * ES : kNowhere;
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int dv = dv0 + 16 * j + r, t = 16 * w + 4 * g4 + e;
      ov[j][e] = dv < a.Dv ? t * (uint32_t)(a.v_s[1] * ES) + dv * ES : kNowhere;
      odo[j][e] = dv < a.Dv ? t * (uint32_t)(a.do_s[1] * ES) + dv * ES : kNowhere;
    }
  const uint32_t om = (2 * w * 64 + l) * 16, od = (16 * w + 4 * g4) * 4,
                 orow = ((16 * w + 4 * g4) * (uint32_t)a.Dvp + dv0 + r) * 4;
  auto load_kq = [&](const Chunk& n) {
    const __amdgpu_buffer_rsrc_t kb = chunk_rows<DT>(a.k, a.k_s, n, hk, (a.Dk + 7) & ~7);
    const __amdgpu_buffer_rsrc_t qb = chunk_rows<DT>(a.q, a.q_s, n, hk, (a.Dk + 7) & ~7);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      xk[s] = buf8<DT>(kb, ok[s]);
      xq[s] = buf8<DT>(qb, oq[s]);
    }
  };
  auto load_v = [&](const Chunk& n) {
    const __amdgpu_buffer_rsrc_t b = chunk_rows<DT>(a.v, a.v_s, n, h, a.Dv);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) xv[j][e] = buf_raw<DT>(b, ov[j][e]);
  };
  auto load_d = [&](const Chunk& n) {
    const __amdgpu_buffer_rsrc_t b = chunk_rows<DT>(a.dout, a.do_s, n, h, a.Dv);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) xd[j][e] = buf_raw<DT>(b, odo[j][e]);
  };
  auto load_rows = [&](float (&x)[NT][4], const float* base, int64_t ch) {
    const __amdgpu_buffer_rsrc_t b = buffer(base + ch * 64 * a.Dvp, 256u * a.Dvp);
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int j = 0; j < NT; ++j) x[j][e] = buf1<CCV_DT_F32>(b, orow + e * 4 * a.Dvp + 64 * j);
  };
  auto load_matrix = [&](Frag<3> (&x)[2], const uint16_t* base, int64_t ch) {
    const __amdgpu_buffer_rsrc_t b = buffer(base + ch * kDeltaMatrix, 2 * kDeltaMatrix);
#pragma unroll
    for (int s = 0; s < 2; ++s) x[s] = buf_planes<3>(b, om + 1024 * s, 8192);
  };
  auto load_dec = [&](int64_t ch) {
    const __amdgpu_buffer_rsrc_t b = buffer(a.dec + ch * kDeltaDec, 4 * kDeltaDec);
    Gates g;
    g.gam = buf_f4(b, od);
    g.del = buf_f4(b, od + 256);
    g.beta = buf_f4(b, od + 512);
    g.last = buf1<CCV_DT_F32>(b, 4 * 63);
    return g;
  };

  if (c0 < c1) {
    const int64_t ch = (int64_t)(c1 - 1) * a.Hv + h;
    k = sq.chunk(seq, c1 - 1);
    load_kq(k);
    load_d(k);
    gn = load_dec(ch);
    load_matrix(xP, a.P, ch);
    load_rows(xN, a.N, ch);
    load_matrix(xW, a.WT, ch);
    load_v(k);
    load_rows(xR, a.R, ch);
  }
  for (int c = c1 - 1; c >= c0; --c) {
    const int64_t ch = (int64_t)c * a.Hv + h;
    const int cn = c > c0 ? c - 1 : c;
    const int64_t chn = (int64_t)cn * a.Hv + h;
    const Chunk kn = sq.chunk(seq, cn);
    gt = gn;
    float* part = a.part + (ch * a.slices + slice) * kDeltaPart;

    // the planes of this chunk
    Frag<NA> kf[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      kf[s] = planes<DT>(xk[s]);
      const Frag<NA> qf = planes<DT>(xq[s]);
#pragma unroll
      for (int p = 0; p < NA; ++p) {
        *reinterpret_cast<bf16x8*>(&Kl[p][16 * w + r][32 * s + 8 * g4]) = kf[s].p[p];
        *reinterpret_cast<bf16x8*>(&Ql[p][16 * w + r][32 * s + 8 * g4]) = qf.p[p];
      }
    }
    load_kq(kn);
    gn = load_dec(chn);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const f32x4 d = {widen<DT>(xd[j][0]), widen<DT>(xd[j][1]), widen<DT>(xd[j][2]), widen<DT>(xd[j][3])};
      put4<NA>(&Dp[0][16 * j + r][16 * w + 4 * g4], CB * LDT, d);
      put4<3>(&Dd[0][16 * j + r][16 * w + 4 * g4], CB * LDT, d * gt.gam * a.scale);
    }
    load_d(kn);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        put4<3>(&Sp[0][16 * j + r][16 * (MT * w + m) + 4 * g4], CB * LDK, S[m][j]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          a.dS[(ch * DKP + 16 * (MT * w + m) + 4 * g4 + e) * a.Dvp + dv0 + 16 * j + r] = S[m][j][e];
      }
    lds_barrier();

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
#pragma unroll
      for (int j = 0; j < NT; ++j) pd[j] = mma<2>(xP[s], get8<NA>(&Dp[0][16 * j + r][32 * s + 8 * g4], CB * LDT), pd[j]);
    }
    f32x4 cs = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      kd[j] *= gt.del;
#pragma unroll
      for (int e = 0; e < 4; ++e) cs[e] = __builtin_fmaf(kd[j][e], xN[j][e], cs[e]);
      put4<3>(&Rp[0][16 * j + r][16 * w + 4 * g4], CB * LDT, pd[j] * a.scale + kd[j]);
    }
    load_matrix(xP, a.P, chn);
    load_rows(xN, a.N, chn);
    lds_barrier();

    // Y, dv
    f32x4 Y[NT], bs = {0, 0, 0, 0}, gs = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < NT; ++j) Y[j] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (2 * s + 1 < w) continue;
#pragma unroll
      for (int j = 0; j < NT; ++j) Y[j] = mma<2>(xW[s], get8<3>(&Rp[0][16 * j + r][32 * s + 8 * g4], CB * LDT), Y[j]);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int dv = dv0 + 16 * j + r;
      const f32x4 dR = Y[j] * gt.beta;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = 16 * w + 4 * g4 + e;
        bs[e] = __builtin_fmaf(Y[j][e], xR[j][e], bs[e]);
        gs[e] = __builtin_fmaf(dR[e], xR[j][e] - widen<DT>(xv[j][e]), gs[e]);
        a.Y[(ch * 64 + t) * a.Dvp + dv] = Y[j][e];
        if (t < k.n && dv < a.Dv) store1<DT>(row_ptr<DT>(a.dv, a.dv_s, k.row, (int64_t)k.t0 + t, h) + dv * ES, dR[e]);
      }
      put4<3>(&Yp[0][16 * j + r][16 * w + 4 * g4], CB * LDT, dR * -gt.gam);
    }
    load_matrix(xW, a.WT, chn);
    load_v(kn);
    load_rows(xR, a.R, chn);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float b = sum16(bs[e]), g = sum16(gs[e]), q = sum16(cs[e]);
      if (r == 0) {
        part[64 + 16 * w + 4 * g4 + e] = b;
        part[128 + 16 * w + 4 * g4 + e] = g;
        part[192 + 16 * w + 4 * g4 + e] = q;
      }
    }
    lds_barrier();

    // dS at the chunk's start
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j) S[m][j] *= gt.last;
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
    k = kn;
    lds_barrier();
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
    const __amdgpu_buffer_rsrc_t kb = half ? chunk_rows<DT>(a.k, a.k_s, k, hk, (a.Dk + 7) & ~7)
                                           : chunk_rows<DT>(a.q, a.q_s, k, hk, (a.Dk + 7) & ~7);
    const uint32_t ks = t * (uint32_t)((half ? a.k_s[1] : a.q_s[1]) * ES);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int d = 32 * s + 8 * g4;
      const Frag<NA> f = planes<DT>(buf8<DT>(kb, d < a.Dk ? ks + d * ES : kNowhere));
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
      const __amdgpu_buffer_rsrc_t Yb = buffer(a.Y + ch * 64 * a.Dvp, 256u * a.Dvp);
      const __amdgpu_buffer_rsrc_t dob = chunk_rows<DT>(a.dout, a.do_s, k, h, (a.Dv + 7) & ~7);
      const uint32_t dos = t * (uint32_t)(a.do_s[1] * ES);
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
        const Frag<NA> of = planes<DT>(buf8<DT>(dob, dv < a.Dv ? dos + dv * ES : kNowhere));
        const uint32_t oy = (t * (uint32_t)a.Dvp + dv) * 4;
        const Frag<3> yf = split8<3>(__builtin_shufflevector(buf_f4(Yb, oy), buf_f4(Yb, oy + 16), 0, 1, 2, 3, 4, 5, 6, 7));
        lds_barrier();
        put4<3>(Ns + sr * LDV + sc, 64 * LDV, n4);
#pragma unroll
        for (int i = 0; i < RS; ++i) put4<OP>(St + (64 * i + sr) * LDV + sc, DKP * LDV, s4[i]);
        lds_barrier();
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
        lds_barrier();
#pragma unroll
        for (int i = 0; i < RS; ++i) put4<OP>(St + (64 * i + sr) * LDV + sc, DKP * LDV, d4[i]);
        lds_barrier();
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
      lds_barrier();
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
      lds_barrier();
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
      lds_barrier();
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
