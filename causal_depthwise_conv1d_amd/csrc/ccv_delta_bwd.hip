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
//   dbeta_i = Y_i . R_i + sum_j e^(Gi - Gj) k_i.k_j dA_ij = Y_i . N_i / beta_i,
// the last since N + A N = beta R.  The gradient of G_i, with c_j = del_j (K dS')_j . N_j and
// sums over j below or above the diagonal:
//   dG_i = scale gam_i dO_i.(Q S)_i + sum_j F_ij q_i.k_j - sum_j F_ji q_j.k_i
//          + (Y_i . N_i - dv_i . v_i) - sum_j E_ji k_j.k_i - c_i,
//   dG_63 += sum_j c_j + gam63 <S, dS'>,          dg_t = sum of dG_i over i >= t;
// the term in brackets is all that k_i's own row of A and of R gives, by the same identity.
// The first step of a sequence without an initial state decays nothing: its dg is 0.
#include "ccv_delta_device.hpp"

namespace ccv {
namespace {

constexpr int LDT = 72;

// Waves 0..3 hold dS, as the forward's hold S; waves 4..7 stay a chunk ahead of them with what
// needs no dS (scale P^T dO, and Q^T (scale gam dO), which dS only has added), and a phase
// behind them with what nothing waits for (the sums of Y.N, dv.v and c over this slice's
// values, dv and Y to memory).  Both sides of such an exchange hold the same elements lane
// by lane, so it takes one 16-byte LDS access a tile and needs no other order than the
// three barriers.  Bound by the chain, as the forward: 2 x 4096 steps, 16 heads of 128 in bf16, 210 us, 3.3 us a
// chunk.
// MAP: what a part of a sequence makes of a gradient of zero at its end; no more than the chain.
template <int DT, int DKP, int NT, bool MAP>
__global__ __launch_bounds__(512, 2) void reverse_kernel(DeltaArgs a, uint32_t heads, uint32_t slices) {
  constexpr int NA = InPlanes<DT>::n, CB = 16 * NT, KS = DKP / 32, MT = DKP / 64, LDK = DKP + 8;
  constexpr int ES = DT == CCV_DT_F32 ? 4 : 2;
  __shared__ __bf16 Sp[3][CB][LDK];        // dS by columns
  __shared__ __bf16 Rp[3][CB][LDT];        // dN
  __shared__ __bf16 Yp[3][CB][LDT];        // -gam beta Y
  __shared__ __bf16 Dp[NA][CB][LDT];       // dO of the next chunk
  __shared__ __bf16 Dd[3][CB][LDT];        // scale gam dO of the next chunk
  __shared__ __bf16 Kl[NA][64][LDK], Ql[NA][64][LDK];
  __shared__ f32x4 Pd[NT][4][64];          // scale P^T dO; then del (K dS'), from the lane that read it
  __shared__ f32x4 Ud[MT][NT][4][64];      // Q^T (scale gam dO); then Y in its first tile, likewise
  uint32_t hs, slice;
  if (!place(a.share, heads, slices, &hs, &slice)) return;
  const int sh = hs / a.Hv, h = hs - sh * a.Hv, hk = h / (a.Hv / a.Hk), dv0 = slice * CB;
  const Part part = part_at(a, sh);
  const int seq = part.seq;
  const int tid = threadIdx.x, w8 = __builtin_amdgcn_readfirstlane(tid >> 6), w = w8 & 3, l = tid & 63, r = l & 15, g4 = l >> 4;

  if (seq >= a.nseq) {                     // steps of no sequence have no gradient
    if (MAP || seq > a.nseq) return;
    const int32_t* begin = a.cstart + (a.nseq + 2);
    for (int64_t i = (int64_t)begin[a.nseq] * CB + tid; i < a.L * CB; i += 512) {
      const int64_t t = i / CB;
      const int d = dv0 + (int)(i - t * CB);
      if (d < a.Dv) store1<DT>(row_ptr<DT>(a.dv, a.dv_s, 0, t, h) + d * ES, 0.0f);
    }
    return;
  }
  if (MAP && part.k == 0) return;          // nothing lies before it
  const Sequence sq = part.sq;
  const int c0 = sq.first, c1 = sq.end;
  const int64_t chl = (int64_t)(c1 - 1) * a.Hv + h;
  const uint32_t om = (2 * w * 64 + l) * 16, od = (16 * w + 4 * g4) * 4;
  const uint32_t on = ((slice * NT * 4 + w) * 64 + l) * 16;
  const auto steps_of = [&](int c) {       // 0 before the first chunk
    if (c < c0) return 0;
    const int64_t left = sq.len - (int64_t)(c - c0) * kDeltaChunk;
    return left < kDeltaChunk ? (int)left : kDeltaChunk;
  };

  if (w8 < 4) {
    // ---- dS: rows 16 (MT w + m) + 4 g4 + e, column 16 j + r ------------------------------
    f32x4 S[MT][NT];
    const f32x4* start = MAP ? nullptr : start_tiles(a, part, h, 1);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
        if (start) {
          S[m][j] = start[((slice * NT + j) * (DKP / 16) + MT * w + m) * 64 + l];
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int dk = 16 * (MT * w + m) + 4 * g4 + e, dv = dv0 + 16 * j + r;
            S[m][j][e] = !MAP && a.dht && dk < a.Dk && dv < a.Dv ? a.dht[seq * a.dht_s[0] + h * a.dht_s[1] + dk * a.dht_s[2] + dv] : 0.0f;
          }
        }
    const auto put_state = [&]() {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j) put4<3>(&Sp[0][16 * j + r][16 * (MT * w + m) + 4 * g4], CB * LDK, S[m][j]);
    };
    Frag<3> xW[2];
    struct Gates {
      f32x4 gam, del, beta;
      float last;
    } gt, gn;
    Rows<DT> K(a.k, a.k_s, sq, hk, (a.Dk + 7) & ~7, c1 - 1);
    Piece<uint16_t> W(a.WT, kDeltaMatrix, a.Hv, chl);
    Piece<float> D(a.dec, kDeltaDec, a.Hv, chl), So(a.dS, (int64_t)DKP * a.Dvp, a.Hv, chl);
    const uint32_t os = ((slice * NT * (DKP / 16) + MT * w) * 64 + l) * 16;
    RowTile<DT, DKP, LDK> kt(w, l, K.stride, a.Dk);
    const auto load_K = [&](int n) {
      kt.load(K.rows(n));
      K.at -= K.step;
    };
    const auto load_gates = [&](int n) {
      const __amdgpu_buffer_rsrc_t d = D.piece(n > 0);
      gn.gam = buf_f4(d, od);
      gn.del = buf_f4(d, od + 256);
      gn.beta = buf_f4(d, od + kDeltaBeta * 4);
      gn.last = buf1<CCV_DT_F32>(d, 4 * 63);
      D.at -= D.step;
    };
    const auto load_W = [&](int n) {
      const __amdgpu_buffer_rsrc_t b = W.piece(n > 0);
#pragma unroll
      for (int s = 0; s < 2; ++s) xW[s] = buf_planes<3>(b, !s && w >= 2 ? kNowhere : om + 1024 * s, 8192);
      W.at -= W.step;
    };
    if (c0 < c1) {
      load_K(steps_of(c1 - 1));
      load_gates(steps_of(c1 - 1));
      load_W(steps_of(c1 - 1));
    }
    put_state();
    lds_barrier();
    lds_barrier();
    for (int c = c1 - 1; c >= c0; --c) {
      const int nn = steps_of(c - 1);
      gt = gn;
      kt.store(&Kl[0][0][0], 64 * LDK);
      load_K(nn);
      // dN = scale P^T dO + del (K dS')
      Sums kd[NT];
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const Frag<NA> kf = get8<NA>(&Kl[0][16 * w + r][32 * s + 8 * g4], 64 * LDK);
#pragma unroll
        for (int j = 0; j < NT; ++j) kd[j].add(kf, get8<3>(&Sp[0][16 * j + r][32 * s + 8 * g4], CB * LDK));
      }
      load_gates(nn);
      {
        const __amdgpu_buffer_rsrc_t sb = So.piece(true);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            if constexpr (!MAP) buf_store_f4(sb, os + (j * (DKP / 16) + m) * 1024, S[m][j]);
            S[m][j] = S[m][j] * gt.last + Ud[m][j][w][l];
          }
        So.at -= So.step;
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const f32x4 x = kd[j].total() * gt.del;
        put4<3>(&Rp[0][16 * j + r][16 * w + 4 * g4], CB * LDT, Pd[j][w][l] + x);
        if constexpr (!MAP) Pd[j][w][l] = x;
      }
      lds_barrier();

      // Y = W^T dN; W^T is upper triangular
      Sums ys[NT];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (2 * s + 1 < w) continue;
#pragma unroll
        for (int j = 0; j < NT; ++j) ys[j].add(xW[s], get8<3>(&Rp[0][16 * j + r][32 * s + 8 * g4], CB * LDT));
      }
      load_W(nn);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const f32x4 y = ys[j].total();
        put4<3>(&Yp[0][16 * j + r][16 * w + 4 * g4], CB * LDT, y * gt.beta * -gt.gam);
        if constexpr (!MAP) Ud[0][j][w][l] = y;
      }
      lds_barrier();

      // dS at the chunk's start
      Sums sn[MT][NT];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Frag<3> yf[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) yf[j] = get8<3>(&Yp[0][16 * j + r][32 * s + 8 * g4], CB * LDT);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const Frag<NA> kf = get8t<NA>(&Kl[0][32 * s][16 * (MT * w + m)], LDK, 64 * LDK, l);
#pragma unroll
          for (int j = 0; j < NT; ++j) sn[m][j].add(kf, yf[j]);
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j) S[m][j] += sn[m][j].total();
      put_state();
      lds_barrier();
    }
    if constexpr (MAP) {
      f32x4* to = reinterpret_cast<f32x4*>(part_map(a, sh, h) + DKP * DKP);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j) to[((slice * NT + j) * (DKP / 16) + MT * w + m) * 64 + l] = S[m][j];
    } else if (a.dh0 && part.k == 0) {
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
  } else {
    // ---- ahead and behind: steps 16 w + 4 g4 + e, column 16 j + r ---------------------------
    typename Stored<DT>::type xd[NT][4], xv[NT][4];
    f32x4 xN[NT];
    Frag<3> xP[2];
    f32x4 gam, beta;
    Rows<DT> Q(a.q, a.q_s, sq, hk, (a.Dk + 7) & ~7, c1 - 1), O(a.dout, a.do_s, sq, h, a.Dv, c1 - 1), V(a.v, a.v_s, sq, h, a.Dv, c1 - 1),
        dV(a.dv, a.dv_s, sq, h, a.Dv, c1 - 1);
    Piece<uint16_t> P(a.P, kDeltaMatrix, a.Hv, chl);
    Piece<float> Dg(a.dec, kDeltaDec, a.Hv, chl), Db(a.dec, kDeltaDec, a.Hv, chl);
    Piece<float> Ni(a.N, 64 * (int64_t)a.Dvp, a.Hv, chl), Yo(a.Y, 64 * (int64_t)a.Dvp, a.Hv, chl);
    const float scale = a.scale;
    RowTile<DT, DKP, LDK> qt(w, l, Q.stride, a.Dk);
    uint32_t ov[NT], oo[NT], odv[NT];      // of the lane's first step; the others follow a stride apart
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int dv = dv0 + 16 * j + r, t = 16 * w + 4 * g4;
      ov[j] = dv < a.Dv ? t * V.stride + dv * ES : kNowhere;
      oo[j] = dv < a.Dv ? t * O.stride + dv * ES : kNowhere;
      odv[j] = dv < a.Dv ? t * dV.stride + dv * ES : kNowhere;
    }
    const auto load_QD = [&](int n) {
      qt.load(Q.rows(n));
      Q.at -= Q.step;
      const __amdgpu_buffer_rsrc_t b = O.rows(n);
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) xd[j][e] = buf_raw<DT>(b, oo[j] == kNowhere ? kNowhere : oo[j] + e * O.stride);
      O.at -= O.step;
      gam = buf_f4(Dg.piece(n > 0), od);
      Dg.at -= Dg.step;
    };
    const auto load_P = [&](int n) {
      const __amdgpu_buffer_rsrc_t b = P.piece(n > 0);
#pragma unroll
      for (int s = 0; s < 2; ++s) xP[s] = buf_planes<3>(b, !s && w >= 2 ? kNowhere : om + 1024 * s, 8192);
      P.at -= P.step;
    };
    const auto load_NV = [&](int n) {
      const __amdgpu_buffer_rsrc_t nb = Ni.piece(n > 0), vb = V.rows(n);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        xN[j] = buf_f4(nb, on + j * 4096);
#pragma unroll
        for (int e = 0; e < 4; ++e) xv[j][e] = buf_raw<DT>(vb, ov[j] == kNowhere ? kNowhere : ov[j] + e * V.stride);
      }
      beta = buf_f4(Db.piece(n > 0), od + kDeltaBeta * 4);
      Ni.at -= Ni.step;
      V.at -= V.step;
      Db.at -= Db.step;
    };
    const auto stage = [&]() {
      qt.store(&Ql[0][0][0], 64 * LDK);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const f32x4 d = {widen<DT>(xd[j][0]), widen<DT>(xd[j][1]), widen<DT>(xd[j][2]), widen<DT>(xd[j][3])};
        put4<NA>(&Dp[0][16 * j + r][16 * w + 4 * g4], CB * LDT, d);
        put4<3>(&Dd[0][16 * j + r][16 * w + 4 * g4], CB * LDT, d * gam * scale);
      }
    };
    f32x4 pd[NT], ud[MT][NT];
    const auto products = [&]() {
      Sums ps[NT], us[MT][NT];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (2 * s + 1 < w) continue;           // P^T is upper triangular
#pragma unroll
        for (int j = 0; j < NT; ++j) ps[j].add(xP[s], get8<NA>(&Dp[0][16 * j + r][32 * s + 8 * g4], CB * LDT));
      }
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const Frag<NA> qf = get8t<NA>(&Ql[0][32 * s][16 * (MT * w + m)], LDK, 64 * LDK, l);
#pragma unroll
          for (int j = 0; j < NT; ++j) us[m][j].add(qf, get8<3>(&Dd[0][16 * j + r][32 * s + 8 * g4], CB * LDT));
        }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        pd[j] = ps[j].total() * scale;
#pragma unroll
        for (int m = 0; m < MT; ++m) ud[m][j] = us[m][j].total();
      }
    };
    const auto hand_over = [&]() {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        Pd[j][w][l] = pd[j];
#pragma unroll
        for (int m = 0; m < MT; ++m) Ud[m][j][w][l] = ud[m][j];
      }
    };
    if (c0 < c1) {
      load_QD(steps_of(c1 - 1));
      load_P(steps_of(c1 - 1));
      if constexpr (!MAP) load_NV(steps_of(c1 - 1));
      stage();
      load_QD(steps_of(c1 - 2));
    }
    lds_barrier();
    if (c0 < c1) {
      products();
      load_P(steps_of(c1 - 2));
      hand_over();
    }
    lds_barrier();
    for (int c = c1 - 1; c >= c0; --c) {
      const int n = steps_of(c);
      stage();                                 // of chunk c - 1; zeros before the first
      load_QD(steps_of(c - 2));
      lds_barrier();
      products();
      load_P(steps_of(c - 2));
      if constexpr (MAP) {
        lds_barrier();
        hand_over();
        lds_barrier();
        continue;
      }
      f32x4 cs = {0, 0, 0, 0}, bs = {0, 0, 0, 0}, gs = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const f32x4 x = Pd[j][w][l];
#pragma unroll
        for (int e = 0; e < 4; ++e) cs[e] = __builtin_fmaf(x[e], xN[j][e], cs[e]);
      }
      lds_barrier();
      const __amdgpu_buffer_rsrc_t yb = Yo.piece(true), vb = dV.rows(n);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const f32x4 y = Ud[0][j][w][l], dR = y * beta;
        buf_store_f4(yb, on + j * 4096, y);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          bs[e] = __builtin_fmaf(y[e], xN[j][e], bs[e]);
          gs[e] = __builtin_fmaf(dR[e], widen<DT>(xv[j][e]), gs[e]);
          buf_store1<DT>(vb, odv[j] == kNowhere ? kNowhere : odv[j] + e * dV.stride, dR[e]);
        }
      }
      Yo.at -= Yo.step;
      dV.at -= dV.step;
      load_NV(steps_of(c - 1));
      hand_over();
      float* part = a.part + (((int64_t)c * a.Hv + h) * a.slices + slice) * kDeltaPart + 16 * w + 4 * g4;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float b = sum16(bs[e]), g = sum16(gs[e]), q = sum16(cs[e]);
        if (r == 0) {
          part[e] = b;
          part[64 + e] = b - g;
          part[128 + e] = q;
        }
      }
      lds_barrier();
    }
  }
}

// The same for fp16 and many heads, as the forward's wave_kernel has it: 16 columns a wave, the chain
//   K dS', P^T dO -> dN,  W^T dN = Y,  Q^T (scale gam dO) and K^T (gam beta Y) -> dS
// in its registers, K and Q shared through LDS; both have their rows in the joined order.  1 x 2048 steps of 256
// heads of 128 in fp16: 592 us against 904 of reverse_kernel, 104 heads 413 against 441, 96 heads, three rounds of
// reverse_kernel's workgroups, 411 against 356.  In bf16 reverse_kernel has LDS for 32 columns a workgroup and needs
// no more (554 and 278 us).
template <int DT, int DKP>
__global__ __launch_bounds__(64 * kColumnWaves, 2) void reverse_wave_kernel(DeltaArgs a, uint32_t heads, uint32_t slices) {
  constexpr int NW = kColumnWaves, NA = InPlanes<DT>::n, KS = DKP / 32, LDK = DKP + 8, CB = 16 * NW, PS = Cut<DT>::n;
  __shared__ uint16_t Kl[2][64][LDK], Ql[2][64][LDK];
  __shared__ float Gl[2][3][64];           // gam, del, beta
  uint32_t hs, slice;
  if (!place(a.share, heads, slices, &hs, &slice)) return;
  const int sh = hs / a.Hv, h = hs - sh * a.Hv, seq = in_order(a, sh), hk = h / (a.Hv / a.Hk);
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, r = l & 15, g4 = l >> 4;
  if (seq >= a.nseq) {                     // steps of no sequence have no gradient
    const int32_t* begin = a.cstart + (a.nseq + 2);
    for (int64_t i = (int64_t)begin[a.nseq] * CB + tid; i < a.L * CB; i += 64 * NW) {
      const int64_t t = i / CB;
      const int d = (int)slice * CB + (int)(i - t * CB);
      if (d < a.Dv) store1<DT>(row_ptr<DT>(a.dv, a.dv_s, 0, t, h) + d * 2, 0.0f);
    }
    return;
  }
  const int ct = slice * NW + w, dv = 16 * ct + r;
  const Sequence sq = sequence_at(a, seq);
  const int c0 = sq.first, c1 = sq.end;
  const int64_t chl = (int64_t)(c1 - 1) * a.Hv + h;

  f32x4 S[2 * KS];                         // dS': tile 2 s + o: keys 32 s + 8 g4 + 4 o + e
#pragma unroll
  for (int m = 0; m < 2 * KS; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int dk = 16 * (m & ~1) + 8 * g4 + 4 * (m & 1) + e;
      S[m][e] = a.dht && dk < a.Dk && dv < a.Dv ? a.dht[seq * a.dht_s[0] + h * a.dht_s[1] + dk * a.dht_s[2] + dv] : 0.0f;
    }
  Rows<DT> K(a.k, a.k_s, sq, hk, (a.Dk + 7) & ~7, c1 - 1), Q(a.q, a.q_s, sq, hk, (a.Dk + 7) & ~7, c1 - 1), V(a.v, a.v_s, sq, h, a.Dv, c1 - 1),
      O(a.dout, a.do_s, sq, h, a.Dv, c1 - 1), dV(a.dv, a.dv_s, sq, h, a.Dv, c1 - 1);
  Piece<uint16_t> W(a.WT, kDeltaMatrix, a.Hv, chl), P(a.P, kDeltaMatrix, a.Hv, chl);
  Piece<float> D(a.dec, kDeltaDec, a.Hv, chl), So(a.dS, (int64_t)DKP * a.Dvp, a.Hv, chl);
  Piece<float> Ni(a.N, 64 * (int64_t)a.Dvp, a.Hv, chl), Yo(a.Y, 64 * (int64_t)a.Dvp, a.Hv, chl),
      Po(a.part, (int64_t)a.slices * kDeltaPart, a.Hv, chl);
  const float scale = a.scale;
  const bool in = dv < a.Dv;
  const uint32_t ov = in ? 8 * g4 * V.stride + dv * 2 : kNowhere, vnext = V.stride;
  const uint32_t oo = in ? 8 * g4 * O.stride + dv * 2 : kNowhere, onext = O.stride;
  const uint32_t odv = in ? 8 * g4 * dV.stride + dv * 2 : kNowhere, dnext = dV.stride;
  // tiles as the workspace has them: row 32 s + 8 g4 + 4 o + e is element e of lane group 2 (g4 % 2) + o of tile 2 s + g4 / 2
  const uint32_t to = ((g4 >> 1) * 64 + 2 * (g4 & 1) * 16 + r) * 16;
  const uint32_t os = ct * (DKP / 16) * 1024 + to, on = ct * 4096 + to;
  const uint32_t op = r == 0 ? (ct * kDeltaPart + 8 * g4) * 4 : kNowhere;      // past the slices: out of bounds too

  RowCopy<DKP, LDK, NW, true> kt(w, l, K.stride, a.Dk), qt(w, l, Q.stride, a.Dk);
  float gates;
  uint16_t xd[4][4];
  const auto steps_of = [&](int c) {       // 0 before the first chunk
    if (c < c0) return 0;
    const int64_t left = sq.len - (int64_t)(c - c0) * kDeltaChunk;
    return left < kDeltaChunk ? (int)left : kDeltaChunk;
  };
  const auto load_rows = [&](int n) {
    kt.load(K.rows(n));
    qt.load(Q.rows(n));
    gates = buf1<CCV_DT_F32>(D.piece(n > 0), tid < 128 ? tid * 4 : tid < 192 ? (kDeltaBeta - 128 + tid) * 4 : kNowhere);
    K.at -= K.step;
    Q.at -= Q.step;
    D.at -= D.step;
  };
  const auto store_rows = [&](int b) {
    kt.store(&Kl[b][0][0]);
    qt.store(&Ql[b][0][0]);
    if (tid < 192) Gl[b][0][tid] = gates;
  };
  const auto load_dO = [&](int n) {
    const __amdgpu_buffer_rsrc_t b = O.rows(n);
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      uint32_t o = anew(oo) + (32 * (it >> 1) + 4 * (it & 1)) * onext;
#pragma unroll
      for (int e = 0; e < 4; ++e, o += onext) xd[it][e] = buf_raw<DT>(b, o);
    }
    O.at -= O.step;
  };
  // an upper triangular matrix in joined rows: row tiles 0 1 by steps 0 .., 0 1 2 3 by steps 32 ..
  const auto load_upper = [&](Frag<3> (&x)[6], Piece<uint16_t>& m) {
    const __amdgpu_buffer_rsrc_t b = m.piece(true);
#pragma unroll
    for (int i = 0; i < 6; ++i) x[i] = buf_planes<3>(b, ((i < 2 ? 2 * i : 2 * i - 3) * 64 + l) * 16, 8192);
    m.at -= m.step;
  };
  if (c0 < c1) {
    load_rows(steps_of(c1 - 1));
    store_rows(0);
    load_rows(steps_of(c1 - 2));           // in the loop's order: the waits of both have to agree
    load_dO(steps_of(c1 - 1));
  }
  for (int c = c1 - 1; c >= c0; --c) {
    const int b = (c1 - 1 - c) & 1, n = steps_of(c);
    const uint16_t *Kb = &Kl[b][0][0], *Qb = &Ql[b][0][0];
    const auto gate = [&](int which, int it) {
      return *reinterpret_cast<const f32x4*>(&Gl[b][which][32 * (it >> 1) + 4 * (it & 1) + 8 * g4]);
    };
    lds_barrier();
    // K dS'
    f32x4 hi[4] = {}, lo[4] = {}, dN[4];
    const int es = column_exponent<DT>(S);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const Cut<DT> x = cut<DT>(join(S[2 * s], S[2 * s + 1]), es);
      u32x4 kf[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) kf[t] = *reinterpret_cast<const u32x4*>(Kb + (16 * t + r) * LDK + 32 * s + 8 * g4);
#pragma unroll
      for (int p = PS - 1; p > 0; --p)
#pragma unroll
        for (int t = 0; t < 4; ++t) lo[t] = mfma16<DT>(kf[t], x.p[p], lo[t]);
#pragma unroll
      for (int t = 0; t < 4; ++t) hi[t] = mfma16<DT>(kf[t], x.p[0], hi[t]);
      keep_order();
    }
    {
      const __amdgpu_buffer_rsrc_t sb = So.piece(true);
#pragma unroll
      for (int m = 0; m < 2 * KS; ++m) buf_store_f4(sb, os + (m >> 1) * 2048 + (m & 1) * 256, S[m]);
      So.at -= So.step;
    }
    f32x4 x[4];
#pragma unroll
    for (int it = 0; it < 4; ++it) x[it] = scaled<DT>(hi[it] + lo[it], es) * gate(1, it);
    Frag<3> xP[6], xW[6];
    __builtin_amdgcn_sched_barrier(0);
    load_upper(xP, P);
    store_rows(b ^ 1);                     // its readers were done at the barrier
    load_rows(steps_of(c - 2));
    // P^T dO, and scale gam dO for the state
    f32x4 pd[4] = {};
    uint32_t two[4][2];                    // dO, two steps a dword
#pragma unroll
    for (int it = 0; it < 4; ++it)
#pragma unroll
      for (int i = 0; i < 2; ++i) two[it][i] = xd[it][2 * i] | (uint32_t)xd[it][2 * i + 1] << 16;
    const auto dO = [&](int it) {
      return f32x4{widen<DT>((uint16_t)two[it][0]), widen<DT>((uint16_t)(two[it][0] >> 16)), widen<DT>((uint16_t)two[it][1]),
                   widen<DT>((uint16_t)(two[it][1] >> 16))};
    };
    {
      Frag<NA> of[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) of[s] = split8<NA>(join(dO(2 * s), dO(2 * s + 1)));
#pragma unroll
      for (int q = 2; q >= 0; --q)
#pragma unroll
        for (int j = 0; j < NA && j <= q; ++j)
#pragma unroll
          for (int x = 0; x < 6; ++x) {
            const int it = x < 2 ? x : x - 2, s = x < 2 ? 0 : 1;
            pd[it] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xP[x].p[q - j], of[s].p[j], pd[it], 0, 0, 0);
          }
    }
    __builtin_amdgcn_sched_barrier(0);
    load_upper(xW, W);
#pragma unroll
    for (int it = 0; it < 4; ++it) dN[it] = pd[it] * scale + x[it];
    // Y = W^T dN
    f32x4 Y[4] = {};
    {
      Frag<3> df[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) df[s] = split8<3>(join(dN[2 * s], dN[2 * s + 1]));
#pragma unroll
      for (int q = 2; q >= 0; --q)
#pragma unroll
        for (int i = 0; i <= q; ++i)
#pragma unroll
          for (int x = 0; x < 6; ++x) {
            const int it = x < 2 ? x : x - 2, s = x < 2 ? 0 : 1;
            Y[it] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xW[x].p[i], df[s].p[q - i], Y[it], 0, 0, 0);
          }
    }
    __builtin_amdgcn_sched_barrier(0);
    f32x4 xN[4];
    uint16_t xv[4][4];
    {
      const __amdgpu_buffer_rsrc_t nb = Ni.piece(true), vb = V.rows(n);
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        xN[it] = buf_f4(nb, on + (it >> 1) * 2048 + (it & 1) * 256);
        uint32_t o = anew(ov) + (32 * (it >> 1) + 4 * (it & 1)) * vnext;
#pragma unroll
        for (int e = 0; e < 4; ++e, o += vnext) xv[it][e] = buf_raw<DT>(vb, o);
      }
      Ni.at -= Ni.step;
      V.at -= V.step;
    }
    // gam63 dS' + Q^T (scale gam dO), then - K^T (gam beta Y)
    const auto add_to_state = [&](const uint16_t* rows, const f32x4 (&y)[4], float last) {
      const int ey = column_exponent<DT>(y);
      Cut<DT> yf[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) yf[s] = cut<DT>(join(y[2 * s], y[2 * s + 1]), ey);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        f32x4 t[2] = {};
        u32x4 f[2][2];
#pragma unroll
        for (int o = 0; o < 2; ++o)
#pragma unroll
          for (int s = 0; s < 2; ++s) f[o][s] = get_joined_t<LDK>(rows, s, k, o, l);
#pragma unroll
        for (int p = PS - 1; p >= 0; --p)
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int o = 0; o < 2; ++o) t[o] = mfma16<DT>(f[o][s], yf[s].p[p], t[o]);
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          t[o] = scaled<DT>(t[o], ey);
#pragma unroll
          for (int e = 0; e < 4; ++e) S[2 * k + o][e] = __builtin_fmaf(S[2 * k + o][e], last, t[o][e]);
        }
        keep_order();
      }
    };
    keep_order();
    {
      f32x4 gd[4];
#pragma unroll
      for (int it = 0; it < 4; ++it) gd[it] = dO(it) * gate(0, it) * scale;
      add_to_state(Qb, gd, Gl[b][0][63]);
    }
    const __amdgpu_buffer_rsrc_t part = Po.piece(true);
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      f32x4 q;
#pragma unroll
      for (int e = 0; e < 4; ++e) q[e] = sum16(x[it][e] * xN[it][e]);
      buf_store_f4(part, op + (128 + 32 * (it >> 1) + 4 * (it & 1)) * 4, q);
    }
    {
      const __amdgpu_buffer_rsrc_t yb = Yo.piece(true), vb = dV.rows(n);
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const f32x4 dR = Y[it] * gate(2, it);
        uint32_t o = anew(odv) + (32 * (it >> 1) + 4 * (it & 1)) * dnext;
        f32x4 bs, bg;
#pragma unroll
        for (int e = 0; e < 4; ++e, o += dnext) {
          buf_store1<DT>(vb, o, dR[e]);
          bs[e] = sum16(Y[it][e] * xN[it][e]);
          bg[e] = bs[e] - sum16(dR[e] * widen<DT>(xv[it][e]));
        }
        buf_store_f4(yb, on + (it >> 1) * 2048 + (it & 1) * 256, Y[it]);
        buf_store_f4(part, op + (32 * (it >> 1) + 4 * (it & 1)) * 4, bs);
        buf_store_f4(part, op + (64 + 32 * (it >> 1) + 4 * (it & 1)) * 4, bg);
        Y[it] = dR * -gate(0, it);
      }
      Yo.at -= Yo.step;
      dV.at -= dV.step;
      Po.at -= Po.step;
    }
    keep_order();
    load_dO(steps_of(c - 1));
    add_to_state(Kb, Y, 1.0f);
  }
  if (a.dh0) {
#pragma unroll
    for (int m = 0; m < 2 * KS; ++m)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int dk = 16 * (m & ~1) + 8 * g4 + 4 * (m & 1) + e;
        if (dk < a.Dk && dv < a.Dv) a.dh0[seq * a.dh0_s[0] + h * a.dh0_s[1] + dk * a.dh0_s[2] + dv] = S[m][e];
      }
  }
}

// ---- dq, dk, dg, dbeta of a chunk ------------------------------------------------------
//
// One workgroup a (chunk, key head): it adds up the key head's value heads in their order, so the
// gradients of shared heads need no atomics.  Eight waves: wave w has the steps of block
// w % 4; waves 0..3 the first half of the keys' columns and F, waves 4..7 the other half
// and E.  Contractions over the values go through LDS 32 values at a time, the next 32
// under way in registers; S, dS', N and Y lie there by values, and the transposing read
// makes fragments of them.  Bound by that staging and its waits, one workgroup a CU: 2 x 4096 steps, 16 heads of
// 128 in bf16, 218 us, 0.6 GB at 2.8 TB/s.
template <int DT, int DKP>
__global__ __launch_bounds__(512) void grads_kernel(DeltaArgs a) {
  constexpr int NA = InPlanes<DT>::n, OP = kOrder + 1, KS = DKP / 32, LDK = DKP + 8, LDO = 40;
  constexpr int ES = DT == CCV_DT_F32 ? 4 : 2, TK = DKP / 32;       // TK: a wave's 16-column tiles of the keys
  constexpr bool TWO = DT != CCV_DT_F32;                            // LDS for S and dS' at once
  constexpr int kS = OP * 32 * LDK, kN = 3 * 32 * LDT, kO = TWO ? NA * 64 * LDO : 0;
  constexpr int kStage = (TWO ? 2 : 1) * kS + 2 * kN + kO, kPair = 2 * OP * 64 * LDT;
  __shared__ __bf16 Kl[NA][64][LDK], Ql[NA][64][LDK];
  __shared__ __bf16 un[kStage > kPair ? kStage : kPair];
  __shared__ __align__(16) float gates[kDeltaDec];  // e^G, e^(G63 - G), -, G as doubles, beta
  __shared__ float rows[64], cols[8][64], dots[8];
  const double* G = reinterpret_cast<const double*>(gates + 192);
  __bf16* St = un;                                  // [OP][32][LDK]
  __bf16* Dt = TWO ? St + kS : St;
  __bf16* Nt = Dt + kS;                             // [3][32][LDT]
  __bf16* Yt = Nt + kN;
  __bf16* Ol = Yt + kN;                             // [NA][64][LDO]: dO, by steps; fp32 has no room for it
  __bf16* Ft = un;                                  // [OP][64][LDT], by columns j
  __bf16* Et = un + OP * 64 * LDT;
  const int c = blockIdx.x / a.Hk, hk = blockIdx.x - c * a.Hk, group = a.Hv / a.Hk;
  const Chunk k = chunk_at(a, c);
  if (k.n <= 0) return;
  const int tid = threadIdx.x, w8 = __builtin_amdgcn_readfirstlane(tid >> 6), w = w8 & 3, half = w8 >> 2, l = tid & 63, r = l & 15,
            g4 = l >> 4;
  const int t = 16 * w + r;
  const bool live = t < k.n;
  f32x4 dq[TK], dk[TK];
#pragma unroll
  for (int n = 0; n < TK; ++n) dq[n] = dk[n] = f32x4{0, 0, 0, 0};

  if (k.seq < a.nseq) {
    RowTile<DT, DKP, LDK> kq(w, l, (uint32_t)((half ? a.k_s[1] : a.q_s[1]) * ES), a.Dk);
    kq.load(half ? chunk_rows<DT>(a.k, a.k_s, k, hk, (a.Dk + 7) & ~7) : chunk_rows<DT>(a.q, a.q_s, k, hk, (a.Dk + 7) & ~7));
    // what a thread moves of 32 values: RS times 4 keys of one value of S and dS', 4 steps of one
    // value of N and Y, and 8 values of one step of dO
    constexpr int RS = DKP / 64, kLanesO = 4;
    const int lv = tid >> 6;                        // its 1 KB tile of the 32 values' (16 of S: RS rounds)
    f32x4 s4[RS], d4[RS], n4, y4;
    u32x4 o4;
    const int orow = TWO ? tid / kLanesO : 64, oc = tid % kLanesO * (16 / ES);
    for (int hg = 0; hg < group; ++hg) {
      const int h = hk * group + hg;
      const int64_t ch = (int64_t)c * a.Hv + h;
      const float* dec = a.dec + ch * kDeltaDec;
      const __amdgpu_buffer_rsrc_t sb = buffer(a.S + ch * DKP * a.Dvp, 4u * DKP * a.Dvp), db = buffer(a.dS + ch * DKP * a.Dvp, 4u * DKP * a.Dvp),
                                   nb = buffer(a.N + ch * 64 * a.Dvp, 256u * a.Dvp), yb = buffer(a.Y + ch * 64 * a.Dvp, 256u * a.Dvp),
                                   ob = chunk_rows<DT>(a.dout, a.do_s, k, h, (a.Dv + 7) & ~7);
      const auto load = [&](int v0) {
        const uint32_t os = (uint32_t)v0 * DKP * 4 + tid * 16, on = (uint32_t)v0 * 256 + tid * 16;
#pragma unroll
        for (int i = 0; i < RS; ++i) {
          s4[i] = buf_f4(sb, os + i * 8192);
          d4[i] = buf_f4(db, os + i * 8192);
        }
        n4 = buf_f4(nb, on);
        y4 = buf_f4(yb, on);
        if constexpr (TWO)
          o4 = buf16(ob, orow < 64 && v0 + oc < a.Dv ? orow * (uint32_t)(a.do_s[1] * ES) + (v0 + oc) * ES : kNowhere);
      };
      load(0);
      if (tid < kDeltaDec) gates[tid] = dec[tid];
      if (hg == 0) kq.store(half ? &Kl[0][0][0] : &Ql[0][0][0], 64 * LDK);
      f32x4 zq[TK], zy[TK], zn[TK], pr[4];
      float dot = 0;
#pragma unroll
      for (int n = 0; n < TK; ++n) zq[n] = zy[n] = zn[n] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int n = 0; n < 4; ++n) pr[n] = f32x4{0, 0, 0, 0};

      for (int v0 = 0; v0 < a.Dvp; v0 += 32) {
        lds_barrier();
        // 1 KB tiles [lane][4 rows]: tile (16 values, 16 keys) of S, (16 values, 16 steps) of N and Y
        const auto put_S = [&](__bf16* to, const f32x4 (&x)[RS]) {
#pragma unroll
          for (int i = 0; i < RS; ++i) {
            const int tile = 8 * i + lv, tv = tile / (DKP / 16), tk = tile % (DKP / 16);
            put4<OP>(to + (16 * tv + r) * LDK + 16 * tk + 4 * g4, 32 * LDK, x[i]);
          }
        };
        put_S(St, s4);
        if constexpr (TWO) put_S(Dt, d4);
        put4<3>(Nt + (16 * (lv >> 2) + r) * LDT + 16 * (lv & 3) + 4 * g4, 32 * LDT, n4);
        put4<3>(Yt + (16 * (lv >> 2) + r) * LDT + 16 * (lv & 3) + 4 * g4, 32 * LDT, y4);
        if constexpr (TWO) {
          if (orow < 64) {
            const Frag<NA> f = planes<DT>(Raw8<DT>{{o4}});
#pragma unroll
            for (int p = 0; p < NA; ++p) *reinterpret_cast<bf16x8*>(Ol + p * 64 * LDO + orow * LDO + oc) = f.p[p];
          }
        }
#pragma unroll
        for (int i = 0; i < RS; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) dot = __builtin_fmaf(s4[i][e], d4[i][e], dot);
        f32x4 later[RS];
#pragma unroll
        for (int i = 0; i < RS; ++i) later[i] = d4[i];
        if (v0 + 32 < a.Dvp) load(v0 + 32);
        lds_barrier();
        Frag<NA> of;
        if constexpr (TWO) of = get8<NA>(Ol + t * LDO + 8 * g4, 64 * LDO);
        else of = planes<DT>(buf8<DT>(ob, v0 + 8 * g4 < a.Dv ? t * (uint32_t)(a.do_s[1] * ES) + (v0 + 8 * g4) * ES : kNowhere));
        const Frag<3> yf = get8t<3>(Yt + 16 * w, LDT, 32 * LDT, l);
        const Frag<OP> nown = get8t<OP>(Nt + 16 * w, LDT, 32 * LDT, l);
#pragma unroll
        for (int n = 0; n < TK; ++n) {
          const Frag<OP> sf = get8t<OP>(St + 16 * (TK * half + n), LDK, 32 * LDK, l);
          zq[n] = mma(sf, of, zq[n]);
          zy[n] = mma(sf, yf, zy[n]);
          if constexpr (TWO) zn[n] = mma(get8t<OP>(Dt + 16 * (TK * half + n), LDK, 32 * LDK, l), nown, zn[n]);
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          if (n > w) continue;
          const Frag<3> nf = get8t<3>(Nt + 16 * n, LDT, 32 * LDT, l);
          if (half) pr[n] = mma(yf, nf, pr[n]);
          else pr[n] = mma(of, nf, pr[n]);
        }
        if constexpr (!TWO) {
          lds_barrier();
          put_S(Dt, later);
          lds_barrier();
#pragma unroll
          for (int n = 0; n < TK; ++n) zn[n] = mma(get8t<OP>(Dt + 16 * (TK * half + n), LDK, 32 * LDK, l), nown, zn[n]);
        }
      }
#pragma unroll
      for (int d = 32; d; d >>= 1) dot += __shfl_xor(dot, d);
      if (l == 0) dots[w8] = dot;
      const float gam = gates[t], del = gates[64 + t], bet = gates[kDeltaBeta + t];
#pragma unroll
      for (int n = 0; n < TK; ++n) {
        dq[n] += zq[n] * (a.scale * gam);
        dk[n] += zn[n] * del - zy[n] * (gam * bet);
      }

      // F (waves 0..3) and E (4..7), their products with Q K^T and K K^T
      lds_barrier();
      f32x4 rs = {0, 0, 0, 0};
      double Gi[4];
      float bi[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        Gi[e] = G[16 * w + 4 * g4 + e];
        bi[e] = half ? -gates[kDeltaBeta + 16 * w + 4 * g4 + e] : a.scale;
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
            x = mma(half ? get8<NA>(&Kl[0][t][32 * s + 8 * g4], 64 * LDK) : get8<NA>(&Ql[0][t][32 * s + 8 * g4], 64 * LDK),
                       get8<NA>(&Kl[0][j][32 * s + 8 * g4], 64 * LDK), x);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = 16 * w + 4 * g4 + e;
            if (i < j || (half && i == j)) continue;
            f[e] = __builtin_amdgcn_exp2f((float)(Gi[e] - G[j])) * pr[n][e] * bi[e];
            if (i > j) {
              rs[e] = __builtin_fmaf(f[e], x[e], rs[e]);
              cs = __builtin_fmaf(f[e], x[e], cs);
            }
          }
        }
        put4<OP>(Pt + j * LDT + 16 * w + 4 * g4, 64 * LDT, f);
        cs = sum4rows(cs);
        if (g4 == 0) cols[w8][j] = cs;
      }
      if (!half) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float rv = sum16(rs[e]);
          if (r == 0) rows[16 * w + 4 * g4 + e] = rv;
        }
      }
      lds_barrier();
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const bool lo = 2 * s <= w, up = 2 * s + 1 >= w;      // rows i >= j; rows j <= i
        // F's fragments, then E's: both at once would not stay in registers
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const __bf16* Mt = e ? Et : Ft;
          Frag<OP> mr, mc;
          if (lo) mr = get8t<OP>(Mt + 32 * s * LDT + 16 * w, LDT, 64 * LDT, l);
          if (up) mc = get8<OP>(Mt + t * LDT + 32 * s + 8 * g4, 64 * LDT);
#pragma unroll
          for (int n = 0; n < TK; ++n) {
            const Frag<NA> kt = get8t<NA>(&Kl[0][32 * s][16 * (TK * half + n)], LDK, 64 * LDK, l);
            if (e) {
              if (lo) dk[n] = mma(kt, mr, dk[n]);
              if (up) dk[n] = mma(kt, mc, dk[n]);
            } else {
              if (lo) dq[n] = mma(kt, mr, dq[n]);
              if (up) dk[n] = mma(get8t<NA>(&Ql[0][32 * s][16 * (TK * half + n)], LDK, 64 * LDK, l), mc, dk[n]);
            }
          }
        }
      }
      if (w8 == 0) {                                          // a step a lane
        float g = rows[l], sd = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          g -= cols[i][l];
          sd += dots[i];
        }
        a.pairs[ch * kDeltaPairs + l] = g;
        if (l == 0) a.pairs[ch * kDeltaPairs + 64] = sd;
      }
      lds_barrier();      // before the next head writes what is read here
    }
  }
  if (live) {
    char* dqp = row_ptr<DT>(a.dq, a.dq_s, k.row, (int64_t)k.t0 + t, hk);
    char* dkp = row_ptr<DT>(a.dk, a.dk_s, k.row, (int64_t)k.t0 + t, hk);
#pragma unroll
    for (int n = 0; n < TK; ++n) {
      const int d = 16 * (TK * half + n) + 4 * g4;
      store4<DT>(dqp + d * ES, dq[n], a.Dk - d, a.vec_dqk);
      store4<DT>(dkp + d * ES, dk[n], a.Dk - d, a.vec_dqk);
    }
  }
}

// dg and dbeta of a chunk and head, a step a lane of one wave: the slices' sums and the pairs'
// joined, then the running sum from the chunk's end (2048 chunks and heads: 9 us).
__global__ __launch_bounds__(256) void gates_kernel(DeltaArgs a, int64_t items) {
  const int64_t ch = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (ch >= items) return;
  const int c = (int)(ch / a.Hv), h = (int)(ch - (int64_t)c * a.Hv), l = threadIdx.x & 63;
  const Chunk k = chunk_at(a, c);
  if (k.n <= 0) return;
  float g = 0, b = 0;
  if (k.seq < a.nseq) {
    const float* part = a.part + ch * a.slices * kDeltaPart;
    const float* pairs = a.pairs + ch * kDeltaPairs;
    const float* dec = a.dec + ch * kDeltaDec;
    const float beta = dec[128 + l], last = dec[63], dot = pairs[64];
    float cj = 0;
    g = pairs[l];
#pragma unroll 4
    for (int i = 0; i < a.slices; ++i) {
      b += part[i * kDeltaPart + l];
      g += part[i * kDeltaPart + 64 + l];
      cj += part[i * kDeltaPart + 128 + l];
    }
    const float* by_state = a.qpart + ch * a.qslices * 64;
#pragma unroll 4
    for (int i = 0; i < a.qslices; ++i) g += by_state[i * 64 + l];
    if (l >= k.n - 1) cj = 0;      // the last step's decay to the end is 1, whatever its g
    float tot = cj;
#pragma unroll
    for (int d = 32; d; d >>= 1) tot += __shfl_xor(tot, d);
    g -= cj;
    if (l == 63) g += tot + last * dot;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const float o = __shfl_down(g, d);
      if (l + d < 64) g += o;
    }
    const int begin = a.packed ? a.cstart[a.nseq + 2 + k.seq] : 0;
    if (l == 0 && k.t0 == begin && !a.h0) g = 0;
    b /= beta;
  }
  if (l < k.n) {
    const int64_t t = (int64_t)k.t0 + l;
    store_gate(a.dg, a.g_dtype, k.row * a.dg_s[0] + t * a.dg_s[1] + h * a.dg_s[2], g);
    store_gate(a.dbeta, a.b_dtype, k.row * a.db_s[0] + t * a.db_s[1] + h * a.db_s[2], b);
  }
}

template <int DT, int DKP, int NT>
void launch_rev(const DeltaArgs& a, hipStream_t st) {
  const uint32_t heads = (a.part_chunks ? (uint32_t)a.parts : (uint32_t)(a.nseq + (a.packed ? 1 : 0))) * a.Hv;
  const uint32_t slices = (a.Dvp + 16 * NT - 1) / (16 * NT);
  const dim3 grid(places(a.share, heads, slices));
  if constexpr (NT == 1) {
    if (a.part_chunks) {
      reverse_kernel<DT, DKP, 1, true><<<grid, 512, 0, st>>>(a, heads, slices);
      join_kernel<DKP, true><<<dim3((uint32_t)a.nseq * a.Hv, a.Dvp / 16), 256, 0, st>>>(a);
    }
  }
  reverse_kernel<DT, DKP, NT, false><<<grid, 512, 0, st>>>(a, heads, slices);
}
template <int DT, int DKP>
void launch_rev_waves(const DeltaArgs& a, hipStream_t st) {
  const uint32_t heads = (uint32_t)(a.nseq + (a.packed ? 1 : 0)) * a.Hv;
  const uint32_t slices = (a.Dvp + 16 * kColumnWaves - 1) / (16 * kColumnWaves);
  reverse_wave_kernel<DT, DKP><<<dim3(places(a.share, heads, slices)), 64 * kColumnWaves, 0, st>>>(a, heads, slices);
}
template <int DT>
void launch_rev(const DeltaArgs& a, int nt, hipStream_t st) {
  if constexpr (DT == CCV_DT_F16) {
    if (a.waves_back) return a.Dkp == 64 ? launch_rev_waves<DT, 64>(a, st) : launch_rev_waves<DT, 128>(a, st);
  }
  if constexpr (DT == CCV_DT_BF16) {       // 32 columns of two or three planes of K and Q exceed the LDS
    if (nt == 2) {
      if (a.Dkp == 64) launch_rev<DT, 64, 2>(a, st);
      else launch_rev<DT, 128, 2>(a, st);
      return;
    }
  }
  if (a.Dkp == 64) launch_rev<DT, 64, 1>(a, st);
  else launch_rev<DT, 128, 1>(a, st);
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
  const int e = (int)hipGetLastError();
  if (e) return e;
  const int64_t items = (int64_t)a.nchunks * a.Hv;
  gates_kernel<<<(uint32_t)((items + 3) / 4), 256, 0, st>>>(a, items);
  return (int)hipGetLastError();
}

}  // namespace ccv
