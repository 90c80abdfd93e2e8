// ccv_delta_scan.hip -- gated delta rule: the pass over a sequence's chunks that carries
// the state, forward.
//
// With gam = e^G, del = e^(G63 - G), W and P of ccv_delta_prep.hip and S the state
// [Dk, Dv] at the chunk's start:
//   R = v - gam K S,  N = W (beta R),  o = scale (gam Q S + P N),  S <- gam63 S + K^T (del N).
// Columns of S (values) do not mix, so a workgroup takes CB = 16 NT of them for one
// sequence and head.  Four of its waves hold the state and share the rows: 16 of a chunk's
// 64 steps and a quarter of the state's rows each, S staying in fp32 accumulators from
// the first chunk to the last.  What a wave needs of the others' rows (S, beta R, N as
// right-hand sides) passes through LDS as bf16 planes, three barriers a chunk.  The other
// four waves make the outputs from the same planes, so that the chain from state to state,
// which nothing else can shorten, holds no work of theirs.
#include "ccv_delta_device.hpp"

namespace ccv {
namespace {

constexpr int LDT = 72;      // row stride of an LDS array of 64 steps

template <int DT, int DKP, int NT, bool BWD>
__global__ __launch_bounds__(512, DT == CCV_DT_BF16 && NT == 1 && !BWD ? 4 : 2) void scan_kernel(DeltaArgs a, uint32_t heads, uint32_t heads_pad) {
  constexpr int NA = InPlanes<DT>::n, CB = 16 * NT, KS = DKP / 32, MT = DKP / 64, LDK = DKP + 8;
  constexpr int OO = OutOrder<DT>::n, ES = DT == CCV_DT_F32 ? 4 : 2;
  __shared__ __bf16 Sp[3][CB][LDK];        // S by columns
  __shared__ __bf16 Rp[3][CB][LDT];        // beta R by columns
  __shared__ __bf16 Kl[NA][64][LDK];
  __shared__ union {                       // Q until the first barrier of a chunk, N from then on
    __bf16 q[NA][64][LDK];
    struct {
      __bf16 p[OO + 1][CB][LDT], d[3][CB][LDT];      // N, del N
    } n;
  } qn;
  auto& Ql = qn.q;
  auto& Np = qn.n.p;
  auto& Nd = qn.n.d;
  const uint32_t hs = blockIdx.x % heads_pad, slice = blockIdx.x / heads_pad;
  if (hs >= heads) return;
  const int seq = hs / a.Hv, h = hs - seq * a.Hv, hk = h / (a.Hv / a.Hk), dv0 = slice * CB;
  const int tid = threadIdx.x, w8 = __builtin_amdgcn_readfirstlane(tid >> 6), w = w8 & 3, l = tid & 63, r = l & 15, g4 = l >> 4;

  if (seq >= a.nseq) {                     // the steps of a packed row that belong to no sequence
    if constexpr (!BWD) {
      const int32_t* begin = a.cstart + (a.nseq + 2);
      for (int64_t i = (int64_t)begin[a.nseq] * CB + tid; i < a.L * CB; i += 512) {
        const int64_t t = i / CB;
        const int d = dv0 + (int)(i - t * CB);
        if (d < a.Dv) store1<DT>(row_ptr<DT>(a.out, a.o_s, 0, t, h) + d * ES, 0.0f);
      }
    }
    return;
  }
  const Sequence sq = sequence_at(a, seq);
  const int c0 = sq.first, c1 = sq.end;
  const int64_t ch0 = (int64_t)c0 * a.Hv + h;
  const int i = 16 * w + r;                // the step whose row of K, Q, W, P this lane holds
  const uint32_t om = (2 * w * 64 + l) * 16;     // its fragments of W and P
  const auto steps = [](int64_t left) { return left < kDeltaChunk ? (int)left : kDeltaChunk; };
  int64_t left = sq.len;                   // steps from the chunk at hand on

  if (w8 < 4) {
    // ---- the state: rows 16 (MT w + m) + 4 g4 + e, column 16 j + r ----------------------
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
    const auto put_state = [&]() {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j) put4<3>(&Sp[0][16 * j + r][16 * (MT * w + m) + 4 * g4], CB * LDK, S[m][j]);
    };
    // What a chunk needs is loaded a chunk ahead, each part as soon as the one before it has
    // been used, so that a load has most of a chunk's time to arrive.
    Frag<3> xW[2];
    uint32_t ov[NT][4];
    typename Stored<DT>::type xv[NT][4];
    struct Gates {
      f32x4 gam, del, beta;
      float last;
    } gt, gn;
    Rows<DT> K(a.k, a.k_s, sq, hk, (a.Dk + 7) & ~7, c0), V(a.v, a.v_s, sq, h, a.Dv, c0);
    Piece<uint16_t> W(a.W, kDeltaMatrix, a.Hv, ch0);
    Piece<float> D(a.dec, kDeltaDec, a.Hv, ch0);
    Piece<float> So(a.S, (int64_t)DKP * a.Dvp, a.Hv, ch0), No(a.N, 64 * (int64_t)a.Dvp, a.Hv, ch0);
    const uint32_t od = (16 * w + 4 * g4) * 4;
    const uint32_t os = ((slice * NT * (DKP / 16) + MT * w) * 64 + l) * 16, on = ((slice * NT * 4 + w) * 64 + l) * 16;
    RowTile<DT, DKP, LDK> kt(w, l, K.stride, a.Dk);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int dv = dv0 + 16 * j + r;
        ov[j][e] = dv < a.Dv ? (16 * w + 4 * g4 + e) * V.stride + dv * ES : kNowhere;
      }
    const auto load_K = [&](int n) {
      kt.load(K.rows(n));
      K.at += K.step;
    };
    const auto load_gates = [&](int n) {
      const __amdgpu_buffer_rsrc_t d = D.piece(n > 0);
      gn.gam = buf_f4(d, od);
      gn.del = buf_f4(d, od + 256);
      gn.beta = buf_f4(d, od + 512);
      gn.last = buf1<CCV_DT_F32>(d, 4 * 63);
      D.at += D.step;
    };
    const auto load_V = [&](int n) {
      const __amdgpu_buffer_rsrc_t b = V.rows(n);
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) xv[j][e] = buf_raw<DT>(b, ov[j][e]);
      V.at += V.step;
    };
    const auto load_W = [&](int n) {
      const __amdgpu_buffer_rsrc_t b = W.piece(n > 0);
#pragma unroll
      for (int s = 0; s < 2; ++s) xW[s] = buf_planes<3>(b, om + 1024 * s, 8192);
      W.at += W.step;
    };
    const auto ahead = [&](int chunks) {       // steps of a chunk further on, 0 past the last
      const int64_t n = left - chunks * kDeltaChunk;
      return n > 0 ? steps(n) : 0;
    };
    if (c0 < c1) {
      load_K(ahead(0));
      load_gates(ahead(0));
      load_V(ahead(0));
      load_W(ahead(0));
    }
    put_state();
    lds_barrier();
    for (int c = c0; c < c1; ++c) {
      const int nn = ahead(1);
      gt = gn;
      kt.store(&Kl[0][0][0], 64 * LDK);
      load_K(nn);
      // K S (rows: steps)
      Sums<2> ks[NT];
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const Frag<NA> kf = get8<NA>(&Kl[0][i][32 * s + 8 * g4], 64 * LDK);
#pragma unroll
        for (int j = 0; j < NT; ++j) ks[j].add(kf, get8<3>(&Sp[0][16 * j + r][32 * s + 8 * g4], CB * LDK));
      }
      load_gates(nn);
      // beta R
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const f32x4 x = ks[j].total();
        f32x4 R;
#pragma unroll
        for (int e = 0; e < 4; ++e) R[e] = __builtin_fmaf(-gt.gam[e], x[e], widen<DT>(xv[j][e]));
        put4<3>(&Rp[0][16 * j + r][16 * w + 4 * g4], CB * LDT, R * gt.beta);
      }
      load_V(nn);
      lds_barrier();
      if constexpr (BWD) {
        const __amdgpu_buffer_rsrc_t sb = So.piece(true);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int m = 0; m < MT; ++m) buf_store_f4(sb, os + (j * (DKP / 16) + m) * 1024, S[m][j]);
        So.at += So.step;
      }

      // N = W (beta R); W is lower triangular
      Sums<2> ws[NT];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (2 * s > w) continue;
#pragma unroll
        for (int j = 0; j < NT; ++j) ws[j].add(xW[s], get8<3>(&Rp[0][16 * j + r][32 * s + 8 * g4], CB * LDT));
      }
      load_W(nn);
      f32x4 N[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        N[j] = ws[j].total();
        put4<3>(&Nd[0][16 * j + r][16 * w + 4 * g4], CB * LDT, N[j] * gt.del);
        if constexpr (!BWD) put4<OO + 1>(&Np[0][16 * j + r][16 * w + 4 * g4], CB * LDT, N[j]);
      }
      lds_barrier();
      if constexpr (BWD) {
        const __amdgpu_buffer_rsrc_t nb = No.piece(true);
#pragma unroll
        for (int j = 0; j < NT; ++j) buf_store_f4(nb, on + j * 4096, N[j]);
        No.at += No.step;
      }

      // the state at the chunk's end
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j) S[m][j] *= gt.last;
      Sums<2> sn[MT][NT];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Frag<3> nf[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) nf[j] = get8<3>(&Nd[0][16 * j + r][32 * s + 8 * g4], CB * LDT);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const Frag<NA> kt = get8t<NA>(&Kl[0][32 * s][16 * (MT * w + m)], LDK, 64 * LDK, l);
#pragma unroll
          for (int j = 0; j < NT; ++j) sn[m][j].add(kt, nf[j]);
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j) S[m][j] += sn[m][j].total();
      put_state();      // nobody has read the planes since the first barrier
      left -= kDeltaChunk;
      lds_barrier();
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
  } else {
    // ---- the outputs: step i, four consecutive values 16 j + 4 g4 a lane; the same barriers ----
    Frag<OO + 1> xP[2];
    Raw4<DT> xd[NT];
    float gam, gam_next;
    uint32_t oo[NT];
    Rows<DT> Q(a.q, a.q_s, sq, hk, (a.Dk + 7) & ~7, c0);
    Rows<DT> O(BWD ? a.dout : a.out, BWD ? a.do_s : a.o_s, sq, h, BWD ? (a.Dv + 7) & ~7 : a.Dv, c0);
    Piece<uint16_t> P(a.P, kDeltaMatrix, a.Hv, ch0);
    Piece<float> D(a.dec, kDeltaDec, a.Hv, ch0);
    const float scale = a.scale;
    const bool vec = a.vec_o;
    const int dleft = a.Dv - dv0 - 4 * g4;
    RowTile<DT, DKP, LDK> qt(w, l, Q.stride, a.Dk);
#pragma unroll
    for (int j = 0; j < NT; ++j) oo[j] = dleft > 16 * j ? i * O.stride + (dv0 + 16 * j + 4 * g4) * ES : kNowhere;
    const auto load_Q = [&](int n) {
      qt.load(Q.rows(n));
      Q.at += Q.step;
      gam_next = buf1<CCV_DT_F32>(D.piece(n > 0), 4 * i);
      D.at += D.step;
    };
    const auto load_P = [&](int n) {
      if constexpr (BWD) {
        const __amdgpu_buffer_rsrc_t b = O.rows(n);
#pragma unroll
        for (int j = 0; j < NT; ++j) xd[j] = buf_raw4<DT>(b, oo[j]);
        O.at += O.step;
      } else {
        const __amdgpu_buffer_rsrc_t b = P.piece(n > 0);
#pragma unroll
        for (int s = 0; s < 2; ++s) xP[s] = buf_planes<OO + 1>(b, om + 1024 * s, 8192);
        P.at += P.step;
      }
    };
    if (c0 < c1) {
      const int n = steps(left);
      load_Q(n);
      load_P(n);
    }
    lds_barrier();
    for (int c = c0; c < c1; ++c) {
      const int n = steps(left);
      left -= kDeltaChunk;
      const int nn = left > 0 ? steps(left) : 0;
      gam = gam_next;
      qt.store(&Ql[0][0][0], 64 * LDK);      // this wave's own rows: no barrier
      Sums<BWD ? 2 : OO> qs[NT];      // S^T Q^T (columns: steps)
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const Frag<NA> qf = get8<NA>(&Ql[0][i][32 * s + 8 * g4], 64 * LDK);
#pragma unroll
        for (int j = 0; j < NT; ++j) qs[j].add(get8<BWD ? 3 : OO + 1>(&Sp[0][16 * j + r][32 * s + 8 * g4], CB * LDK), qf);
      }
      load_Q(nn);
      lds_barrier();
      if constexpr (BWD) {
        // scale gam dO . (Q S): the part of dG that comes by the state
        float dot = 0;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const f32x4 x = qs[j].total(), d = widen4<DT>(xd[j]);
#pragma unroll
          for (int e = 0; e < 4; ++e) dot = __builtin_fmaf(d[e], x[e], dot);
        }
        load_P(nn);
        dot = sum4rows(dot) * gam * scale;
        if (g4 == 0) a.part[(((int64_t)c * a.Hv + h) * a.slices + slice) * kDeltaPart + i] = dot;
        lds_barrier();
      } else {
        f32x4 o[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) o[j] = qs[j].total() * gam;
        lds_barrier();
        Sums<OO> ps[NT];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (2 * s > w) continue;
#pragma unroll
          for (int j = 0; j < NT; ++j) ps[j].add(get8<OO + 1>(&Np[0][16 * j + r][32 * s + 8 * g4], CB * LDT), xP[s]);
        }
        load_P(nn);
        const __amdgpu_buffer_rsrc_t b = O.rows(n);
#pragma unroll
        for (int j = 0; j < NT; ++j) buf_store4<DT>(b, oo[j], (o[j] + ps[j].total()) * scale, dleft - 16 * j, vec);
        O.at += O.step;
      }
      lds_barrier();
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
  if (bwd) scan_kernel<DT, DKP, NT, true><<<grid, 512, 0, st>>>(a, heads, pad);
  else scan_kernel<DT, DKP, NT, false><<<grid, 512, 0, st>>>(a, heads, pad);
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
