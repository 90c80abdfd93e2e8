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
//
// What bounds it is that chain: 4 x 4096 steps, 16 heads of 128 in bf16 take 204 us, 3.2 us a chunk,
// of which the matrix units are busy 24 % and LDS 52 %.  NT is 2 where blocks of 16 columns are more
// than the CUs, since K, Q, W and P are then staged for 32 columns at once, and 1 below: 1 x 2048 steps of 34 heads of
// 128 in bf16, forward, backward's forward pass and pass from the end: 94, 102, 127 us with 2, 97, 126, 173 with 1;
// 32 heads: 93, 99, 117 with 2, 63, 70, 94 with 1.  fp32, and the backward's passes in fp16, have LDS
// for 1 only.  Held to 128 registers, for two workgroups a CU, the forward with NT 1 in bf16 is slower: 2 x 4096
// steps of 16 heads of 128 take 127 us, 124 without.
#include "ccv_delta_device.hpp"

namespace ccv {
namespace {

constexpr int LDT = 80;      // row stride of an LDS array of 64 steps

// kMap: what a part of a sequence makes of any state, S -> T S + B: the columns of T are the chain's result from
// those of the identity, without values, and those of B from zeros; only the waves of the state.
enum Mode { kForward, kBackward, kMap };

template <int DT, int DKP, int NT, Mode MODE>
__global__ __launch_bounds__(MODE == kMap ? 256 : 512, MODE == kMap ? 1 : 2) void scan_kernel(DeltaArgs a, uint32_t heads, uint32_t slices) {
  constexpr int NA = InPlanes<DT>::n, CB = 16 * NT, KS = DKP / 32, MT = DKP / 64, LDK = DKP + 16;
  constexpr bool BWD = MODE == kBackward;
  constexpr int ES = DT == CCV_DT_F32 ? 4 : 2;
  __shared__ __bf16 Sp[3][CB][LDK];        // S by columns
  __shared__ __bf16 Rp[3][CB][LDT];        // beta R by columns
  __shared__ __bf16 Kl[NA][64][LDK];
  __shared__ union {                       // Q until the first barrier of a chunk, N from then on
    __bf16 q[MODE == kMap ? 1 : NA][MODE == kMap ? 1 : 64][LDK];
    struct {
      __bf16 p[3][CB][LDT], d[3][CB][LDT];      // N, del N
    } n;
  } qn;
  auto& Ql = qn.q;
  auto& Np = qn.n.p;
  auto& Nd = qn.n.d;
  uint32_t hs, slice;
  if (!place(a.share, heads, slices, &hs, &slice)) return;
  const int sh = hs / a.Hv, h = hs - sh * a.Hv, hk = h / (a.Hv / a.Hk), dv0 = slice * CB - (MODE == kMap ? DKP : 0);
  const Part part = part_at(a, sh);
  const int seq = part.seq;
  const int tid = threadIdx.x, w8 = __builtin_amdgcn_readfirstlane(tid >> 6), w = w8 & 3, l = tid & 63, r = l & 15, g4 = l >> 4;

  if (seq >= a.nseq) {                     // the steps of a packed row that belong to no sequence
    if constexpr (MODE == kForward) {
      if (seq > a.nseq) return;
      const int32_t* begin = a.cstart + (a.nseq + 2);
      for (int64_t i = (int64_t)begin[a.nseq] * CB + tid; i < a.L * CB; i += 512) {
        const int64_t t = i / CB;
        const int d = dv0 + (int)(i - t * CB);
        if (d < a.Dv) store1<DT>(row_ptr<DT>(a.out, a.o_s, 0, t, h) + d * ES, 0.0f);
      }
    }
    return;
  }
  if (MODE == kMap && part.last && (!a.dS || !part.k || dv0 >= 0)) return;   // its T serves the backward only, its B nobody
  const Sequence sq = part.sq;
  const int c0 = sq.first, c1 = sq.end;
  const int64_t ch0 = (int64_t)c0 * a.Hv + h;
  const int i = 16 * w + r;                // the step whose row of K, Q, W, P this lane holds
  const uint32_t om = (2 * w * 64 + l) * 16;     // its fragments of W and P
  const auto steps = [](int64_t left) { return left < kDeltaChunk ? (int)left : kDeltaChunk; };
  int64_t left = sq.len;                   // steps from the chunk at hand on

  if (w8 < 4) {
    // ---- the state: rows 16 (MT w + m) + 4 g4 + e, column 16 j + r ----------------------
    f32x4 S[MT][NT];
    const f32x4* start = MODE == kMap ? nullptr : start_tiles(a, part, h, -1);
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
            if constexpr (MODE == kMap) S[m][j][e] = dk == dv + DKP ? 1.0f : 0.0f;
            else S[m][j][e] = a.h0 && dk < a.Dk && dv < a.Dv ? a.h0[seq * a.h0_s[0] + h * a.h0_s[1] + dk * a.h0_s[2] + dv] : 0.0f;
          }
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
        ov[j][e] = dv >= 0 && dv < a.Dv ? (16 * w + 4 * g4 + e) * V.stride + dv * ES : kNowhere;
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
      for (int s = 0; s < 2; ++s) xW[s] = buf_planes<3>(b, s && w < 2 ? kNowhere : om + 1024 * s, 8192);
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
      Sums ks[NT];
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
      Sums ws[NT];
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
        if constexpr (MODE == kForward) put4<3>(&Np[0][16 * j + r][16 * w + 4 * g4], CB * LDT, N[j]);
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
      Sums sn[MT][NT];
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
    if constexpr (MODE == kMap) {
      float* to = part_map(a, sh, h);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if (dv0 < 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) to[map_at<DKP>(16 * (MT * w + m) + 4 * g4 + e, slice * CB + 16 * j + r)] = S[m][j][e];
          } else {
            reinterpret_cast<f32x4*>(to + DKP * DKP)[((dv0 / 16 + j) * (DKP / 16) + MT * w + m) * 64 + l] = S[m][j];
          }
        }
    } else if (a.ht && part.last) {
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
  } else if constexpr (MODE != kMap) {
    // ---- the outputs: step i, four consecutive values 16 j + 4 g4 a lane; the same barriers ----
    Frag<3> xP[2];
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
        for (int s = 0; s < 2; ++s) xP[s] = buf_planes<3>(b, s && w < 2 ? kNowhere : om + 1024 * s, 8192);
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
      Sums qs[NT];      // S^T Q^T (columns: steps)
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const Frag<NA> qf = get8<NA>(&Ql[0][i][32 * s + 8 * g4], 64 * LDK);
#pragma unroll
        for (int j = 0; j < NT; ++j) qs[j].add(get8<3>(&Sp[0][16 * j + r][32 * s + 8 * g4], CB * LDK), qf);
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
        if (g4 == 0) a.qpart[(((int64_t)c * a.Hv + h) * a.qslices + slice) * 64 + i] = dot;
        lds_barrier();
      } else {
        f32x4 o[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) o[j] = qs[j].total() * gam;
        lds_barrier();
        Sums ps[NT];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (2 * s > w) continue;
#pragma unroll
          for (int j = 0; j < NT; ++j) ps[j].add(get8<3>(&Np[0][16 * j + r][32 * s + 8 * g4], CB * LDT), xP[s]);
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

// ---- 16-bit inputs: 16 columns a wave --------------------------------------------------------
//
// A wave holds 16 columns of the state to their full height, so that all of the chain above stays
// in its registers (see joined()): K S is R's rows, R the right-hand side of W R, N that of
// K^T (del N) and the left-hand side of P N.  What the waves share are K and Q, which are needed
// by rows and, K, by columns: a chunk's rows lie in LDS, two chunks in turn, one barrier a chunk.
//
// A chunk takes longer so (4.8 us: all of a column's 132 to 182 matrix instructions in one wave) but costs
// the CU less: nothing is exchanged, and K and Q are staged once for 64 columns.  It pays once scan_kernel's
// workgroups of 32 columns are more than the CUs: 1 x 2048 steps of 72 heads of 128, 576 waves, forward and the
// backward's forward pass: 148 and 186 us against 176 and 215 (bf16), 153 and 179 against 230 and 260 (fp16); 64 heads:
// 146 and 177 against 94 and 120, 150 and 170 against 128 and 182; 256 heads: 271 against 371 and 482 forward.  65536
// packed steps, 64 sequences, 20 heads in fp16: 840 to 1000 us.  Bound by the instructions of two waves a SIMD and the
// loads of W and P between them; 256 registers a wave leave no room to fetch those a chunk ahead.
template <int DT, int DKP, bool BWD>
__global__ __launch_bounds__(64 * kColumnWaves, 2) void wave_kernel(DeltaArgs a, uint32_t heads, uint32_t slices) {
  constexpr int NW = kColumnWaves, KS = DKP / 32, LDK = DKP + 8, CB = 16 * NW, PS = Cut<DT>::n;
  __shared__ uint16_t Kl[2][64][LDK], Ql[2][64][LDK];
  __shared__ float Gl[2][3][64];            // gam, del, beta
  uint32_t hs, slice;
  if (!place(a.share, heads, slices, &hs, &slice)) return;
  const int sh = hs / a.Hv, h = hs - sh * a.Hv, seq = in_order(a, sh), hk = h / (a.Hv / a.Hk);
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, r = l & 15, g4 = l >> 4;
  if (seq >= a.nseq) {                     // the steps of a packed row that belong to no sequence
    if constexpr (!BWD) {
      const int32_t* begin = a.cstart + (a.nseq + 2);
      for (int64_t i = (int64_t)begin[a.nseq] * CB + tid; i < a.L * CB; i += 64 * NW) {
        const int64_t t = i / CB;
        const int d = (int)slice * CB + (int)(i - t * CB);
        if (d < a.Dv) store1<DT>(row_ptr<DT>(a.out, a.o_s, 0, t, h) + d * 2, 0.0f);
      }
    }
    return;
  }
  const int ct = slice * NW + w, dv0 = 16 * ct, dv = dv0 + r;      // this wave's columns, and the lane's
  const Sequence sq = sequence_at(a, seq);
  const int c0 = sq.first, c1 = sq.end;
  const int64_t ch0 = (int64_t)c0 * a.Hv + h;

  f32x4 S[2 * KS];                         // tile 2 s + o: keys 32 s + 8 g4 + 4 o + e
#pragma unroll
  for (int m = 0; m < 2 * KS; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int dk = 16 * (m & ~1) + 8 * g4 + 4 * (m & 1) + e;
      S[m][e] = a.h0 && dk < a.Dk && dv < a.Dv ? a.h0[seq * a.h0_s[0] + h * a.h0_s[1] + dk * a.h0_s[2] + dv] : 0.0f;
    }
  Rows<DT> K(a.k, a.k_s, sq, hk, (a.Dk + 7) & ~7, c0), Q(a.q, a.q_s, sq, hk, (a.Dk + 7) & ~7, c0), V(a.v, a.v_s, sq, h, a.Dv, c0);
  Rows<DT> O(BWD ? a.dout : a.out, BWD ? a.do_s : a.o_s, sq, h, BWD ? (a.Dv + 7) & ~7 : a.Dv, c0);
  Piece<uint16_t> W(a.W, kDeltaMatrix, a.Hv, ch0), P(a.P, kDeltaMatrix, a.Hv, ch0);
  Piece<float> D(a.dec, kDeltaDec, a.Hv, ch0);
  Piece<float> So(a.S, (int64_t)DKP * a.Dvp, a.Hv, ch0), No(a.N, 64 * (int64_t)a.Dvp, a.Hv, ch0),
      Po(a.qpart, (int64_t)a.qslices * 64, a.Hv, ch0);
  const float scale = a.scale;
  const bool vec = a.vec_o;
  const int dleft = a.Dv - dv0 - 4 * g4;
  const uint32_t oo = dleft > 0 ? r * O.stride + (dv0 + 4 * g4) * 2 : kNowhere, onext = 16 * O.stride;
  const uint32_t ov = dv < a.Dv ? 8 * g4 * V.stride + dv * 2 : kNowhere, vnext = V.stride;
  // tiles as the workspace has them: row 32 s + 8 g4 + 4 o + e is element e of lane group 2 (g4 % 2) + o of tile 2 s + g4 / 2
  const uint32_t to = ((g4 >> 1) * 64 + 2 * (g4 & 1) * 16 + r) * 16;
  const uint32_t os = ct * (DKP / 16) * 1024 + to, on = ct * 4096 + to;
  const uint32_t op = g4 == 0 ? (ct * 64 + r) * 4 : kNowhere;      // past the slices: out of bounds too

  RowCopy<DKP, LDK, NW, true> kt(w, l, K.stride, a.Dk);
  RowCopy<DKP, LDK, NW, false> qt(w, l, Q.stride, a.Dk);
  Frag<3> xW[6];
  Frag<3> xP[6];
  uint16_t xv[4][4];
  Raw4<DT> xd[4];
  float gates;                             // one of a chunk's gam, del, beta, on the way to LDS
  int64_t left = sq.len;                   // steps from the chunk at hand on
  const auto ahead = [&](int chunks) {     // steps of a chunk further on, 0 past the last
    const int64_t n = left - chunks * kDeltaChunk;
    return n <= 0 ? 0 : n < kDeltaChunk ? (int)n : kDeltaChunk;
  };
  const auto load_rows = [&](int n) {
    kt.load(K.rows(n));
    qt.load(Q.rows(n));
    gates = buf1<CCV_DT_F32>(D.piece(n > 0), tid < 192 ? tid * 4 : kNowhere);
    K.at += K.step;
    Q.at += Q.step;
    D.at += D.step;
  };
  const auto store_rows = [&](int b) {
    kt.store(&Kl[b][0][0]);
    qt.store(&Ql[b][0][0]);
    if (tid < 192) Gl[b][0][tid] = gates;
  };
  const auto load_V = [&](int n) {
    const __amdgpu_buffer_rsrc_t b = V.rows(n);
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      uint32_t o = anew(ov) + (32 * (it >> 1) + 4 * (it & 1)) * vnext;
#pragma unroll
      for (int e = 0; e < 4; ++e, o += vnext) xv[it][e] = buf_raw<DT>(b, o);
    }
    V.at += V.step;
  };
  const auto load_W = [&](int n) {
    const __amdgpu_buffer_rsrc_t b = W.piece(n > 0);
#pragma unroll
    for (int i = 0; i < 6; ++i) xW[i] = buf_planes<3>(b, ((i < 4 ? 2 * i : 2 * i - 3) * 64 + l) * 16, 8192);
    W.at += W.step;
  };
  const auto load_P = [&](int n) {
    if constexpr (BWD) {
      const __amdgpu_buffer_rsrc_t b = O.rows(n);
#pragma unroll
      for (int t = 0; t < 4; ++t) xd[t] = buf_raw4<DT>(b, anew(oo) + t * onext);
      O.at += O.step;
    } else {
      const __amdgpu_buffer_rsrc_t b = P.piece(n > 0);
#pragma unroll
      for (int i = 0; i < 6; ++i) xP[i] = buf_planes<3>(b, ((i < 4 ? 2 * i : 2 * i - 3) * 64 + l) * 16, 8192);
      P.at += P.step;
    }
  };
  if (c0 < c1) {
    load_rows(ahead(0));
    store_rows(0);
    load_rows(ahead(1));                   // in the loop's order: the waits of both have to agree
    load_V(ahead(0));
  }
  for (int c = c0; c < c1; ++c) {
    const int b = (c - c0) & 1, n = ahead(0), nn = ahead(1);
    const uint16_t *Kb = &Kl[b][0][0], *Qb = &Ql[b][0][0];
    const auto gate = [&](int which, int it) {
      return *reinterpret_cast<const f32x4*>(&Gl[b][which][32 * (it >> 1) + 4 * (it & 1) + 8 * g4]);
    };
    lds_barrier();
    // K S, and (Q S)^T
    f32x4 hi[4] = {}, lo[4] = {}, qs[4] = {};
    const int es = column_exponent<DT>(S);
    u32x4 kf[4], qf[4];
    const auto read_rows = [&](int s) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        kf[t] = *reinterpret_cast<const u32x4*>(Kb + (16 * t + r) * LDK + 32 * s + 8 * g4);
        qf[t] = *reinterpret_cast<const u32x4*>(Qb + (16 * t + r) * LDK + 32 * s + 8 * g4);
      }
    };
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      read_rows(s);
      const Cut<DT> x = cut<DT>(join(S[2 * s], S[2 * s + 1]), es);
#pragma unroll
      for (int p = PS - 1; p > 0; --p)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          lo[t] = mfma16<DT>(kf[t], x.p[p], lo[t]);
          qs[t] = mfma16<DT>(x.p[p], qf[t], qs[t]);
        }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        hi[t] = mfma16<DT>(kf[t], x.p[0], hi[t]);
        qs[t] = mfma16<DT>(x.p[0], qf[t], qs[t]);
      }
    }
    load_W(n);
    store_rows(b ^ 1);                     // its readers were done at the barrier
    load_rows(ahead(2));
    if constexpr (BWD) {
      const __amdgpu_buffer_rsrc_t sb = So.piece(true);
#pragma unroll
      for (int m = 0; m < 2 * KS; ++m) buf_store_f4(sb, os + (m >> 1) * 2048 + (m & 1) * 256, S[m]);
      So.at += So.step;
    }
    // beta R
    Frag<3> rf[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      f32x4 R[2];
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const int it = 2 * s + o;
        const f32x4 x = scaled<DT>(hi[it] + lo[it], es), gam = gate(0, it), beta = gate(2, it);
#pragma unroll
        for (int e = 0; e < 4; ++e) R[o][e] = __builtin_fmaf(-gam[e], x[e], widen<DT>(xv[it][e])) * beta[e];
      }
      rf[s] = split8<3>(join(R[0], R[1]));
    }
    load_V(nn);
    u32x4 tf[2][2];
    const auto read_columns = [&](int c) {
#pragma unroll
      for (int o = 0; o < 2; ++o)
#pragma unroll
        for (int s = 0; s < 2; ++s) tf[o][s] = get_joined_t<LDK>(Kb, s, c, o, l);
    };
    // N = W (beta R); W is lower triangular
    f32x4 N[4] = {};
#pragma unroll
    for (int q = 2; q >= 0; --q)
#pragma unroll
      for (int i = 0; i <= q; ++i)
#pragma unroll
        for (int x = 0; x < 6; ++x) {        // row tiles 0 1 2 3 2 3, steps 0 0 0 0 32 32 ..
          const int it = x < 4 ? x : x - 2, s = x / 4;
          N[it] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xW[x].p[i], rf[s].p[q - i], N[it], 0, 0, 0);
        }
    load_P(n);
    if constexpr (BWD) {
      const __amdgpu_buffer_rsrc_t nb = No.piece(true);
#pragma unroll
      for (int it = 0; it < 4; ++it) buf_store_f4(nb, on + (it >> 1) * 2048 + (it & 1) * 256, N[it]);
      No.at += No.step;
    }
    // the state at the chunk's end
    {
      f32x4 y[4];
#pragma unroll
      for (int it = 0; it < 4; ++it) y[it] = N[it] * gate(1, it);
      const int ey = column_exponent<DT>(y);
      const float last = Gl[b][0][63];
      Cut<DT> yf[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) yf[s] = cut<DT>(join(y[2 * s], y[2 * s + 1]), ey);
#pragma unroll
      for (int c = 0; c < KS; ++c) {
        read_columns(c);
        f32x4 t[2] = {};
#pragma unroll
        for (int p = PS - 1; p >= 0; --p)
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int o = 0; o < 2; ++o) t[o] = mfma16<DT>(tf[o][s], yf[s].p[p], t[o]);
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          t[o] = scaled<DT>(t[o], ey);
#pragma unroll
          for (int e = 0; e < 4; ++e) S[2 * c + o][e] = __builtin_fmaf(S[2 * c + o][e], last, t[o][e]);
        }
      }
    }
    int er[4] = {};                        // the rows of (Q S)^T are columns of S
    if constexpr (DT == CCV_DT_F16) {
#pragma unroll
      for (int e = 0; e < 4; ++e) er[e] = __shfl(es, 4 * g4 + e);
    }
    if constexpr (BWD) {
      // scale gam dO . (Q S): the part of dG that comes by the state
      const __amdgpu_buffer_rsrc_t part = Po.piece(true);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const f32x4 d = widen4<DT>(xd[t]);
        float dot = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) dot = __builtin_fmaf(d[e], scaled<DT>(qs[t][e], er[e]), dot);
        dot = sum4rows(dot) * Gl[b][0][16 * t + r] * scale;
        buf_store1<CCV_DT_F32>(part, op + 64 * t, dot);
      }
      Po.at += Po.step;
    } else {
      // the outputs: step 16 t + r, four consecutive values a lane
      const __amdgpu_buffer_rsrc_t ob = O.rows(n);
      Frag<3> nf[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) nf[s] = split8<3>(join(N[2 * s], N[2 * s + 1]));
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float gam = Gl[b][0][16 * t + r];
#pragma unroll
        for (int e = 0; e < 4; ++e) qs[t][e] = scaled<DT>(qs[t][e], er[e]) * gam;
      }
      // the low planes last: they arrive last (65536 packed steps, 20 heads in fp16: 920 us, 1015 with them first)
#pragma unroll
      for (int q = 0; q <= kOrder; ++q)
#pragma unroll
        for (int i = q; i >= 0; --i)
#pragma unroll
          for (int x = 0; x < 6; ++x) {
            const int t = x < 4 ? x : x - 2, s = x / 4;
            qs[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(nf[s].p[i], xP[x].p[q - i], qs[t], 0, 0, 0);
          }
#pragma unroll
      for (int t = 0; t < 4; ++t) buf_store4<DT>(ob, anew(oo) + t * onext, qs[t] * scale, dleft, vec);
      O.at += O.step;
    }
    left -= kDeltaChunk;
  }
  if (a.ht) {
#pragma unroll
    for (int m = 0; m < 2 * KS; ++m)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int dk = 16 * (m & ~1) + 8 * g4 + 4 * (m & 1) + e;
        if (dk < a.Dk && dv < a.Dv) a.ht[seq * a.ht_s[0] + h * a.ht_s[1] + dk * a.ht_s[2] + dv] = S[m][e];
      }
  }
}

template <int DT, int DKP>
void launch_waves(const DeltaArgs& a, bool bwd, hipStream_t st) {
  constexpr int NW = kColumnWaves;
  const uint32_t heads = (uint32_t)(a.nseq + (a.packed ? 1 : 0)) * a.Hv;
  const uint32_t slices = (a.Dvp + 16 * NW - 1) / (16 * NW);
  const dim3 grid(places(a.share, heads, slices));
  if (bwd) wave_kernel<DT, DKP, true><<<grid, 64 * NW, 0, st>>>(a, heads, slices);
  else wave_kernel<DT, DKP, false><<<grid, 64 * NW, 0, st>>>(a, heads, slices);
}
uint32_t parts_of(const DeltaArgs& a) { return a.part_chunks ? (uint32_t)a.parts : (uint32_t)(a.nseq + (a.packed ? 1 : 0)); }

template <int DT, int DKP>
void launch_map(const DeltaArgs& a, hipStream_t st) {
  const uint32_t heads = (uint32_t)a.parts * a.Hv, slices = (DKP + a.Dvp) / 16;
  scan_kernel<DT, DKP, 1, kMap><<<dim3(places(a.share, heads, slices)), 256, 0, st>>>(a, heads, slices);
  join_kernel<DKP, false><<<dim3((uint32_t)a.nseq * a.Hv, a.Dvp / 16), 256, 0, st>>>(a);
}
template <int DT>
void launch_map(const DeltaArgs& a, hipStream_t st) {
  if (a.Dkp == 64) launch_map<DT, 64>(a, st);
  else launch_map<DT, 128>(a, st);
}

template <int DT, int DKP, int NT>
void launch(const DeltaArgs& a, bool bwd, hipStream_t st) {
  const uint32_t heads = parts_of(a) * a.Hv;
  const uint32_t slices = (a.Dvp + 16 * NT - 1) / (16 * NT);
  const dim3 grid(places(a.share, heads, slices));
  if (bwd) scan_kernel<DT, DKP, NT, kBackward><<<grid, 512, 0, st>>>(a, heads, slices);
  else scan_kernel<DT, DKP, NT, kForward><<<grid, 512, 0, st>>>(a, heads, slices);
}
template <int DT>
void launch(const DeltaArgs& a, bool bwd, int nt, hipStream_t st) {
  if constexpr (DT != CCV_DT_F32) {
    if (a.waves) return a.Dkp == 64 ? launch_waves<DT, 64>(a, bwd, st) : launch_waves<DT, 128>(a, bwd, st);
  }
  if constexpr (DT != CCV_DT_F32) {
    if (nt == 2) return a.Dkp == 64 ? launch<DT, 64, 2>(a, bwd, st) : launch<DT, 128, 2>(a, bwd, st);
  }
  if (a.Dkp == 64) launch<DT, 64, 1>(a, bwd, st);
  else launch<DT, 128, 1>(a, bwd, st);
}

}  // namespace

int launch_delta_carry(const DeltaArgs& a, void* stream) {
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (a.x_dtype == CCV_DT_F32) launch_map<CCV_DT_F32>(a, st);
  else if (a.x_dtype == CCV_DT_F16) launch_map<CCV_DT_F16>(a, st);
  else launch_map<CCV_DT_BF16>(a, st);
  return (int)hipGetLastError();
}

int launch_delta_scan(const DeltaArgs& a, bool backward, int nt, void* stream) {
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (a.x_dtype == CCV_DT_F32) launch<CCV_DT_F32>(a, backward, nt, st);
  else if (a.x_dtype == CCV_DT_F16) launch<CCV_DT_F16>(a, backward, nt, st);
  else launch<CCV_DT_BF16>(a, backward, nt, st);
  return (int)hipGetLastError();
}

}  // namespace ccv
