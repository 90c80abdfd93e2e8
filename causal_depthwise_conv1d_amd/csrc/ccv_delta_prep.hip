// ccv_delta_prep.hip -- gated delta rule: the part of a chunk that no state enters.
//
// For the 64 steps of a chunk and one value head, with G the running sum of g inside the
// chunk:   A_ij = beta_i e^(G_i - G_j) k_i.k_j  (i > j),   P_ij = e^(G_i - G_j) q_i.k_j  (i >= j),
//          W = (1 + A)^-1.
// Bound by memory, and by the latency of a chunk's few steps one after the other: 35 KB of LDS let four
// workgroups of 16-bit inputs share a CU.  W and P go out as three bf16 planes, both without the quarter
// above the diagonal blocks of 32, which is zero.  4 x 4096 steps, 16 heads of 128 in bf16: 67 us, 300 MB at 4.5 TB/s
// (with P in two planes 62, then 78 with whole planes and K's and W's LDS apart).  65536 packed steps, 10 key
// and 20 value heads in fp16: 270 to 330 us.
// G is summed in 64 bits, so that differences of steps that lie far down a strongly
// decaying chunk keep 32 bits.  A decay of g < -2000 (and -inf, a forgotten state) counts
// as -2000: e^-2000 is 0 in fp32 with room to spare, and no inf - inf arises.
#include "ccv_delta_device.hpp"

#include <type_traits>

namespace ccv {
namespace {

// ---- rows that 16-byte loads cannot take, copied -------------------------------------
template <class T>
__global__ __launch_bounds__(256) void pack_kernel(DeltaPackArgs a) {
  const int64_t n = a.rows * a.Dp;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / a.Dp, d = i - r * a.Dp, bh = r / a.L, b = bh / a.H;
    const T* src = static_cast<const T*>(a.src) + b * a.s[0] + (r - bh * a.L) * a.s[1] + (bh - b * a.H) * a.s[2];
    static_cast<T*>(a.dst)[i] = d < a.D ? src[d] : T{0};
  }
}

// ---- packed rows: the chunks of each sequence ---------------------------------------
//
// Sequence s holds the steps [cu[s], cu[s + 1]); the offsets count as their running maximum,
// clamped to [0, L], so that no table can lead outside the row.  The steps past the last
// sequence are sequence `nseq`, whose outputs are zeros.  One workgroup: the longest part
// is a binary search a chunk (64 sequences of 65536 steps: 7 us, 7 of 3011 steps: 4 us).
struct Most { static __device__ inline int of(int x, int y) { return x > y ? x : y; } };
struct Sum { static __device__ inline int of(int x, int y) { return x + y; } };

// Running results over the workgroup's 1024 threads of values that are not negative, from `from` on, which becomes
// the result of all.  `wave` may be used again after the next barrier.
template <class OP>
__device__ inline int running(int x, int& from, int (&wave)[16]) {
  const auto row = [](int v, auto ctrl, auto rows) {
    return OP::of(v, __builtin_amdgcn_update_dpp(0, v, ctrl.value, rows.value, 0xf, false));
  };
  using std::integral_constant;
  x = row(x, integral_constant<int, 0x111>(), integral_constant<int, 0xf>());      // rows of 16: 1, 2, 4, 8 lanes back
  x = row(x, integral_constant<int, 0x112>(), integral_constant<int, 0xf>());
  x = row(x, integral_constant<int, 0x114>(), integral_constant<int, 0xf>());
  x = row(x, integral_constant<int, 0x118>(), integral_constant<int, 0xf>());
  x = row(x, integral_constant<int, 0x142>(), integral_constant<int, 0xa>());      // a row's last lane to the next row
  x = row(x, integral_constant<int, 0x143>(), integral_constant<int, 0xc>());      // lane 31 to the upper half
  const int w = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 63) wave[w] = x;
  __syncthreads();
  int before = from, all = from;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    if (k == w) before = all;
    all = OP::of(all, wave[k]);
  }
  from = all;
  return OP::of(before, x);
}

__global__ __launch_bounds__(1024) void table_kernel(DeltaArgs a) {
  __shared__ int waves[3][16], count[1024], at[1024], ends[1024];
  const int tid = threadIdx.x, n = a.nseq + 1, L = (int)a.L;
  int32_t* begin = a.cstart + (a.nseq + 2);
  int last = 0, chunks = 0, parts = 0;
  count[tid] = 0;
  // the order in which the passes over the chunks take the sequences: longest first, so that no long one
  // starts when the others are done (which of two of one length comes first changes no result)
  const auto bucket = [](int chunks) { return chunks < 1023 ? 1023 - chunks : 0; };
  for (int base = 0; base < n; base += 1024) {
    const int i = base + tid, before = last;
    int e = 0;
    if (i < a.nseq) {
      const int x = a.cu[i + 1];
      e = x < 0 ? 0 : x > L ? L : x;
    } else if (i == a.nseq) {
      e = L;
    }
    const int end = running<Most>(e, last, waves[0]);
    ends[tid] = end;
    __syncthreads();
    const int t0 = tid ? ends[tid - 1] : before;
    const int c = i < n ? (end - t0 + kDeltaChunk - 1) / kDeltaChunk : 0;
    const int upto = running<Sum>(c, chunks, waves[1]);
    if (i < n) {
      a.cstart[i + 1] = upto;
      begin[i] = t0;
      if (i == a.nseq) begin[n] = L;
      else atomicAdd(&count[bucket(c)], 1);
    }
    if (a.part_chunks) {      // the parts of each sequence, one at least
      const int p = i < a.nseq ? (c + a.part_chunks - 1) / a.part_chunks : 1;
      const int up = running<Sum>(i < n ? (p > 1 ? p : 1) : 0, parts, waves[2]);
      if (i < n) a.pstart[i + 1] = up;
    }
    __syncthreads();
  }
  if (tid == 0) {
    a.cstart[0] = 0;
    if (a.part_chunks) a.pstart[0] = 0;
    a.order[a.nseq] = a.nseq;
  }
  int zero = 0;
  at[tid] = running<Sum>(count[tid], zero, waves[0]) - count[tid];
  __threadfence_block();
  __syncthreads();
  for (int s = tid; s < a.nseq; s += 1024) a.order[atomicAdd(&at[bucket(a.cstart[s + 1] - a.cstart[s])], 1)] = s;
  // the last of the first `n` entries of an increasing table that is <= x
  const auto find = [&](const int32_t* table, int x) {
    int lo = 0, hi = a.nseq;
    while (lo < hi) {
      const int m = (lo + hi + 1) >> 1;
      if (table[m] <= x) lo = m;
      else hi = m - 1;
    }
    return lo;
  };
  for (int p = tid; a.part_chunks && p < a.parts; p += 1024) {
    const int s = find(a.pstart, p);
    a.ptable[2 * p] = p < parts ? s : n;
    a.ptable[2 * p + 1] = p < parts ? p - a.pstart[s] : 0;
  }
  for (int c = tid; c < a.nchunks; c += 1024) {
    int s = a.nseq, t0 = 0, len = 0;
    if (c < chunks) {
      s = find(a.cstart, c);
      t0 = begin[s] + (c - a.cstart[s]) * kDeltaChunk;
      len = begin[s + 1] - t0;
      len = len < kDeltaChunk ? len : kDeltaChunk;
    }
    a.table[4 * c] = s;
    a.table[4 * c + 1] = t0;
    a.table[4 * c + 2] = len;
    a.table[4 * c + 3] = 0;
  }
}

// ---- A, P and W of a chunk -----------------------------------------------------------
//
// One workgroup a (chunk, head); wave w holds rows 16 w .. 16 w + 15 of every 64 x 64 matrix.
// W by blocks: each wave solves its 16 x 16 diagonal block by substitution (a lane a
// column), then blocks join in pairs, [X 0; Y Z]^-1 = [X' 0; -Z' Y X' Z'], on the fp32
// matrix instruction, whose accumulator layout is the next product's operand.
template <int DT, int DKP, bool BWD>
__global__ __launch_bounds__(256) void prep_kernel(DeltaArgs a) {
  // 16-bit rows go through LDS as they are, and are multiplied in their own type: exact products
  constexpr int RT = DT == CCV_DT_F32 ? DT : CCV_DT_BF16, NA = InPlanes<RT>::n, LDK = DKP + 8, LDA = 68, ES = DT == CCV_DT_F32 ? 4 : 2;
  __shared__ union { __bf16 k[NA][64][LDK]; float w[64][LDA]; } kw;    // K's planes, then W
  auto& Kp = kw.k;
  auto& Wl = kw.w;
  __shared__ float Al[64][LDA];                                        // A, then P
  __shared__ double G[64];
  __shared__ float bt[64];
  uint32_t item, slice;
  if (!place(a.share_prep, (uint32_t)a.nchunks * a.Hv, 1, &item, &slice)) return;
  const int ch = item, c = ch / a.Hv, h = ch - c * a.Hv, hk = h / (a.Hv / a.Hk);
  const Chunk k = chunk_at(a, c);
  if (k.n <= 0 || k.seq >= a.nseq) return;
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, r = l & 15, g4 = l >> 4;

  // gates: wave 0, a step a lane
  if (w == 0) {
    double g = 0;
    float b = 0, given = 0;
    if (l < k.n) {
      const int64_t t = k.t0 + l;
      float x = load_param(a.g, a.g_dtype, k.row * a.g_s[0] + t * a.g_s[1] + h * a.g_s[2]);
      x = x < -2000.0f ? -2000.0f : x;
      g = (double)x * 1.4426950408889634;
      b = given = load_param(a.beta, a.b_dtype, k.row * a.b_s[0] + t * a.b_s[1] + h * a.b_s[2]);
      // the backward divides N by beta (dbeta = Y . N / beta): a beta of 0 is there, for N, the smallest that
      // keeps N / beta in fp32, and N stays below anything it is added to; what is a multiple of beta itself,
      // dv among it, takes beta as given
      if (BWD && __builtin_fabsf(b) < 1e-30f) b = __builtin_copysignf(1e-30f, b);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double o = __shfl_up(g, d);
      if (l >= d) g += o;
    }
    const double last = __shfl(g, 63);
    G[l] = g;
    bt[l] = b;
    float* dec = a.dec + (int64_t)ch * kDeltaDec;
    dec[l] = __builtin_amdgcn_exp2f((float)g);
    dec[64 + l] = __builtin_amdgcn_exp2f((float)(last - g));
    dec[128 + l] = b;
    dec[kDeltaBeta + l] = given;
    reinterpret_cast<double*>(dec + 192)[l] = g;
  }

  // K's planes into LDS, and Q's; this wave's 16 rows of Q then stay in registers
  const int row = 16 * w + r;
  Frag<NA> qf[DKP / 32];
  {
    RowTile<RT, DKP, LDK> kt(w, l, (uint32_t)(a.k_s[1] * ES), a.Dk), qt(w, l, (uint32_t)(a.q_s[1] * ES), a.Dk);
    kt.load(chunk_rows<DT>(a.k, a.k_s, k, hk, (a.Dk + 7) & ~7));
    qt.load(chunk_rows<DT>(a.q, a.q_s, k, hk, (a.Dk + 7) & ~7));
    qt.store(&Kp[0][0][0], 64 * LDK);          // each wave's own rows
#pragma unroll
    for (int s = 0; s < DKP / 32; ++s) qf[s] = get8<NA>(&Kp[0][row][32 * s + 8 * g4], 64 * LDK);
    kt.store(&Kp[0][0][0], 64 * LDK);
  }
  __syncthreads();

  f32x4 pv[4];
  double Gi[4];
  float bi[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    Gi[e] = G[16 * w + 4 * g4 + e];
    bi[e] = bt[16 * w + 4 * g4 + e];
  }
#pragma unroll
  for (int jb = 0; jb < 4; ++jb) {
    f32x4 kk = {0, 0, 0, 0}, qk = {0, 0, 0, 0};
    const int j = 16 * jb + r;
    if (jb <= w) {
#pragma unroll
      for (int s = 0; s < DKP / 32; ++s) {
        const Frag<NA> bf = get8<NA>(&Kp[0][j][32 * s + 8 * g4], 64 * LDK);
        const Frag<NA> af = get8<NA>(&Kp[0][row][32 * s + 8 * g4], 64 * LDK);
        if constexpr (DT == CCV_DT_F32) {
          kk = mma(af, bf, kk);
          qk = mma(qf[s], bf, qk);
        } else {
          const u32x4 y = __builtin_bit_cast(u32x4, bf.p[0]);
          kk = mfma16<DT>(__builtin_bit_cast(u32x4, af.p[0]), y, kk);
          qk = mfma16<DT>(__builtin_bit_cast(u32x4, qf[s].p[0]), y, qk);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 16 * w + 4 * g4 + e;
      const float d = i >= j ? __builtin_amdgcn_exp2f((float)(Gi[e] - G[j])) : 0.0f;
      pv[jb][e] = i >= j ? d * qk[e] : 0.0f;
      Al[i][j] = i > j ? bi[e] * d * kk[e] : 0.0f;
    }
  }
  __syncthreads();
  // what of W's rows lies right of the diagonal blocks
#pragma unroll
  for (int jb = 1; jb < 4; ++jb)
    if (jb > w) *reinterpret_cast<f32x4*>(&Wl[16 * w + r][16 * jb + 4 * g4]) = f32x4{0, 0, 0, 0};

  // diagonal blocks: column r of block w, the four groups of lanes alike
  {
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float acc = i == r ? 1.0f : 0.0f;
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (j < i) acc = __builtin_fmaf(-Al[16 * w + i][16 * w + j], x[j], acc);
      x[i] = acc;
      if (i / 4 == g4) Wl[16 * w + i][16 * w + r] = acc;
    }
  }
  __syncthreads();
  if (w < 2) {                                       // blocks of 32
    const int r0 = 32 * w, r1 = r0 + 16;
    f32x4 t = {0, 0, 0, 0}, y = {0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < 4; ++s)
      t = __builtin_amdgcn_mfma_f32_16x16x4f32(Al[r1 + r][r0 + 4 * s + g4], Wl[r0 + 4 * s + g4][r0 + r], t, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      y = __builtin_amdgcn_mfma_f32_16x16x4f32(Wl[r1 + r][r1 + 4 * g4 + e], t[e], y, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < 4; ++e) Wl[r1 + 4 * g4 + e][r0 + r] = -y[e];
  }
  __syncthreads();
  {                                                  // 64: wave w makes block (w / 2, w % 2) of the lower left
    const int rb = w >> 1, cb = w & 1;
    f32x4 y = {0, 0, 0, 0};
    for (int s = 0; s <= rb; ++s) {
      f32x4 t = {0, 0, 0, 0};
      for (int u = cb; u < 2; ++u)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          t = __builtin_amdgcn_mfma_f32_16x16x4f32(Al[32 + 16 * s + r][16 * u + 4 * q + g4],
                                                   Wl[16 * u + 4 * q + g4][16 * cb + r], t, 0, 0, 0);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        y = __builtin_amdgcn_mfma_f32_16x16x4f32(Wl[32 + 16 * rb + r][32 + 16 * s + 4 * g4 + e], t[e], y, 0, 0, 0);
    }
    // rows 32.. of columns 0..31 are read by nobody in this step
#pragma unroll
    for (int e = 0; e < 4; ++e) Wl[32 + 16 * rb + 4 * g4 + e][16 * cb + r] = -y[e];
  }
  __syncthreads();
#pragma unroll
  for (int jb = 0; jb < 4; ++jb)
#pragma unroll
    for (int e = 0; e < 4; ++e) Al[16 * w + 4 * g4 + e][16 * jb + r] = pv[jb][e];
  __syncthreads();
  // out as planes: a thread takes 8 consecutive elements of two rows (columns when transposed)
  const auto write = [&](uint16_t* out, const float (*m)[LDA], auto nplanes, bool transposed, bool join = false) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = i * 256 + tid, ro = transposed ? e & 63 : e >> 3, co = 8 * (transposed ? e >> 6 : e & 7);
      if (transposed ? ro >= 32 && co < 32 : ro < 32 && co >= 32) continue;      // the zero quarter: nobody reads it
      f32x8 x;
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = transposed ? m[co + q][ro] : m[ro][co + q];
      const auto f = split8<nplanes.value>(x);
#pragma unroll
      for (int p = 0; p < nplanes.value; ++p)
        *reinterpret_cast<bf16x8*>(out + (int64_t)ch * kDeltaMatrix + p * 4096 + fragment_at(join ? joined(ro) : ro, co)) = f.p[p];
    }
  };
  write(a.W, Wl, std::integral_constant<int, 3>(), false, a.waves);
  if constexpr (BWD) {
    write(a.WT, Wl, std::integral_constant<int, 3>(), true, a.waves_back);
    write(a.P, Al, std::integral_constant<int, 3>(), true, a.waves_back);
  } else {
    write(a.P, Al, std::integral_constant<int, 3>(), false);
  }
}

template <int DT, int DKP>
void launch_prep(const DeltaArgs& a, bool bwd, hipStream_t st) {
  const dim3 grid(places(a.share_prep, (int64_t)a.nchunks * a.Hv, 1));
  if (bwd) prep_kernel<DT, DKP, true><<<grid, 256, 0, st>>>(a);
  else prep_kernel<DT, DKP, false><<<grid, 256, 0, st>>>(a);
}
template <int DT>
void launch_prep(const DeltaArgs& a, bool bwd, hipStream_t st) {
  if (a.Dkp == 64) launch_prep<DT, 64>(a, bwd, st);
  else launch_prep<DT, 128>(a, bwd, st);
}

}  // namespace

int launch_delta_pack(const DeltaPackArgs& a, void* stream) {
  const int64_t need = (a.rows * a.Dp + 255) / 256;
  const uint32_t grid = (uint32_t)(need < 65536 ? need : 65536);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (a.dtype == CCV_DT_F32) pack_kernel<uint32_t><<<grid, 256, 0, st>>>(a);
  else pack_kernel<uint16_t><<<grid, 256, 0, st>>>(a);
  return (int)hipGetLastError();
}

int launch_delta_table(const DeltaArgs& a, void* stream) {
  table_kernel<<<1, 1024, 0, static_cast<hipStream_t>(stream)>>>(a);
  return (int)hipGetLastError();
}

int launch_delta_prep(const DeltaArgs& a, bool backward, void* stream) {
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (a.x_dtype == CCV_DT_F32) launch_prep<CCV_DT_F32>(a, backward, st);
  else if (a.x_dtype == CCV_DT_F16) launch_prep<CCV_DT_F16>(a, backward, st);
  else launch_prep<CCV_DT_BF16>(a, backward, st);
  return (int)hipGetLastError();
}

}  // namespace ccv
