// ccv_delta_launch.hpp -- launch descriptors of the gated delta rule's kernels, seen
// by the host validation code and the kernels.  No HIP types.
#pragma once

#include <stdint.h>

namespace ccv {

constexpr int kDeltaChunk = 64;       // steps a chunk: one wave's lanes, four 16-row matrix tiles
constexpr int kDeltaMatrix = 3 * 64 * 64;   // elements of a chunk's W or P
constexpr int kDeltaDec = 384;        // fp32 values of a chunk's gates in the workspace
constexpr int kDeltaBeta = 320;       // where beta as given stands among them
constexpr int kDeltaPart = 192;       // fp32 sums of a chunk and slice: 64 each of Y.N, Y.N - dv.v, c
constexpr int kDeltaPairs = 128;      // fp32 values: 64 of dG, one dot product, and room
constexpr int kDeltaMaxDk = 128;      // key width (the state's rows are spread over a workgroup's registers)

// One forward or backward call.  Strides are in elements: (row, step, head), unit inside
// a head; states (sequence, head, key), unit along the values.
struct DeltaArgs {
  const void *q, *k, *v, *g, *beta, *dout;
  void* out;                                    // [B, L, Hv, Dv]; nullptr in the backward
  int64_t q_s[3], k_s[3], v_s[3], g_s[3], b_s[3], o_s[3], do_s[3];
  const float* h0;  int64_t h0_s[3];            // nullptr: zeros
  float* ht;        int64_t ht_s[3];            // nullptr: not wanted
  const float* dht; int64_t dht_s[3];
  float* dh0;       int64_t dh0_s[3];
  void *dq, *dk, *dv, *dg, *dbeta;
  int64_t dq_s[3], dk_s[3], dv_s[3], dg_s[3], db_s[3];
  const int32_t* cu;                            // [nseq + 1] or nullptr
  int64_t L;
  int32_t nseq;                                 // sequences: N of a packed row, else B
  int32_t packed;
  int32_t chunks_per_row;                       // ceil(L / 64), not packed
  int32_t nchunks;                              // upper bound of the chunks of all sequences
  int32_t Hk, Hv, Dk, Dv;
  int32_t Dvp;                                  // Dv rounded up to 32: the workspace's value width
  int32_t x_dtype, g_dtype, b_dtype;
  int32_t vec_o, vec_dqk;                       // rows of out, of dq and dk, may be written as whole vectors
  float scale;
  // workspace (element counts below), ch = chunk * Hv + head
  int32_t* table;                               // packed: [nchunks] x (sequence, first step, steps, -)
  int32_t* cstart;                              // packed: [nseq + 2] first chunk of each sequence
  int32_t* order;                               // packed: [nseq + 1] the sequences, longest first
  // few heads: the passes over the chunks take parts of `part_chunks` chunks (0: whole sequences)
  int32_t part_chunks, parts, parts_per_row;    // parts: upper bound over all sequences
  int32_t* pstart;                              // packed: [nseq + 2] first part of each sequence
  int32_t* ptable;                              // packed: [parts] x (sequence, part of it)
  float* carry;                                 // [part][head]: the map of the state over a part, S -> T S + B: Dkp x Dkp of T, Dkp x Dvp of B
  uint16_t* W;                                  // [ch][3][64 x 64, fragment_at]: (1 + A)^-1 as bf16 planes
  uint16_t* P;                                  // likewise, kDeltaMatrix a chunk and head; the backward holds it transposed
  uint16_t* WT;                                 // backward: W transposed
  float* dec;                                   // [ch][kDeltaDec]: e^G, e^(G63 - G), N's beta (ccv_delta_prep.hip), G log2(e) as 64 doubles, beta
  // backward, in 16 x 16 tiles as a wave's accumulators hold them, [tile][lane][4 rows], tiles of
  // one 16 values together:
  float *S, *dS;                                // [ch][Dvp / 16][Dkp / 16] tiles: state at a chunk's start, gradient at its end
  float *N, *Y;                                 // [ch][Dvp / 16][4] tiles
  float* part;                                  // backward: [ch][slices][kDeltaPart] sums over a slice's values
  float* qpart;                                 // backward: [ch][qslices][64] dG by the state, likewise
  float* pairs;                                 // backward: [ch][kDeltaPairs] dG by pairs of steps; <S, dS'>
  int32_t share, share_prep;                    // value heads of one key head that go to one die together, or 1
  int32_t Dkp, slices, qslices;                 // value slices of the pass from the end, and of the forward one
  int32_t waves;                                // the forward pass holds whole columns a wave; W has its rows in joined() order
  int32_t waves_back;                           // the backward's pass likewise, W and P transposed
};

// Single steps against states in a cache.
struct DeltaStepArgs {
  const void *q, *k, *v, *g, *beta;
  void* out;
  int64_t q_s[3], k_s[3], v_s[3], g_s[3], b_s[3], o_s[3];   // (row, step, head)
  float* state; int64_t st_s[3];                            // (slot, head, key)
  const int32_t* slots;                                     // [B] or nullptr: row b uses slot b
  int64_t nslots;
  int32_t B, T, Hk, Hv, Dk, Dv;
  int32_t x_dtype, g_dtype, b_dtype, vec;
  float scale;
};

// A [B, L, H, D] array into one of Dp >= D elements a head, zeros behind the D: rows of odd widths, strides or
// addresses, made ready for 16-byte loads.  The copy is [B, H, L, Dp], so that its steps lie as near to each other as
// the 32-bit offsets over 64 of them need, however many heads there are.
struct DeltaPackArgs {
  const void* src; int64_t s[3];
  void* dst;
  int64_t rows, L;      // rows = B * L * H
  int32_t H, D, Dp, dtype;
};

// Each returns a hipError_t value (0 = success).
int launch_delta_pack(const DeltaPackArgs& a, void* stream);
int launch_delta_table(const DeltaArgs& a, void* stream);
int launch_delta_prep(const DeltaArgs& a, bool backward, void* stream);
int launch_delta_carry(const DeltaArgs& a, void* stream);
int launch_delta_scan(const DeltaArgs& a, bool backward, int nt, void* stream);
int launch_delta_reverse(const DeltaArgs& a, int nt, void* stream);
int launch_delta_grads(const DeltaArgs& a, void* stream);
int launch_delta_step(const DeltaStepArgs& a, void* stream);

}  // namespace ccv
