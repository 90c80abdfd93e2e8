// ccv_linrec_launch.hpp -- launch descriptors of the gated linear recurrence, seen by the host
// validation code and the kernels.  No HIP types.
#pragma once

#include <stdint.h>

#include "ccv.h"

namespace ccv {

// A tile is 64 channels of 128 steps, one workgroup's work: 16 rows of lanes, each with 8 consecutive
// steps of its two channels a lane.
constexpr int kLrChannels = 64;
constexpr int kLrRows = 16;
constexpr int kLrTile = CCV_LINREC_CHUNK;
constexpr int kLrSteps = kLrTile / kLrRows;
// Tiles in a row of them that look at each other's maps directly.
constexpr int kLrGroup = 32;

struct LinrecArgs {
  const void *x, *g, *dout;
  void *out, *dx, *dg;
  int64_t x_s[2], g_s[2], o_s[2], do_s[2], dx_s[2], dg_s[2];      // (row, step)
  const float *init, *dfinal;         // [sequences, C], rows init_s and df_s apart, or nullptr
  float *final, *dinit;
  int64_t init_s, final_s, df_s, di_s;
  const int32_t* cu;                  // [nseq + 1] or nullptr
  int32_t* sid;                       // packed: each step's sequence, -1 past the last
  float* carries;                     // [B, chunks, C]: the state before each tile
  uint64_t* ticket;                   // of tiles
  uint64_t* words;                    // [chains, tiles][64] maps of tiles, then [chains, groups][64] states
  uint64_t* clear;                    // tickets and words: all bits set by launch_linrec_prepare
  int64_t B, L, C, nseq;
  int64_t clear_count;
  uint32_t tiles, cblocks, chains, groups;
  int32_t x_dtype, g_dtype, normalize;
};

struct LinrecStepArgs {
  const void *x, *g;
  void* out;
  int64_t x_s[2], g_s[2], o_s[2];
  float* state;
  int64_t st_s;
  const int32_t* slots;
  int64_t B, T, C, nslots;
  int32_t x_dtype, g_dtype, normalize;
};

// Each returns a hipError_t value (0 = success).
int launch_linrec_prepare(const LinrecArgs& a, const float* from, int64_t from_s, float* to, int64_t to_s, void* stream);
int launch_linrec_fwd(const LinrecArgs& a, void* stream);
int launch_linrec_bwd(const LinrecArgs& a, void* stream);
int launch_linrec_step(const LinrecStepArgs& a, void* stream);

}  // namespace ccv
