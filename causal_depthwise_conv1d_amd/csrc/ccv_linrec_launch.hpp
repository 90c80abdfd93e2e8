// ccv_linrec_launch.hpp -- launch descriptors of the gated linear recurrence, seen by the host
// validation code and the kernels.  No HIP types.
#pragma once

#include <stdint.h>

#include "ccv.h"

#ifdef __HIPCC__
#define LR_HOST_DEVICE __host__ __device__
#else
#define LR_HOST_DEVICE
#endif

namespace ccv {

// A tile is 64 channels of 128 steps, one workgroup's work: 16 rows of lanes, each with 8 consecutive
// steps of its two channels a lane.
constexpr int kLrChannels = 64;
constexpr int kLrRows = 16;
constexpr int kLrTile = CCV_LINREC_CHUNK;
constexpr int kLrSteps = kLrTile / kLrRows;
constexpr int kLrWaves = kLrRows / 2;
// Tiles of a chain in a group, and groups in a stretch: a word for each wave of a workgroup to wait for.
constexpr uint32_t kLrGroup = kLrWaves, kLrStretch = kLrWaves;
// Queues of tickets, at most, and the words from one's counter to the next: 128 bytes.
constexpr uint32_t kLrQueues = 8, kLrTicketWords = 16;

// A divisor as the kernels use it: n / d = (t + ((n - t) >> first)) >> second with t the upper half of n magic.
struct LrDivisor { uint32_t magic, first, second; };

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
  uint64_t* ticket;                   // counters of the queues
  uint64_t* words;                    // [chains, tiles][64] maps of tiles, [chains, groups][64] of groups, [chains, stretches][64] states
  uint64_t* clear;                    // tickets and words: all bits set by launch_linrec_prepare
  int64_t B, L, C, nseq;
  int64_t clear_count;
  uint32_t tiles, cblocks, chains, groups, stretches;
  uint32_t queues, fewer, longer;     // queues of neighbouring chains: fewer + 1 in the first `longer`, fewer in the others
  LrDivisor by_more, by_fewer, by_cblocks;
  int32_t x_dtype, g_dtype, normalize;

  LR_HOST_DEVICE uint32_t first_chain(uint32_t queue) const { return queue * fewer + (queue < longer ? queue : longer); }
  LR_HOST_DEVICE uint32_t chains_of(uint32_t queue) const { return fewer + (queue < longer ? 1 : 0); }
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
