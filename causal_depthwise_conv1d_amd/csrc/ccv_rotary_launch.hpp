// ccv_rotary_launch.hpp -- launch descriptor of rotary positions, seen by the host validation code
// and the kernels.  No HIP types.
#pragma once

#include <stdint.h>

namespace ccv {

struct RotaryArgs {
  const void* in[2];                  // queries and keys
  void* out[2];
  int64_t in_s[2][3], out_s[2][3];    // (row, step, head)
  const int32_t* pos;
  int64_t pos_s[2];
  const double* freq;                 // [half], radians a position
  int64_t tokens;                     // B L
  int32_t L, heads[2];                // heads of the queries and of the keys
  int32_t D, half;                    // 2 half elements of a head are turned
  int32_t x_dtype, interleaved;
  float scale, sign;                  // sign -1: turned back
  bool in_place;                      // both outputs are their inputs, or absent: what is not turned stays
  int32_t span;                       // tokens a workgroup
  int32_t units;                      // of a head that threads take by vectors, the turned ones first; 0: element by element
  int32_t turned_units;
};

constexpr int kRotaryAngles = 1024;   // of a workgroup, at most

// Returns a hipError_t value (0 = success).
int launch_rotary(const RotaryArgs& a, void* stream);

}  // namespace ccv
