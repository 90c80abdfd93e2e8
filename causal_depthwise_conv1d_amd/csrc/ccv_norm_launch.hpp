// ccv_norm_launch.hpp -- launch descriptors of layer norm and of the sequence tables, seen
// by the host validation code and the kernels.  No HIP types.
#pragma once

#include <stdint.h>

namespace ccv {

// Rows are numbered r = i * n1 + j, row (i, j) of x starting at i * s[0] + j * s[1]
// elements (n1 = 0: row r at r * s[1], in every view); elements of a row are unit-stride.
struct NormArgs {
  const void *x, *w, *b, *dout;
  void *out, *dx, *dw, *db;
  int64_t x_s[2], o_s[2], do_s[2], dx_s[2];
  float *mean, *rstd;                 // [rows]; written by the forward when wanted, read by the backward
  int64_t rows;
  uint32_t n1;
  int32_t width, x_dtype, w_dtype;
  float eps;
  float* part;                        // backward: [groups][2][width] partial sums of dw, db
  int32_t groups;                     // workgroups of the backward's first kernel
};

// The terms of a column's sum that are added up one after the other before their sum joins those before it: with
// millions of rows, one chain over all of a thread's would round each term to the whole sum's spacing.  Threads that
// hold their rows in registers have no room for a second sum: there it is the workgroups that get more, beyond
// kNormRows rows a thread (1024 of them are the fastest: 4194304 x 64 in fp32 takes 664 us, 710 with 2048).
constexpr int kNormRun = 128;
constexpr int kNormRows = 1024;

// How a call is laid out: `lanes` threads a row, each holding `nv` 16-byte vectors of it;
// lanes 0: rows too wide for that or narrower than a vector, walked in pieces.  Four vectors
// in each of 16 threads would need a workgroup to have 16 rows' sums of dw and db in 200
// registers a thread: one in 64 threads is faster (60000 x 333 bf16, backward: 29 us, not 46).
struct NormShape { int32_t lanes, nv; };

inline NormShape norm_shape(int64_t width, int elt) {
  const int64_t v = 16 / elt;
  if (width < v) return {0, 0};
  for (int32_t lanes : {16, 64, 256, 512})
    for (int32_t nv : {1, 2, 4})
      if (width <= lanes * nv * v && !(lanes == 16 && nv == 4)) return {lanes, nv};
  return {0, 0};
}

struct TablesArgs {
  const int32_t* lengths;
  int32_t *cu, *seq, *pos;            // [n + 1], [total] or nullptr, [total] or nullptr
  int64_t n, total;
};

// Each returns a hipError_t value (0 = success).
int launch_norm_fwd(const NormArgs& a, int cus, void* stream);
int launch_norm_bwd(const NormArgs& a, void* stream);
int launch_tables(const TablesArgs& a, void* stream);

}  // namespace ccv
