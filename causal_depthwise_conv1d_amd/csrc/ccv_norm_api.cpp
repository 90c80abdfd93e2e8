// ccv_norm_api.cpp -- C ABI of layer norm, of group norm and of the sequence tables: argument
// checks and launches.  The operations are stated in ccv.h beside ccv_norm_fwd, ccv_norm_bwd,
// ccv_group_norm_fwd, ccv_group_norm_bwd and ccv_seq_tables.  Host code; nothing here touches a device except the launches.
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "ccv.h"
#include "ccv_checks.hpp"
#include "ccv_launch.hpp"
#include "ccv_norm_launch.hpp"

namespace {

using namespace ccv;
using namespace ccv::checks;

constexpr int64_t kGroups = 1024;    // workgroups, and so partial rows, of the backward, unless it has very many rows

struct Rows {
  const void* p;
  const int64_t* s;
};

int check_rows(const Rows& r, int64_t n0, int64_t n1, int64_t width, int es, bool written) {
  if (r.s[0] < 0 || r.s[1] < 0) return CCV_E_LAYOUT;
  const int64_t n[3] = {n0, n1, width}, s[3] = {r.s[0], r.s[1], 1};
  if (!fits_bytes(max_offset(n, s), es)) return CCV_E_SHAPE;
  return !written || non_overlapping(n, s) ? CCV_OK : CCV_E_LAYOUT;
}

int check_common(int64_t n0, int64_t n1, int64_t width, int x_dtype, int w_dtype, float eps) {
  if (n0 < 0 || n1 < 0 || width < 0 || width > INT32_MAX / 2) return CCV_E_SHAPE;
  if (x_dtype < 0 || x_dtype > 2 || w_dtype < 0 || w_dtype > 2) return CCV_E_DTYPE;
  if (!(eps >= 0.0f) || isinf(eps)) return CCV_E_UNSUPPORTED;
  int64_t rows;
  return __builtin_mul_overflow(n0, n1, &rows) || rows > INT32_MAX ? CCV_E_SHAPE : CCV_OK;
}

// Whether row (i, j) lies at (i n1 + j) s[1], as far as there are such rows; one group of rows, or
// groups of one, then take the stride that counts.
bool flat(const int64_t s[2], int64_t n0, int64_t n1) { return n0 <= 1 || n1 <= 1 || s[0] == n1 * s[1]; }

int validate_fwd(const ccv_norm_fwd_args_t* p, NormArgs* a) {
  if (!p) return CCV_E_NULL;
  if (p->struct_size != (int64_t)sizeof(ccv_norm_fwd_args_t)) return CCV_E_ABI;
  int st = check_common(p->n0, p->n1, p->width, p->x_dtype, p->w_dtype, p->eps);
  if (st != CCV_OK) return st;
  *a = NormArgs{};
  if (p->n0 * p->n1 == 0 || p->width == 0) return CCV_OK;
  if (!p->x || !p->out) return CCV_E_NULL;
  const int es = elt_size(p->x_dtype);
  const Rows x{p->x, p->x_stride}, o{p->out, p->out_stride};
  if ((st = check_rows(x, p->n0, p->n1, p->width, es, false)) != CCV_OK) return st;
  if ((st = check_rows(o, p->n0, p->n1, p->width, es, true)) != CCV_OK) return st;
  for (const void* q : {(const void*)p->out, (const void*)p->mean, (const void*)p->rstd})
    if (q && (q == p->x || q == p->weight || q == p->bias)) return CCV_E_ALIAS;
  if ((p->mean && (p->mean == p->rstd || p->mean == p->out)) || (p->rstd && p->rstd == p->out)) return CCV_E_ALIAS;
  a->x = p->x;
  a->w = p->weight;
  a->b = p->bias;
  a->out = p->out;
  a->mean = p->mean;
  a->rstd = p->rstd;
  for (int i = 0; i < 2; ++i) {
    a->x_s[i] = p->x_stride[i];
    a->o_s[i] = p->out_stride[i];
  }
  a->rows = p->n0 * p->n1;
  a->n1 = (uint32_t)p->n1;
  if (flat(a->x_s, p->n0, p->n1) && flat(a->o_s, p->n0, p->n1)) {
    a->n1 = 0;
    if (p->n1 == 1) {
      a->x_s[1] = a->x_s[0];
      a->o_s[1] = a->o_s[0];
    }
  }
  a->width = (int32_t)p->width;
  a->x_dtype = p->x_dtype;
  a->w_dtype = p->w_dtype;
  a->eps = p->eps;
  return CCV_OK;
}

int validate_bwd(const ccv_norm_bwd_args_t* p, NormArgs* a, int64_t* bytes, bool with_ws) {
  if (!p) return CCV_E_NULL;
  if (p->struct_size != (int64_t)sizeof(ccv_norm_bwd_args_t)) return CCV_E_ABI;
  int st = check_common(p->n0, p->n1, p->width, p->x_dtype, p->w_dtype, 0.0f);
  if (st != CCV_OK) return st;
  *a = NormArgs{};
  *bytes = 0;
  if (p->width == 0) return CCV_OK;
  const int64_t rows = p->n0 * p->n1;
  const int es = elt_size(p->x_dtype);
  if (rows > 0) {
    if (!p->x || !p->dout || !p->mean || !p->rstd) return CCV_E_NULL;
    const Rows x{p->x, p->x_stride}, d{p->dout, p->dout_stride}, o{p->dx, p->dx_stride};
    if ((st = check_rows(x, p->n0, p->n1, p->width, es, false)) != CCV_OK) return st;
    if ((st = check_rows(d, p->n0, p->n1, p->width, es, false)) != CCV_OK) return st;
    if (p->dx) {
      if ((st = check_rows(o, p->n0, p->n1, p->width, es, true)) != CCV_OK) return st;
    }
  }
  const void* written[] = {p->dx, p->dweight, p->dbias};
  for (int i = 0; i < 3; ++i) {
    if (!written[i]) continue;
    for (const void* q : {p->x, p->weight, p->dout, (const void*)p->mean, (const void*)p->rstd})
      if (q == written[i]) return CCV_E_ALIAS;
    for (int j = 0; j < i; ++j)
      if (written[j] == written[i]) return CCV_E_ALIAS;
  }
  a->x = p->x;
  a->w = p->weight;
  a->dout = p->dout;
  a->dx = p->dx;
  a->dw = p->dweight;
  a->db = p->dbias;
  a->mean = const_cast<float*>(p->mean);
  a->rstd = const_cast<float*>(p->rstd);
  for (int i = 0; i < 2; ++i) {
    a->x_s[i] = p->x_stride[i];
    a->do_s[i] = p->dout_stride[i];
    a->dx_s[i] = p->dx_stride[i];
  }
  a->rows = rows;
  a->n1 = p->n1 > 0 ? (uint32_t)p->n1 : 1;
  if (flat(a->x_s, p->n0, p->n1) && flat(a->do_s, p->n0, p->n1) && (!p->dx || flat(a->dx_s, p->n0, p->n1))) {
    a->n1 = 0;
    if (p->n1 == 1) {
      a->x_s[1] = a->x_s[0];
      a->do_s[1] = a->do_s[0];
      a->dx_s[1] = a->dx_s[0];
    }
  }
  a->width = (int32_t)p->width;
  a->x_dtype = p->x_dtype;
  a->w_dtype = p->w_dtype;
  if (p->dweight || p->dbias) {
    const NormShape s = norm_shape(p->width, es);
    const int64_t per = s.lanes && s.lanes < 256 ? 256 / s.lanes : 1, need = (rows + per - 1) / per;
    // rows walked by one workgroup share a partial row; the column sums of very wide rows take 64
    const int64_t most = s.lanes ? std::max(kGroups, (need + kNormRows - 1) / kNormRows) : p->width * es < 16 ? kGroups : 64;
    a->groups = (int32_t)(need < most ? need : most);
    *bytes = (int64_t)a->groups * 2 * p->width * 4;
    if (with_ws && *bytes) {
      if (!p->workspace) return CCV_E_NULL;
      if (!aligned16(p->workspace)) return CCV_E_LAYOUT;
      if (p->workspace_bytes < *bytes) return CCV_E_SHAPE;
    }
    a->part = static_cast<float*>(p->workspace);
  } else {
    a->groups = (int32_t)(rows < kGroups ? rows : kGroups);
  }
  return CCV_OK;
}

// ---- group norm

int check_group_rows(const void* p, int64_t s, int64_t rows, int64_t C, int es, bool written) {
  if (!p) return CCV_OK;
  const int64_t st[2] = {0, s};
  return check_rows(Rows{p, st}, 1, rows, C, es, written);
}

int check_group_common(int64_t rows, int64_t groups, int64_t width, int x_dtype, int w_dtype, int activation, float eps) {
  if (rows < 0 || groups < 1 || width < 0 || rows > INT32_MAX || groups > (1 << 24) || width > (1 << 24) || groups * width > (1 << 24)) return CCV_E_SHAPE;
  if (x_dtype < 0 || x_dtype > 2 || w_dtype < 0 || w_dtype > 2) return CCV_E_DTYPE;
  if (activation != CCV_ACT_NONE && activation != CCV_ACT_SILU) return CCV_E_UNSUPPORTED;
  return !(eps >= 0.0f) || isinf(eps) ? CCV_E_UNSUPPORTED : CCV_OK;
}

// Walkers of a group: with `slots` groups under way a workgroup and about `blocks` workgroups; `least` rows each.
int32_t group_walkers(int64_t rows, int64_t groups, int64_t slots, int64_t blocks, int64_t least) {
  const int64_t most = std::max<int64_t>(1, blocks * slots / groups), need = (rows + least - 1) / least;
  return (int32_t)std::max<int64_t>(1, std::min(most, need));
}

int validate_group_fwd(const ccv_group_norm_fwd_args_t* p, GroupNormArgs* a) {
  if (!p) return CCV_E_NULL;
  if (p->struct_size != (int64_t)sizeof(ccv_group_norm_fwd_args_t)) return CCV_E_ABI;
  int st = check_group_common(p->rows, p->groups, p->width, p->x_dtype, p->w_dtype, p->activation, p->eps);
  if (st != CCV_OK) return st;
  *a = GroupNormArgs{};
  if (p->rows == 0 || p->width == 0) return CCV_OK;
  if (!p->x || !p->out) return CCV_E_NULL;
  const int es = elt_size(p->x_dtype);
  const int64_t C = p->groups * p->width;
  if ((st = check_group_rows(p->x, p->x_stride, p->rows, C, es, false)) != CCV_OK) return st;
  if ((st = check_group_rows(p->gate, p->gate_stride, p->rows, C, es, false)) != CCV_OK) return st;
  if ((st = check_group_rows(p->out, p->out_stride, p->rows, C, es, true)) != CCV_OK) return st;
  const void* written[] = {p->out, p->mean, p->rstd};
  for (int i = 0; i < 3; ++i) {
    if (!written[i]) continue;
    for (const void* q : {p->x, p->weight, p->bias, p->gate})
      if (q == written[i]) return CCV_E_ALIAS;
    for (int j = 0; j < i; ++j)
      if (written[j] == written[i]) return CCV_E_ALIAS;
  }
  a->x = p->x;
  a->w = p->weight;
  a->b = p->bias;
  a->z = p->gate;
  a->out = p->out;
  a->mean = p->mean;
  a->rstd = p->rstd;
  a->x_s = p->x_stride;
  a->z_s = p->gate_stride;
  a->o_s = p->out_stride;
  a->rows = p->rows;
  a->groups = (int32_t)p->groups;
  a->width = (int32_t)p->width;
  a->x_dtype = p->x_dtype;
  a->w_dtype = p->w_dtype;
  a->silu = p->activation == CCV_ACT_SILU;
  a->eps = p->eps;
  return CCV_OK;
}

int validate_group_bwd(const ccv_group_norm_bwd_args_t* p, GroupNormArgs* a, int64_t* bytes, bool with_ws) {
  if (!p) return CCV_E_NULL;
  if (p->struct_size != (int64_t)sizeof(ccv_group_norm_bwd_args_t)) return CCV_E_ABI;
  int st = check_group_common(p->rows, p->groups, p->width, p->x_dtype, p->w_dtype, p->activation, 0.0f);
  if (st != CCV_OK) return st;
  *a = GroupNormArgs{};
  *bytes = 0;
  if (p->dgate && !p->gate && p->rows > 0) return CCV_E_UNSUPPORTED;
  if (p->width == 0) return CCV_OK;
  const int es = elt_size(p->x_dtype);
  const int64_t C = p->groups * p->width;
  if (p->rows > 0) {
    if (!p->x || !p->dout || !p->mean || !p->rstd) return CCV_E_NULL;
    if ((st = check_group_rows(p->x, p->x_stride, p->rows, C, es, false)) != CCV_OK) return st;
    if ((st = check_group_rows(p->gate, p->gate_stride, p->rows, C, es, false)) != CCV_OK) return st;
    if ((st = check_group_rows(p->dout, p->dout_stride, p->rows, C, es, false)) != CCV_OK) return st;
    if ((st = check_group_rows(p->dx, p->dx_stride, p->rows, C, es, true)) != CCV_OK) return st;
    if ((st = check_group_rows(p->dgate, p->dgate_stride, p->rows, C, es, true)) != CCV_OK) return st;
  }
  const void* written[] = {p->dx, p->dgate, p->dweight, p->dbias};
  for (int i = 0; i < 4; ++i) {
    if (!written[i]) continue;
    for (const void* q : {p->x, p->weight, p->bias, p->gate, p->dout, (const void*)p->mean, (const void*)p->rstd})
      if (q == written[i]) return CCV_E_ALIAS;
    for (int j = 0; j < i; ++j)
      if (written[j] == written[i]) return CCV_E_ALIAS;
  }
  a->x = p->x;
  a->w = p->weight;
  a->b = p->bias;
  a->z = p->gate;
  a->dout = p->dout;
  a->dx = p->dx;
  a->dz = p->dgate;
  a->dw = p->dweight;
  a->db = p->dbias;
  a->mean = const_cast<float*>(p->mean);
  a->rstd = const_cast<float*>(p->rstd);
  a->x_s = p->x_stride;
  a->z_s = p->gate_stride;
  a->do_s = p->dout_stride;
  a->dx_s = p->dx_stride;
  a->dz_s = p->dgate_stride;
  a->rows = p->rows;
  a->groups = (int32_t)p->groups;
  a->width = (int32_t)p->width;
  a->x_dtype = p->x_dtype;
  a->w_dtype = p->w_dtype;
  a->silu = p->activation == CCV_ACT_SILU;
  const NormShape s = group_norm_shape(p->width, es);
  if (p->rows == 0) {
    a->walkers = 0;
  } else if (s.lanes) {
    // no more than a launch has threads for, at least 128; such calls' arrays are larger than the memory
    const int64_t most = ((int64_t)1 << 31) / (p->groups * s.lanes);
    a->walkers = std::max(group_walkers(p->rows, p->groups, 256 / s.lanes, kGroups, 4), (int32_t)((p->rows + kNormRows - 1) / kNormRows));
    a->walkers = (int32_t)std::min<int64_t>(a->walkers, most);
  } else {
    a->walkers = (int32_t)std::min<int64_t>(p->rows, 64);
  }
  if (p->dweight || p->dbias) {
    *bytes = (int64_t)a->walkers * 2 * C * 4;
    if (with_ws && *bytes) {
      if (!p->workspace) return CCV_E_NULL;
      if (!aligned16(p->workspace)) return CCV_E_LAYOUT;
      if (p->workspace_bytes < *bytes) return CCV_E_SHAPE;
    }
    a->part = static_cast<float*>(p->workspace);
  }
  return CCV_OK;
}

int validate_tables(const ccv_seq_tables_args_t* p, TablesArgs* a) {
  if (!p) return CCV_E_NULL;
  if (p->struct_size != (int64_t)sizeof(ccv_seq_tables_args_t)) return CCV_E_ABI;
  if (p->N < 0 || p->total < 0 || p->N > INT32_MAX - 1024 || p->total > INT32_MAX - 8192) return CCV_E_SHAPE;
  if ((p->N > 0 && !p->lengths) || !p->cu_seqlens) return CCV_E_NULL;
  const void* w[] = {p->cu_seqlens, p->seq_idx, p->positions};
  for (int i = 0; i < 3; ++i) {
    if (w[i] && w[i] == p->lengths) return CCV_E_ALIAS;
    for (int j = 0; j < i; ++j)
      if (w[i] && w[i] == w[j]) return CCV_E_ALIAS;
  }
  *a = TablesArgs{p->lengths, p->cu_seqlens, p->seq_idx, p->positions, p->N, p->total};
  return CCV_OK;
}

}  // namespace

extern "C" {

int ccv_norm_fwd_check(const ccv_norm_fwd_args_t* args) {
  NormArgs a;
  return validate_fwd(args, &a);
}

int ccv_norm_fwd(const ccv_norm_fwd_args_t* args, void* hip_stream) {
  NormArgs a;
  const int st = validate_fwd(args, &a);
  if (st != CCV_OK || a.rows == 0) return st;
  const int cus = device_cu_count(hip_stream);
  if (cus < 0) return CCV_E_HIP;
  return launch_norm_fwd(a, cu_count(cus), hip_stream) == 0 ? CCV_OK : CCV_E_HIP;
}

int ccv_norm_bwd_check(const ccv_norm_bwd_args_t* args) {
  NormArgs a;
  int64_t bytes;
  return validate_bwd(args, &a, &bytes, true);
}

int64_t ccv_norm_bwd_workspace_size(const ccv_norm_bwd_args_t* args) {
  NormArgs a;
  int64_t bytes;
  const int st = validate_bwd(args, &a, &bytes, false);
  return st != CCV_OK ? st : bytes;
}

int ccv_norm_bwd(const ccv_norm_bwd_args_t* args, void* hip_stream) {
  NormArgs a;
  int64_t bytes;
  const int st = validate_bwd(args, &a, &bytes, true);
  if (st != CCV_OK || a.width == 0) return st;
  if (a.rows == 0 && !a.dw && !a.db) return CCV_OK;
  return launch_norm_bwd(a, hip_stream) == 0 ? CCV_OK : CCV_E_HIP;
}

int ccv_group_norm_fwd_check(const ccv_group_norm_fwd_args_t* args) {
  GroupNormArgs a;
  return validate_group_fwd(args, &a);
}

int ccv_group_norm_fwd(const ccv_group_norm_fwd_args_t* args, void* hip_stream) {
  GroupNormArgs a;
  const int st = validate_group_fwd(args, &a);
  if (st != CCV_OK || a.rows == 0) return st;
  const int cus = device_cu_count(hip_stream);
  if (cus < 0) return CCV_E_HIP;
  const NormShape s = group_norm_shape(a.width, elt_size(a.x_dtype));
  if (s.lanes) a.walkers = group_walkers(a.rows, a.groups, 256 / s.lanes, (int64_t)cu_count(cus) * 8, 1);
  return launch_group_norm_fwd(a, hip_stream) == 0 ? CCV_OK : CCV_E_HIP;
}

int ccv_group_norm_bwd_check(const ccv_group_norm_bwd_args_t* args) {
  GroupNormArgs a;
  int64_t bytes;
  return validate_group_bwd(args, &a, &bytes, true);
}

int64_t ccv_group_norm_bwd_workspace_size(const ccv_group_norm_bwd_args_t* args) {
  GroupNormArgs a;
  int64_t bytes;
  const int st = validate_group_bwd(args, &a, &bytes, false);
  return st != CCV_OK ? st : bytes;
}

int ccv_group_norm_bwd(const ccv_group_norm_bwd_args_t* args, void* hip_stream) {
  GroupNormArgs a;
  int64_t bytes;
  const int st = validate_group_bwd(args, &a, &bytes, true);
  if (st != CCV_OK || a.width == 0) return st;
  if (!a.dw && !a.db && (a.rows == 0 || (!a.dx && !a.dz))) return CCV_OK;
  return launch_group_norm_bwd(a, hip_stream) == 0 ? CCV_OK : CCV_E_HIP;
}

int ccv_seq_tables_check(const ccv_seq_tables_args_t* args) {
  TablesArgs a;
  return validate_tables(args, &a);
}

int ccv_seq_tables(const ccv_seq_tables_args_t* args, void* hip_stream) {
  TablesArgs a;
  const int st = validate_tables(args, &a);
  if (st != CCV_OK) return st;
  return launch_tables(a, hip_stream) == 0 ? CCV_OK : CCV_E_HIP;
}

}  // extern "C"
