// ccv_rotary_api.cpp -- C ABI of rotary positions: argument checks and the launch.  The operation is
// stated in ccv.h beside ccv_rotary.  Host code; nothing here touches a device except the launch.
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "ccv.h"
#include "ccv_checks.hpp"
#include "ccv_rotary_launch.hpp"

namespace {

using namespace ccv;
using namespace ccv::checks;

// A [B, L, H, D] array with unit stride inside a head.
int check_heads(const int64_t s[3], int64_t B, int64_t L, int64_t H, int64_t D, int es, bool written) {
  for (int i = 0; i < 3; ++i)
    if (s[i] < 0) return CCV_E_LAYOUT;
  const int64_t n[3] = {B, L, H};
  int64_t reach = max_offset(n, s);
  if (reach < 0 || __builtin_add_overflow(reach, D - 1, &reach) || !fits_bytes(reach, es)) return CCV_E_SHAPE;
  if (!written) return CCV_OK;
  // four dimensions: the head's elements lie before every other stride, and those are checked in its units
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && s[i] < D) return CCV_E_LAYOUT;
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int p, int q) { return s[p] < s[q]; });
  int64_t used = D - 1;
  for (int i = 0; i < 3; ++i) {
    const int d = order[i];
    if (n[d] <= 1) continue;
    if (s[d] <= used) return CCV_E_LAYOUT;
    used += (n[d] - 1) * s[d];
  }
  return CCV_OK;
}

int validate(const ccv_rotary_args_t* p, RotaryArgs* a) {
  if (!p) return CCV_E_NULL;
  if (p->struct_size != (int64_t)sizeof(ccv_rotary_args_t)) return CCV_E_ABI;
  *a = RotaryArgs{};
  if (p->B < 0 || p->L < 0 || p->Hq < 0 || p->Hk < 0 || p->D < 1 || p->turned < 0 || p->turned > p->D || p->turned % 2) return CCV_E_SHAPE;
  if (p->D > 2048) return CCV_E_UNSUPPORTED;
  if (p->Hq > 65536 || p->Hk > 65536) return CCV_E_SHAPE;
  if (p->x_dtype < 0 || p->x_dtype > 2) return CCV_E_DTYPE;
  if ((p->interleaved != 0 && p->interleaved != 1) || (p->inverse != 0 && p->inverse != 1) || !isfinite(p->scale)) return CCV_E_UNSUPPORTED;
  int64_t tokens;
  if (__builtin_mul_overflow(p->B, p->L, &tokens) || tokens > INT32_MAX) return CCV_E_SHAPE;
  if (tokens == 0 || p->Hq + p->Hk == 0) return CCV_OK;
  const int es = elt_size(p->x_dtype);
  const int64_t heads[2] = {p->Hq, p->Hk};
  const void* in[2] = {p->q, p->k};
  void* out[2] = {p->q_out, p->k_out};
  const int64_t *in_s[2] = {p->q_stride, p->k_stride}, *out_s[2] = {p->q_out_stride, p->k_out_stride};
  bool in_place = true;
  for (int i = 0; i < 2; ++i) {
    if (heads[i] == 0) continue;
    if (!in[i] || !out[i]) return CCV_E_NULL;
    int st = check_heads(in_s[i], p->B, p->L, heads[i], p->D, es, false);
    if (st == CCV_OK) st = check_heads(out_s[i], p->B, p->L, heads[i], p->D, es, true);
    if (st != CCV_OK) return st;
    if (out[i] == in[i]) {
      const int64_t n[3] = {p->B, p->L, heads[i]};
      for (int d = 0; d < 3; ++d)
        if (n[d] > 1 && in_s[i][d] != out_s[i][d]) return CCV_E_ALIAS;
    } else {
      in_place = false;
    }
    if (out[i] == p->positions || out[i] == p->frequencies) return CCV_E_ALIAS;
  }
  if (p->Hq && p->Hk && (p->q_out == p->k_out || p->q_out == p->k || p->k_out == p->q)) return CCV_E_ALIAS;
  const int64_t pn[3] = {1, p->B, p->L}, ps[3] = {0, p->pos_stride[0], p->pos_stride[1]};
  if (p->turned > 0) {
    if (!p->positions || !p->frequencies) return CCV_E_NULL;
    if (ps[1] < 0 || ps[2] < 0) return CCV_E_LAYOUT;
    if (!fits_bytes(max_offset(pn, ps), 4)) return CCV_E_SHAPE;
  }
  for (int i = 0; i < 2; ++i) {
    a->in[i] = in[i];
    a->out[i] = out[i];
    a->heads[i] = (int32_t)heads[i];
    for (int d = 0; d < 3; ++d) {
      a->in_s[i][d] = in_s[i][d];
      a->out_s[i][d] = out_s[i][d];
    }
  }
  a->pos = p->positions;
  a->pos_s[0] = p->pos_stride[0];
  a->pos_s[1] = p->pos_stride[1];
  a->freq = p->frequencies;
  a->tokens = tokens;
  a->L = (int32_t)p->L;
  a->D = (int32_t)p->D;
  a->half = (int32_t)(p->turned / 2);
  a->x_dtype = p->x_dtype;
  a->interleaved = p->interleaved;
  a->scale = p->scale;
  a->sign = p->inverse ? -1.0f : 1.0f;
  // Vectors where each part of a head holds one; a part that is no multiple ends with a vector that shares elements with the
  // one before, which an array turned in place does not bear.
  const bool some_in_place = (p->Hq && p->q == p->q_out) || (p->Hk && p->k == p->k_out);
  const int v = 16 / es, turned = p->interleaved ? 2 * a->half : a->half, rest = a->D - 2 * a->half;
  const auto whole = [&](int n) { return n == 0 || (n >= v && (n % v == 0 || !some_in_place)); };
  int units = 0;
  if (whole(turned) && (in_place || whole(rest))) {
    a->turned_units = (turned + v - 1) / v;
    units = a->turned_units + (in_place ? 0 : (rest + v - 1) / v);
    if (units <= 256) a->units = units;
  }
  a->in_place = in_place;
  // about four units a thread, as far as the angles fit
  const int64_t each = (int64_t)std::max(a->units, 1) * (heads[0] + heads[1]);
  const int64_t span = a->units ? std::max<int64_t>(1, 1024 / each) : std::max<int64_t>(1, 2048 / ((int64_t)a->D * (heads[0] + heads[1])));
  a->span = (int32_t)std::min<int64_t>(span, kRotaryAngles / std::max(a->half, 1));
  if ((tokens + a->span - 1) / a->span >= (int64_t)1 << 24) return CCV_E_SHAPE;      // a launch has fewer than 2^32 threads
  if (units == 0 && in_place && turned == 0) a->tokens = 0;      // nothing is turned and nothing is copied
  return CCV_OK;
}

}  // namespace

extern "C" {

int ccv_rotary_check(const ccv_rotary_args_t* args) {
  RotaryArgs a;
  return validate(args, &a);
}

int ccv_rotary(const ccv_rotary_args_t* args, void* hip_stream) {
  RotaryArgs a;
  const int st = validate(args, &a);
  if (st != CCV_OK || a.tokens == 0 || a.heads[0] + a.heads[1] == 0) return st;
  return launch_rotary(a, hip_stream) == 0 ? CCV_OK : CCV_E_HIP;
}

}  // extern "C"
