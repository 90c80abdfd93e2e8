// ccv_linrec_api.cpp -- C ABI of the gated linear recurrence: argument checks, workspace layout and
// launches.  The operation is stated in ccv.h beside ccv_linrec_fwd.  Host code; nothing here
// touches a device except the launches.
#include <stdint.h>

#include <algorithm>
#include <initializer_list>

#include "ccv.h"
#include "ccv_checks.hpp"
#include "ccv_launch.hpp"
#include "ccv_linrec_launch.hpp"

namespace {

using namespace ccv;
using namespace ccv::checks;

constexpr int64_t kMostBlocks = ((int64_t)1 << 32) / 512 - 1;      // a launch has fewer than 2^32 threads
constexpr int64_t kMostStep = (int64_t)32 << 20;                   // bytes between steps: a lane's offsets are 32-bit
constexpr int64_t kTicketWords = kLrQueues * kLrTicketWords;

// A [B, L, C] array with unit stride along the channels.
int check_steps(const int64_t s[2], int64_t B, int64_t L, int64_t C, int es, bool written) {
  if (s[0] < 0 || s[1] < 0) return CCV_E_LAYOUT;
  const int64_t n[3] = {B, L, C}, st[3] = {s[0], s[1], 1};
  if (!fits_bytes(max_offset(n, st), es)) return CCV_E_SHAPE;
  if (L > 1 && s[1] > kMostStep / es) return CCV_E_LAYOUT;
  return !written || non_overlapping(n, st) ? CCV_OK : CCV_E_LAYOUT;
}

// Rows of C states.
int check_states(const void* p, int64_t s, int64_t rows, int64_t C, bool written) {
  if (!p) return CCV_OK;
  if (s < 0) return CCV_E_LAYOUT;
  const int64_t n[3] = {1, rows, C}, st[3] = {0, s, 1};
  if (!fits_bytes(max_offset(n, st), 4)) return CCV_E_SHAPE;
  return !written || non_overlapping(n, st) ? CCV_OK : CCV_E_LAYOUT;
}

int check_sizes(int64_t B, int64_t L, int64_t C, int64_t N, const void* cu, int x_dtype, int g_dtype, int normalize) {
  if (B < 0 || L < 0 || C < 0 || N < 0 || L > INT32_MAX - 8192 || C > (1 << 24) || B > INT32_MAX || N > INT32_MAX - 8192) return CCV_E_SHAPE;
  if (x_dtype < 0 || x_dtype > 2 || g_dtype < 0 || g_dtype > 2) return CCV_E_DTYPE;
  if (normalize != 0 && normalize != 1) return CCV_E_UNSUPPORTED;
  if (cu ? B != 1 : N != 0) return CCV_E_SHAPE;
  return CCV_OK;
}

int64_t ceil_div(int64_t n, int64_t d) { return (n + d - 1) / d; }

// Division by an invariant as Granlund and Montgomery (1994) have it: exact for all 32-bit n.
LrDivisor divisor(uint32_t d) {
  uint32_t l = 0;
  while (l < 32 && ((uint64_t)1 << l) < d) ++l;
  return {(uint32_t)((((((uint64_t)1 << l) - d) << 32) / d) + 1), l < 1 ? l : 1, l > 0 ? l - 1 : 0};
}

// The tiles of a walk and the words that they need; false when there are too many.
bool tile(LinrecArgs* a, int64_t* words) {
  *words = 0;
  if (a->L == 0) return true;                  // no tiles, however many rows and channels
  const int64_t tiles = ceil_div(a->L, kLrTile), cblocks = ceil_div(a->C, kLrChannels);
  int64_t chains, blocks;
  if (__builtin_mul_overflow(a->B, cblocks, &chains) || __builtin_mul_overflow(chains, tiles, &blocks) || blocks > kMostBlocks) return false;
  a->tiles = (uint32_t)tiles;
  a->cblocks = (uint32_t)cblocks;
  a->chains = (uint32_t)chains;
  a->queues = (uint32_t)std::min<int64_t>(chains, kLrQueues);
  a->fewer = a->chains / a->queues;
  a->longer = a->chains % a->queues;
  a->by_more = divisor(a->fewer + 1);
  a->by_fewer = divisor(a->fewer);
  a->by_cblocks = divisor(a->cblocks);
  a->groups = (uint32_t)ceil_div(tiles, kLrGroup);
  a->stretches = (uint32_t)ceil_div(a->groups, kLrStretch);
  *words = tiles > 1 ? kTicketWords + (blocks + chains * (a->groups + a->stretches)) * kLrChannels : 0;
  return true;
}

int64_t align16(int64_t n) { return (n + 15) & ~(int64_t)15; }

bool hits(const void* w, std::initializer_list<const void*> others) {
  for (const void* q : others)
    if (w && w == q) return true;
  return false;
}

int validate_fwd(const ccv_linrec_fwd_args_t* p, LinrecArgs* a, int64_t* bytes, bool with_ws) {
  if (!p) return CCV_E_NULL;
  if (p->struct_size != (int64_t)sizeof(ccv_linrec_fwd_args_t)) return CCV_E_ABI;
  int st = check_sizes(p->B, p->L, p->C, p->N, p->cu_seqlens, p->x_dtype, p->g_dtype, p->normalize);
  if (st != CCV_OK) return st;
  *a = LinrecArgs{};
  *bytes = 0;
  const int64_t seqs = p->cu_seqlens ? p->N : p->B;
  if (p->C == 0 || p->B == 0) return CCV_OK;
  if (p->L > 0 && (!p->x || !p->g || !p->out)) return CCV_E_NULL;
  const int xs = elt_size(p->x_dtype), gs = elt_size(p->g_dtype);
  if (p->L > 0) {
    if ((st = check_steps(p->x_stride, p->B, p->L, p->C, xs, false)) != CCV_OK) return st;
    if ((st = check_steps(p->g_stride, p->B, p->L, p->C, gs, false)) != CCV_OK) return st;
    if ((st = check_steps(p->out_stride, p->B, p->L, p->C, xs, true)) != CCV_OK) return st;
  }
  if ((st = check_states(p->initial_state, p->init_stride, seqs, p->C, false)) != CCV_OK) return st;
  if ((st = check_states(p->final_state, p->final_stride, seqs, p->C, true)) != CCV_OK) return st;
  if (p->final_state && p->final_state == p->initial_state && seqs > 1 && p->final_stride != p->init_stride) return CCV_E_ALIAS;
  if (hits(p->out, {p->x, p->g, p->cu_seqlens, p->initial_state, p->final_state, p->carries})) return CCV_E_ALIAS;
  if (hits(p->final_state, {p->x, p->g, p->cu_seqlens, p->carries}) || hits(p->carries, {p->x, p->g, p->cu_seqlens, p->initial_state}))
    return CCV_E_ALIAS;
  a->x = p->x;
  a->g = p->g;
  a->out = p->out;
  for (int i = 0; i < 2; ++i) {
    a->x_s[i] = p->x_stride[i];
    a->g_s[i] = p->g_stride[i];
    a->o_s[i] = p->out_stride[i];
  }
  a->init = p->initial_state;
  a->init_s = p->init_stride;
  a->final = p->final_state;
  a->final_s = p->final_stride;
  a->cu = p->cu_seqlens;
  a->carries = p->carries;
  a->B = p->B;
  a->L = p->L;
  a->C = p->C;
  a->nseq = p->N;
  a->x_dtype = p->x_dtype;
  a->g_dtype = p->g_dtype;
  a->normalize = p->normalize;
  if (!tile(a, &a->clear_count)) return CCV_E_SHAPE;
  const int64_t sid = p->cu_seqlens ? 4 * p->L : 0;
  *bytes = 8 * a->clear_count + sid;
  if (with_ws && *bytes) {
    if (!p->workspace) return CCV_E_NULL;
    if (!aligned16(p->workspace)) return CCV_E_LAYOUT;
    if (p->workspace_bytes < *bytes) return CCV_E_SHAPE;
  }
  a->clear = a->ticket = static_cast<uint64_t*>(p->workspace);
  if (p->workspace) {
    a->words = a->ticket + kTicketWords;
    if (sid) a->sid = reinterpret_cast<int32_t*>(static_cast<char*>(p->workspace) + 8 * a->clear_count);
  }
  return CCV_OK;
}

// a: the backward's walk; f: the forward's, which makes the carries where none are given.
int validate_bwd(const ccv_linrec_bwd_args_t* p, LinrecArgs* a, LinrecArgs* f, int64_t* bytes, bool with_ws) {
  if (!p) return CCV_E_NULL;
  if (p->struct_size != (int64_t)sizeof(ccv_linrec_bwd_args_t)) return CCV_E_ABI;
  int st = check_sizes(p->B, p->L, p->C, p->N, p->cu_seqlens, p->x_dtype, p->g_dtype, p->normalize);
  if (st != CCV_OK) return st;
  if (p->dinitial_state && !p->initial_state) return CCV_E_UNSUPPORTED;
  *a = LinrecArgs{};
  *bytes = 0;
  const int64_t seqs = p->cu_seqlens ? p->N : p->B;
  if (p->C == 0 || p->B == 0) return CCV_OK;
  if (p->L > 0 && (!p->x || !p->g || !p->dout || !p->dx || !p->dg)) return CCV_E_NULL;
  const int xs = elt_size(p->x_dtype), gs = elt_size(p->g_dtype);
  if (p->L > 0) {
    if ((st = check_steps(p->x_stride, p->B, p->L, p->C, xs, false)) != CCV_OK) return st;
    if ((st = check_steps(p->g_stride, p->B, p->L, p->C, gs, false)) != CCV_OK) return st;
    if ((st = check_steps(p->dout_stride, p->B, p->L, p->C, xs, false)) != CCV_OK) return st;
    if ((st = check_steps(p->dx_stride, p->B, p->L, p->C, xs, true)) != CCV_OK) return st;
    if ((st = check_steps(p->dg_stride, p->B, p->L, p->C, gs, true)) != CCV_OK) return st;
  }
  if ((st = check_states(p->initial_state, p->init_stride, seqs, p->C, false)) != CCV_OK) return st;
  if ((st = check_states(p->dfinal_state, p->dfinal_stride, seqs, p->C, false)) != CCV_OK) return st;
  if ((st = check_states(p->dinitial_state, p->dinit_stride, seqs, p->C, true)) != CCV_OK) return st;
  const auto inputs = {p->x, p->g, p->dout, (const void*)p->cu_seqlens, (const void*)p->initial_state, (const void*)p->dfinal_state, (const void*)p->carries};
  if (hits(p->dx, inputs) || hits(p->dg, inputs) || hits(p->dinitial_state, inputs) || hits(p->dx, {p->dg, p->dinitial_state}) || hits(p->dg, {p->dinitial_state}))
    return CCV_E_ALIAS;
  a->x = p->x;
  a->g = p->g;
  a->dout = p->dout;
  a->dx = p->dx;
  a->dg = p->dg;
  for (int i = 0; i < 2; ++i) {
    a->x_s[i] = p->x_stride[i];
    a->g_s[i] = p->g_stride[i];
    a->do_s[i] = p->dout_stride[i];
    a->dx_s[i] = p->dx_stride[i];
    a->dg_s[i] = p->dg_stride[i];
  }
  a->init = p->initial_state;
  a->init_s = p->init_stride;
  a->dfinal = p->dfinal_state;
  a->df_s = p->dfinal_stride;
  a->dinit = p->dinitial_state;
  a->di_s = p->dinit_stride;
  a->cu = p->cu_seqlens;
  a->carries = const_cast<float*>(p->carries);
  a->B = p->B;
  a->L = p->L;
  a->C = p->C;
  a->nseq = p->N;
  a->x_dtype = p->x_dtype;
  a->g_dtype = p->g_dtype;
  a->normalize = p->normalize;
  *f = *a;
  int64_t words, more = 0;
  if (!tile(a, &words) || (!p->carries && !tile(f, &more))) return CCV_E_SHAPE;
  a->clear_count = words + more;
  const int64_t sid = p->cu_seqlens ? align16(4 * p->L) : 0, carries = p->carries ? 0 : (int64_t)a->B * a->tiles * a->C * 4;
  *bytes = 8 * a->clear_count + sid + carries;
  if (with_ws && *bytes) {
    if (!p->workspace) return CCV_E_NULL;
    if (!aligned16(p->workspace)) return CCV_E_LAYOUT;
    if (p->workspace_bytes < *bytes) return CCV_E_SHAPE;
  }
  if (char* ws = static_cast<char*>(p->workspace)) {
    a->clear = a->ticket = reinterpret_cast<uint64_t*>(ws);
    a->words = a->ticket + kTicketWords;
    f->ticket = a->ticket + words;
    f->words = f->ticket + kTicketWords;
    if (sid) a->sid = f->sid = reinterpret_cast<int32_t*>(ws + 8 * a->clear_count);
    if (carries) a->carries = f->carries = reinterpret_cast<float*>(ws + 8 * a->clear_count + sid);
  }
  return CCV_OK;
}

int validate_step(const ccv_linrec_update_args_t* p, LinrecStepArgs* a) {
  if (!p) return CCV_E_NULL;
  if (p->struct_size != (int64_t)sizeof(ccv_linrec_update_args_t)) return CCV_E_ABI;
  int st = check_sizes(p->B, p->L, p->C, 0, nullptr, p->x_dtype, p->g_dtype, p->normalize);
  if (st != CCV_OK) return st;
  if (p->slots < 0) return CCV_E_SHAPE;
  *a = LinrecStepArgs{};
  if (p->B == 0 || p->L == 0 || p->C == 0) return CCV_OK;
  if (!p->x || !p->g || !p->out || (!p->state && p->slots > 0)) return CCV_E_NULL;
  if (!p->state_indices && p->B > p->slots) return CCV_E_SHAPE;
  const int xs = elt_size(p->x_dtype), gs = elt_size(p->g_dtype);
  if ((st = check_steps(p->x_stride, p->B, p->L, p->C, xs, false)) != CCV_OK) return st;
  if ((st = check_steps(p->g_stride, p->B, p->L, p->C, gs, false)) != CCV_OK) return st;
  if ((st = check_steps(p->out_stride, p->B, p->L, p->C, xs, true)) != CCV_OK) return st;
  if ((st = check_states(p->state, p->state_stride, p->slots, p->C, true)) != CCV_OK) return st;
  if (hits(p->out, {p->x, p->g, p->state, p->state_indices}) || hits(p->state, {p->x, p->g, p->state_indices})) return CCV_E_ALIAS;
  if ((p->C + 1) / 2 * p->B / 256 >= kMostBlocks) return CCV_E_SHAPE;
  *a = LinrecStepArgs{p->x, p->g, p->out, {p->x_stride[0], p->x_stride[1]}, {p->g_stride[0], p->g_stride[1]},
                      {p->out_stride[0], p->out_stride[1]}, p->state, p->state_stride, p->state_indices,
                      p->B, p->L, p->C, p->slots, p->x_dtype, p->g_dtype, p->normalize};
  return CCV_OK;
}

}  // namespace

extern "C" {

int ccv_linrec_fwd_check(const ccv_linrec_fwd_args_t* args) {
  LinrecArgs a;
  int64_t bytes;
  return validate_fwd(args, &a, &bytes, true);
}

int64_t ccv_linrec_fwd_workspace_size(const ccv_linrec_fwd_args_t* args) {
  LinrecArgs a;
  int64_t bytes;
  const int st = validate_fwd(args, &a, &bytes, false);
  return st != CCV_OK ? st : bytes;
}

int ccv_linrec_fwd(const ccv_linrec_fwd_args_t* args, void* hip_stream) {
  LinrecArgs a;
  int64_t bytes;
  const int st = validate_fwd(args, &a, &bytes, true);
  if (st != CCV_OK || a.B == 0 || a.C == 0) return st;
  if (a.clear_count || a.cu || (a.L == 0 && a.final))
    if (launch_linrec_prepare(a, a.init, a.init_s, a.final, a.final_s, hip_stream)) return CCV_E_HIP;
  if (a.L == 0) return CCV_OK;
  return launch_linrec_fwd(a, hip_stream) == 0 ? CCV_OK : CCV_E_HIP;
}

int ccv_linrec_bwd_check(const ccv_linrec_bwd_args_t* args) {
  LinrecArgs a, f;
  int64_t bytes;
  return validate_bwd(args, &a, &f, &bytes, true);
}

int64_t ccv_linrec_bwd_workspace_size(const ccv_linrec_bwd_args_t* args) {
  LinrecArgs a, f;
  int64_t bytes;
  const int st = validate_bwd(args, &a, &f, &bytes, false);
  return st != CCV_OK ? st : bytes;
}

int ccv_linrec_bwd(const ccv_linrec_bwd_args_t* args, void* hip_stream) {
  LinrecArgs a, f;
  int64_t bytes;
  const int st = validate_bwd(args, &a, &f, &bytes, true);
  if (st != CCV_OK || a.B == 0 || a.C == 0) return st;
  if (a.clear_count || a.cu || (a.L == 0 && a.dinit))
    if (launch_linrec_prepare(a, a.dfinal, a.df_s, a.dinit, a.di_s, hip_stream)) return CCV_E_HIP;
  if (a.L == 0) return CCV_OK;
  if (!args->carries && launch_linrec_fwd(f, hip_stream)) return CCV_E_HIP;
  return launch_linrec_bwd(a, hip_stream) == 0 ? CCV_OK : CCV_E_HIP;
}

int ccv_linrec_update_check(const ccv_linrec_update_args_t* args) {
  LinrecStepArgs a;
  return validate_step(args, &a);
}

int ccv_linrec_update(const ccv_linrec_update_args_t* args, void* hip_stream) {
  LinrecStepArgs a;
  const int st = validate_step(args, &a);
  if (st != CCV_OK || a.B == 0) return st;
  return launch_linrec_step(a, hip_stream) == 0 ? CCV_OK : CCV_E_HIP;
}

}  // extern "C"
