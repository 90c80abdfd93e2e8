// ccv_delta_api.cpp -- C ABI of the gated delta rule: argument checks, the workspace's
// layout and the launches.  The operation and its contract are stated in ccv.h beside
// ccv_delta_fwd, ccv_delta_bwd and ccv_delta_update.  Host code; nothing here touches a
// device except the launches.
#include <stdint.h>

#include <algorithm>

#include "ccv.h"
#include "ccv_checks.hpp"
#include "ccv_delta_launch.hpp"
#include "ccv_launch.hpp"

namespace {

using namespace ccv;
using namespace ccv::checks;

// A strided view: up to four extents with their element strides, outermost first, the
// innermost of unit stride.
struct View {
  const void* p;
  int64_t n[4], s[4];
  int elt;
};

View view(const void* p, int64_t a, int64_t b, int64_t c, int64_t d, const int64_t s[3], int elt) {
  return {p, {a, b, c, d}, {s[0], s[1], s[2], 1}, elt};
}

// A negative stride, or offsets that do not fit.
int check_view(const View& v) {
  int64_t total = 0;
  for (int i = 0; i < 4; ++i) {
    if (v.s[i] < 0) return CCV_E_LAYOUT;
    if (v.n[i] <= 1) continue;
    int64_t p;
    if (__builtin_mul_overflow(v.n[i] - 1, v.s[i], &p) || __builtin_add_overflow(total, p, &total)) return CCV_E_SHAPE;
  }
  return fits_bytes(total, v.elt) ? CCV_OK : CCV_E_SHAPE;
}

// No two indexes share an element, by the sufficient test of checks::non_overlapping.
bool apart(const View& v) {
  int o[4] = {0, 1, 2, 3};
  std::sort(o, o + 4, [&](int p, int q) { return v.s[p] < v.s[q]; });
  int64_t reach = 0;
  for (int i : o) {
    if (v.n[i] <= 1) continue;
    if (v.s[i] <= reach) return false;
    reach += (v.n[i] - 1) * v.s[i];
  }
  return true;
}

int check_written(const View& v) {
  const int st = check_view(v);
  return st != CCV_OK ? st : apart(v) ? CCV_OK : CCV_E_LAYOUT;
}

// Rows of `unit` elements move as whole vectors of `bytes` bytes.
bool vectors(const View& v, int unit, int bytes) {
  if (v.n[3] % unit != 0 || ((uintptr_t)v.p & (uintptr_t)(bytes - 1)) != 0) return false;
  for (int i = 0; i < 3; ++i)
    if (v.n[i] > 1 && (v.s[i] * v.elt) % bytes != 0) return false;
  return true;
}

constexpr int64_t kMostStep = 1 << 25;      // bytes from step to step, so that 64 of them fit 31 bits

// Whether the kernels' buffer loads take the view's rows as they are: steps apart from each
// other and near enough for a 32-bit offset over 64 of them, `unit` elements a load.
bool loadable(const View& v, int unit, int bytes) {
  return vectors(v, unit, bytes) && (v.n[1] <= 1 || (v.s[1] >= v.n[3] && v.s[1] <= kMostStep / v.elt));
}

bool dtype_ok(int d) { return d >= 0 && d <= 2; }
int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Hands out 256-byte aligned pieces of the workspace; with a null base it only measures.
struct Pieces {
  char* base;
  int64_t used;
  bool over;
  template <class T>
  void take(T** p, int64_t count, int64_t each) {
    int64_t n;
    if (__builtin_mul_overflow(count, each, &n) || __builtin_mul_overflow(n, (int64_t)sizeof(T), &n) || n > INT64_MAX / 64) {
      over = true;
      return;
    }
    *p = base ? reinterpret_cast<T*>(base + used) : nullptr;
    if (__builtin_add_overflow(used, round_up(n, 256), &used)) over = true;
  }
};

// The sizes that forward and backward share.
struct Sizes {
  int64_t B, L, N, Hk, Hv, Dk, Dv;
  const int32_t* cu;
  int x_dtype, g_dtype, b_dtype;
};

int check_sizes(const Sizes& z) {
  if (z.B < 0 || z.L < 0 || z.N < 0 || z.Hk < 1 || z.Hv < 1 || z.Dk < 1 || z.Dv < 1) return CCV_E_SHAPE;
  if (z.Hv % z.Hk != 0) return CCV_E_SHAPE;
  if (z.cu ? z.B != 1 : z.N != 0) return CCV_E_SHAPE;
  if (!dtype_ok(z.x_dtype) || !dtype_ok(z.g_dtype) || !dtype_ok(z.b_dtype)) return CCV_E_DTYPE;
  if (z.Dk > kDeltaMaxDk) return CCV_E_UNSUPPORTED;
  const int64_t most = INT32_MAX - 2 * kDeltaChunk;
  if (z.L > most || z.B > most || z.N > most || z.Hv > most || z.Dv > (1 << 20)) return CCV_E_SHAPE;
  return CCV_OK;
}

// What validate leaves to be launched.
struct Work {
  DeltaArgs a;
  int nt;
  int64_t bytes;
  bool chunks, states;     // there are steps; there are states to be written without any
  bool pack[4];            // q, k, v, dout: need a copy before the kernels' loads take them
  void* packed[4];
};

// Fills the counts and the workspace's pieces.
int plan(const Sizes& z, bool bwd, void* ws, Work* out, const bool (&pack)[4]) {
  DeltaArgs* a = &out->a;
  int* nt = &out->nt;
  *a = DeltaArgs{};
  const bool packed = z.cu && z.L > 0;
  a->cu = z.cu;
  a->packed = packed;
  a->L = z.L;
  a->nseq = (int32_t)(z.cu ? z.N : z.B);
  a->chunks_per_row = packed ? 0 : (int32_t)((z.L + kDeltaChunk - 1) / kDeltaChunk);
  const int64_t nch = packed ? z.L / kDeltaChunk + z.N + 1 : z.B * a->chunks_per_row;
  a->Hk = (int32_t)z.Hk;
  a->Hv = (int32_t)z.Hv;
  a->Dk = (int32_t)z.Dk;
  a->Dv = (int32_t)z.Dv;
  a->Dkp = z.Dk <= 64 ? 64 : 128;
  a->Dvp = (int32_t)round_up(z.Dv, 32);
  a->x_dtype = z.x_dtype;
  a->g_dtype = z.g_dtype;
  a->b_dtype = z.b_dtype;
  int64_t heads, groups;
  if (__builtin_mul_overflow(nch, z.Hv, &heads) || heads > INT32_MAX) return CCV_E_SHAPE;
  if (__builtin_mul_overflow((int64_t)a->nseq + 1, z.Hv, &groups) || groups > INT32_MAX / 2) return CCV_E_SHAPE;
  groups = round_up(groups, 8);
  if (groups * (a->Dvp / 16) > INT32_MAX) return CCV_E_SHAPE;
  a->nchunks = (int32_t)nch;
  // key heads enough for the chip's eight dies to get as many each
  a->share = (int64_t)a->nseq * z.Hk >= 64 ? (int32_t)(z.Hv / z.Hk) : 1;
  a->share_prep = nch * z.Hk >= 64 ? (int32_t)(z.Hv / z.Hk) : 1;
  // Which kernels, by the blocks of 16 values that there are: 32 values a workgroup once 16 would be more workgroups
  // than the chip's 256 CUs, whole columns a wave once 32 would be, and in the pass from the end once 16 would be three
  // rounds of them.  Both sides of each bound stand measured beside the kernels (ccv_delta_scan.hip, ccv_delta_bwd.hip).
  const int64_t blocks = (int64_t)a->nseq * z.Hv * (a->Dvp / 16);
  a->waves = z.x_dtype != CCV_F32 && blocks > 512;
  a->waves_back = z.x_dtype == CCV_F16 && blocks > 768;
  *nt = z.x_dtype == CCV_F32 || (bwd && z.x_dtype != CCV_BF16) || blocks <= 256 ? 1 : 2;
  // Few heads: a sequence in parts that run side by side, once for the map of the state that each is and
  // once from the states that these give.  A chunk of the chain costs the same in both, so parts pay
  // where a sequence is several times twice its part: forward, fp32 1 x 2048, one head of 64, parts of 4
  // chunks: 30 us against 58 of the chain; bf16 1 x 8192, 2 heads of 128, parts of 8: 80 against 216;
  // 1 x 32768, 8 heads, parts of 128: 580 against 875.
  const int64_t side = std::max<int64_t>(1, 256 / (z.Hv * (a->Dvp / 16)));
  const int64_t each = std::max<int64_t>(4, (nch + side - 1) / side);
  if (!a->waves && a->nseq > 0 && nch >= 4 * each * a->nseq) {
    a->part_chunks = (int32_t)each;
    a->parts_per_row = packed ? 0 : (int32_t)((a->chunks_per_row + each - 1) / each);
    a->parts = packed ? (int32_t)(nch / each + z.N + 1) : a->nseq * a->parts_per_row;
    *nt = 1;
  }
  a->slices = a->Dvp / (16 * *nt);
  a->qslices = a->waves ? a->Dvp / 16 : a->slices;

  Pieces w{static_cast<char*>(ws), 0, false};
  if (packed) {
    w.take(&a->table, nch, 4);
    w.take(&a->cstart, a->nseq + 2, 2);
    w.take(&a->order, a->nseq + 1, 1);
    if (a->part_chunks) {
      w.take(&a->pstart, a->nseq + 2, 1);
      w.take(&a->ptable, a->parts, 2);
    }
  }
  if (a->part_chunks) w.take(&a->carry, (int64_t)a->parts * z.Hv, (int64_t)a->Dkp * (a->Dkp + a->Dvp));
  w.take(&a->W, heads, kDeltaMatrix);
  w.take(&a->P, heads, kDeltaMatrix);
  w.take(&a->dec, heads, kDeltaDec);
  if (bwd) {
    w.take(&a->WT, heads, kDeltaMatrix);
    w.take(&a->S, heads, (int64_t)a->Dkp * a->Dvp);
    w.take(&a->dS, heads, (int64_t)a->Dkp * a->Dvp);
    w.take(&a->N, heads, 64 * (int64_t)a->Dvp);
    w.take(&a->Y, heads, 64 * (int64_t)a->Dvp);
    w.take(&a->pairs, heads, kDeltaPairs);
    w.take(&a->part, heads, a->slices * kDeltaPart);
    w.take(&a->qpart, heads, a->qslices * 64);
  }
  const int64_t steps = z.B * z.L, wk = z.Hk * round_up(z.Dk, 8), wv = z.Hv * round_up(z.Dv, 8);
  char* p[4] = {};
  for (int i = 0; i < 4; ++i)
    if (pack[i]) w.take(&p[i], steps, (i < 2 ? wk : wv) * elt_size(z.x_dtype));
  if (w.over) return CCV_E_SHAPE;
  for (int i = 0; i < 4; ++i) {
    out->pack[i] = pack[i];
    out->packed[i] = p[i];
  }
  out->bytes = w.used;
  return CCV_OK;
}

void copy3(int64_t to[3], const int64_t from[3]) {
  for (int i = 0; i < 3; ++i) to[i] = from[i];
}

int check_workspace(const void* ws, int64_t given, int64_t need) {
  if (need == 0) return CCV_OK;
  if (!ws) return CCV_E_NULL;
  if (!aligned16(ws)) return CCV_E_LAYOUT;
  return given < need ? CCV_E_SHAPE : CCV_OK;
}

int validate_fwd(const ccv_delta_fwd_args_t* p, Work* w, bool with_ws) {
  if (!p) return CCV_E_NULL;
  if (p->struct_size != (int64_t)sizeof(ccv_delta_fwd_args_t)) return CCV_E_ABI;
  const Sizes z{p->B, p->L, p->N, p->Hk, p->Hv, p->Dk, p->Dv, p->cu_seqlens, p->x_dtype, p->g_dtype, p->beta_dtype};
  int st = check_sizes(z);
  if (st != CCV_OK) return st;
  const int es = elt_size(p->x_dtype);
  const bool pack[4] = {!loadable(view(p->q, p->B, p->L, p->Hk, p->Dk, p->q_stride, es), 8, 16),
                        !loadable(view(p->k, p->B, p->L, p->Hk, p->Dk, p->k_stride, es), 8, 16),
                        !loadable(view(p->v, p->B, p->L, p->Hv, p->Dv, p->v_stride, es), 1, es), false};
  if (p->L > 1 && p->out_stride[1] > kMostStep / es) return CCV_E_LAYOUT;
  st = plan(z, false, with_ws ? p->workspace : nullptr, w, pack);
  if (st != CCV_OK) return st;
  DeltaArgs& a = w->a;
  w->chunks = p->B > 0 && p->L > 0;
  w->states = p->final_state && a.nseq > 0;
  const View q = view(p->q, p->B, p->L, p->Hk, p->Dk, p->q_stride, es), k = view(p->k, p->B, p->L, p->Hk, p->Dk, p->k_stride, es),
             v = view(p->v, p->B, p->L, p->Hv, p->Dv, p->v_stride, es), o = view(p->out, p->B, p->L, p->Hv, p->Dv, p->out_stride, es),
             g = view(p->g, p->B, p->L, p->Hv, 1, p->g_stride, 4), b = view(p->beta, p->B, p->L, p->Hv, 1, p->beta_stride, 4),
             h0 = view(p->initial_state, a.nseq, p->Hv, p->Dk, p->Dv, p->init_stride, 4),
             ht = view(p->final_state, a.nseq, p->Hv, p->Dk, p->Dv, p->final_stride, 4);
  if (w->chunks) {
    if (!p->q || !p->k || !p->v || !p->g || !p->beta || !p->out) return CCV_E_NULL;
    for (const View& x : {q, k, v, g, b})
      if ((st = check_view(x)) != CCV_OK) return st;
    if ((st = check_written(o)) != CCV_OK) return st;
    for (const void* x : {p->q, p->k, p->v, p->g, p->beta, (const void*)p->initial_state, (const void*)p->final_state})
      if (x == p->out) return CCV_E_ALIAS;
  }
  if (p->initial_state && (st = check_view(h0)) != CCV_OK) return st;
  if (p->final_state) {
    if ((st = check_written(ht)) != CCV_OK) return st;
    for (const void* x : {p->q, p->k, p->v, p->g, p->beta})
      if (x == p->final_state) return CCV_E_ALIAS;
    if (p->final_state == p->initial_state)      // in place, element by element
      for (int i = 0; i < 3; ++i)
        if (ht.n[i] > 1 && ht.s[i] != h0.s[i]) return CCV_E_ALIAS;
  }
  if (!w->chunks) w->bytes = 0;
  if (with_ws && (st = check_workspace(p->workspace, p->workspace_bytes, w->bytes)) != CCV_OK) return st;
  a.q = p->q;
  a.k = p->k;
  a.v = p->v;
  a.g = p->g;
  a.beta = p->beta;
  a.out = p->out;
  a.h0 = p->initial_state;
  a.ht = p->final_state;
  copy3(a.q_s, p->q_stride);
  copy3(a.k_s, p->k_stride);
  copy3(a.v_s, p->v_stride);
  copy3(a.g_s, p->g_stride);
  copy3(a.b_s, p->beta_stride);
  copy3(a.o_s, p->out_stride);
  copy3(a.h0_s, p->init_stride);
  copy3(a.ht_s, p->final_stride);
  a.scale = p->scale;
  a.vec_o = vectors(o, 4, 4 * es);
  return CCV_OK;
}

int validate_bwd(const ccv_delta_bwd_args_t* p, Work* w, bool with_ws) {
  if (!p) return CCV_E_NULL;
  if (p->struct_size != (int64_t)sizeof(ccv_delta_bwd_args_t)) return CCV_E_ABI;
  const Sizes z{p->B, p->L, p->N, p->Hk, p->Hv, p->Dk, p->Dv, p->cu_seqlens, p->x_dtype, p->g_dtype, p->beta_dtype};
  int st = check_sizes(z);
  if (st != CCV_OK) return st;
  const int es = elt_size(p->x_dtype);
  const bool pack[4] = {!loadable(view(p->q, p->B, p->L, p->Hk, p->Dk, p->q_stride, es), 8, 16),
                        !loadable(view(p->k, p->B, p->L, p->Hk, p->Dk, p->k_stride, es), 8, 16),
                        !loadable(view(p->v, p->B, p->L, p->Hv, p->Dv, p->v_stride, es), 1, es),
                        !loadable(view(p->dout, p->B, p->L, p->Hv, p->Dv, p->dout_stride, es), 8, 16)};
  // dv goes out through a buffer descriptor too
  if (p->L > 1 && p->dv_stride[1] > kMostStep / es) return CCV_E_LAYOUT;
  st = plan(z, true, with_ws ? p->workspace : nullptr, w, pack);
  if (st != CCV_OK) return st;
  DeltaArgs& a = w->a;
  w->chunks = p->B > 0 && p->L > 0;
  w->states = p->dinitial_state && a.nseq > 0;
  const View q = view(p->q, p->B, p->L, p->Hk, p->Dk, p->q_stride, es), k = view(p->k, p->B, p->L, p->Hk, p->Dk, p->k_stride, es),
             v = view(p->v, p->B, p->L, p->Hv, p->Dv, p->v_stride, es), d = view(p->dout, p->B, p->L, p->Hv, p->Dv, p->dout_stride, es),
             g = view(p->g, p->B, p->L, p->Hv, 1, p->g_stride, 4), b = view(p->beta, p->B, p->L, p->Hv, 1, p->beta_stride, 4),
             h0 = view(p->initial_state, a.nseq, p->Hv, p->Dk, p->Dv, p->init_stride, 4),
             dht = view(p->dfinal_state, a.nseq, p->Hv, p->Dk, p->Dv, p->dfinal_stride, 4),
             dh0 = view(p->dinitial_state, a.nseq, p->Hv, p->Dk, p->Dv, p->dinit_stride, 4),
             dq = view(p->dq, p->B, p->L, p->Hk, p->Dk, p->dq_stride, es), dk = view(p->dk, p->B, p->L, p->Hk, p->Dk, p->dk_stride, es),
             dv = view(p->dv, p->B, p->L, p->Hv, p->Dv, p->dv_stride, es), dg = view(p->dg, p->B, p->L, p->Hv, 1, p->dg_stride, 4),
             db = view(p->dbeta, p->B, p->L, p->Hv, 1, p->dbeta_stride, 4);
  if (p->dinitial_state && !p->initial_state) return CCV_E_UNSUPPORTED;
  if (w->chunks) {
    if (!p->q || !p->k || !p->v || !p->g || !p->beta || !p->dout || !p->dq || !p->dk || !p->dv || !p->dg || !p->dbeta)
      return CCV_E_NULL;
    for (const View& x : {q, k, v, g, b, d})
      if ((st = check_view(x)) != CCV_OK) return st;
    const View written[] = {dq, dk, dv, dg, db, dh0};
    for (int i = 0; i < 6; ++i) {
      if (!written[i].p) continue;
      if ((st = check_written(written[i])) != CCV_OK) return st;
      for (const void* x : {p->q, p->k, p->v, p->g, p->beta, p->dout, (const void*)p->initial_state, (const void*)p->dfinal_state})
        if (x && x == written[i].p && !(i == 5 && x == (const void*)p->dfinal_state)) return CCV_E_ALIAS;
      for (int j = 0; j < i; ++j)
        if (written[j].p == written[i].p) return CCV_E_ALIAS;
    }
  }
  if (p->initial_state && (st = check_view(h0)) != CCV_OK) return st;
  if (p->dfinal_state && (st = check_view(dht)) != CCV_OK) return st;
  if (p->dinitial_state) {
    if ((st = check_written(dh0)) != CCV_OK) return st;
    if (p->dinitial_state == p->initial_state) return CCV_E_ALIAS;
    if (p->dinitial_state == p->dfinal_state)
      for (int i = 0; i < 3; ++i)
        if (dh0.n[i] > 1 && dh0.s[i] != dht.s[i]) return CCV_E_ALIAS;
  }
  if (!w->chunks) w->bytes = 0;
  if (with_ws && (st = check_workspace(p->workspace, p->workspace_bytes, w->bytes)) != CCV_OK) return st;
  a.q = p->q;
  a.k = p->k;
  a.v = p->v;
  a.g = p->g;
  a.beta = p->beta;
  a.dout = p->dout;
  a.h0 = p->initial_state;
  a.dht = p->dfinal_state;
  a.dh0 = p->dinitial_state;
  a.dq = p->dq;
  a.dk = p->dk;
  a.dv = p->dv;
  a.dg = p->dg;
  a.dbeta = p->dbeta;
  copy3(a.q_s, p->q_stride);
  copy3(a.k_s, p->k_stride);
  copy3(a.v_s, p->v_stride);
  copy3(a.g_s, p->g_stride);
  copy3(a.b_s, p->beta_stride);
  copy3(a.do_s, p->dout_stride);
  copy3(a.h0_s, p->init_stride);
  copy3(a.dht_s, p->dfinal_stride);
  copy3(a.dh0_s, p->dinit_stride);
  copy3(a.dq_s, p->dq_stride);
  copy3(a.dk_s, p->dk_stride);
  copy3(a.dv_s, p->dv_stride);
  copy3(a.dg_s, p->dg_stride);
  copy3(a.db_s, p->dbeta_stride);
  a.scale = p->scale;
  a.vec_dqk = vectors(dq, 4, 4 * es) && vectors(dk, 4, 4 * es);
  return CCV_OK;
}

int validate_step(const ccv_delta_update_args_t* p, DeltaStepArgs* a, bool* work) {
  if (!p) return CCV_E_NULL;
  if (p->struct_size != (int64_t)sizeof(ccv_delta_update_args_t)) return CCV_E_ABI;
  int st = check_sizes({p->B, p->L, 0, p->Hk, p->Hv, p->Dk, p->Dv, nullptr, p->x_dtype, p->g_dtype, p->beta_dtype});
  if (st != CCV_OK) return st;
  if (p->slots < 0) return CCV_E_SHAPE;
  if (!p->state_indices && p->B > p->slots) return CCV_E_SHAPE;
  *work = p->B > 0 && p->L > 0;
  if (!*work) return CCV_OK;
  if (!p->q || !p->k || !p->v || !p->g || !p->beta || !p->out || (!p->state && p->slots > 0)) return CCV_E_NULL;
  const int es = elt_size(p->x_dtype);
  const View q = view(p->q, p->B, p->L, p->Hk, p->Dk, p->q_stride, es), k = view(p->k, p->B, p->L, p->Hk, p->Dk, p->k_stride, es),
             v = view(p->v, p->B, p->L, p->Hv, p->Dv, p->v_stride, es), o = view(p->out, p->B, p->L, p->Hv, p->Dv, p->out_stride, es),
             g = view(p->g, p->B, p->L, p->Hv, 1, p->g_stride, 4), b = view(p->beta, p->B, p->L, p->Hv, 1, p->beta_stride, 4),
             s = view(p->state, p->slots, p->Hv, p->Dk, p->Dv, p->state_stride, 4);
  for (const View& x : {q, k, v, g, b})
    if ((st = check_view(x)) != CCV_OK) return st;
  if ((st = check_written(o)) != CCV_OK || (st = check_written(s)) != CCV_OK) return st;
  for (const void* x : {p->q, p->k, p->v, p->g, p->beta})
    if (x == p->out || x == (const void*)p->state) return CCV_E_ALIAS;
  if (p->out == (void*)p->state) return CCV_E_ALIAS;
  int64_t items;
  if (__builtin_mul_overflow(p->B, p->Hv, &items) || __builtin_mul_overflow(items, (p->Dv + 31) / 32, &items) ||
      items / 4 >= INT32_MAX)
    return CCV_E_SHAPE;
  *a = DeltaStepArgs{};
  a->q = p->q;
  a->k = p->k;
  a->v = p->v;
  a->g = p->g;
  a->beta = p->beta;
  a->out = p->out;
  a->state = p->state;
  a->slots = p->state_indices;
  a->nslots = p->slots;
  copy3(a->q_s, p->q_stride);
  copy3(a->k_s, p->k_stride);
  copy3(a->v_s, p->v_stride);
  copy3(a->g_s, p->g_stride);
  copy3(a->b_s, p->beta_stride);
  copy3(a->o_s, p->out_stride);
  copy3(a->st_s, p->state_stride);
  a->B = (int32_t)p->B;
  a->T = (int32_t)p->L;
  a->Hk = (int32_t)p->Hk;
  a->Hv = (int32_t)p->Hv;
  a->Dk = (int32_t)p->Dk;
  a->Dv = (int32_t)p->Dv;
  a->x_dtype = p->x_dtype;
  a->g_dtype = p->g_dtype;
  a->b_dtype = p->beta_dtype;
  a->scale = p->scale;
  a->vec = vectors(q, 4, 4 * es) && vectors(k, 4, 4 * es) && vectors(v, 4, 4 * es) && vectors(o, 4, 4 * es) && vectors(s, 4, 16);
  return CCV_OK;
}

// Copies what the kernels' loads cannot take, and points the call at the copies.
int pack(Work* w, void* stream) {
  DeltaArgs& a = w->a;
  if (a.L == 1) {                // a stride that is never used may be anything: the kernels' bound on
    a.q_s[1] = a.k_s[1] = kDeltaMaxDk;      // a chunk's rows counts on steps that lie apart
    a.v_s[1] = a.do_s[1] = a.o_s[1] = a.dv_s[1] = round_up(a.Dv, 8);
  }
  const int64_t B = a.packed ? 1 : a.nseq;
  const auto one = [&](const void** src, int64_t* s, int32_t H, int32_t D, void* dst) {
    const int32_t Dp = (int32_t)round_up(D, 8);
    DeltaPackArgs p{*src, {s[0], s[1], s[2]}, dst, B * a.L * H, a.L, H, D, Dp, a.x_dtype};
    *src = dst;
    s[1] = Dp;
    s[2] = a.L * Dp;
    s[0] = s[2] * H;
    return launch_delta_pack(p, stream);
  };
  int e = 0;
  if (w->pack[0]) e = one(&a.q, a.q_s, a.Hk, a.Dk, w->packed[0]);
  if (!e && w->pack[1]) e = one(&a.k, a.k_s, a.Hk, a.Dk, w->packed[1]);
  if (!e && w->pack[2]) e = one(&a.v, a.v_s, a.Hv, a.Dv, w->packed[2]);
  if (!e && w->pack[3]) e = one(&a.dout, a.do_s, a.Hv, a.Dv, w->packed[3]);
  return e;
}

}  // namespace

extern "C" {

int ccv_delta_fwd_check(const ccv_delta_fwd_args_t* args) {
  Work w;
  return validate_fwd(args, &w, true);
}

int64_t ccv_delta_fwd_workspace_size(const ccv_delta_fwd_args_t* args) {
  Work w;
  const int st = validate_fwd(args, &w, false);
  return st != CCV_OK ? st : w.bytes;
}

int ccv_delta_fwd(const ccv_delta_fwd_args_t* args, void* hip_stream) {
  Work w;
  const int st = validate_fwd(args, &w, true);
  if (st != CCV_OK) return st;
  if (!w.chunks && !w.states) return CCV_OK;
  if (w.chunks) {
    if (pack(&w, hip_stream) != 0) return CCV_E_HIP;
    if (w.a.packed && launch_delta_table(w.a, hip_stream) != 0) return CCV_E_HIP;
    if (launch_delta_prep(w.a, false, hip_stream) != 0) return CCV_E_HIP;
    if (w.a.part_chunks && launch_delta_carry(w.a, hip_stream) != 0) return CCV_E_HIP;
  }
  return launch_delta_scan(w.a, false, w.nt, hip_stream) == 0 ? CCV_OK : CCV_E_HIP;
}

int ccv_delta_bwd_check(const ccv_delta_bwd_args_t* args) {
  Work w;
  return validate_bwd(args, &w, true);
}

int64_t ccv_delta_bwd_workspace_size(const ccv_delta_bwd_args_t* args) {
  Work w;
  const int st = validate_bwd(args, &w, false);
  return st != CCV_OK ? st : w.bytes;
}

int ccv_delta_bwd(const ccv_delta_bwd_args_t* args, void* hip_stream) {
  Work w;
  const int st = validate_bwd(args, &w, true);
  if (st != CCV_OK) return st;
  if (!w.chunks && !w.states) return CCV_OK;
  if (w.chunks) {
    if (pack(&w, hip_stream) != 0) return CCV_E_HIP;
    if (w.a.packed && launch_delta_table(w.a, hip_stream) != 0) return CCV_E_HIP;
    if (launch_delta_prep(w.a, true, hip_stream) != 0) return CCV_E_HIP;
    if (w.a.part_chunks && launch_delta_carry(w.a, hip_stream) != 0) return CCV_E_HIP;
    if (launch_delta_scan(w.a, true, w.nt, hip_stream) != 0) return CCV_E_HIP;
  }
  if (launch_delta_reverse(w.a, w.nt, hip_stream) != 0) return CCV_E_HIP;
  if (!w.chunks) return CCV_OK;
  return launch_delta_grads(w.a, hip_stream) == 0 ? CCV_OK : CCV_E_HIP;
}

int ccv_delta_update_check(const ccv_delta_update_args_t* args) {
  DeltaStepArgs a;
  bool work;
  return validate_step(args, &a, &work);
}

int ccv_delta_update(const ccv_delta_update_args_t* args, void* hip_stream) {
  DeltaStepArgs a;
  bool work;
  const int st = validate_step(args, &a, &work);
  if (st != CCV_OK || !work) return st;
  return launch_delta_step(a, hip_stream) == 0 ? CCV_OK : CCV_E_HIP;
}

}  // extern "C"
