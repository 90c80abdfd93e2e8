// ccv_tables.hip -- the tables of a packed row, from its sequences' lengths.
//
//   cu[0] = 0, cu[s + 1] = cu[s] + lengths[s];  a step t in [cu[s], cu[s + 1]) has
//   seq[t] = s and pos[t] = t - cu[s]; a step past cu[n] has seq -1 and pos 0.
// Lengths count as 0 when negative, and sums stop at `total`.  One launch: every workgroup
// adds up all lengths for itself (n is small beside the row, and they stay in L2), so none
// waits for another; it keeps the offsets of a piece of 4096 sequences at a time in LDS, and
// writes its own steps of a piece, four a thread, as it passes it.  Bound by the latency of
// that: 64 sequences of 65536 steps 5.4 us, 4001 of 1048576 (8 MB) 7.2 us (with pieces of 1024
// sequences and one step a thread at a time 7.1 and 13).
#include "ccv_delta_device.hpp"
#include "ccv_norm_launch.hpp"

namespace ccv {
namespace {

constexpr int kTile = 4096;      // steps a workgroup writes, four a thread
constexpr int kPiece = 4096;     // lengths it adds up at a time, four a thread

// Sums stop at `most` < 2^31: adding so stays associative.
__device__ inline uint32_t add(uint32_t x, uint32_t y, uint32_t most) { return min(x + y, most); }

// Inclusive sums over a wave's lanes: four steps inside rows of 16, then each row's last to the rows after it.
template <int CTRL, int ROWS>
__device__ inline uint32_t step(uint32_t x, uint32_t most) {
  return add(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xf, false), most);
}
__device__ inline uint32_t wave_sums(uint32_t x, uint32_t most) {
  x = step<0x111, 0xf>(x, most);     // row_shr 1, 2, 4, 8
  x = step<0x112, 0xf>(x, most);
  x = step<0x114, 0xf>(x, most);
  x = step<0x118, 0xf>(x, most);
  x = step<0x142, 0xa>(x, most);     // lane 15 of a row to the next, rows 1 and 3
  return step<0x143, 0xc>(x, most);  // lane 31 to rows 2 and 3
}

__global__ __launch_bounds__(1024) void tables_kernel(TablesArgs a) {
  __shared__ uint32_t wave[16];
  __shared__ uint32_t start[kPiece + 1];
  const int tid = threadIdx.x, l = tid & 63, w = tid >> 6;
  const uint32_t most = (uint32_t)a.total;
  const uint32_t lo = blockIdx.x * (uint32_t)kTile, hi = min(lo + kTile, most);
  const bool first = blockIdx.x == 0;
  uint32_t carry = 0;
  if (first && tid == 0) a.cu[0] = 0;
  for (int64_t base = 0; base < a.n; base += kPiece) {
    uint32_t x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t i = base + 4 * tid + j;
      const int32_t v = i < a.n ? a.lengths[i] : 0;
      x[j] = v < 0 ? 0 : min((uint32_t)v, most);
    }
#pragma unroll
    for (int j = 1; j < 4; ++j) x[j] = add(x[j], x[j - 1], most);
    const uint32_t sum = wave_sums(x[3], most);
    if (l == 63) wave[w] = sum;
    uint32_t before = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)sum, 0x138, 0xf, 0xf, false);      // wave_shr 1
    __syncthreads();
    uint32_t all = carry;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      if (k == w) before = add(before, all, most);
      all = add(all, wave[k], most);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t end = add(x[j], before, most);
      start[4 * tid + j + 1] = end;
      if (first && base + 4 * tid + j < a.n) a.cu[base + 4 * tid + j + 1] = (int)end;
    }
    if (tid == 0) start[0] = carry;
    __syncthreads();
    // this piece's steps among the workgroup's own
    const uint32_t p0 = max(carry, lo), p1 = min(all, hi), t = lo + 4 * tid;
    if (t < p1 && t + 4 > p0) {
      int s0[4] = {0, 0, 0, 0};                       // the last sequence that starts at or before the step
#pragma unroll
      for (int d = kPiece / 2; d; d >>= 1)
#pragma unroll
        for (int j = 0; j < 4; ++j) s0[j] += start[s0[j] + d] <= t + j ? d : 0;
      int id[4], at[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        id[j] = (int)base + s0[j];
        at[j] = (int)(t + j - start[s0[j]]);
      }
      if (t >= p0 && t + 4 <= p1) {
        if (a.seq) store16(a.seq + t, u32x4{(uint32_t)id[0], (uint32_t)id[1], (uint32_t)id[2], (uint32_t)id[3]});
        if (a.pos) store16(a.pos + t, u32x4{(uint32_t)at[0], (uint32_t)at[1], (uint32_t)at[2], (uint32_t)at[3]});
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (t + j >= p0 && t + j < p1) {
            if (a.seq) a.seq[t + j] = id[j];
            if (a.pos) a.pos[t + j] = at[j];
          }
      }
    }
    carry = all;
    __syncthreads();
    if (!first && carry >= hi) return;                // the same value in every thread
  }
  for (uint32_t t = max(carry, lo) + tid; t < hi; t += 1024) {
    if (a.seq) a.seq[t] = -1;
    if (a.pos) a.pos[t] = 0;
  }
}

}  // namespace

int launch_tables(const TablesArgs& a, void* stream) {
  const int64_t g = (a.total + kTile - 1) / kTile;
  tables_kernel<<<(uint32_t)(g > 0 ? g : 1), 1024, 0, static_cast<hipStream_t>(stream)>>>(a);
  return (int)hipGetLastError();
}

}  // namespace ccv
