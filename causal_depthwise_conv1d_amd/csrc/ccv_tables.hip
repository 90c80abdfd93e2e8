// ccv_tables.hip -- the tables of a packed row, from its sequences' lengths.
//
//   cu[0] = 0, cu[s + 1] = cu[s] + lengths[s];  a step t in [cu[s], cu[s + 1]) has
//   seq[t] = s and pos[t] = t - cu[s]; a step past cu[n] has seq -1 and pos 0.
// Lengths count as 0 when negative, and sums stop at `total`.  One launch: every workgroup
// adds up all lengths for itself (n is small beside the row, and they stay in L2), so none
// waits for another; it keeps the offsets of its own steps' sequences in LDS, a piece of
// 1024 sequences at a time, and writes the steps of a piece as it passes it.  Bound by the latency of
// that: 64 sequences of 65536 steps 7 us, 4001 of 1048576 (8 MB) 13 us.
#include "ccv_delta_device.hpp"
#include "ccv_norm_launch.hpp"

namespace ccv {
namespace {

constexpr int kTile = 4096;      // steps a workgroup writes

__global__ __launch_bounds__(1024) void tables_kernel(TablesArgs a) {
  __shared__ int64_t wave[16];
  __shared__ int start[1025];
  const int tid = threadIdx.x, l = tid & 63, w = tid >> 6;
  const int64_t lo = (int64_t)blockIdx.x * kTile, hi = lo + kTile < a.total ? lo + kTile : a.total;
  const bool first = blockIdx.x == 0;
  int64_t carry = 0;
  if (first && tid == 0) a.cu[0] = 0;
  for (int64_t base = 0; base < a.n; base += 1024) {
    const int64_t i = base + tid;
    int64_t x = i < a.n ? a.lengths[i] : 0;
    x = x < 0 ? 0 : x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t o = __shfl_up(x, d);
      if (l >= d) x += o;
    }
    if (l == 63) wave[w] = x;
    __syncthreads();
    int64_t before = carry, all = carry;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      if (k < w) before += wave[k];
      all += wave[k];
    }
    const int64_t end = x + before < a.total ? x + before : a.total;
    start[tid + 1] = (int)end;
    if (tid == 0) start[0] = (int)(carry < a.total ? carry : a.total);
    if (first && i < a.n) a.cu[i + 1] = (int)end;
    __syncthreads();
    // this piece's steps among the workgroup's own
    const int64_t p0 = start[0] > lo ? start[0] : lo, p1 = start[1024] < hi ? start[1024] : hi;
    for (int64_t t = p0 + tid; t < p1; t += 1024) {
      int s0 = 0, s1 = 1023;                          // the last sequence that starts at or before t
      while (s0 < s1) {
        const int m = (s0 + s1 + 1) >> 1;
        if (start[m] <= t) s0 = m;
        else s1 = m - 1;
      }
      if (a.seq) a.seq[t] = (int)(base + s0);
      if (a.pos) a.pos[t] = (int)(t - start[s0]);
    }
    carry = all;
    __syncthreads();
    if (!first && carry >= hi) return;                // the same value in every thread
  }
  for (int64_t t = (carry > lo ? carry : lo) + tid; t < hi; t += 1024) {
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
