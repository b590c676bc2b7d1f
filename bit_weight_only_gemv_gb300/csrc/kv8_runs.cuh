// Equal runs of work over ragged sequences: a list of entries (a sequence, or
// a (sequence, head)) of known weights is cut into consecutive runs of equal
// length, one a CTA, and each CTA finds its own from the weights alone.
#pragma once

#include "kv8.cuh"

namespace w4 {
namespace kv8 {

// A row tile of a sequence: its rows' positions and the slices they see.
struct Tile {
  int lo, hi;        // first (down to a slice) and one past the last visible token of any row
  int pmin, pmax;    // positions of its first and last row
  int slices;
};

// a / b, whose quotient fits an int.
__device__ __forceinline__ int quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (int)((uint32_t)a / (uint32_t)b) : (int)(a / b);
}

// Rows rt * rows .. of the n G query rows that a key head has in a sequence.
__device__ __forceinline__ Tile tile_of(const Seq& s, int G, int window, int rt, int rows, int slice) {
  Tile t;
  const int R = s.n * G;
  const int r0 = rt * rows, r1 = min(R, r0 + rows) - 1;
  t.pmin = s.len - s.n + (s.n == 1 ? 0 : r0 / G);
  t.pmax = s.len - s.n + (s.n == 1 ? 0 : r1 / G);
  t.lo = window > 0 ? (int)max(0LL, (long long)t.pmin + 1 - window) / slice * slice : 0;
  t.hi = t.pmax + 1;
  // at least one slice, if an empty one: the rows are written too
  t.slices = max(1, t.hi > t.lo ? (t.hi - t.lo + slice - 1) / slice : 0);
  return t;
}

// Slices of all row tiles of a sequence, for one head.
__device__ __forceinline__ long long head_slices(const Seq& s, int G, int window, int rows, int slice) {
  const int rts = (s.n * G + rows - 1) / rows;
  long long sum = 0;
  for (int rt = 0; rt < rts; ++rt) sum += tile_of(s, G, window, rt, rows, slice).slices;
  return sum;
}

// This CTA's run [g0, g1) of the `total`, the entry that holds g0 and the
// offset in it; ctas: how many CTAs have one.
struct Run {
  long long total, g0, g1, off;
  int ctas, entry;

  // the CTA whose run holds item g
  __host__ __device__ __forceinline__ int holder(long long g) const {
    if (total <= kNarrow) return (int)(((uint32_t)(g + 1) * (uint32_t)ctas - 1) / (uint32_t)total);
    return (int)(((g + 1) * ctas - 1) / total);
  }
  __host__ __device__ __forceinline__ long long start(int c) const {
    if (total <= kNarrow) return (uint32_t)total * (uint32_t)c / (uint32_t)ctas;
    return total * c / ctas;
  }
  // items u0 .. u0 + n - 1 are all of the runs' (a number read back from
  // memory: a call that gave up may have left another one's there)
  __host__ __device__ __forceinline__ bool holds(long long u0, int n) const {
    return u0 >= 0 && n <= total && u0 <= total - n;
  }
  static constexpr long long kNarrow = 1 << 22;   // times at most 1023 CTAs: 32 bits do
};

// Every thread of the CTA calls (kWarps warps; sm: 2 kWarps + 2 words of
// shared memory); weight(e, &units) is entry e's length, and adds its units'
// number.  Runs have about min_run items at least, but there are as many as
// there are units when CTAs for that many exist (a CTA takes units one after
// the other: 12 sequences of 3 tokens took 55 us in one).  false: this CTA has
// no run.
template <int kWarps, typename Weight>
__device__ bool find_run(int E, int min_run, Weight weight, long long* sm, Run* r) {
  constexpr int kThreads = 32 * kWarps;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long first = 0, mine = 0;
  int units = 0;
  const bool small = E <= 32;   // every warp by itself
  if (small) {
    first = lane < E ? weight(lane, &units) : 0;
    mine = first;
  } else {
    for (int e = tid; e < E; e += kThreads) mine += weight(e, &units);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  units = __reduce_add_sync(0xffffffffu, units);
  if (!small) {
    if (lane == 0) sm[warp] = mine;
    if (lane == 0) sm[kWarps + warp] = units;
    __syncthreads();
    mine = 0;
    long long all = 0;
    for (int w = 0; w < kWarps; ++w) {
      mine += sm[w];
      all += sm[kWarps + w];
    }
    units = (int)min(all, (long long)gridDim.x);
    __syncthreads();
  }
  r->total = mine;
  r->ctas = (int)min(min((long long)gridDim.x, mine),
                     max((mine + min_run - 1) / min_run, (long long)units));
  if ((int)blockIdx.x >= r->ctas) return false;
  r->g0 = r->start(blockIdx.x);
  r->g1 = r->start(blockIdx.x + 1);
  if (small) {
    long long inc = first;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += t;
    }
    const bool here = first > 0 && r->g0 >= inc - first && r->g0 < inc;
    const int at = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
    r->entry = at;
    r->off = r->g0 - __shfl_sync(0xffffffffu, inc - first, at);
    return true;
  }
  long long base = 0;
  for (int e0 = 0; e0 < E; e0 += kThreads) {
    int none = 0;
    const long long w = e0 + tid < E ? weight(e0 + tid, &none) : 0;
    long long inc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += t;
    }
    if (lane == 31) sm[warp] = inc;
    __syncthreads();
    long long all = 0;
    for (int v = 0; v < kWarps; ++v) {
      if (v < warp) inc += sm[v];
      all += sm[v];
    }
    const bool here = w > 0 && r->g0 >= base + inc - w && r->g0 < base + inc;
    if (here) {
      sm[kWarps] = e0 + tid;
      sm[kWarps + 1] = r->g0 - (base + inc - w);
    }
    if (__syncthreads_or(here)) {
      r->entry = (int)sm[kWarps];
      r->off = sm[kWarps + 1];
      __syncthreads();
      return true;
    }
    base += all;
    __syncthreads();
  }
  return false;
}

}  // namespace kv8
}  // namespace w4
