// Choosing what to read and what to keep of an 8-bit cache: the pages of
// highest score bound (w4_kv8_select) and the tokens of most accumulated
// weight (w4_kv8_evict), with the gather of the kept tokens into fresh pages.
//
// Both choices are the same operation on a list of keys: the `count` largest,
// ties from the lowest index on, given back in ascending index order.  Keys
// are fp32 values mapped to uint32 in order.  Up to 16384 keys stay in the
// registers, consecutive ones in a thread.  Three radix passes (11, 11 and 10
// bits, a shared-memory histogram each) find the count-th largest key T and
// how many keys equal to T are taken, then one prefix sum gives every thread
// its place.  Longer lists are read from memory in each pass and written in
// rounds.  Measured: scores of 16 x 8 x 1024 pages (33 MB of ranges) 13.8 us, their
// choices 8, in front of the attention's 42 (60 together); 8 x 8 lists of 16k
// weights 15 us and the gather of 4096 tokens each 27 us, 5 TB/s (41 together).
#include "kv8.cuh"

namespace w4 {
namespace kv8 {
namespace {

constexpr int kTopThreads = 1024;
constexpr int kBins = 2048;

// fp32 -> uint32 in the order of the values, below kForced; -0 and 0 are one
// key, and every NaN, of either sign, is the highest.
constexpr uint32_t kForced = 0xFFFFFFFFu;
constexpr uint32_t kNoPage = 0x7FABCDEFu;   // a NaN no product gives
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t b = __float_as_uint(f);
  if (b == 0x80000000u) return 0x80000000u;
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return kForced - 1;
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// A constant as an argument.
template <int N>
struct Const {
  static constexpr int value = N;
};

struct TopShared {
  uint32_t hist[kBins];
  uint32_t warp_sum[32];
  uint32_t prefix, remaining;
};

// Inclusive sums over the CTA of two small counts packed in one word each
// (kTopThreads threads, every thread calls); returns this thread's exclusive
// sum, *total the whole.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* warp_sum, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  __syncthreads();   // earlier readers of warp_sum are done
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  // every warp sums the warps' sums by itself
  uint32_t w = lane < (int)(blockDim.x >> 5) ? warp_sum[lane] : 0u;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t t = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += t;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const uint32_t base = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  return (warp > 0 ? base : 0u) + inc - v;
}

// The count-th largest key (there are more than `count`), and in *ties how
// many of the keys equal to it belong to the `count`.  keys(add) calls
// add(key) for every key that the thread sees, the same ones each time.
template <typename Keys>
__device__ uint32_t threshold(TopShared& sh, int count, Keys keys, int* ties) {
  const int tid = threadIdx.x, nth = blockDim.x;
  uint32_t prefix = 0, mask = 0, remaining = (uint32_t)count;
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int bins = pass == 2 ? 1024 : 2048;
    for (int i = tid; i < bins; i += nth) sh.hist[i] = 0;
    __syncthreads();
    keys([&](uint32_t u) {
      if ((u & mask) == prefix) atomicAdd(&sh.hist[(u >> shift) & (bins - 1)], 1u);
    });
    __syncthreads();
    // from the highest bin down: the one where the running count reaches
    // `remaining`; a thread owns `per` consecutive bins
    const int per = (bins + nth - 1) / nth;
    uint32_t mine = 0;
    for (int j = 0; j < per; ++j)
      if (tid * per + j < bins) mine += sh.hist[bins - 1 - tid * per - j];
    uint32_t total;
    uint32_t before = block_scan(mine, sh.warp_sum, &total);
    if (before < remaining && before + mine >= remaining) {
      for (int j = 0; j < per; ++j) {
        const uint32_t c = sh.hist[bins - 1 - tid * per - j];
        if (before < remaining && before + c >= remaining) {
          sh.prefix = prefix | ((uint32_t)(bins - 1 - tid * per - j) << shift);
          sh.remaining = remaining - before;
        }
        before += c;
      }
    }
    __syncthreads();
    prefix = sh.prefix;
    remaining = sh.remaining;
    mask |= (uint32_t)(bins - 1) << shift;
    __syncthreads();
  }
  *ties = (int)remaining;
  return prefix;
}

// Calls emit(rank, index) for the `count` largest of key(0) .. key(n - 1)
// (count <= n), rank ascending with the index.  Every thread of the CTA calls.
template <typename Key, typename Emit>
__device__ void top_indexes(TopShared& sh, int n, int count, Key key, Emit emit) {
  const int tid = threadIdx.x, nth = blockDim.x;
  uint32_t T = 0, ties = 0;   // threshold key, and how many equal ones are taken
  if (count < n) {
    int t = 0;
    T = threshold(
        sh, count,
        [&](auto add) {
          for (int i = tid; i < n; i += nth) add(key(i));
        },
        &t);
    ties = (uint32_t)t;
  }
  // ordered pass: rounds of nth consecutive indexes
  uint32_t taken = 0, seen_ties = 0;
  for (int i0 = 0; i0 < n; i0 += nth) {
    const int i = i0 + tid;
    const uint32_t u = i < n ? key(i) : 0u;
    const bool above = i < n && (count >= n || u > T);
    const bool tie = i < n && count < n && u == T;
    uint32_t total;
    const uint32_t ex = block_scan((above ? 1u : 0u) | (tie ? 1u << 16 : 0u), sh.warp_sum, &total);
    const uint32_t tie_rank = seen_ties + (ex >> 16);
    // every taken tie before this index has a tie rank below `ties`
    const uint32_t rank = taken + (ex & 0xFFFFu) + (min(ties, tie_rank) - min(ties, seen_ties));
    if (above || (tie && tie_rank < ties)) emit((int)rank, i);
    const uint32_t t_all = total >> 16;
    taken += (total & 0xFFFFu) + (min(ties, seen_ties + t_all) - min(ties, seen_ties));
    seen_ties += t_all;
  }
}

// The same for keys in registers: thread t holds keys t * kPer .. of n (0 past
// the end), at most 16384 in all.  Calls emit(rank, k) for the thread's k-th key.
template <int kPer, typename Emit>
__device__ void top_registers(TopShared& sh, const uint32_t (&key)[kPer], int n, int count, Emit emit) {
  const int tid = threadIdx.x;
  const int have = max(0, min(kPer, n - tid * kPer));
  const bool all = count >= n;
  uint32_t T = 0;
  int ties = 0;   // keys equal to T that are taken
  if (!all)
    T = threshold(
        sh, count,
        [&](auto add) {
#pragma unroll
          for (int k = 0; k < kPer; ++k)
            if (k < have) add(key[k]);
        },
        &ties);
  // keys above T, and of those equal to T the first ones
  uint32_t above = 0, equal = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k)
    if (k < have) {
      if (all || key[k] > T) ++above;
      else if (key[k] == T) ++equal;
    }
  uint32_t total;
  const uint32_t ex = block_scan(above | equal << 16, sh.warp_sum, &total);
  int rank = (int)(ex & 0xFFFFu), tie = (int)(ex >> 16);
  rank += min(tie, ties);
#pragma unroll
  for (int k = 0; k < kPer; ++k)
    if (k < have) {
      if (all || key[k] > T) {
        emit(rank++, k);
      } else if (key[k] == T) {
        if (tie < ties) emit(rank++, k);
        ++tie;
      }
    }
}

// ------------------------------------------------------------------ select
struct SelectParams {
  Cache c;
  Batch bt;
  const __nv_bfloat16* q;
  long long q_stride;
  int G;
  int32_t* sel;
  int32_t* n_sel;
  int max_sel, sink, recent;
  float* scores;      // [B][H][scores_row]
  long long scores_row;
  int chunk;          // pages scored by one CTA
  int32_t* status;
};

// The query of a (sequence, head) as the pages are scored with: sums of the
// group's positive and negative parts, 8 bits, [down | up] as the ranges lie.
// part: one float per warp.
__device__ void group_query(const SelectParams& p, const Seq& s, int h, float* part, int8_t (&qi)[2][256]) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, D = p.c.D;
  float up = 0.0f, down = 0.0f;
  if (tid < D && s.n > 0) {
    const __nv_bfloat16* q = p.q + (long long)s.row0 * p.q_stride + (long long)h * p.G * D + tid;
#pragma unroll 8
    for (int g = 0; g < p.G; ++g) {
      const float x = __bfloat162float(q[g * D]);
      up += fmaxf(x, 0.0f);
      down += fminf(x, 0.0f);
    }
  }
  float m = fmaxf(up, -down);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) part[warp] = m;
  __syncthreads();
  m = 0.0f;
  for (int w = 0; w < (D + 31) / 32; ++w) m = fmaxf(m, part[w]);
  const float step = pow2_step(fminf(m, 3.0e38f));
  if (tid < D) {
    qi[0][tid] = (int8_t)__float2int_rn(fmaxf(__fdiv_rn(down, step), -127.0f));
    qi[1][tid] = (int8_t)__float2int_rn(fminf(__fdiv_rn(up, step), 127.0f));
  }
  __syncthreads();
}

// Scores of `chunk` pages of a (sequence, head).  A page's two range rows are
// 2 D consecutive bytes: 16 bytes a lane, the codes made signed by one XOR,
// four products an instruction; whole numbers below 2^24, so the sum's order
// does not matter and its conversion is exact.  The bytes of the ranges bound
// it once there are enough of them; four pages a lane are in flight.
constexpr int kScoreThreads = 256;

__global__ void __launch_bounds__(kScoreThreads) score_kernel(const SelectParams p) {
  __shared__ float part[kScoreThreads / 32];
  __shared__ __align__(16) int8_t qi[2][256];
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Seq s = sequence(p.bt, p.c.P, b);
  const int P = p.c.P, D = p.c.D;
  if (!s.ok) {
    if (tid == 0 && blockIdx.x == 0 && h == 0) report(p.status, W4_ERR_INDEX);
    return;
  }
  const int np = (s.len + P - 1) / P;
  const int c0 = blockIdx.x * p.chunk, c1 = min(np, c0 + p.chunk);
  if (c0 >= c1) return;
  const long long bh = (long long)b * p.c.H + h;
  float* scores = p.scores + bh * p.scores_row;
  const int32_t* table = p.bt.table + (long long)b * p.bt.max_pages;
  const int lanes = 2 * D / 16;             // lanes of a page: 8, 16 or 32
  const int sub = lane / lanes, l = lane % lanes;
  const int per = kScoreThreads / lanes;    // pages of the CTA at a time
  constexpr int kDeep = 4;
  int4 r[kDeep];
  float ks[kDeep];
  auto load = [&](int i0) {
    int page[kDeep];
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const int i = i0 + k * per + sub;
      page[k] = i < c1 ? __ldg(table + i) : 0;
    }
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const bool ok = page[k] >= 0 && page[k] < p.c.num_pages;
      if (!ok) page[k] = 0;
      r[k] = __ldg(reinterpret_cast<const int4*>(p.c.ranges + p.c.pair(page[k], h) * 2 * D) + l);
      // a page that is none: a mark that the choice refuses (no score is it)
      ks[k] = ok ? __ldg(p.c.ks + p.c.pair(page[k], h)) : __uint_as_float(kNoPage);
    }
  };
  int i0 = c0 + warp * (32 / lanes);
  load(i0);                                 // on their way while the query is summed
  group_query(p, s, h, part, qi);
  const int4 qw = *reinterpret_cast<const int4*>(&qi[l * 16 / D][l * 16 % D]);
  while (true) {
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const int i = i0 + k * per + sub;
      int acc = __dp4a(r[k].x ^ (int)0x80808080, qw.x, 0);
      acc = __dp4a(r[k].y ^ (int)0x80808080, qw.y, acc);
      acc = __dp4a(r[k].z ^ (int)0x80808080, qw.z, acc);
      acc = __dp4a(r[k].w ^ (int)0x80808080, qw.w, acc);
      for (int o = lanes >> 1; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
      const float v = __float_as_uint(ks[k]) == kNoPage ? ks[k] : (float)acc * ks[k];
      if (l == 0 && i < c1) scores[i] = v;
    }
    i0 += kDeep * per;
    if (i0 >= c1) break;
    load(i0);
  }
}

// The choice of one (sequence, head).
__global__ void __launch_bounds__(kTopThreads) choose_kernel(const SelectParams p) {
  __shared__ TopShared sh;
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const Seq s = sequence(p.bt, p.c.P, b);
  if (!s.ok) return;   // said by the scores
  const int np = (s.len + p.c.P - 1) / p.c.P;
  const long long bh = (long long)b * p.c.H + h;
  const float* scores = p.scores + bh * p.scores_row;
  const int count = min(np, p.max_sel);
  int32_t* sel = p.sel + bh * p.max_sel;
  bool bad = false;
  auto key = [&](int i) {
    const float v = __ldcg(scores + i);
    bad |= __float_as_uint(v) == kNoPage;
    return i < p.sink || i >= np - p.recent ? kForced : order_key(v);
  };
  auto in_registers = [&](auto kPer) {
    constexpr int per = decltype(kPer)::value;
    uint32_t keys[per];
#pragma unroll
    for (int k = 0; k < per; ++k) keys[k] = tid * per + k < np ? key(tid * per + k) : 0u;
    if (__syncthreads_or(bad)) return false;
    top_registers<per>(sh, keys, np, count, [&](int rank, int k) { sel[rank] = tid * per + k; });
    return true;
  };
  bool fine;
  const int nth = blockDim.x;
  if (np <= 4 * nth) {
    fine = in_registers(Const<4>());
  } else if (np <= 16 * nth) {
    fine = in_registers(Const<16>());
  } else {
    for (int i = tid; i < np; i += nth) key(i);
    fine = !__syncthreads_or(bad);
    if (fine) top_indexes(sh, np, count, key, [&](int rank, int i) { sel[rank] = i; });
  }
  if (!fine) {
    if (tid == 0) report(p.status, W4_ERR_INDEX);
    return;
  }
  for (int i = count + tid; i < p.max_sel; i += nth) sel[i] = -1;
  if (tid == 0) p.n_sel[bh] = count;
}

// ------------------------------------------------------------------ evict
struct EvictParams {
  Cache c;
  Batch bt;
  const int32_t* dst_table;
  int dst_pages;
  int32_t* kept;
  int32_t* new_lens;
  int budget, sink, recent;
  int32_t* go;        // [B][H]
  uint32_t* keys;     // [B][H][keys_row]: of sequences too long for registers
  long long keys_row;
  int32_t* status;
};

// One CTA per (sequence, head): the kept positions.  Sixteen consecutive
// tokens lie in one page: a thread that holds that many reads them as four
// 16-byte words.  go[b][h] tells the gather whether there are any (1) or the
// sequence was refused (0).
__global__ void __launch_bounds__(kTopThreads) evict_top_kernel(const EvictParams p) {
  __shared__ TopShared sh;
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int P = p.c.P;
  const int len = __ldg(p.bt.lens + b);
  const long long bh = (long long)b * p.c.H + h;
  const int32_t* table = p.bt.table + (long long)b * p.bt.max_pages;
  bool bad = len < 0 || len > p.bt.max_len;
  const int n = bad ? 0 : len, count = min(n, p.budget);
  int32_t* kept = p.kept + bh * p.budget;
  auto in_registers = [&](auto kPer) {
    constexpr int per = decltype(kPer)::value;
    uint32_t keys[per];
    const int t0 = tid * per;
#pragma unroll
    for (int k = 0; k < per; ++k) keys[k] = 0u;
    if (t0 < n) {
      const int page = __ldg(table + t0 / P);
      if (page < 0 || page >= p.c.num_pages) {
        bad = true;
      } else {
        const float* w = p.c.weight + p.c.pair(page, h) * P + t0 % P;
        float v[per];
        if (per == 16 && (reinterpret_cast<uintptr_t>(p.c.weight) & 15) == 0) {
#pragma unroll
          for (int k = 0; k < per; k += 4) {
            const float4 x = *reinterpret_cast<const float4*>(w + k);
            v[k] = x.x;
            v[k + 1] = x.y;
            v[k + 2] = x.z;
            v[k + 3] = x.w;
          }
        } else {
#pragma unroll
          for (int k = 0; k < per; ++k) v[k] = w[k];
        }
#pragma unroll
        for (int k = 0; k < per; ++k)
          if (t0 + k < n)
            keys[k] = t0 + k < p.sink || t0 + k >= n - p.recent ? kForced : order_key(v[k]);
      }
    }
    if (__syncthreads_or(bad)) return false;
    top_registers<per>(sh, keys, n, count, [&](int rank, int k) { kept[rank] = t0 + k; });
    return true;
  };
  bool fine;
  const int nth = blockDim.x;
  if (n <= 4 * nth) {
    fine = in_registers(Const<4>());
  } else if (n <= 16 * nth) {
    fine = in_registers(Const<16>());
  } else {
    uint32_t* keys = p.keys + bh * p.keys_row;
    for (int t = tid; t < n; t += nth) {
      const int page = __ldg(table + t / P);
      uint32_t u = kForced;
      if (page < 0 || page >= p.c.num_pages)
        bad = true;
      else if (t >= p.sink && t < n - p.recent)
        u = order_key(p.c.weight[p.c.pair(page, h) * P + t % P]);
      keys[t] = u;
    }
    fine = !__syncthreads_or(bad);
    if (fine)
      top_indexes(
          sh, n, count, [&](int i) { return keys[i]; },
          [&](int rank, int i) { kept[rank] = i; });
  }
  if (tid == 0) {
    p.go[bh] = fine;
    if (!fine) report(p.status, W4_ERR_INDEX);
    if (fine && h == 0) p.new_lens[b] = count;
  }
  if (!fine) return;
  for (int i = count + tid; i < p.budget; i += nth) kept[i] = -1;
}

// One warp per (destination page, head, sequence): its tokens' places and
// steps, then the codes, rescaled where the token's step is not the block's,
// 16 bytes a lane and four rows in flight for keys and values each.  No
// barriers: the bytes moved bound it.
constexpr int kMoveWarps = 4;

__global__ void __launch_bounds__(32 * kMoveWarps) evict_move_kernel(const EvictParams p) {
  struct Token {
    long long from;   // byte offset of its codes
    float ks, vs;     // step ratios
  };
  __shared__ Token tokens[kMoveWarps][128];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j = blockIdx.x * kMoveWarps + warp, h = blockIdx.y, b = blockIdx.z;
  const int P = p.c.P, D = p.c.D;
  const long long bh = (long long)b * p.c.H + h;
  if (j >= p.dst_pages || __ldcg(p.go + bh) != 1) return;   // refused before
  const int count = min(__ldg(p.bt.lens + b), p.budget);
  const int n = min(P, count - j * P);
  if (n <= 0) return;
  const int dst = __ldg(p.dst_table + (long long)b * p.dst_pages + j);
  if (dst < 0 || dst >= p.c.num_pages) {
    if (lane == 0) report(p.status, W4_ERR_INDEX);
    return;
  }
  Token* tk = tokens[warp];
  float mk = 0.0f, mv = 0.0f;
  for (int i = lane; i < n; i += 32) {
    const int t = __ldcg(p.kept + bh * p.budget + (long long)j * P + i);
    const int page = __ldg(p.bt.table + (long long)b * p.bt.max_pages + t / P);   // checked before
    const long long pr = p.c.pair(page, h);
    const Token x = {p.c.block(page, h) + (long long)(t % P) * D, p.c.ks[pr], p.c.vs[pr]};
    p.c.weight[p.c.pair(dst, h) * P + i] = p.c.weight[pr * P + t % P];
    mk = fmaxf(mk, x.ks);
    mv = fmaxf(mv, x.vs);
    tk[i] = x;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, o));
    mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, o));
  }
  for (int i = lane; i < n; i += 32) {   // steps to ratios
    tk[i].ks = mk > 0.0f ? __fdiv_rn(tk[i].ks, mk) : 0.0f;
    tk[i].vs = mv > 0.0f ? __fdiv_rn(tk[i].vs, mv) : 0.0f;
  }
  if (lane == 0) {
    p.c.ks[p.c.pair(dst, h)] = mk;
    p.c.vs[p.c.pair(dst, h)] = mv;
  }
  __syncwarp();
  const int vecs = D / 16, col = lane % vecs, r0 = lane / vecs, rstep = 32 / vecs;
  const long long to = p.c.block(dst, h) + col * 16;
  uint32_t lo[4] = {~0u, ~0u, ~0u, ~0u}, hi[4] = {0, 0, 0, 0};
  auto rescaled = [](uint4 w, float ratio) {
    uint32_t x[4] = {w.x, w.y, w.z, w.w};
    if (ratio != 1.0f) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t y = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          y |= to_code((float)((int)((x[i] >> (8 * e)) & 0xFF) - 128) * ratio) << (8 * e);
        x[i] = y;
      }
    }
    return make_uint4(x[0], x[1], x[2], x[3]);
  };
  constexpr int kDeep = 4;
  for (int r = r0; r < n; r += kDeep * rstep) {
    uint4 k[kDeep], v[kDeep];
#pragma unroll
    for (int z = 0; z < kDeep; ++z) {
      if (r + z * rstep < n) {
        const long long from = tk[r + z * rstep].from + col * 16;
        k[z] = __ldcs(reinterpret_cast<const uint4*>(p.c.kc + from));
        v[z] = __ldcs(reinterpret_cast<const uint4*>(p.c.vc + from));
      }
    }
#pragma unroll
    for (int z = 0; z < kDeep; ++z) {
      const int rr = r + z * rstep;
      if (rr < n) {
        const uint4 a = rescaled(k[z], tk[rr].ks), c = rescaled(v[z], tk[rr].vs);
        *reinterpret_cast<uint4*>(p.c.kc + to + (long long)rr * D) = a;
        *reinterpret_cast<uint4*>(p.c.vc + to + (long long)rr * D) = c;
        const uint32_t x[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lo[i] = __vminu4(lo[i], x[i]);
          hi[i] = __vmaxu4(hi[i], x[i]);
        }
      }
    }
  }
  if (p.c.ranges == nullptr) return;
  for (int o = vecs; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = __vminu4(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o));
      hi[i] = __vmaxu4(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o));
    }
  if (r0 == 0) {
    uint4* rg = reinterpret_cast<uint4*>(p.c.ranges + p.c.pair(dst, h) * 2 * D) + col;
    rg[0] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    rg[vecs] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  }
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// Threads of a choice among n keys: a small CTA's barriers are cheaper, and
// 1024 threads hold 16 keys each at most.
int choice_threads(int n) { return n <= 1024 ? 256 : n <= 8192 ? 512 : kTopThreads; }

long long scores_row(const Batch& b) { return (b.max_pages + 3) / 4 * 4; }

long long evict_row(const Batch& b) { return (b.max_len + 63) / 64 * 64; }

}  // namespace
}  // namespace kv8
}  // namespace w4

using namespace w4;

extern "C" size_t w4_kv8_select_workspace_bytes(const w4_kv8_cache* cache,
                                                const w4_kv8_batch* batch) {
  kv8::Cache c;
  kv8::Batch b;
  if (kv8::view(cache, batch, &c, &b) != W4_OK) return 0;
  return kv8::kHeadBytes + kv8::up256((size_t)b.B * c.H * kv8::scores_row(b) * 4);
}

extern "C" w4_status w4_kv8_select(int32_t* sel, int32_t* n_sel, int max_sel, int sink, int recent,
                                   const void* q, size_t q_row_stride, int q_heads,
                                   const w4_kv8_cache* cache, const w4_kv8_batch* batch,
                                   void* workspace, size_t workspace_bytes, int32_t* status_dev,
                                   unsigned flags, w4_stream_t stream) {
  kv8::SelectParams p = {};
  w4_status st = kv8::view(cache, batch, &p.c, &p.bt);
  if (st != W4_OK) return st;
  if (sel == nullptr || n_sel == nullptr || p.c.ranges == nullptr ||
      (flags & ~W4_FLAG_PDL) != 0 || sink < 0 || recent < 0 || max_sel < 1 ||
      (long long)sink + recent > max_sel)
    return W4_ERR_ARG;
  if ((st = kv8::check_q(q, q_row_stride, q_heads, p.c)) != W4_OK) return st;
  if (p.bt.max_new != 1 || max_sel > (1 << 24)) return W4_ERR_SHAPE;
  if (kv8::misaligned(sel, 4) || kv8::misaligned(n_sel, 4) || kv8::misaligned(workspace, 16))
    return W4_ERR_ALIGN;
  if (workspace == nullptr || workspace_bytes < w4_kv8_select_workspace_bytes(cache, batch))
    return W4_ERR_WORKSPACE;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride = (long long)q_row_stride;
  p.G = q_heads / p.c.H;
  p.sel = sel;
  p.n_sel = n_sel;
  p.max_sel = max_sel;
  p.sink = sink;
  p.recent = recent;
  p.scores = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kv8::kHeadBytes);
  p.scores_row = kv8::scores_row(p.bt);
  p.status = status_dev;
  // about eight CTAs an SM, of at least 32 and at most 1024 pages
  const int pages = max(1, (p.bt.max_len + p.c.P - 1) / p.c.P);
  const long long most = (long long)pages * p.c.H * p.bt.B;
  p.chunk = 32;
  while (p.chunk < 1024 && most / p.chunk > 1400) p.chunk *= 2;
  st = kv8::launch(kv8::score_kernel,
                   dim3((unsigned)((pages + p.chunk - 1) / p.chunk), (unsigned)p.c.H,
                        (unsigned)p.bt.B),
                   kv8::kScoreThreads, 0, stream, p);
  if (st != W4_OK) return st;
  return kv8::launch(kv8::choose_kernel, dim3((unsigned)p.c.H, (unsigned)p.bt.B),
                     kv8::choice_threads(pages), 0, stream, p);
}

extern "C" size_t w4_kv8_evict_workspace_bytes(const w4_kv8_cache* cache,
                                               const w4_kv8_batch* batch, int budget) {
  kv8::Cache c;
  kv8::Batch b;
  if (kv8::view(cache, batch, &c, &b) != W4_OK || budget < 1) return 0;
  return kv8::kHeadBytes + kv8::up256((size_t)b.B * c.H * 4) +
         (size_t)b.B * c.H * kv8::evict_row(b) * 4;
}

extern "C" w4_status w4_kv8_evict(const int32_t* dst_table, int32_t* kept, int32_t* new_lens,
                                  int budget, int sink, int recent, const w4_kv8_cache* cache,
                                  const w4_kv8_batch* batch, void* workspace,
                                  size_t workspace_bytes, int32_t* status_dev, unsigned flags,
                                  w4_stream_t stream) {
  kv8::EvictParams p = {};
  const w4_status st = kv8::view(cache, batch, &p.c, &p.bt);
  if (st != W4_OK) return st;
  if (dst_table == nullptr || kept == nullptr || new_lens == nullptr || p.c.weight == nullptr ||
      (flags & ~W4_FLAG_PDL) != 0 || sink < 0 || recent < 0 || budget < 1 ||
      (long long)sink + recent > budget || new_lens == p.bt.lens || dst_table == p.bt.table)
    return W4_ERR_ARG;
  if (budget > (1 << 24)) return W4_ERR_SHAPE;
  if (kv8::misaligned(dst_table, 4) || kv8::misaligned(kept, 4) || kv8::misaligned(new_lens, 4) ||
      kv8::misaligned(workspace, 16))
    return W4_ERR_ALIGN;
  if (workspace == nullptr || workspace_bytes < w4_kv8_evict_workspace_bytes(cache, batch, budget))
    return W4_ERR_WORKSPACE;
  p.dst_table = dst_table;
  p.dst_pages = (budget + p.c.P - 1) / p.c.P;
  p.kept = kept;
  p.new_lens = new_lens;
  p.budget = budget;
  p.sink = sink;
  p.recent = recent;
  uint8_t* ws = static_cast<uint8_t*>(workspace) + kv8::kHeadBytes;
  p.go = reinterpret_cast<int32_t*>(ws);
  p.keys = reinterpret_cast<uint32_t*>(ws + kv8::up256((size_t)p.bt.B * p.c.H * 4));
  p.keys_row = kv8::evict_row(p.bt);
  p.status = status_dev;
  w4_status r = kv8::launch(kv8::evict_top_kernel, dim3((unsigned)p.c.H, (unsigned)p.bt.B),
                            kv8::choice_threads(p.bt.max_len), 0, stream, p);
  if (r != W4_OK) return r;
  const int pages = (min(budget, max(1, p.bt.max_len)) + p.c.P - 1) / p.c.P;
  return kv8::launch(kv8::evict_move_kernel,
                     dim3((unsigned)((pages + kv8::kMoveWarps - 1) / kv8::kMoveWarps),
                          (unsigned)p.c.H, (unsigned)p.bt.B),
                     32 * kv8::kMoveWarps, 0, stream, p);
}
