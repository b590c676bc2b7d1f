// Choosing what to read and what to keep of an 8-bit cache: the pages of
// highest score bound (w4_kv8_select) and the tokens of most accumulated
// weight (w4_kv8_evict), with the gather of the kept tokens into fresh pages.
//
// Both choices are the same operation on a list of keys: the `count` largest,
// ties from the lowest index on, given back in ascending index order.  Keys
// are fp32 values mapped to uint32 in order; three radix passes (11, 11 and
// 10 bits, a shared-memory histogram each) find the count-th largest key T
// and how many keys equal to T are taken, then one ordered pass with prefix
// sums writes the indexes.
#include "kv8.cuh"

namespace w4 {
namespace kv8 {
namespace {

constexpr int kTopThreads = 1024;
constexpr int kBins = 2048;

// fp32 -> uint32 in the order of the values (-NaN lowest, NaN highest), below
// kForced; -0 and 0 are one key.
constexpr uint32_t kForced = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t b = __float_as_uint(f);
  if (b == 0x80000000u) return 0x80000000u;
  return (b & 0x80000000u) ? ~b : min(b | 0x80000000u, kForced - 1);
}

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
  uint32_t base = 0, all = 0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
    const uint32_t s = warp_sum[w];
    if (w < warp) base += s;
    all += s;
  }
  *total = all;
  return base + inc - v;
}

// Calls emit(rank, index) for the `count` largest of key(0) .. key(n - 1)
// (count <= n), rank ascending with the index.  Every thread of the CTA calls.
template <typename Key, typename Emit>
__device__ void top_indexes(TopShared& sh, int n, int count, Key key, Emit emit) {
  const int tid = threadIdx.x, nth = blockDim.x;
  uint32_t T = 0, ties = 0;   // threshold key, and how many equal ones are taken
  if (count < n) {
    uint32_t prefix = 0, mask = 0, remaining = (uint32_t)count;
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const int bins = pass == 2 ? 1024 : 2048;
      for (int i = tid; i < bins; i += nth) sh.hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < n; i += nth) {
        const uint32_t u = key(i);
        if ((u & mask) == prefix) atomicAdd(&sh.hist[(u >> shift) & (bins - 1)], 1u);
      }
      __syncthreads();
      // from the highest bin down: the bin where the running count reaches
      // `remaining`.  Thread t owns bins top, top - 1 (of its pair).
      const int per = bins / kTopThreads > 0 ? bins / kTopThreads : 1;
      uint32_t mine = 0;
      if (tid * per < bins)
        for (int j = 0; j < per; ++j) mine += sh.hist[bins - 1 - tid * per - j];
      uint32_t total;
      uint32_t before = block_scan(mine, sh.warp_sum, &total);
      if (tid * per < bins) {
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
    T = prefix;
    ties = remaining;
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
  float* scores;      // [B][H][max_pages]
  int32_t* arrived;   // [B][H], zero between calls
  int chunk;          // pages scored by one CTA
  int32_t* status;
};

// One CTA scores `chunk` pages of a (sequence, head); the last of a
// (sequence, head)'s CTAs to finish chooses.  A page's two range rows are 2 D
// consecutive bytes: 16 bytes a lane, the codes made signed by one XOR, four
// products an instruction; whole numbers below 2^24, so the sum's order does
// not matter and its conversion is exact.
__global__ void __launch_bounds__(kTopThreads) select_kernel(const SelectParams p) {
  __shared__ TopShared sh;
  __shared__ float part[32];
  __shared__ __align__(16) int8_t qi[2][256];   // [down | up] rows, as the ranges are laid out
  __shared__ int last;
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Seq s = sequence(p.bt, p.c.P, b);
  const int P = p.c.P, D = p.c.D;
  int np = s.ok ? (s.len + P - 1) / P : -1;
  if (np > p.bt.max_pages) np = -1;
  if (np < 0) {
    if (tid == 0 && blockIdx.x == 0) report(p.status, W4_ERR_INDEX);
    return;
  }
  const int c0 = blockIdx.x * p.chunk, c1 = min(np, c0 + p.chunk);
  const int ctas = max(1, (np + p.chunk - 1) / p.chunk);   // that take part
  if ((int)blockIdx.x >= ctas) return;
  // an entry in no use is refused before anything is written; each CTA
  // checks its own pages and leaves a mark in the scores
  const long long bh = (long long)b * p.c.H + h;
  float* scores = p.scores + bh * p.bt.max_pages;
  // the group's query rows: sums of their positive and negative parts
  float up = 0.0f, down = 0.0f;
  if (tid < D && s.n > 0) {
    const __nv_bfloat16* q = p.q + (long long)s.row0 * p.q_stride + (long long)h * p.G * D + tid;
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
  const int lanes = 2 * D / 16;             // lanes of a page: 8, 16 or 32
  const int sub = lane / lanes, l = lane % lanes;
  const int row = l * 16 / D, off = l * 16 % D;
  const int4 qw = *reinterpret_cast<const int4*>(&qi[row][off]);
  const int per_warp = 32 / lanes;
  const int32_t* table = p.bt.table + (long long)b * p.bt.max_pages;
  bool bad = false;
  for (int i = c0 + warp * per_warp + sub; i - sub < c1; i += (kTopThreads / 32) * per_warp) {
    const int page = i < c1 ? __ldg(table + i) : 0;
    const bool ok = page >= 0 && page < p.c.num_pages;
    bad |= !ok;
    int acc = 0;
    float ks = 0.0f;
    if (ok && i < c1) {
      const int4 r = __ldg(reinterpret_cast<const int4*>(p.c.ranges + p.c.pair(page, h) * 2 * D) + l);
      ks = __ldg(p.c.ks + p.c.pair(page, h));
      acc = __dp4a(r.x ^ (int)0x80808080, qw.x, acc);
      acc = __dp4a(r.y ^ (int)0x80808080, qw.y, acc);
      acc = __dp4a(r.z ^ (int)0x80808080, qw.z, acc);
      acc = __dp4a(r.w ^ (int)0x80808080, qw.w, acc);
    }
    for (int o = lanes >> 1; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (l == 0 && i < c1) scores[i] = (float)acc * ks;
  }
  if (bad) report(p.status, W4_ERR_INDEX);
  const int any_bad = __syncthreads_or(bad);
  if (tid == 0) {
    // low half: CTAs that finished; high half: those that met a bad page
    const int add = 1 + (any_bad ? 1 << 16 : 0);
    const int was = atomic_add_acq_rel_gpu(p.arrived + bh, add);
    last = (was & 0xFFFF) + 1 == ctas ? 1 + ((was + add) >> 16 != 0) : 0;
    if (last) p.arrived[bh] = 0;
  }
  __syncthreads();
  if (last != 1) return;   // not the last, or a page of the sequence is not one
  const int count = min(np, p.max_sel);
  int32_t* sel = p.sel + bh * p.max_sel;
  top_indexes(
      sh, np, count,
      [&](int i) {
        return i < p.sink || i >= np - p.recent ? kForced : order_key(__ldcg(scores + i));
      },
      [&](int rank, int i) { sel[rank] = i; });
  for (int i = count + tid; i < p.max_sel; i += kTopThreads) sel[i] = -1;
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
  uint32_t* keys;     // [B][H][max_len rounded up]
  long long keys_row;
  int32_t* status;
};

// One CTA per (sequence, head): the kept positions.  keys[0] afterwards tells
// the gather whether there are any (kForced) or the sequence was refused (0).
__global__ void __launch_bounds__(kTopThreads) evict_top_kernel(const EvictParams p) {
  __shared__ TopShared sh;
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int P = p.c.P;
  const int len = __ldg(p.bt.lens + b);
  const long long bh = (long long)b * p.c.H + h;
  uint32_t* keys = p.keys + bh * p.keys_row;
  const int32_t* table = p.bt.table + (long long)b * p.bt.max_pages;
  const bool in = len >= 0 && len <= p.bt.max_len;
  bool bad = !in;
  if (in) {
    for (int t = tid; t < len; t += kTopThreads) {
      const int page = __ldg(table + t / P);
      uint32_t u = kForced;
      if (page < 0 || page >= p.c.num_pages)
        bad = true;
      else if (t >= p.sink && t < len - p.recent)
        u = order_key(p.c.weight[p.c.pair(page, h) * P + t % P]);
      keys[t] = u;
    }
  }
  bad = __syncthreads_or(bad);
  if (bad) {
    if (tid == 0) {
      report(p.status, W4_ERR_INDEX);
      keys[0] = 0u;   // the gather's sign that this (sequence, head) is left alone
    }
    return;
  }
  const int count = min(len, p.budget);
  int32_t* kept = p.kept + bh * p.budget;
  top_indexes(
      sh, len, count, [&](int i) { return keys[i]; },
      [&](int rank, int i) { kept[rank] = i; });
  for (int i = count + tid; i < p.budget; i += kTopThreads) kept[i] = -1;
  if (h == 0 && tid == 0) p.new_lens[b] = count;
  __syncthreads();
  if (tid == 0) keys[0] = kForced;
}

// One CTA per (destination page, head, sequence): the block's tokens, its
// steps, then the codes rescaled, 16 bytes a thread.
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictParams p) {
  __shared__ long long src_blk[128];   // byte offset of each token's codes
  __shared__ float src_ks[128], src_vs[128];
  __shared__ float steps[2];
  __shared__ __align__(16) uint8_t lo_sm[256 * 16], hi_sm[256 * 16];
  pdl_launch_dependents();
  pdl_wait();
  const int j = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int P = p.c.P, D = p.c.D;
  const long long bh = (long long)b * p.c.H + h;
  if (__ldcg(p.keys + bh * p.keys_row) != kForced) return;   // refused before
  const int count = min(__ldg(p.bt.lens + b), p.budget);
  const int n = min(P, count - j * P);
  if (n <= 0) return;
  const int dst = __ldg(p.dst_table + (long long)b * p.dst_pages + j);
  if (dst < 0 || dst >= p.c.num_pages) {
    if (tid == 0) report(p.status, W4_ERR_INDEX);
    return;
  }
  if (tid < n) {
    const int t = __ldcg(p.kept + bh * p.budget + (long long)j * P + tid);
    const int page = __ldg(p.bt.table + (long long)b * p.bt.max_pages + t / P);   // checked before
    src_blk[tid] = p.c.block(page, h) + (long long)(t % P) * D;
    src_ks[tid] = p.c.ks[p.c.pair(page, h)];
    src_vs[tid] = p.c.vs[p.c.pair(page, h)];
    p.c.weight[p.c.pair(dst, h) * P + tid] = p.c.weight[p.c.pair(page, h) * P + t % P];
  }
  __syncthreads();
  if (tid < 64) {   // one warp each for keys and values
    const float* s = tid < 32 ? src_ks : src_vs;
    float m = 0.0f;
    for (int i = tid & 31; i < n; i += 32) m = fmaxf(m, s[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((tid & 31) == 0) steps[tid >> 5] = m;
  }
  __syncthreads();
  if (tid == 0) {
    p.c.ks[p.c.pair(dst, h)] = steps[0];
    p.c.vs[p.c.pair(dst, h)] = steps[1];
  }
  const int vecs = D / 16, col = tid % vecs, r0 = tid / vecs, rstep = 256 / vecs;
  const long long to = p.c.block(dst, h);
  uint32_t lo[4] = {~0u, ~0u, ~0u, ~0u}, hi[4] = {0, 0, 0, 0};
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const uint8_t* src = kv ? p.c.vc : p.c.kc;
    uint8_t* out = (kv ? p.c.vc : p.c.kc) + to;
    const float step = steps[kv];
    for (int r = r0; r < n; r += rstep) {
      uint4 w = *reinterpret_cast<const uint4*>(src + src_blk[r] + col * 16);
      const float s0 = kv ? src_vs[r] : src_ks[r];
      uint32_t x[4] = {w.x, w.y, w.z, w.w};
      if (s0 != step) {
        const float ratio = step > 0.0f ? __fdiv_rn(s0, step) : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t y = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            y |= to_code((float)((int)((x[i] >> (8 * e)) & 0xFF) - 128) * ratio) << (8 * e);
          x[i] = y;
        }
      }
      *reinterpret_cast<uint4*>(out + (long long)r * D + col * 16) =
          make_uint4(x[0], x[1], x[2], x[3]);
      if (kv == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lo[i] = __vminu4(lo[i], x[i]);
          hi[i] = __vmaxu4(hi[i], x[i]);
        }
      }
    }
  }
  if (p.c.ranges == nullptr) return;
  uint4* ls = reinterpret_cast<uint4*>(lo_sm);
  uint4* hs = reinterpret_cast<uint4*>(hi_sm);
  ls[tid] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  hs[tid] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  __syncthreads();
  if (tid < 2 * vecs) {
    const bool is_hi = tid >= vecs;
    const uint4* s = is_hi ? hs : ls;
    uint4 a = s[col];
    for (int r = 1; r < rstep; ++r) {
      const uint4 o = s[r * vecs + col];
      a.x = is_hi ? __vmaxu4(a.x, o.x) : __vminu4(a.x, o.x);
      a.y = is_hi ? __vmaxu4(a.y, o.y) : __vminu4(a.y, o.y);
      a.z = is_hi ? __vmaxu4(a.z, o.z) : __vminu4(a.z, o.z);
      a.w = is_hi ? __vmaxu4(a.w, o.w) : __vminu4(a.w, o.w);
    }
    *(reinterpret_cast<uint4*>(p.c.ranges + p.c.pair(dst, h) * 2 * D) + tid) = a;
  }
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

size_t select_scores_bytes(const Cache& c, const Batch& b) {
  return up256((size_t)b.B * c.H * b.max_pages * 4);
}

}  // namespace
}  // namespace kv8
}  // namespace w4

using namespace w4;

extern "C" size_t w4_kv8_select_workspace_bytes(const w4_kv8_cache* cache,
                                                const w4_kv8_batch* batch) {
  kv8::Cache c;
  kv8::Batch b;
  if (kv8::view(cache, batch, &c, &b) != W4_OK) return 0;
  return kv8::up256((size_t)b.B * c.H * 4) + kv8::select_scores_bytes(c, b);
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
  p.arrived = static_cast<int32_t*>(workspace);
  p.scores = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) +
                                      kv8::up256((size_t)p.bt.B * p.c.H * 4));
  const int pages = max(1, (p.bt.max_len + p.c.P - 1) / p.c.P);
  p.chunk = 1024;
  while ((pages + p.chunk - 1) / p.chunk > 16384) p.chunk *= 2;   // `arrived` counts in 16 bits
  p.status = status_dev;
  return kv8::launch(kv8::select_kernel,
                     dim3((unsigned)((pages + p.chunk - 1) / p.chunk), (unsigned)p.c.H,
                          (unsigned)p.bt.B),
                     kv8::kTopThreads, 0, (flags & W4_FLAG_PDL) != 0, stream, p);
}

extern "C" size_t w4_kv8_evict_workspace_bytes(const w4_kv8_cache* cache,
                                               const w4_kv8_batch* batch, int budget) {
  kv8::Cache c;
  kv8::Batch b;
  if (kv8::view(cache, batch, &c, &b) != W4_OK || budget < 1) return 0;
  return (size_t)b.B * c.H * kv8::up256((size_t)(b.max_len + 1) * 4);
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
  p.keys = static_cast<uint32_t*>(workspace);
  p.keys_row = (long long)(kv8::up256((size_t)(p.bt.max_len + 1) * 4) / 4);
  p.status = status_dev;
  w4_status r = kv8::launch(kv8::evict_top_kernel, dim3((unsigned)p.c.H, (unsigned)p.bt.B),
                            kv8::kTopThreads, 0, (flags & W4_FLAG_PDL) != 0, stream, p);
  if (r != W4_OK) return r;
  const int most = min(budget, max(1, p.bt.max_len));
  return kv8::launch(kv8::evict_move_kernel,
                     dim3((unsigned)((most + p.c.P - 1) / p.c.P), (unsigned)p.c.H,
                          (unsigned)p.bt.B),
                     256, 0, true, stream, p);
}
