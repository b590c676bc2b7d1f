// Who has which page of the 8-bit cache: forks, growth and compaction
// (w4_kv8_fork, w4_kv8_reserve, w4_kv8_compact).
//
// Each call decides in one cluster of kRanks CTAs, whose barrier separates its
// phases: counts of references by atomics (whole numbers, so their order does
// not matter), decisions in row order by block scans that every CTA repeats,
// free pages in page order by a scan over the cluster's contiguous shares of
// the pages.  Tables are walked in pieces of kPiece entries, one piece a warp,
// so that one long row has as many readers as many short ones.  What has to be
// copied goes into a list in the workspace; copy_kernel moves it in every
// cache, one warp for the keys or values of one (page, head).
#include "kv8.cuh"

namespace w4 {
namespace kv8 {
namespace {

constexpr int kRanks = 8, kPlanThreads = 1024;
constexpr int kAll = kRanks * kPlanThreads;
constexpr int kPiece = 128;
constexpr int kRowsEach = W4_KV8_MAX_BATCH / kPlanThreads;   // rows a thread decides
constexpr unsigned kFull = 0xffffffffu;

// Areas of the workspace past its head.
struct Scratch {
  int32_t* n_copies;   // [1]
  int32_t* row_pages;  // [rows]: pages a row names, -1: it breaks its bounds
  int32_t* count;      // [pages]
  int32_t* first;      // [pages]
  int32_t* src;        // copies
  int32_t* dst;
  int32_t* tokens;
};

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

size_t carve(void* ws, int batch, int num_pages, Scratch* s) {
  uint8_t* base = static_cast<uint8_t*>(ws);
  size_t at = kHeadBytes;
  auto take = [&](size_t n) {
    int32_t* p = base == nullptr ? nullptr : reinterpret_cast<int32_t*>(base + at);
    at += up256(n * 4);
    return p;
  };
  const size_t pages = (size_t)num_pages, list = batch > num_pages ? (size_t)batch : pages;
  Scratch t;
  t.n_copies = take(1);
  t.row_pages = take((size_t)batch);
  t.count = take(pages);
  t.first = take(pages);
  t.src = take(list);
  t.dst = take(list);
  t.tokens = take(list);
  if (s != nullptr) *s = t;
  return at;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Everything that the cluster's threads wrote before is seen after (global
// memory through L2: what other CTAs write is read by __ldcg).
__device__ __forceinline__ void cluster_sync() {
  __threadfence();
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ int remote(const int* p, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return (int)v;
}

// Exclusive sum over the block's threads; *total the block's.  red: 33 words.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* red, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(kFull, s, o);
    if (lane >= o) s += u;
  }
  __syncthreads();
  if (lane == 31) red[warp] = s;
  __syncthreads();
  if (warp == 0) {
    T w = red[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T u = __shfl_up_sync(kFull, w, o);
      if (lane >= o) w += u;
    }
    red[lane] = w;
  }
  __syncthreads();
  *total = red[31];
  return s - v + (warp > 0 ? red[warp - 1] : T(0));
}

struct Rows {
  const int32_t* table;
  const int32_t* lens;
  int batch, max_pages, shift;   // tokens of a page: 1 << shift
  int num_pages;

  __device__ __forceinline__ int pages(int len) const {   // -1: out of bounds
    return len < 0 || (long long)len > ((long long)max_pages << shift)
               ? -1
               : (int)(((long long)len + (1 << shift) - 1) >> shift);
  }
};

// Pages of every old row into s.row_pages, -1 where its length or one of its
// entries breaks its bounds.  Ends in a cluster barrier.
__device__ void check_rows(const Rows& r, const Scratch& s, uint32_t rank, int32_t* status) {
  const int gt = rank * kPlanThreads + threadIdx.x;
  for (int b = gt; b < r.batch; b += kAll) {
    const int np = r.pages(__ldg(r.lens + b));
    s.row_pages[b] = np;
    if (np < 0) report(status, W4_ERR_INDEX);
  }
  cluster_sync();
  const int lane = threadIdx.x & 31;
  const long long pieces = (r.max_pages + kPiece - 1) / kPiece;
  for (long long i = gt >> 5; i < pieces * r.batch; i += kAll / 32) {
    const int b = (int)(i / pieces), at = (int)(i % pieces) * kPiece;
    const int np = min(r.pages(__ldg(r.lens + b)), at + kPiece);
    bool bad = false;
    for (int e = at + lane; e < np; e += 32) {
      const int pg = __ldg(r.table + (long long)b * r.max_pages + e);
      bad |= pg < 0 || pg >= r.num_pages;
    }
    if (__any_sync(kFull, bad) && lane == 0) {
      s.row_pages[b] = -1;
      report(status, W4_ERR_INDEX);
    }
  }
  cluster_sync();
}

// This thread's share of the pages, in page order over the cluster.
__device__ __forceinline__ void my_share(int num_pages, uint32_t rank, int* lo, int* hi) {
  const long long each = ((long long)num_pages + kAll - 1) / kAll;
  const long long a = ((long long)rank * kPlanThreads + threadIdx.x) * each;
  *lo = (int)min(a, (long long)num_pages);
  *hi = (int)min(a + each, (long long)num_pages);
}

// Sum of `mine` (the same in all threads of a CTA) over the ranks before this
// one, and over all.  slot: shared memory of this use alone.
__device__ __forceinline__ int before_rank(int mine, int* slot, uint32_t rank, int* total) {
  if (threadIdx.x == 0) *slot = mine;
  cluster_sync();
  int before = 0, all = 0;
  for (int i = 0; i < kRanks; ++i) {
    const int v = remote(slot, i);
    all += v;
    if (i < (int)rank) before += v;
  }
  *total = all;
  return before;
}

// The lowest `want` free pages into list, in order; false (everywhere) if there
// are fewer.  Ends in a cluster barrier: what every rank read before the call
// may be written after it.
__device__ bool take_free(const int32_t* refs, int num_pages, long long want, int32_t* list,
                          uint32_t rank, int* red, int* slot) {
  if (want == 0) {
    cluster_sync();
    return true;
  }
  int lo, hi;
  my_share(num_pages, rank, &lo, &hi);
  int free = 0;
  for (int i = lo; i < hi; ++i) free += __ldcg(refs + i) == 0;
  int total, all;
  int at = block_scan(free, red, &total);
  at += before_rank(total, slot, rank, &all);
  const bool ok = all >= want;
  if (ok && free > 0 && at < want)
    for (int i = lo; i < hi && at < want; ++i)
      if (__ldcg(refs + i) == 0) list[at++] = i;
  cluster_sync();
  return ok;
}

struct ForkParams {
  Rows old;
  const int32_t* refs;
  const int32_t* parents;
  int32_t* new_table;
  int32_t* new_lens;
  int32_t* new_refs;
  int new_batch;
  Scratch s;
  int32_t* status;
};

__global__ void __cluster_dims__(kRanks, 1, 1) __launch_bounds__(kPlanThreads)
    fork_kernel(ForkParams p) {
  __shared__ int red[33], slot;
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t rank = cluster_rank();
  const int gt = rank * kPlanThreads + threadIdx.x, lane = threadIdx.x & 31;
  const Rows& r = p.old;
  for (int i = gt; i < r.num_pages; i += kAll) {
    p.new_refs[i] = __ldg(p.refs + i);
    p.s.count[i] = 0;
    p.s.first[i] = 0x7fffffff;
  }
  check_rows(r, p.s, rank, p.status);
  // the old rows' names go, the new rows' come
  const long long pieces = (r.max_pages + kPiece - 1) / kPiece;
  const int rows = max(r.batch, p.new_batch);
  for (long long i = gt >> 5; i < pieces * rows; i += kAll / 32) {
    const int b = (int)(i / pieces), at = (int)(i % pieces) * kPiece;
    const int par = b < p.new_batch ? __ldg(p.parents + b) : -1;
    int had = b < r.batch ? __ldcg(p.s.row_pages + b) : 0, np = 0, len = 0;
    bool ok = par >= -1 && par < r.batch;
    if (ok && par >= 0) {
      np = __ldcg(p.s.row_pages + par);
      len = __ldg(r.lens + par);
      ok = np >= 0;
    }
    if (!ok) {
      if (at == 0 && lane == 0) {
        p.new_lens[b] = -1;
        report(p.status, W4_ERR_INDEX);
      }
      continue;
    }
    if (par != b)
      for (int e = at + lane; e < min(had, at + kPiece); e += 32)
        atomicSub(p.new_refs + __ldg(r.table + (long long)b * r.max_pages + e), 1);
    if (b >= p.new_batch) continue;
    for (int e = at + lane; e < min(np, at + kPiece); e += 32) {
      const int pg = __ldg(r.table + (long long)par * r.max_pages + e);
      p.new_table[(long long)b * r.max_pages + e] = pg;
      if (par != b) atomicAdd(p.new_refs + pg, 1);
      if (e == np - 1 && (len & ((1 << r.shift) - 1)) != 0) {   // a page to be written to
        atomicAdd(p.s.count + pg, 1);
        atomicMin(p.s.first + pg, b);
      }
    }
    if (at == 0 && lane == 0) p.new_lens[b] = len;
  }
  cluster_sync();
  // rows that need a page of their own, in order
  int page[kRowsEach], used[kRowsEach], last[kRowsEach], mine = 0;
#pragma unroll
  for (int z = 0; z < kRowsEach; ++z) {
    const int b = threadIdx.x * kRowsEach + z;
    page[z] = -1;
    if (b >= p.new_batch) continue;
    const int len = __ldcg(p.new_lens + b);
    used[z] = len & ((1 << r.shift) - 1);
    if (len <= 0 || used[z] == 0) continue;
    last[z] = r.pages(len) - 1;
    const int pg = __ldcg(p.new_table + (long long)b * r.max_pages + last[z]);
    if (__ldcg(p.s.count + pg) == __ldcg(p.new_refs + pg) && __ldcg(p.s.first + pg) == b) continue;
    page[z] = pg;
    ++mine;
  }
  int want;
  int at = block_scan(mine, red, &want);
  const bool ok = take_free(p.new_refs, r.num_pages, want, p.s.dst, rank, red, &slot);
  if (rank == 0) {
    if (threadIdx.x == 0) {
      *p.s.n_copies = ok ? want : 0;
      if (!ok) report(p.status, W4_ERR_STATE);
    }
    if (!ok) {
      for (int b = threadIdx.x; b < p.new_batch; b += kPlanThreads) p.new_lens[b] = -1;
    } else {
#pragma unroll
      for (int z = 0; z < kRowsEach; ++z) {
        if (page[z] < 0) continue;
        const int to = __ldcg(p.s.dst + at);
        p.new_table[(long long)(threadIdx.x * kRowsEach + z) * r.max_pages + last[z]] = to;
        atomicSub(p.new_refs + page[z], 1);
        p.new_refs[to] = 1;
        p.s.src[at] = page[z];
        p.s.tokens[at] = used[z];
        ++at;
      }
    }
  }
}

struct ReserveParams {
  Rows r;
  int32_t* table;
  int32_t* lens;
  int32_t* refs;
  const int32_t* grow;
  Scratch s;
  int32_t* status;
};

__global__ void __cluster_dims__(kRanks, 1, 1) __launch_bounds__(kPlanThreads)
    reserve_kernel(ReserveParams p) {
  __shared__ long long red64[33];
  __shared__ int red[33], slot;
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t rank = cluster_rank();
  int from[kRowsEach], to[kRowsEach], len[kRowsEach];
  long long mine = 0;
#pragma unroll
  for (int z = 0; z < kRowsEach; ++z) {
    const int b = threadIdx.x * kRowsEach + z;
    from[z] = to[z] = len[z] = -1;
    if (b >= p.r.batch) continue;
    const int now = __ldcg(p.lens + b);
    const int g = p.grow != nullptr ? __ldg(p.grow + b) : now > 0;
    const long long then = (long long)now + g;
    const int a = p.r.pages(now);
    const int e = g < 0 || then > 0x7fffffffll ? -1 : p.r.pages((int)then);
    if (a < 0 || e < 0) {
      if (rank == 0) report(p.status, W4_ERR_INDEX);
      continue;
    }
    from[z] = a;
    to[z] = e;
    len[z] = (int)then;
    mine += e - a;
  }
  long long want;
  long long at = block_scan(mine, red64, &want);
  const bool ok = take_free(p.refs, p.r.num_pages, want, p.s.dst, rank, red, &slot);
  if (rank != 0) return;
  if (!ok) {
    if (threadIdx.x == 0) report(p.status, W4_ERR_STATE);
    return;
  }
#pragma unroll
  for (int z = 0; z < kRowsEach; ++z) {
    if (len[z] < 0) continue;
    const int b = threadIdx.x * kRowsEach + z;
    for (int e = from[z]; e < to[z]; ++e) {
      const int pg = __ldcg(p.s.dst + at++);
      p.table[(long long)b * p.r.max_pages + e] = pg;
      p.refs[pg] = 1;
    }
    p.lens[b] = len[z];
  }
}

struct CompactParams {
  Rows r;
  const int32_t* refs;
  int32_t* new_table;
  int32_t* new_refs;
  int32_t* used;
  Scratch s;
  int32_t* status;
};

__global__ void __cluster_dims__(kRanks, 1, 1) __launch_bounds__(kPlanThreads)
    compact_kernel(CompactParams p) {
  __shared__ int red[33], slot[3];
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t rank = cluster_rank();
  const int gt = rank * kPlanThreads + threadIdx.x, lane = threadIdx.x & 31;
  const Rows& r = p.r;
  int32_t* to = p.s.first;   // where each page goes
  for (int i = gt; i < r.num_pages; i += kAll) {
    p.new_refs[i] = __ldg(p.refs + i);
    p.s.count[i] = 0;
    to[i] = i;
  }
  if (gt == 0) *p.used = 0;
  check_rows(r, p.s, rank, p.status);
  const long long pieces = (r.max_pages + kPiece - 1) / kPiece;
  for (long long i = gt >> 5; i < pieces * r.batch; i += kAll / 32) {
    const int b = (int)(i / pieces), at = (int)(i % pieces) * kPiece;
    const int np = min(__ldcg(p.s.row_pages + b), at + kPiece);
    for (int e = at + lane; e < np; e += 32)
      atomicAdd(p.s.count + __ldg(r.table + (long long)b * r.max_pages + e), 1);
  }
  int lo, hi;
  my_share(r.num_pages, rank, &lo, &hi);
  int live = 0, total, n;
  for (int i = lo; i < hi; ++i) live += __ldg(p.refs + i) != 0;
  block_scan(live, red, &total);
  before_rank(total, slot, rank, &n);   // a barrier: the counts are complete
  int from = 0, hole = 0;
  for (int i = lo; i < hi; ++i) {
    const int c = __ldg(p.refs + i);
    from += i >= n && c != 0 && __ldcg(p.s.count + i) == c;
    hole += i < n && c == 0;
  }
  int moves, holes;
  int fat = block_scan(from, red, &total);
  fat += before_rank(total, slot + 1, rank, &moves);
  int hat = block_scan(hole, red, &total);
  hat += before_rank(total, slot + 2, rank, &holes);
  for (int i = lo; i < hi; ++i) {
    const int c = __ldg(p.refs + i);
    if (i >= n && c != 0 && __ldcg(p.s.count + i) == c) p.s.src[fat++] = i;
    if (i < n && c == 0 && hat < moves) p.s.dst[hat++] = i;
  }
  cluster_sync();
  for (int j = gt; j < moves; j += kAll) {
    const int a = __ldcg(p.s.src + j), b = __ldcg(p.s.dst + j);
    to[a] = b;
    p.new_refs[b] = __ldg(p.refs + a);
    p.new_refs[a] = 0;
    p.s.tokens[j] = 1 << r.shift;
  }
  if (gt == 0) *p.s.n_copies = moves;
  cluster_sync();
  for (long long i = gt >> 5; i < pieces * r.batch; i += kAll / 32) {
    const int b = (int)(i / pieces), at = (int)(i % pieces) * kPiece;
    const int np = min(__ldcg(p.s.row_pages + b), at + kPiece);
    for (int e = at + lane; e < np; e += 32) {
      const long long o = (long long)b * r.max_pages + e;
      p.new_table[o] = __ldcg(to + __ldg(r.table + o));
    }
  }
  int most = 0;
  for (int i = lo; i < hi; ++i)
    if (__ldcg(p.new_refs + i) != 0) most = i + 1;
  most = __reduce_max_sync(kFull, most);
  if (lane == 0 && most > 0) atomicMax(p.used, most);
}

// ---------------------------------------------------------------- copies
constexpr int kCopyThreads = 256;

struct One {   // one cache's arrays
  uint8_t* kc;
  uint8_t* vc;
  float* ks;
  float* vs;
  uint8_t* ranges;
  float* weight;
  long long page_stride, head_stride;
};
struct CopyParams {
  One c[W4_KV8_MAX_CACHES];
  int n, H, P, D;
  const int32_t* n_copies;
  const int32_t* src;
  const int32_t* dst;
  const int32_t* tokens;
};

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warps = gridDim.x * (kCopyThreads / 32);
  const long long items = (long long)__ldg(p.n_copies) * p.n * p.H * 2;
  for (long long i = (long long)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); i < items;
       i += warps) {
    const bool is_v = i & 1;
    long long j = i >> 1;
    const int h = (int)(j % p.H);
    j /= p.H;
    const One& c = p.c[j % p.n];
    j /= p.n;
    const int from = __ldg(p.src + j), to = __ldg(p.dst + j), tokens = __ldg(p.tokens + j);
    uint8_t* codes = (is_v ? c.vc : c.kc) + h * c.head_stride;
    const uint4* a = reinterpret_cast<const uint4*>(codes + from * c.page_stride);
    uint4* b = reinterpret_cast<uint4*>(codes + to * c.page_stride);
    const int n = tokens * p.D / 16;
#pragma unroll 4
    for (int e = lane; e < n; e += 32) b[e] = a[e];
    const long long ph = (long long)from * p.H + h, qh = (long long)to * p.H + h;
    if (is_v) {
      if (lane == 0) c.vs[qh] = c.vs[ph];
      if (c.weight != nullptr)
        for (int e = lane; e < tokens; e += 32) c.weight[qh * p.P + e] = c.weight[ph * p.P + e];
    } else {
      if (lane == 0) c.ks[qh] = c.ks[ph];
      if (c.ranges != nullptr)
        for (int e = lane; e < p.D / 8; e += 32)
          reinterpret_cast<uint4*>(c.ranges + qh * 2 * p.D)[e] =
              reinterpret_cast<const uint4*>(c.ranges + ph * 2 * p.D)[e];
    }
  }
}

// host: the caches of a call, all alike.
w4_status view_caches(const w4_kv8_cache* caches, int n, CopyParams* p, int* num_pages) {
  if (caches == nullptr || n < 1) return W4_ERR_ARG;
  if (n > W4_KV8_MAX_CACHES) return W4_ERR_SHAPE;
  for (int i = 0; i < n; ++i) {
    // the checks of a cache, with a batch that passes its own
    const w4_kv8_batch one = {reinterpret_cast<const int32_t*>(16), reinterpret_cast<const int32_t*>(16),
                              nullptr, 1, 1, 1, 1, 0};
    Cache c;
    Batch b;
    const w4_status st = view(caches + i, &one, &c, &b);
    if (st != W4_OK) return st;
    if (i == 0) {
      p->H = c.H;
      p->P = c.P;
      p->D = c.D;
      *num_pages = c.num_pages;
    } else if (c.H != p->H || c.P != p->P || c.D != p->D || c.num_pages != *num_pages) {
      return W4_ERR_SHAPE;
    }
    p->c[i] = {c.kc, c.vc, c.ks, c.vs, c.ranges, c.weight, c.page_stride, c.head_stride};
  }
  p->n = n;
  return W4_OK;
}

bool overlap(const void* a, const void* b, size_t na, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

w4_status check_table(const int32_t* table, const int32_t* lens, const int32_t* refs, int batch,
                      int max_pages, int num_pages, int P) {
  if (table == nullptr || lens == nullptr || refs == nullptr || batch < 1 || max_pages < 1 ||
      num_pages < 1)
    return W4_ERR_ARG;
  if (batch > W4_KV8_MAX_BATCH || (P != 16 && P != 32 && P != 64 && P != 128)) return W4_ERR_SHAPE;
  if (misaligned(table, 4) || misaligned(lens, 4) || misaligned(refs, 4)) return W4_ERR_ALIGN;
  return W4_OK;
}

int log2_of(int p) { return p == 16 ? 4 : p == 32 ? 5 : p == 64 ? 6 : 7; }

// At most this many copies: a CTA for every eight warps' worth, as many as stay resident.
w4_status copy(const CopyParams& p, long long most, w4_stream_t stream) {
  const long long items = most * p.n * p.H * 2, ctas = (items + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
  return launch(copy_kernel, dim3((unsigned)min(ctas, 152ll * 8)), kCopyThreads, 0, stream, p);
}

}  // namespace
}  // namespace kv8
}  // namespace w4

using namespace w4;

extern "C" size_t w4_kv8_pages_workspace_bytes(int batch, int num_pages) {
  if (batch < 1 || batch > W4_KV8_MAX_BATCH || num_pages < 1) return 0;
  return kv8::carve(nullptr, batch, num_pages, nullptr);
}

extern "C" w4_status w4_kv8_fork(int32_t* new_table, int32_t* new_lens, int32_t* new_refs,
                                 int new_batch, const int32_t* parents, const int32_t* table,
                                 const int32_t* lens, const int32_t* refs, int batch,
                                 int max_pages, const w4_kv8_cache* caches, int n_caches,
                                 void* workspace, size_t workspace_bytes, int32_t* status_dev,
                                 unsigned flags, w4_stream_t stream) {
  kv8::CopyParams c = {};
  int num = 0;
  w4_status st = kv8::view_caches(caches, n_caches, &c, &num);
  if (st != W4_OK) return st;
  if ((st = kv8::check_table(table, lens, refs, batch, max_pages, num, c.P)) != W4_OK) return st;
  if (new_table == nullptr || new_lens == nullptr || new_refs == nullptr || parents == nullptr ||
      new_batch < 1 || (flags & ~W4_FLAG_PDL) != 0)
    return W4_ERR_ARG;
  if (new_batch > W4_KV8_MAX_BATCH) return W4_ERR_SHAPE;
  if (kv8::misaligned(new_table, 4) || kv8::misaligned(new_lens, 4) ||
      kv8::misaligned(new_refs, 4) || kv8::misaligned(parents, 4) || kv8::misaligned(workspace, 16))
    return W4_ERR_ALIGN;
  const size_t row = (size_t)max_pages * 4;
  if (kv8::overlap(table, new_table, row * batch, row * new_batch) ||
      kv8::overlap(lens, new_lens, 4 * (size_t)batch, 4 * (size_t)new_batch) ||
      kv8::overlap(refs, new_refs, 4 * (size_t)num, 4 * (size_t)num))
    return W4_ERR_ARG;
  const int most = batch > new_batch ? batch : new_batch;
  if (workspace == nullptr || workspace_bytes < w4_kv8_pages_workspace_bytes(most, num))
    return W4_ERR_WORKSPACE;
  kv8::ForkParams p = {};
  p.old = {table, lens, batch, max_pages, kv8::log2_of(c.P), num};
  p.refs = refs;
  p.parents = parents;
  p.new_table = new_table;
  p.new_lens = new_lens;
  p.new_refs = new_refs;
  p.new_batch = new_batch;
  kv8::carve(workspace, most, num, &p.s);
  p.status = status_dev;
  st = kv8::launch(kv8::fork_kernel, dim3(kv8::kRanks), kv8::kPlanThreads, 0, stream, p);
  if (st != W4_OK) return st;
  c.n_copies = p.s.n_copies;
  c.src = p.s.src;
  c.dst = p.s.dst;
  c.tokens = p.s.tokens;
  return kv8::copy(c, new_batch, stream);
}

extern "C" w4_status w4_kv8_reserve(int32_t* table, int32_t* lens, int32_t* refs,
                                    const int32_t* grow, int batch, int max_pages, int num_pages,
                                    int page_tokens, void* workspace, size_t workspace_bytes,
                                    int32_t* status_dev, unsigned flags, w4_stream_t stream) {
  const w4_status st =
      kv8::check_table(table, lens, refs, batch, max_pages, num_pages, page_tokens);
  if (st != W4_OK) return st;
  if ((flags & ~W4_FLAG_PDL) != 0) return W4_ERR_ARG;
  if (kv8::misaligned(grow, 4) || kv8::misaligned(workspace, 16)) return W4_ERR_ALIGN;
  if (workspace == nullptr || workspace_bytes < w4_kv8_pages_workspace_bytes(batch, num_pages))
    return W4_ERR_WORKSPACE;
  kv8::ReserveParams p = {};
  p.r = {table, lens, batch, max_pages, kv8::log2_of(page_tokens), num_pages};
  p.table = table;
  p.lens = lens;
  p.refs = refs;
  p.grow = grow;
  kv8::carve(workspace, batch, num_pages, &p.s);
  p.status = status_dev;
  return kv8::launch(kv8::reserve_kernel, dim3(kv8::kRanks), kv8::kPlanThreads, 0, stream, p);
}

extern "C" w4_status w4_kv8_compact(int32_t* new_table, int32_t* new_refs, int32_t* used,
                                    const int32_t* table, const int32_t* lens,
                                    const int32_t* refs, int batch, int max_pages,
                                    const w4_kv8_cache* caches, int n_caches, void* workspace,
                                    size_t workspace_bytes, int32_t* status_dev, unsigned flags,
                                    w4_stream_t stream) {
  kv8::CopyParams c = {};
  int num = 0;
  w4_status st = kv8::view_caches(caches, n_caches, &c, &num);
  if (st != W4_OK) return st;
  if ((st = kv8::check_table(table, lens, refs, batch, max_pages, num, c.P)) != W4_OK) return st;
  if (new_table == nullptr || new_refs == nullptr || used == nullptr ||
      (flags & ~W4_FLAG_PDL) != 0)
    return W4_ERR_ARG;
  if (kv8::misaligned(new_table, 4) || kv8::misaligned(new_refs, 4) || kv8::misaligned(used, 4) ||
      kv8::misaligned(workspace, 16))
    return W4_ERR_ALIGN;
  const size_t all = (size_t)max_pages * 4 * batch;
  if (kv8::overlap(table, new_table, all, all) ||
      kv8::overlap(refs, new_refs, 4 * (size_t)num, 4 * (size_t)num))
    return W4_ERR_ARG;
  if (workspace == nullptr || workspace_bytes < w4_kv8_pages_workspace_bytes(batch, num))
    return W4_ERR_WORKSPACE;
  kv8::CompactParams p = {};
  p.r = {table, lens, batch, max_pages, kv8::log2_of(c.P), num};
  p.refs = refs;
  p.new_table = new_table;
  p.new_refs = new_refs;
  p.used = used;
  kv8::carve(workspace, batch, num, &p.s);
  p.status = status_dev;
  st = kv8::launch(kv8::compact_kernel, dim3(kv8::kRanks), kv8::kPlanThreads, 0, stream, p);
  if (st != W4_OK) return st;
  c.n_copies = p.s.n_copies;
  c.src = p.s.src;
  c.dst = p.s.dst;
  c.tokens = p.s.tokens;
  return kv8::copy(c, num / 2 + 1, stream);
}
