// Who has which page of the 8-bit cache: forks, growth and compaction
// (w4_kv8_fork, w4_kv8_reserve, w4_kv8_compact).
//
// Each call decides in one kernel whose barriers separate its phases: counts of
// references by atomics (whole numbers, so their order does not matter),
// decisions in row order by block scans, free pages in page order by a scan over
// contiguous shares of the pages.  A small pool is decided by one CTA with its
// counts in shared memory, a large one by a cluster of 8 with counts in the
// workspace (Team<R>; every CTA repeats the scans over rows).  Latency bounds
// both: a phase is a chain of a barrier and one or two loads.  Tables are
// walked in pieces of kPiece entries, one piece a warp, so that one long row has
// as many readers as many short ones.  What has to be copied goes into a list in
// the workspace; copy_kernel moves it in every cache, one warp for the keys or
// values of one (page, head), four 16-byte loads a lane in flight.
// Four beams forked and grown 9.8 us, 128 beams over 30 layers 21 us (27 with
// everything cold), 3400 pages of 16 layers made dense 147 us, 7.4 TB/s.  Growth by
// many pages is serial: a prompt of 131072 tokens in pages of 16 takes 249 us in a small
// pool and 1290 in a large one, where each free page comes through L2.
#include <initializer_list>
#include <mutex>

#include "kv8.cuh"

namespace w4 {
namespace kv8 {
namespace {

constexpr int kRanks = 8, kPlanThreads = 1024;
constexpr int kPiece = 128;
constexpr int kTogether = 4;   // pieces, or pages, of a warp or thread that are on their way at once
// One CTA's largest pool (three counts a page in its shared memory) and most pieces of a table: a
// fork of 128 pieces takes it 11.5 us, the cluster 18; of 512 pieces 30 and 21.
constexpr int kOnePages = 16384;
constexpr long long kOnePieces = 256;
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
// The threads that decide: one CTA, or a cluster of R.  sync(): what any of them wrote before is
// seen after; words that others wrote are read by get(), through L2 where they may be global.
template <int R>
struct Team {
  static constexpr int kAll = R * kPlanThreads;
  static __device__ __forceinline__ uint32_t rank() {
    if constexpr (R == 1) return 0;
    return cluster_rank();
  }
  static __device__ __forceinline__ void sync() {
    if constexpr (R == 1) {
      __syncthreads();
    } else {
      asm volatile("barrier.cluster.arrive.release;" ::: "memory");
      asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    }
  }
  static __device__ __forceinline__ int get(const int32_t* p) {
    if constexpr (R == 1) return *p;
    return __ldcg(p);
  }
};
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

// The pieces of a warp: every 32nd (or 256th) of the rows' pieces in turn, without a division each.
struct Pieces {
  int each, row, piece, row_step, piece_step;

  __device__ __forceinline__ Pieces(int max_pages, int warp, int warps) {
    each = (max_pages - 1) / kPiece + 1;
    row = warp;
    piece = 0;
    row_step = warps;
    piece_step = 0;
    if (each > 1) {   // divisions that a CTA of 32 warps feels
      row = warp / each;
      piece = warp - row * each;
      row_step = warps / each;
      piece_step = warps - row_step * each;
    }
  }
  __device__ __forceinline__ void next() {
    row += row_step;
    piece += piece_step;
    if (piece >= each) {
      piece -= each;
      ++row;
    }
  }
};

// A lane's entries of a piece, all on their way at once; kNone past the row's pages.
constexpr int kNone = (int)0x80000000;
__device__ __forceinline__ void load_piece(const Rows& r, int b, int first, int pages, int (&pg)[kPiece / 32]) {
  const int32_t* row = r.table + (long long)b * r.max_pages + first;
#pragma unroll
  for (int z = 0; z < kPiece / 32; ++z) pg[z] = first + 32 * z < pages ? load_in(row + 32 * z) : kNone;
}

// Pages of every old row into row_pages, -1 where its length or one of its
// entries breaks its bounds.  len: the length of row gt, if there is one.  Ends in a barrier.
template <int R>
__device__ __forceinline__ void check_rows(const Rows& r, int len, int32_t* row_pages, uint32_t rank,
                                           int32_t* status) {
  using T = Team<R>;
  const int gt = rank * kPlanThreads + threadIdx.x;
  static_assert(W4_KV8_MAX_BATCH <= kRanks * kPlanThreads && kOnePieces <= kPlanThreads, "a row a thread");
  if (gt < r.batch) {
    const int np = r.pages(len);
    row_pages[gt] = np;
    if (np < 0) report(status, W4_ERR_INDEX);
  }
  T::sync();
  const int lane = threadIdx.x & 31;
  // several pieces' entries on their way at once: in a cold table each is a trip to memory
  for (Pieces i(r.max_pages, gt >> 5, T::kAll / 32); i.row < r.batch;) {
    int pg[kTogether][kPiece / 32], row[kTogether];
#pragma unroll
    for (int y = 0; y < kTogether; ++y) {
      row[y] = i.row;
      const bool there = i.row < r.batch;
      load_piece(r, there ? i.row : 0, i.piece * kPiece + lane, there ? T::get(row_pages + i.row) : 0, pg[y]);
      i.next();
    }
#pragma unroll
    for (int y = 0; y < kTogether; ++y) {
      bool bad = false;
#pragma unroll
      for (int z = 0; z < kPiece / 32; ++z)
        bad |= pg[y][z] != kNone && (pg[y][z] < 0 || pg[y][z] >= r.num_pages);
      if (__any_sync(kFull, bad) && lane == 0) {
        row_pages[row[y]] = -1;
        report(status, W4_ERR_INDEX);
      }
    }
  }
  T::sync();
}

// This thread's share of the pages, in page order over the team.
template <int R>
__device__ __forceinline__ void my_share(int num_pages, uint32_t rank, int* lo, int* hi) {
  const long long all = Team<R>::kAll;
  const long long each = ((num_pages + all - 1) / all) | 1;   // odd: no two threads of a warp in one bank
  const long long a = ((long long)rank * kPlanThreads + threadIdx.x) * each;
  *lo = (int)min(a, (long long)num_pages);
  *hi = (int)min(a + each, (long long)num_pages);
}

// Sum of `mine` (the same in all threads of a CTA) over the ranks before this
// one, and over all.  slot: shared memory of this use alone.  A barrier.
template <int R>
__device__ __forceinline__ int before_rank(int mine, int* slot, uint32_t rank, int* total) {
  if constexpr (R == 1) {
    __syncthreads();
    *total = mine;
    return 0;
  }
  if (threadIdx.x == 0) *slot = mine;
  Team<R>::sync();
  int before = 0, all = 0;
  for (int i = 0; i < R; ++i) {
    const int v = remote(slot, i);
    all += v;
    if (i < (int)rank) before += v;
  }
  *total = all;
  return before;
}

// Free pages of this thread's share.
template <int R>
__device__ __forceinline__ int count_free(const int32_t* refs, int num_pages, uint32_t rank) {
  int lo, hi, free = 0;
  my_share<R>(num_pages, rank, &lo, &hi);
#pragma unroll 4
  for (int i = lo; i < hi; ++i) free += Team<R>::get(refs + i) == 0;
  return free;
}

// The lowest `want` free pages into list, in order; false (everywhere) if there
// are fewer.  free: count_free().  Ends in a barrier: what every rank read before
// the call may be written after it.
template <int R>
__device__ __forceinline__ bool take_free(const int32_t* refs, int num_pages, long long want, int free,
                                          int32_t* list, uint32_t rank, int* red, int* slot) {
  using T = Team<R>;
  if (want == 0) {
    T::sync();
    return true;
  }
  int total, all;
  int at = block_scan(free, red, &total);
  at += before_rank<R>(total, slot, rank, &all);
  const bool ok = all >= want;
  if (ok && free > 0 && at < want) {
    int lo, hi;
    my_share<R>(num_pages, rank, &lo, &hi);
    for (int i = lo; i < hi && at < want; ++i)
      if (T::get(refs + i) == 0) list[at++] = i;
  }
  T::sync();
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

template <int R>
__global__ void __launch_bounds__(kPlanThreads, 1) fork_kernel(const __grid_constant__ ForkParams p) {
  using T = Team<R>;
  extern __shared__ int32_t sm[];
  __shared__ int red[33], slot;
  // one CTA: what it knows of its rows (old ones' pages; new ones' lengths, last pages and parents)
  // and the pages that it takes
  __shared__ int32_t of_rows[5][R == 1 ? kOnePieces : 1];
  pdl_wait();
  const uint32_t rank = T::rank();
  const int gt = rank * kPlanThreads + threadIdx.x, lane = threadIdx.x & 31;
  const Rows& r = p.old;
  int32_t* refs = R == 1 ? sm : p.new_refs;
  int32_t* count = R == 1 ? sm + r.num_pages : p.s.count;
  int32_t* first = R == 1 ? sm + 2 * r.num_pages : p.s.first;
  int32_t* row_pages = R == 1 ? of_rows[0] : p.s.row_pages;
  int32_t* new_lens = R == 1 ? of_rows[1] : p.new_lens;
  int32_t* list = R == 1 ? of_rows[3] : p.s.dst;
  const int32_t* parents = R == 1 ? of_rows[4] : p.parents;
  // what a call starts from comes in one trip to memory
  const int len = gt < r.batch ? load_in(r.lens + gt) : 0;
  const int parent = R == 1 && gt < p.new_batch ? load_in(p.parents + gt) : 0;
  for (int i0 = gt; i0 < r.num_pages; i0 += kTogether * T::kAll) {
    int v[kTogether];
#pragma unroll
    for (int z = 0; z < kTogether; ++z)
      if (i0 + z * T::kAll < r.num_pages) v[z] = load_in(p.refs + i0 + z * T::kAll);
#pragma unroll
    for (int z = 0; z < kTogether; ++z) {
      const int i = i0 + z * T::kAll;
      if (i >= r.num_pages) break;
      refs[i] = v[z];
      count[i] = 0;
      first[i] = 0x7fffffff;
    }
  }
  if constexpr (R == 1)
    if (gt < p.new_batch) of_rows[4][gt] = parent;
  check_rows<R>(r, len, row_pages, rank, p.status);
  // the old rows' names go, the new rows' come
  const int rows = max(r.batch, p.new_batch);
  for (Pieces i(r.max_pages, gt >> 5, T::kAll / 32); i.row < rows; i.next()) {
    const int b = i.row, at = i.piece * kPiece;
    const int par = b < p.new_batch ? T::get(parents + b) : -1;
    const int had = b < r.batch ? T::get(row_pages + b) : 0;
    int np = 0, len = 0;
    bool ok = par >= -1 && par < r.batch;
    if (ok && par >= 0) {
      np = T::get(row_pages + par);
      len = load_in(r.lens + par);
      ok = np >= 0;
    }
    if (!ok) {
      if (at == 0 && lane == 0) {
        new_lens[b] = -1;
        report(p.status, W4_ERR_INDEX);
      }
      continue;
    }
    int mine[kPiece / 32], come[kPiece / 32];
    load_piece(r, b, at + lane, par != b ? had : 0, mine);
    load_piece(r, par, at + lane, np, come);
    int32_t* row = p.new_table + (long long)b * r.max_pages + at + lane;
#pragma unroll
    for (int z = 0; z < kPiece / 32; ++z) {
      if (at + 32 * z >= max(had, np)) break;
      if (mine[z] != kNone) atomicSub(refs + mine[z], 1);
      const int pg = come[z], e = at + lane + 32 * z;
      if (pg == kNone) continue;
      row[32 * z] = pg;
      if (par != b) atomicAdd(refs + pg, 1);
      if (e == np - 1 && (len & ((1 << r.shift) - 1)) != 0) {   // a page to be written to
        atomicAdd(count + pg, 1);
        atomicMin(first + pg, b);
        if constexpr (R == 1) of_rows[2][b] = pg;
      }
    }
    if (at == 0 && lane == 0 && b < p.new_batch) new_lens[b] = len;
  }
  T::sync();
  // rows that need a page of their own, in order
  int page[kRowsEach], used[kRowsEach], last[kRowsEach], mine = 0;
#pragma unroll
  for (int z = 0; z < kRowsEach; ++z) {
    const int b = threadIdx.x * kRowsEach + z;
    page[z] = -1;
    if (b >= p.new_batch) continue;
    const int len = T::get(new_lens + b);
    used[z] = len & ((1 << r.shift) - 1);
    if (len <= 0 || used[z] == 0) continue;
    last[z] = r.pages(len) - 1;
    const int pg = R == 1 ? of_rows[2][b]
                          : T::get(p.new_table + (long long)b * r.max_pages + last[z]);
    if (T::get(count + pg) == T::get(refs + pg) && T::get(first + pg) == b) continue;
    page[z] = pg;
    ++mine;
  }
  int want;
  int at = block_scan(mine, red, &want);
  const int free = want != 0 ? count_free<R>(refs, r.num_pages, rank) : 0;
  const bool ok = take_free<R>(refs, r.num_pages, want, free, list, rank, red, &slot);
  if (rank != 0) return;
  if (threadIdx.x == 0) {
    *p.s.n_copies = ok ? want : 0;
    if (!ok) report(p.status, W4_ERR_STATE);
  }
  if (!ok) {
    for (int b = threadIdx.x; b < p.new_batch; b += kPlanThreads) p.new_lens[b] = -1;
    return;
  }
#pragma unroll
  for (int z = 0; z < kRowsEach; ++z) {
    if (page[z] < 0) continue;
    const int to = T::get(list + at);
    p.new_table[(long long)(threadIdx.x * kRowsEach + z) * r.max_pages + last[z]] = to;
    atomicSub(refs + page[z], 1);
    refs[to] = 1;
    p.s.src[at] = page[z];
    if constexpr (R == 1) p.s.dst[at] = to;
    p.s.tokens[at] = used[z];
    ++at;
  }
  if constexpr (R == 1) {
    for (int b = threadIdx.x; b < p.new_batch; b += kPlanThreads) p.new_lens[b] = new_lens[b];
    __syncthreads();
    for (int i = threadIdx.x; i < r.num_pages; i += kPlanThreads) p.new_refs[i] = refs[i];
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

template <int R>
__global__ void __launch_bounds__(kPlanThreads, 1) reserve_kernel(const __grid_constant__ ReserveParams p) {
  using T = Team<R>;
  __shared__ long long red64[33];
  __shared__ int red[33], slot;
  pdl_wait();
  const uint32_t rank = T::rank();
  const int free = count_free<R>(p.refs, p.r.num_pages, rank);   // needed by most calls; beside the lengths
  int from[kRowsEach], to[kRowsEach], len[kRowsEach];
  long long mine = 0;
#pragma unroll
  for (int z = 0; z < kRowsEach; ++z) {
    const int b = threadIdx.x * kRowsEach + z;
    from[z] = to[z] = len[z] = -1;
    if (b >= p.r.batch) continue;
    const int now = load_in(p.lens + b);
    const int g = p.grow != nullptr ? load_in(p.grow + b) : now > 0;
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
  const bool ok = take_free<R>(p.refs, p.r.num_pages, want, free, p.s.dst, rank, red, &slot);
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
      const int pg = T::get(p.s.dst + at++);
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

template <int R>
__global__ void __launch_bounds__(kPlanThreads, 1) compact_kernel(const __grid_constant__ CompactParams p) {
  using T = Team<R>;
  extern __shared__ int32_t sm[];
  __shared__ int red[33], slot[3];
  __shared__ int32_t of_rows[R == 1 ? kOnePieces : 1];
  pdl_wait();
  const uint32_t rank = T::rank();
  const int gt = rank * kPlanThreads + threadIdx.x, lane = threadIdx.x & 31;
  const Rows& r = p.r;
  int32_t* refs = R == 1 ? sm : p.new_refs;
  int32_t* count = R == 1 ? sm + r.num_pages : p.s.count;
  int32_t* to = R == 1 ? sm + 2 * r.num_pages : p.s.first;   // where each page goes
  const int len = gt < r.batch ? load_in(r.lens + gt) : 0;
  for (int i0 = gt; i0 < r.num_pages; i0 += kTogether * T::kAll) {
    int v[kTogether];
#pragma unroll
    for (int z = 0; z < kTogether; ++z)
      if (i0 + z * T::kAll < r.num_pages) v[z] = load_in(p.refs + i0 + z * T::kAll);
#pragma unroll
    for (int z = 0; z < kTogether; ++z) {
      const int i = i0 + z * T::kAll;
      if (i >= r.num_pages) break;
      refs[i] = v[z];
      count[i] = 0;
      to[i] = i;
    }
  }
  int32_t* row_pages = R == 1 ? of_rows : p.s.row_pages;
  if (gt == 0) *p.used = 0;
  check_rows<R>(r, len, row_pages, rank, p.status);
  for (Pieces i(r.max_pages, gt >> 5, T::kAll / 32); i.row < r.batch; i.next()) {
    const int b = i.row, at = i.piece * kPiece;
    int pg[kPiece / 32];
    load_piece(r, b, at + lane, T::get(row_pages + b), pg);
#pragma unroll
    for (int z = 0; z < kPiece / 32; ++z)
      if (pg[z] != kNone) atomicAdd(count + pg[z], 1);
  }
  int lo, hi;
  my_share<R>(r.num_pages, rank, &lo, &hi);
  int live = 0, total, n;
  for (int i = lo; i < hi; ++i) live += T::get(refs + i) != 0;
  block_scan(live, red, &total);
  before_rank<R>(total, slot, rank, &n);   // a barrier: the counts are complete
  int from = 0, hole = 0;
  for (int i = lo; i < hi; ++i) {
    const int c = T::get(refs + i);
    from += i >= n && c != 0 && T::get(count + i) == c;
    hole += i < n && c == 0;
  }
  int moves, holes;
  int fat = block_scan(from, red, &total);
  fat += before_rank<R>(total, slot + 1, rank, &moves);
  int hat = block_scan(hole, red, &total);
  hat += before_rank<R>(total, slot + 2, rank, &holes);
  for (int i = lo; i < hi; ++i) {
    const int c = T::get(refs + i);
    if (i >= n && c != 0 && T::get(count + i) == c) p.s.src[fat++] = i;
    if (i < n && c == 0 && hat < moves) p.s.dst[hat++] = i;
  }
  T::sync();
  for (int j = gt; j < moves; j += T::kAll) {
    const int a = T::get(p.s.src + j), b = T::get(p.s.dst + j);
    to[a] = b;
    refs[b] = T::get(refs + a);
    refs[a] = 0;
    p.s.tokens[j] = 1 << r.shift;
  }
  if (gt == 0) *p.s.n_copies = moves;
  T::sync();
  for (Pieces i(r.max_pages, gt >> 5, T::kAll / 32); i.row < r.batch; i.next()) {
    const int b = i.row, at = i.piece * kPiece;
    int pg[kPiece / 32];
    load_piece(r, b, at + lane, T::get(row_pages + b), pg);
#pragma unroll
    for (int z = 0; z < kPiece / 32; ++z)
      if (pg[z] != kNone)
        p.new_table[(long long)b * r.max_pages + at + lane + 32 * z] = T::get(to + pg[z]);
  }
  int most = 0;
  for (int i = lo; i < hi; ++i)
    if (T::get(refs + i) != 0) most = i + 1;
  most = __reduce_max_sync(kFull, most);
  if (lane == 0 && most > 0) atomicMax(p.used, most);
  if constexpr (R == 1)
    for (int i = threadIdx.x; i < r.num_pages; i += kPlanThreads) p.new_refs[i] = refs[i];
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
  pdl_wait();
  const int lane = threadIdx.x & 31, copies = load_in(p.n_copies);
  // the warp's items: (copy, cache, head, keys or values) in turn, without a division each
  const int warps = gridDim.x * (kCopyThreads / 32), first = blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5);
  int kv = first & 1, h = (first >> 1) % p.H, l = (first >> 1) / p.H % p.n, j = (first >> 1) / p.H / p.n;
  const int kv_step = warps & 1, h_step = (warps >> 1) % p.H, l_step = (warps >> 1) / p.H % p.n,
            j_step = (warps >> 1) / p.H / p.n;
  auto next = [&]() {
    kv += kv_step;
    h += h_step + (kv >> 1);
    kv &= 1;
    int carry = h >= p.H;
    h -= carry ? p.H : 0;
    l += l_step + carry;
    carry = l >= p.n;
    l -= carry ? p.n : 0;
    j += j_step + carry;
  };
  for (; j < copies; next()) {
    const bool is_v = kv != 0;
    const One& c = p.c[l];
    const int from = load_in(p.src + j), to = load_in(p.dst + j), tokens = load_in(p.tokens + j);
    uint8_t* codes = (is_v ? c.vc : c.kc) + h * c.head_stride;
    const uint4* a = reinterpret_cast<const uint4*>(codes + from * c.page_stride);
    uint4* b = reinterpret_cast<uint4*>(codes + to * c.page_stride);
    const int n = tokens * p.D / 16;
    const long long ph = (long long)from * p.H + h, qh = (long long)to * p.H + h;
    // what goes with the codes, on its way with the first of them
    float step = 0.0f, weight[4] = {};
    uint4 range = {};
    const bool ranged = !is_v && c.ranges != nullptr && lane < p.D / 8;
    const bool weighed = is_v && c.weight != nullptr;
    if (lane == 0) step = (is_v ? c.vs : c.ks)[ph];
    if (ranged) range = reinterpret_cast<const uint4*>(c.ranges + ph * 2 * p.D)[lane];
    if (weighed)
#pragma unroll
      for (int z = 0; z < 4; ++z)
        if (lane + 32 * z < tokens) weight[z] = c.weight[ph * p.P + lane + 32 * z];
    int e = lane;
    for (; e + 96 < n; e += 128) {
      uint4 v[4];
#pragma unroll
      for (int z = 0; z < 4; ++z) v[z] = a[e + 32 * z];
#pragma unroll
      for (int z = 0; z < 4; ++z) b[e + 32 * z] = v[z];
    }
    uint4 v[3];
#pragma unroll
    for (int z = 0; z < 3; ++z)
      if (e + 32 * z < n) v[z] = a[e + 32 * z];
#pragma unroll
    for (int z = 0; z < 3; ++z)
      if (e + 32 * z < n) b[e + 32 * z] = v[z];
    if (lane == 0) (is_v ? c.vs : c.ks)[qh] = step;
    if (ranged) reinterpret_cast<uint4*>(c.ranges + qh * 2 * p.D)[lane] = range;
    if (weighed)
#pragma unroll
      for (int z = 0; z < 4; ++z)
        if (lane + 32 * z < tokens) c.weight[qh * p.P + lane + 32 * z] = weight[z];
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

struct Span {
  const void* p;
  size_t words;
};

// Whether one of the call's outputs overlaps another one or an input (read by some CTAs while others
// write).
bool overlap(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  auto meet = [](const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + 4 * b.words && y < x + 4 * a.words;
  };
  for (const Span& o : outs) {
    for (const Span& i : ins)
      if (meet(o, i)) return true;
    for (const Span& other : outs)
      if (&other != &o && meet(o, other)) return true;
  }
  return false;
}

w4_status check_table(const int32_t* table, const int32_t* lens, const int32_t* refs, int batch,
                      int max_pages, int num_pages, int P) {
  if (table == nullptr || lens == nullptr || refs == nullptr || batch < 1 || max_pages < 1 ||
      num_pages < 1)
    return W4_ERR_ARG;
  if (batch > W4_KV8_MAX_BATCH || max_pages > (1 << 26) || num_pages > (1 << 30) || (P != 16 && P != 32 && P != 64 && P != 128))
    return W4_ERR_SHAPE;
  if (misaligned(table, 4) || misaligned(lens, 4) || misaligned(refs, 4)) return W4_ERR_ALIGN;
  return W4_OK;
}

int log2_of(int p) { return p == 16 ? 4 : p == 32 ? 5 : p == 64 ? 6 : 7; }

// At most this many copies: a CTA for every eight warps' worth, as many as stay resident.
w4_status copy(const CopyParams& p, long long most, w4_stream_t stream) {
  const long long items = most * p.n * p.H * 2, ctas = (items + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
  return launch(copy_kernel, dim3((unsigned)min(ctas, 152ll * 8)), kCopyThreads, 0, stream, p);
}

// The decision of a call: by one CTA where the pool and the table are small.
template <typename P>
w4_status decide(void (*one)(P), void (*team)(P), const P& p, long long rows, int max_pages, int num_pages,
                 int words, w4_stream_t stream) {
  const long long pieces = (max_pages + kPiece - 1) / kPiece;
  if (num_pages <= kOnePages && rows * pieces <= kOnePieces) {
    const size_t smem = (size_t)words * 4 * num_pages;
    if (smem > 24 << 10) {   // once for each device and kernel: more shared memory than the default
      static std::mutex mu;
      static bool done[64] = {};
      int dev = 0;
      if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return W4_ERR_DEVICE;
      std::lock_guard<std::mutex> lock(mu);
      if (!done[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(one, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   words * 4 * kOnePages);
        if (e != cudaSuccess) {
          note_cuda_error(e);
          (void)cudaGetLastError();
          return W4_ERR_LAUNCH;
        }
        done[dev] = true;
      }
    }
    return launch(one, dim3(1), kPlanThreads, smem, stream, p);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kRanks);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kRanks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, team, p);
  if (e != cudaSuccess) {
    note_cuda_error(e);
    (void)cudaGetLastError();
    return W4_ERR_LAUNCH;
  }
  return W4_OK;
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
  const size_t row = (size_t)max_pages, nb = (size_t)new_batch, ob = (size_t)batch, pages = (size_t)num;
  if (kv8::overlap({{new_table, row * nb}, {new_lens, nb}, {new_refs, pages}},
                   {{table, row * ob}, {lens, ob}, {refs, pages}, {parents, nb}}))
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
  st = kv8::decide(kv8::fork_kernel<1>, kv8::fork_kernel<kv8::kRanks>, p, most, max_pages, num, 3, stream);
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
  return kv8::decide(kv8::reserve_kernel<1>, kv8::reserve_kernel<kv8::kRanks>, p, 1, 1, num_pages, 0, stream);
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
  const size_t all = (size_t)max_pages * batch, pages = (size_t)num;
  if (kv8::overlap({{new_table, all}, {new_refs, pages}, {used, 1}},
                   {{table, all}, {lens, (size_t)batch}, {refs, pages}}))
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
  st = kv8::decide(kv8::compact_kernel<1>, kv8::compact_kernel<kv8::kRanks>, p, batch, max_pages, num, 3, stream);
  if (st != W4_OK) return st;
  c.n_copies = p.s.n_copies;
  c.src = p.s.src;
  c.dst = p.s.dst;
  c.tokens = p.s.tokens;
  return kv8::copy(c, num / 2 + 1, stream);
}
