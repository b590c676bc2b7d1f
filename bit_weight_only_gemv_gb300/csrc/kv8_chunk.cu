// Attention over the 8-bit cache for prompt chunks (many query rows on a key
// head) on the 5th-generation tensor cores (tcgen05, sm_103a).
//
// The rows of a (sequence, key head) are its tokens times the group's query
// heads, 128 to a tile.  A CTA takes one or two row tiles against a run of
// key tiles, with a running maximum m and sum l:
//
//   S = Q K^T          kind::f16, bf16 operands (a code is exact in bf16)
//   P = 2^(scale log2(e) ks S - m) vs
//   O += P V           kind::tf32, P from tensor memory, codes exact
//
// P stays in tensor memory in S's own columns, as fp32 bits rounded to tf32:
// 11 significant bits at every magnitude, so no weight is lost however far
// below the row's largest it lies, and no conversion or packing is needed.  That
// costs PV twice the tensor time of a 16-bit P; as the softmax warps are the
// limit, little of that shows.  For the same reason m need not be
// the maximum: it is the largest score of the row's first 32 keys, and moves
// (with O and l rescaled) only when a score passes it by 2^60.
//
// Roles: four softmax warps per row tile (a thread owns a row, so maxima and
// sums need no exchange), six warps that expand the codes (K to bf16, V to
// fp32 transposed, both in the 128-byte-swizzled K-major layout), one warp
// that issues the MMAs, one that issues the tiled copies of pages.  Two row
// tiles take turns: while one's scores go through the softmax, the tensor
// cores work for the other.  A unit of one row tile gives its key tiles to
// the two softmax groups in turn and joins them at the end.
//
// Work is cut into equal runs of key tiles over all units, one run a CTA
// (kv8_runs.cuh); parts of a cut unit meet in the workspace and are joined in
// order by a second small kernel.  Every wait is bounded.
//
// 256 rows of 32 heads on 8 of 128 channels against 16k keys: 112 us, 0.61
// PFLOP/s.  Of about 3400 cycles per 64 keys a softmax group computes 2300 (four
// warps, one per scheduler, beside the expansion and the issuing), the tensor
// cores 1792 for both groups; one issuing warp keeps up (one per group: 133 us), and
// neither 64 scores in registers at once (121 us) nor 128-key tiles (145 us)
// were faster.
#include <algorithm>
#include <mutex>

#include "gemv_host.h"
#include "kv8_attn.h"
#include "kv8_runs.cuh"
#include "kv8_tc.cuh"

namespace w4 {
namespace kv8 {
namespace {

using tc::kWaitCycles;
using tc::tc_fence_after;
using tc::tc_fence_before;
using tc::wait_bar;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kPass = 60.0f;        // log2 of how far a score may pass m
constexpr float kFar = 1152921504606846976.0f;   // 2^60
constexpr float kRound = 1.0f + 0.72f / 2048.0f;
constexpr int kRowTile = 128;
constexpr int kKeys = 64;             // keys of a tile
constexpr int kMetaRing = 16;         // tiles described ahead of their softmax
constexpr int kUnitRing = 32;         // units of which a refusal is remembered
// Key tiles of a CTA's run, at least: 128 rows of 8 heads on 2 of 64 channels
// against 4k keys 31.6 us (2: 48.5, 8: 28.4, 16: 33.4), 64 rows of 16 on 4 of 256
// against 1000 28.8 (2: 28.5, 8: 33.4, 16: 35.6), 256 rows of 16 on 4 of 128 against
// 2000 32.4 (2: 34.7, 8: 34.2, 16: 42.3).
constexpr int kMinTiles = 4;

// The same for roles that work ahead of the others: they leave the issue slots
// to those while they wait.
__device__ __forceinline__ bool wait_idle(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    __nanosleep(64);
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag != 0) return false;
    if (clock64() - t0 > kWaitCycles) return false;
  }
}

template <int D>
struct Shape {
  static constexpr int kGroups = D == 256 ? 1 : 2;   // softmax groups (and O accumulators)
  static constexpr int kRows = kRowTile * kGroups;   // query rows of a unit
  static constexpr int kSoftWarps = 4 * kGroups;
  static constexpr int kConvWarp = kSoftWarps;
  static constexpr int kConvWarps = 6;               // 16 warps in all with two groups
  static constexpr int kMmaWarp = kConvWarp + kConvWarps;
  static constexpr int kCopyWarp = kMmaWarp + 1;
  static constexpr int kWarps = kCopyWarp + 1;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kBuf = D == 256 ? 1 : 2;      // expanded tiles of K, and of V
  static constexpr int kRaw = D == 256 ? 2 : 4;      // copied tiles of K, and of V
  static constexpr int kQTile = kRowTile * D * 2;    // bytes
  static constexpr int kKTile = kKeys * D * 2;
  static constexpr int kVTile = kKeys * D * 4;
  static constexpr int kRawTile = kKeys * D;
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + kGroups * kQTile;
  static constexpr int kV = kK + kBuf * kKTile;
  static constexpr int kRawK = kV + kBuf * kVTile;
  static constexpr int kRawV = kRawK + kRaw * kRawTile;
  static constexpr int kMeta = kRawV + kRaw * kRawTile;   // [kMetaRing][4] (ks, vs) of 16 keys
  static constexpr int kPages = kMeta + kMetaRing * 4 * 8;  // [kMetaRing][4]
  static constexpr int kBars = kPages + kMetaRing * 4 * 4;
  static constexpr int kMisc = kBars + 40 * 8;
  static constexpr int kEnd = kMisc + 512 + 1024;
  // more than half an SM's: each CTA holds all of its tensor memory
  static constexpr int kSmem = kEnd > 117248 ? kEnd : 117248;
  static_assert(kSmem <= 232448 && 2 * kSmem > 232448, "shared memory");
  // tensor memory columns: S (and P) regions of a tile, then O
  static constexpr int kRegions = 2 * kGroups;
  static constexpr int kOCol = kRegions * kKeys;
  static_assert(kOCol + kGroups * D <= 512, "tensor memory");
};

// barriers
enum {
  kRawKFull = 0,   // [4] by stage
  kRawKEmpty = 4,
  kRawVFull = 8,
  kRawVEmpty = 12,
  kQReady = 16, kQFree,
  kKReady = 18,    // [2] by buffer
  kKFree = 20,
  kVReady = 22,
  kVFree = 24,
  kSFull = 26,     // [4] by S region
  kPFull = 30,
  kODone = 34,     // [2] by group
  kOFree = 36,
  kEpi = 38,
  kBarCount
};

struct ChunkParams {
  CUtensorMap tm_k, tm_v;
  Cache c;
  Batch bt;
  ChunkArgs a;
  int G;
  int rts;            // row tiles (units) of a (sequence, head), at most
  long long* cut;     // [2 + B * H * rts]: total and CTAs of the runs, then each unit's
                      // first item, -1 where the unit's outputs are written already
  float* parts;       // [4 * CTAs][rows][D]
  float* part_stats;  // [4 * CTAs][rows][2]: m, l (l = -1: refused)
};

// One unit of a run: a row tile (pair) of a (sequence, head), key tiles i0 .. i1 - 1 of it.
struct Unit {
  Seq s;
  Tile t;
  int b, h, rt, i0, i1, rows, R;   // rows: of this unit; R: of the (sequence, head)
  long long u0;                    // item of the unit's tile 0
  __device__ __forceinline__ bool whole() const { return i0 == 0 && i1 == t.slices; }
  __device__ __forceinline__ int tiles() const { return i1 - i0; }
};

template <int D>
__device__ __forceinline__ long long entry_tiles(const ChunkParams& p, int b, int* units) {
  using S = Shape<D>;
  const Seq s = sequence(p.bt, p.c.P, b);
  if (!s.ok || s.n == 0) return 0;
  *units += (s.n * p.G + S::kRows - 1) / S::kRows * p.c.H;
  return head_slices(s, p.G, p.a.window, S::kRows, kKeys) * p.c.H;
}

// Walks the units of a run; every role walks alike.
struct Walk {
  long long g, off;
  int entry;
};

template <int D>
__device__ __noinline__ bool next_unit(const ChunkParams& p, const Run& run, Walk& w, Unit& u) {
  using S = Shape<D>;
  if (w.g >= run.g1) return false;
  u.b = w.entry;
  u.s = sequence(p.bt, p.c.P, u.b);
  u.R = u.s.n * p.G;
  const long long per = head_slices(u.s, p.G, p.a.window, S::kRows, kKeys);
  u.h = (int)(w.off / per);
  long long rem = w.off - per * u.h;
  u.rt = 0;
  u.t = tile_of(u.s, p.G, p.a.window, 0, S::kRows, kKeys);
  while (rem >= u.t.slices) {
    rem -= u.t.slices;
    u.t = tile_of(u.s, p.G, p.a.window, ++u.rt, S::kRows, kKeys);
  }
  u.rows = min(S::kRows, u.R - u.rt * S::kRows);
  u.i0 = (int)rem;
  u.i1 = (int)min((long long)u.t.slices, rem + run.g1 - w.g);
  u.u0 = w.g - rem;
  const long long step = u.i1 - u.i0;
  w.g += step;
  w.off += step;
  if (w.off == per * p.c.H && w.g < run.g1) {
    w.off = 0;
    int none = 0;
    do ++w.entry;
    while (entry_tiles<D>(p, w.entry, &none) == 0);
  }
  return true;
}

// 2^(x factor - m) in place, 0 for the columns outside lo .. hi (cut: there
// are some in the warp's rows); returns the sum.
__device__ __forceinline__ float weights(float* x, float f0, float f1, float m, bool cut, int lo,
                                         int hi) {
  const uint64_t a0 = pack2(f0, f0), a1 = pack2(f1, f1), c = pack2(-m, -m);
#pragma unroll
  for (int e = 0; e < 32; e += 2)
    unpack2(fma2(pack2(x[e], x[e + 1]), e < 16 ? a0 : a1, c), x[e], x[e + 1]);
  if (cut) {
    const uint32_t seen = columns(lo, hi);
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (!(seen >> e & 1u)) x[e] = -INFINITY;
  }
  uint64_t s0 = 0, s1 = 0;   // two sums of pairs
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
#pragma unroll
    for (int k = 0; k < 4; ++k) x[e + k] = exp2_fast(x[e + k]);
    s0 = add2(s0, pack2(x[e], x[e + 1]));
    s1 = add2(s1, pack2(x[e + 2], x[e + 3]));
  }
  float a, b;
  unpack2(add2(s0, s1), a, b);
  return a + b;
}

// Multiply 32 columns from `col` on by this thread's factor.
__device__ __forceinline__ void tmem_scale32(uint32_t col, float factor) {
  float v[32];
  tc::tmem_ld<32>(col, v);
  tc::tmem_wait_ld<32>(v);
#pragma unroll
  for (int e = 0; e < 32; ++e) v[e] *= factor;
  tmem_st32(col, v);
}

__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int x, int tok, int h,
                                       int page, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(tok), "r"(h), "r"(page), "r"(bar)
      : "memory");
}

__device__ __forceinline__ uint2 pack_bf16x4(const float* v, float f) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0] * f, v[1] * f);
  const __nv_bfloat162 b = __floats2bfloat162_rn(v[2] * f, v[3] * f);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// A constant as an argument.
template <int N>
struct Const {
  static constexpr int value = N;
  __device__ __forceinline__ constexpr operator int() const { return N; }
};

// Parity of the n-th use (from 0) of a ring of N barriers, and of the use
// before it (the first passes at once).
template <int N>
__device__ __forceinline__ uint32_t use(uint32_t n) { return (n / N) & 1u; }
template <int N>
__device__ __forceinline__ uint32_t before(uint32_t n) { return ((n / N) & 1u) ^ 1u; }

// A part's m and l against its largest weight, not against an m that may lie
// 2^60 below it, so that the join's factors reach as far down as fp32 does: l's
// power of two is that weight, or above it by the weights' number.  Returns
// the factor that brings the part's values along.
__device__ __forceinline__ float settle(float2& s) {
  const int e = (int)(__float_as_uint(s.y) >> 23 & 0xFF) - 127;
  if (e <= 0 || e >= 127) return 1.0f;
  const float f = __uint_as_float((uint32_t)(127 - e) << 23);
  s.x += (float)e;
  s.y *= f;
  return f;
}

// Four channels of one row from its parts, in order: part(k) is the row's
// place in the k-th.
template <int D, typename Part>
__device__ __forceinline__ void join_row(const ChunkParams& p, const Seq& s, int h, int row, int c4,
                                         int parts, Part part) {
  const float2* stats = reinterpret_cast<const float2*>(p.part_stats);
  float M = -INFINITY, L = 0.0f;
  bool none = false;
  for (int k = 0; k < parts; ++k) {
    const float2 s2 = __ldcg(stats + part(k));
    M = fmaxf(M, s2.x);
    none |= s2.y < 0.0f;
  }
  if (none) return;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int k = 0; k < parts; ++k) {
    const long long q = part(k);
    const float2 s2 = __ldcg(stats + q);
    const float4 v = __ldcg(reinterpret_cast<const float4*>(p.parts + q * D + 4 * c4));
    const float w = s2.x == -INFINITY ? (s2.y == 0.0f ? 0.0f : 1.0f) : exp2_fast(s2.x - M);
    L += w * s2.y;
    a.x += w * v.x;
    a.y += w * v.y;
    a.z += w * v.z;
    a.w += w * v.w;
  }
  const long long to = (long long)(s.row0 + row / p.G) * p.a.Hq + h * p.G + row % p.G;
  const float o4[4] = {a.x, a.y, a.z, a.w};
  *reinterpret_cast<uint2*>(p.a.out + to * D + 4 * c4) =
      pack_bf16x4(o4, L == 0.0f ? 0.0f : 1.0f / L);
  if (c4 == 0 && p.a.lse != nullptr) p.a.lse[to] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
}

template <int D>
__global__ void __launch_bounds__(Shape<D>::kThreads, 1)
    attn_chunk_kernel(const __grid_constant__ ChunkParams p) {
  using S = Shape<D>;
  constexpr int kGroups = S::kGroups, kBuf = S::kBuf, kRaw = S::kRaw;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_addr(smem_raw) & 1023u)) & 1023u;
  uint8_t* sm = smem_raw + pad;
  const uint32_t sb = smem_addr(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bars = sb + S::kBars;
  auto bar = [&](int i) { return bars + 8 * i; };
  float2* meta = reinterpret_cast<float2*>(sm + S::kMeta);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + S::kMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + S::kMisc + 4);
  volatile int* refused = reinterpret_cast<volatile int*>(sm + S::kMisc + 16);   // [kUnitRing]
  long long* scan = reinterpret_cast<long long*>(sm + S::kMisc + 16 + 4 * kUnitRing);

  if (tid == 0) {
    for (int i = 0; i < kBarCount; ++i) {
      const bool conv = (i >= kRawKEmpty && i < kRawVFull) || i == kQReady ||
                        (i >= kRawVEmpty && i < kQReady) || i == kKReady || i == kKReady + 1 ||
                        i == kVReady || i == kVReady + 1;
      const bool soft = (i >= kPFull && i < kODone) || i == kOFree || i == kOFree + 1;
      mbar_init(bar(i), conv ? S::kConvWarps : soft ? 4 : i == kEpi ? S::kSoftWarps : 1);
    }
    *abort_flag = 0;
    for (int i = 0; i < kUnitRing; ++i) refused[i] = 0;
    mbar_init_fence();
  }
  if (warp == S::kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // only now that the tensor memory is held: a dependent that allocates some
  // and shares the SM could else take columns first and wait for this grid,
  // while this CTA's allocation waits for those columns
  pdl_launch_dependents();
  constexpr uint32_t tmem = 0;   // all 512 columns: they begin at 0
  pdl_wait();
  if (blockIdx.x == 0)
    for (int b = tid; b < p.bt.B; b += S::kThreads)
      if (!sequence(p.bt, p.c.P, b).ok) report(p.a.status, W4_ERR_INDEX);
  Run run;
  const bool any = find_run<S::kWarps>(
      p.bt.B, kMinTiles, [&](int e, int* units) { return entry_tiles<D>(p, e, units); }, scan, &run);
  Walk walk = {any ? run.g0 : 0, any ? run.off : 0, any ? run.entry : 0};
  if (!any) run.g1 = 0;
  Unit u;
  bool ok = *tmem_slot == 0;
  __syncthreads();

  if (warp == S::kCopyWarp) {
    // ------------------------------------------------------------- pages
    // Tiles of K run two ahead of those of V, as they are needed.
    const int box = min(p.c.P, kKeys);   // tokens of one copy
    const int boxes = kKeys / box;
    int* pages = reinterpret_cast<int*>(sm + S::kPages);
    uint32_t nk = 0, nv = 0;             // tiles copied
    for (int unit = 0; ok && next_unit<D>(p, run, walk, u); ++unit) {
      const int32_t* table = p.bt.table + (long long)u.b * p.bt.max_pages;
      const int n = u.tiles();
      auto copy = [&](bool keys, int i, uint32_t serial) {
        const int full = keys ? kRawKFull : kRawVFull, st = serial % kRaw;
        if (!wait_idle(bar((keys ? kRawKEmpty : kRawVEmpty) + st), before<kRaw>(serial), abort_flag))
          return false;
        const int tok = u.t.lo + (u.i0 + i) * kKeys + lane * box;
        const int at = (serial % kMetaRing) * 4 + lane * (box / 16);
        int page = -1;
        if (lane < boxes) {
          if (!keys) {
            page = pages[at];
          } else {
            float2 m = make_float2(0.0f, 0.0f);
            if (tok < u.t.hi) {
              page = load_in(table + tok / p.c.P);
              if (page < 0 || page >= p.c.num_pages) {
                page = -1;
                refused[unit % kUnitRing] = 1;
              } else {
                m = make_float2(p.c.ks[p.c.pair(page, u.h)], p.c.vs[p.c.pair(page, u.h)]);
              }
            }
            for (int e = 0; e < box / 16; ++e) meta[at + e] = m;
            pages[at] = page;
          }
        }
        const int c = __popc(__ballot_sync(0xffffffffu, page >= 0));
        if (lane == 0) {
          if (c > 0) mbar_arrive_expect_tx(bar(full + st), (uint32_t)(c * box * D));
          else mbar_arrive(bar(full + st));
        }
        __syncwarp();
        if (page >= 0) {
          const uint32_t dst = sb + (keys ? S::kRawK : S::kRawV) + st * S::kRawTile;
#pragma unroll
          for (int x = 0; x < D; x += 128)
            tma_4d(dst + x * kKeys + lane * box * (D < 128 ? D : 128), keys ? &p.tm_k : &p.tm_v, x,
                   tok % p.c.P, u.h, page, bar(full + st));
        }
        __syncwarp();
        return true;
      };
      ok = copy(true, 0, nk++);
      if (ok && n > 1) ok = copy(true, 1, nk++);
      for (int i = 0; ok && i < n; ++i) {
        ok = copy(false, i, nv++);
        if (ok && i + 2 < n) ok = copy(true, i + 2, nk++);
      }
    }
    // after a failure: what is in flight lands before the CTA leaves
    if (!ok) {
      const long long t0 = clock64();
      while (clock64() - t0 < (1 << 20)) {
      }
    }
  } else if (warp == S::kMmaWarp) {
    // -------------------------------------------------------- MMA issuer
    constexpr uint32_t kDescS = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kKeys >> 3) << 17) |
                                ((uint32_t)(kRowTile >> 4) << 24);
    constexpr uint32_t kDescO = (1u << 4) | (2u << 7) | (2u << 10) | ((uint32_t)(D >> 3) << 17) |
                                ((uint32_t)(kRowTile >> 4) << 24);
    // The jobs of a unit go round in steps whose S region, K and V buffers and
    // row tile are compile-time constants: the descriptors are then a uniform
    // base plus constants, and an MMA issues in a few instructions.
    const uint64_t dq = desc_sw128(sb + S::kQ), dk = desc_sw128(sb + S::kK), dv = desc_sw128(sb + S::kV);
    uint32_t units = 0;
    uint32_t k_par = 0, v_par = 0, p_par = 0, o_par = 0;   // next parity of each barrier
    int last_buf = -1;                                     // of the last commit on kVFree
    auto take = [&](uint32_t& mask, int i) {
      const uint32_t p = (mask >> i) & 1u;
      mask ^= 1u << i;
      return p;
    };
    for (; ok && next_unit<D>(p, run, walk, u); ++units) {
      const bool two = kGroups == 2 && u.rows > kRowTile;   // two row tiles
      const int jobs = two ? 2 * u.tiles() : u.tiles();
      if (!wait_bar(bar(kQReady), use<1>(units), abort_flag)) {
        ok = false;
        break;
      }
      // S of a job: key tile in buffer kB, row tile kT, into region kR
      auto scores = [&](auto kR, auto kB, auto kT, bool first, bool last, bool end) {
        if (first && !wait_bar(bar(kKReady + kB), take(k_par, kB), abort_flag)) return false;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ss_f16(tmem + kR * kKeys,
                     dq + kT * (S::kQTile / 16) + (k >> 2) * (kRowTile * 128 / 16) + (k & 3) * 2,
                     dk + kB * (S::kKTile / 16) + (k >> 2) * (kKeys * 128 / 16) + (k & 3) * 2, kDescS,
                     k > 0);
        mma_commit(bar(kSFull + kR));
        if (last) mma_commit(bar(kKFree + kB));
        if (end) mma_commit(bar(kQFree));
        return true;
      };
      // O of a job: weights in region kR, value tile in buffer kB, group kG
      auto values = [&](auto kR, auto kB, auto kG, bool begin, bool first, bool last) {
        if (begin && !wait_bar(bar(kOFree + kG), take(o_par, kG) ^ 1u, abort_flag)) return false;
        if (first && !wait_bar(bar(kVReady + kB), take(v_par, kB), abort_flag)) return false;
        if (!wait_bar(bar(kPFull + kR), take(p_par, kR), abort_flag)) return false;
        tc_fence_after();
        const uint32_t acc = begin ? 0u : 1u;
#pragma unroll
        for (int k = 0; k < kKeys / 8; ++k)
          mma_ts_tf32(tmem + S::kOCol + kG * D, tmem + kR * kKeys + 8 * k,
                      dv + kB * (S::kVTile / 16) + (k >> 2) * (D * 128 / 16) + (k & 3) * 2, kDescO,
                      k > 0 ? 1u : acc);
        mma_commit(bar(kODone + kG));
        if (last) mma_commit(bar(kVFree + kB));
        if (last) last_buf = kB;
        return true;
      };
      if (two) {
        // job j: key tile j / 2, row tile (and group) j % 2, region j % 4; scores four ahead
        auto step = [&](auto kZ, int j, int at) {   // at: the job whose scores, or weights
          constexpr int z = decltype(kZ)::value;
          using R = Const<z>;
          using B = Const<(z >> 1) % kBuf>;
          using T = Const<z & 1>;
          if (at >= jobs) return true;
          if (j < 0) return scores(R(), B(), T(), (z & 1) == 0, (z & 1) == 1, at == jobs - 1);
          return values(R(), B(), T(), at < 2, (z & 1) == 0, (z & 1) == 1);
        };
        ok = step(Const<0>(), -1, 0) && step(Const<1>(), -1, 1) && step(Const<2>(), -1, 2) &&
             step(Const<3>(), -1, 3);
        for (int j = 0; ok && j < jobs; j += 4)
          ok = step(Const<0>(), 0, j) && step(Const<0>(), -1, j + 4) && step(Const<1>(), 0, j + 1) &&
               step(Const<1>(), -1, j + 5) && step(Const<2>(), 0, j + 2) &&
               step(Const<2>(), -1, j + 6) && step(Const<3>(), 0, j + 3) &&
               step(Const<3>(), -1, j + 7);
      } else {
        // job j: key tile j, region j % 2; scores two ahead
        auto step = [&](auto kZ, int j, int at) {
          constexpr int z = decltype(kZ)::value;
          using R = Const<z>;
          using B = Const<z % kBuf>;
          using G = Const<z % kGroups>;
          if (at >= jobs) return true;
          if (j < 0) return scores(R(), B(), Const<0>(), true, true, at == jobs - 1);
          return values(R(), B(), G(), at < kGroups, true, true);
        };
        ok = step(Const<0>(), -1, 0) && step(Const<1>(), -1, 1);
        for (int j = 0; ok && j < jobs; j += 2)
          ok = step(Const<0>(), 0, j) && step(Const<0>(), -1, j + 2) && step(Const<1>(), 0, j + 1) &&
               step(Const<1>(), -1, j + 3);
      }
    }
    // the last commits land before the CTA may leave
    if (ok) {
      if (last_buf >= 0)
        mbar_wait_bounded(bar(kVFree + last_buf), ((v_par >> last_buf) & 1u) ^ 1u, kWaitCycles);
    } else {
      const long long t0 = clock64();
      while (clock64() - t0 < (1 << 20)) {
      }
    }
  } else if (warp >= S::kConvWarp) {
    // ---------------------------------------------------------- expansion
    const int w = warp - S::kConvWarp, ct = tid - 32 * S::kConvWarp;
    constexpr int kQThreads = 128;       // that copy query rows (a power of two)
    uint32_t nk = 0, nv = 0;             // tiles expanded
    uint32_t kf_par = 3, vf_par = 3;     // next parity of each kKFree, kVFree (the first passes at once)
    for (uint32_t units = 0; ok && next_unit<D>(p, run, walk, u); ++units) {
      if (!wait_idle(bar(kQFree), before<1>(units), abort_flag)) {
        ok = false;
        break;
      }
      // query rows as they are; rows past the unit's are zero
      const int qtiles = u.rows > kRowTile ? 2 : 1;
      // (a thread keeps its 16-byte column and finds the next row's token and
      // head by addition)
      if (ct < kQThreads) {
        constexpr int kStep = kQThreads / (D / 8);   // rows
        const int ch = ct % (D / 8);
        int r = ct / (D / 8), row = u.rt * S::kRows + r;
        int t = row / p.G, g = row - t * p.G;
        const __nv_bfloat16* src = p.a.q + (long long)(u.s.row0 + t) * p.a.q_stride +
                                   (long long)(u.h * p.G + g) * D + ch * 8;
#pragma unroll 4
        for (; r < qtiles * kRowTile; r += kStep) {
          const bool in = r < u.rows;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                           sb + S::kQ + (r >> 7) * S::kQTile + (ch >> 3) * (kRowTile * 128) +
                           (r & 127) * 128 + (((ch & 7) ^ (r & 7)) << 4)),
                       "l"(in ? src : p.a.q), "r"(in ? 16 : 0)
                       : "memory");
          g += kStep;
          src += kStep * D;
          while (g >= p.G) {
            g -= p.G;
            src += p.a.q_stride - (long long)p.G * D;
          }
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kQReady));

      // keys: 8 rows by 4 chunks of 16 codes at a time (no bank conflicts on
      // either side), 32 bytes of bf16 each
      auto keys = [&](int i) {
        const uint32_t st = nk % kRaw, buf = i % kBuf;
        if (!wait_idle(bar(kRawKFull + st), use<kRaw>(nk), abort_flag) ||
            !wait_idle(bar(kKFree + buf), (kf_par >> buf) & 1u, abort_flag))
          return false;
        kf_par ^= 1u << buf;
        const uint32_t raw = sb + S::kRawK + st * S::kRawTile, to0 = sb + S::kK + buf * S::kKTile;
#pragma unroll
        for (int x = w; x < (kKeys / 8) * (D / 64); x += S::kConvWarps) {
          const int row = 8 * (x % (kKeys / 8)) + (lane & 7), c = 4 * (x / (kKeys / 8)) + (lane >> 3);
          const uint4 v = lds128(
              raw + (D == 64 ? row * 64 + ((c ^ ((row >> 1) & 3)) << 4)
                             : (c >> 3) * (kKeys * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4)));
          const uint32_t to = to0 + (c >> 2) * (kKeys * 128) + row * 128;
          const int e = 2 * (c & 3);
          sts128(to + ((e ^ (row & 7)) << 4), codes_bf16(v.x, 0x4140), codes_bf16(v.x, 0x4342),
                 codes_bf16(v.y, 0x4140), codes_bf16(v.y, 0x4342));
          sts128(to + (((e + 1) ^ (row & 7)) << 4), codes_bf16(v.z, 0x4140),
                 codes_bf16(v.z, 0x4342), codes_bf16(v.w, 0x4140), codes_bf16(v.w, 0x4342));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(kKReady + buf));
          mbar_arrive(bar(kRawKEmpty + st));
        }
        ++nk;
        return true;
      };
      // values: four tokens of a channel side by side as fp32 (a byte under
      // 0x4B0000 reads 2^23 + u); lanes start at different channels of their
      // word so that the stores meet no bank conflict
      auto vals = [&](int i) {
        const uint32_t st = nv % kRaw, buf = i % kBuf;
        if (!wait_idle(bar(kRawVFull + st), use<kRaw>(nv), abort_flag) ||
            !wait_idle(bar(kVFree + buf), (vf_par >> buf) & 1u, abort_flag))
          return false;
        vf_par ^= 1u << buf;
        const uint32_t raw = sb + S::kRawV + st * S::kRawTile, to0 = sb + S::kV + buf * S::kVTile;
        constexpr int kWords = D == 64 ? 16 : 32;         // words of a raw row
        constexpr int kSub = 32 / kWords;                 // token groups of a warp at a time
        const uint64_t zero = pack2(-8388736.0f, -8388736.0f);
#pragma unroll
        for (int x = w; x < kKeys / 4 / kSub * ((D + 127) / 128); x += S::kConvWarps) {
          const int g = x % (kKeys / 4 / kSub), half = x / (kKeys / 4 / kSub);
          const int tok = 4 * (g * kSub + lane / kWords), wd = lane % kWords;
          uint32_t v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int t = tok + e;
            v[e] = lds32(raw +
                         (D == 64 ? t * 64 + (((wd >> 2) ^ ((t >> 1) & 3)) << 4)
                                  : half * (kKeys * 128) + t * 128 + (((wd >> 2) ^ (t & 7)) << 4)) +
                         (wd & 3) * 4);
          }
#pragma unroll
          for (int dd = 0; dd < 4; ++dd) {
            const int d = (dd + (lane >> 1)) & 3, ch = 128 * half + 4 * wd + d;
            float f[4];
#pragma unroll
            for (int e = 0; e < 4; e += 2)
              unpack2(add2(pack2(__uint_as_float(__byte_perm(v[e], 0x4B000000u, 0x7440 + d)),
                                 __uint_as_float(__byte_perm(v[e + 1], 0x4B000000u, 0x7440 + d))),
                           zero),
                      f[e], f[e + 1]);
            sts128(to0 + (tok >> 5) * (D * 128) + ch * 128 + ((((tok & 31) >> 2) ^ (ch & 7)) << 4),
                   __float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                   __float_as_uint(f[3]));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(kVReady + buf));
          mbar_arrive(bar(kRawVEmpty + st));
        }
        ++nv;
        return true;
      };
      const int n = u.tiles();
      ok = keys(0) && (n < 2 || keys(1));
      for (int i = 0; ok && i < n; ++i) ok = vals(i) && (i + 2 >= n || keys(i + 2));
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int grp = warp >> 2;                                     // 0 .. kGroups - 1
    const int r = tid & 127;                                       // row in the tile
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ocol = tmem + lanes + S::kOCol + grp * D;
    const float f = p.a.scale * kLog2e;
    uint32_t s_par = 0;                  // next parity of each region's barrier
    uint32_t o_done = 0;                 // PVs of this group, units before this one
    int serial = 0, unit = 0;            // key tiles and units walked
    for (; ok && next_unit<D>(p, run, walk, u); ++unit) {
      const bool two = kGroups == 2 && u.rows > kRowTile;
      const int row = u.rt * S::kRows + (two ? grp * kRowTile : 0) + r;   // of the (sequence, head)
      const int pos = u.s.len - u.s.n + min(row, u.R - 1) / p.G;
      const int tok_lo = u.t.lo + u.i0 * kKeys, n = u.tiles(), win = p.a.window;
      float m = 0.0f, l = 0.0f;
      bool have = false;     // m is some score's
      int done = 0;          // jobs of this group whose PV may be under way
      const int step = kGroups == 2 && !two ? 2 : 1;               // the other group has the others
      for (int i = step == 2 ? grp : 0; i < n; i += step) {
        const int reg = two ? 2 * (i & 1) + grp : i & 1;
        const uint32_t scol = tmem + lanes + reg * kKeys;
        const int tok0 = tok_lo + i * kKeys;
        const float2* mt = meta + ((serial + i) % kMetaRing) * 4;
        if (!wait_bar(bar(kSFull + reg), (s_par >> reg) & 1u, abort_flag)) {
          ok = false;
          break;
        }
        s_par ^= 1u << reg;
        tc_fence_after();
        // the tile's columns that the row sees
        const int hi = pos - tok0, lo = win > 0 ? hi - win + 1 : 0;
        const bool cut = __any_sync(0xffffffffu, hi < kKeys - 1 || lo > 0);
#pragma unroll 1
        for (int c0 = 0; c0 < kKeys; c0 += 32) {
          float y[32];
          const float2 m0 = mt[c0 / 16], m1 = mt[c0 / 16 + 1];
          const float f0 = f * m0.x, f1 = f * m1.x;
          float sum;
#pragma unroll 1
          for (bool again = false;; again = true) {
            tc::tmem_ld<32>(scol + c0, y);
            tc::tmem_wait_ld<32>(y);
            sum = weights(y, f0, f1, m, cut, lo - c0, hi - c0);
            // a score far past m shows in the sum (once m has moved, the sum
            // is what it is: not a number, say)
            if (again || !__any_sync(0xffffffffu, !have || !(sum <= kFar))) break;
            tc::tmem_ld<32>(scol + c0, y);
            tc::tmem_wait_ld<32>(y);
            float mx = -INFINITY;
            const uint32_t seen = columns(lo - c0, hi - c0);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              mx = fmaxf(mx, seen >> e & 1u ? y[e] * (e < 16 ? f0 : f1) : -INFINITY);
            float up = 0.0f;
            if (!have) {
              have = mx > -INFINITY;
              m = have ? mx : 0.0f;
            } else if (mx - m > kPass) {
              up = ceilf(mx - m);   // whole, so that rescaling is exact
              m += up;
              up = fminf(up, 252.0f);
            }
            // what was weighed against the old m: earlier columns, O and l.  Twice
            // where m moves further than one factor reaches: what stands 2^60 above
            // the old m shows down to 2^-126 of the new one.
            while (__any_sync(0xffffffffu, up > 0.0f)) {
              const float keep = exp2_fast(-fminf(up, 126.0f));
              up = fmaxf(up - 126.0f, 0.0f);
              l *= keep;
              tmem_wait_st();
              for (int c = 0; c < c0; c += 32) tmem_scale32(scol + c, keep);
              if (done > 0) {
                // the last PV of this group has to be complete
                if (!wait_bar(bar(kODone + grp), (o_done + done - 1) & 1u, abort_flag)) ok = false;
                tc_fence_after();
                for (int c = 0; c < D; c += 32) tmem_scale32(ocol + c, keep);
              }
              tmem_wait_st();
            }
          }
          l += sum;
          // times the block's step; the MMA drops 13 bits of what it reads,
          // and the factor's last part makes that a rounding: the mean error is
          // nil, and a weight of 11 bits stays what it is
          const uint64_t v0 = pack2(m0.y * kRound, m0.y * kRound);
          const uint64_t v1 = pack2(m1.y * kRound, m1.y * kRound);
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            unpack2(mul2(pack2(y[e], y[e + 1]), e < 16 ? v0 : v1), y[e], y[e + 1]);
          tmem_st32(scol + c0, y);
        }
        if (!ok) break;
        tmem_wait_st();
        tc_fence_before();
        // A wait tells phases apart by one bit: the PV before this one is seen
        // to complete before this one may begin (it has had the whole softmax).
        if (done > 0 && !wait_bar(bar(kODone + grp), (o_done + done - 1) & 1u, abort_flag)) {
          ok = false;
          break;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kPFull + reg));
        ++done;
      }
      serial += n;
      if (!ok) break;
      // ---------------------------------------------------------- epilogue
      if (done > 0 && !wait_bar(bar(kODone + grp), (o_done + done - 1) & 1u, abort_flag)) {
        ok = false;
        break;
      }
      o_done += done;
      tc_fence_after();
      const bool no = refused[unit % kUnitRing] != 0;
      const bool direct = u.whole() && (two || kGroups == 1);
      // a whole unit of one row tile: the groups' parts meet right here, in
      // two places of this CTA's own in turn
      const bool pair = u.whole() && !direct;
      const int slot = pair ? 2 * gridDim.x + 2 * blockIdx.x + (unit & 1)
                            : 2 * blockIdx.x + (u.i0 == 0 ? 1 : 0);
      const int prow = (kGroups == 2 ? grp * kRowTile : 0) + r;
      const bool mine = row < u.R;
      if (!have) m = -INFINITY;
      const long long at = mine ? (long long)(u.s.row0 + row / p.G) * p.a.Hq + u.h * p.G + row % p.G : 0;
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      float2 kept = make_float2(m, l);
      const float part_scale = direct ? inv : settle(kept);
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float o[32];
        if (done > 0) {
          tc::tmem_ld<32>(ocol + c, o);
          tc::tmem_wait_ld<32>(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.0f;
        }
        if (direct) {
          if (mine && !no) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              const uint2 a = pack_bf16x4(o + e, inv), b = pack_bf16x4(o + e + 4, inv);
              *reinterpret_cast<uint4*>(p.a.out + at * D + c + e) = make_uint4(a.x, a.y, b.x, b.y);
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(p.parts + ((long long)slot * S::kRows + prow) * D + c + e) =
                make_float4(o[e] * part_scale, o[e + 1] * part_scale, o[e + 2] * part_scale,
                            o[e + 3] * part_scale);
        }
      }
      tc_fence_before();
      __syncwarp();
      // (a group without a tile in this unit holds up no PV)
      if (lane == 0 && done > 0) mbar_arrive(bar(kOFree + grp));
      if (direct) {
        if (mine && !no && p.a.lse != nullptr)
          p.a.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
      } else {
        *reinterpret_cast<float2*>(p.part_stats + ((long long)slot * S::kRows + prow) * 2) =
            make_float2(kept.x, no ? -1.0f : kept.y);
      }
      // the unit's first CTA says where its parts are
      if (tid == 0 && u.i0 == 0)
        p.cut[2 + ((long long)u.b * p.c.H + u.h) * p.rts + u.rt] = u.whole() ? -1 : u.u0;
      // all softmax warps have read `refused` and written their parts
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kEpi));
      if (!wait_bar(bar(kEpi), use<1>(unit), abort_flag)) {
        ok = false;
        break;
      }
      if (tid == 0) {
        if (no) report(p.a.status, W4_ERR_INDEX);
        refused[unit % kUnitRing] = 0;
      }
      if (pair && !no) {
        const long long base = (long long)slot * S::kRows;
        for (int x = tid; x < u.rows * (D / 4); x += 32 * S::kSoftWarps)
          join_row<D>(p, u.s, u.h, u.rt * S::kRows + x / (D / 4), x % (D / 4), 2, [&](int k) {
            return base + x / (D / 4) + k * kRowTile;
          });
      }
    }
    if (tid == 0 && blockIdx.x == 0) {   // also when a wait ran out
      p.cut[0] = run.total;
      p.cut[1] = run.ctas;
    }
  }
  if (!ok) {
    if (*abort_flag == 0) report(p.a.status, W4_ERR_TIMEOUT);
    *abort_flag = 1;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == S::kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(*tmem_slot)
                 : "memory");
}

// Joins the parts of cut units: one CTA per 4 rows.  Reading and adding
// them all from one SM would take longer than computing them did.
constexpr int kJoinRows = 4;
constexpr int kJoinThreads = 128;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const __grid_constant__ ChunkParams p) {
  using S = Shape<D>;
  pdl_launch_dependents();
  pdl_wait();
  constexpr int kSlabs = S::kRows / kJoinRows;
  const int rt = blockIdx.x / kSlabs, slab = blockIdx.x % kSlabs, h = blockIdx.y, b = blockIdx.z;
  const Seq s = sequence(p.bt, p.c.P, b);
  const int R = s.n * p.G, row0 = rt * S::kRows + slab * kJoinRows;
  if (!s.ok || row0 >= R) return;
  const long long u0 = p.cut[2 + ((long long)b * p.c.H + h) * p.rts + rt];
  if (u0 < 0) return;
  Run run;
  run.total = p.cut[0];
  run.ctas = (int)p.cut[1];
  const Tile t = tile_of(s, p.G, p.a.window, rt, S::kRows, kKeys);
  // a unit whose CTA gave up waiting has no start of this call's: whatever
  // stands there may not be taken for parts (the status says W4_ERR_TIMEOUT)
  if (!run.holds(u0, t.slices)) return;
  const int c0 = run.holder(u0), c1 = run.holder(u0 + t.slices - 1);
  // of one row tile, each CTA holds two parts (one per softmax group)
  const int subs = S::kGroups == 2 && R - rt * S::kRows <= kRowTile ? 2 : 1;
  const int parts = (c1 - c0 + 1) * subs;
#pragma unroll 2
  for (int x = threadIdx.x; x < kJoinRows * (D / 4); x += kJoinThreads) {
    const int r = x / (D / 4), c4 = x % (D / 4), row = row0 + r;
    if (row >= R) break;
    auto part = [&](int k) {
      const int c = c0 + (subs == 2 ? k >> 1 : k), sub = subs == 2 ? k & 1 : 0;
      // the first CTA's part began the unit, the others' runs began inside it
      return (long long)(c == c0 ? 2 * c + 1 : 2 * c) * S::kRows + slab * kJoinRows + r +
             sub * kRowTile;
    };
    join_row<D>(p, s, h, row, c4, parts, part);
  }
}

// ================================================================= host side
size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

struct Plan {
  int rows, rts;
  size_t cut, parts, stats, bytes;
};

Plan plan_chunk(const Cache& c, const Batch& b, int G, int sms) {
  Plan pl;
  pl.rows = c.D == 256 ? Shape<256>::kRows : Shape<128>::kRows;
  pl.rts = (int)(((long long)b.max_new * G + pl.rows - 1) / pl.rows);
  pl.cut = up256(((size_t)b.B * c.H * pl.rts + 2) * 8);
  pl.parts = up256((size_t)4 * sms * pl.rows * c.D * 4);
  pl.stats = up256((size_t)4 * sms * pl.rows * 8);
  pl.bytes = kHeadBytes + pl.cut + pl.parts + pl.stats;
  return pl;
}

template <int D>
w4_status launch_chunk(ChunkParams& p, int sms, int dev, w4_stream_t stream) {
  using S = Shape<D>;
  static std::mutex mu;
  static bool done[64] = {};
  if (dev < 0 || dev >= 64) return W4_ERR_DEVICE;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      const cudaError_t e = cudaFuncSetAttribute(
          attn_chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
      if (e != cudaSuccess) {
        note_cuda_error(e);
        (void)cudaGetLastError();
        return W4_ERR_LAUNCH;
      }
      done[dev] = true;
    }
  }
  const int box = std::min(p.c.P, kKeys);
  if (!tensor_map(&p.tm_k, p.c.kc, p.c, box) || !tensor_map(&p.tm_v, p.c.vc, p.c, box)) {
    note_cuda_error(cudaErrorInvalidValue);
    return W4_ERR_LAUNCH;
  }
  const w4_status st =
      launch(attn_chunk_kernel<D>, dim3((unsigned)sms), S::kThreads, S::kSmem, stream, p);
  if (st != W4_OK) return st;
  return launch(attn_join_kernel<D>,
                dim3((unsigned)(p.rts * (S::kRows / kJoinRows)), (unsigned)p.c.H, (unsigned)p.bt.B),
                kJoinThreads, 0, stream, p);
}

}  // namespace

size_t chunk_workspace_bytes(const Cache& c, const Batch& b, int G, int sms) {
  return plan_chunk(c, b, G, sms).bytes;
}

w4_status chunk_attn(const Cache& c, const Batch& b, const ChunkArgs& a, void* workspace, int sms,
                     int dev, w4_stream_t stream) {
  ChunkParams p = {};
  p.c = c;
  p.bt = b;
  p.a = a;
  p.G = a.Hq / c.H;
  const Plan pl = plan_chunk(c, b, p.G, sms);
  p.rts = pl.rts;
  uint8_t* ws = static_cast<uint8_t*>(workspace) + kHeadBytes;
  p.cut = reinterpret_cast<long long*>(ws);
  p.parts = reinterpret_cast<float*>(ws + pl.cut);
  p.part_stats = reinterpret_cast<float*>(ws + pl.cut + pl.parts);
  switch (c.D) {
    case 64: return launch_chunk<64>(p, sms, dev, stream);
    case 128: return launch_chunk<128>(p, sms, dev, stream);
    default: return launch_chunk<256>(p, sms, dev, stream);
  }
}

}  // namespace kv8
}  // namespace w4
