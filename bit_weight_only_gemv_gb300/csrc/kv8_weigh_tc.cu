// Accumulated attention weights (w4_kv8_weigh) for prompt chunks, on the
// 5th-generation tensor cores (tcgen05, sm_103a).
//
// S^T = K q^T with tokens as the MMA's 128 rows: a token's scores lie along
// one thread's columns of tensor memory, so that its weights
//   2^(scale log2(e) ks S - log2(e) lse)
// add up in that thread's registers, in a fixed order of rows, without any
// exchange.  A unit of work is 256 tokens (128 of 256-channel heads), whose keys
// are expanded to bf16 once, against all query rows that see one of them, 128
// at a time: two row tiles' keys share each query tile, which halves what the
// queries cost in L2 traffic.  A CTA takes every gridDim.x-th unit and loads
// a unit's keys while the one before is worked on.
//
// Roles: eight warps per key tile that exponentiate and add (a thread has a
// token and half of the columns), four that bring keys in, one that issues the
// copies of query tiles, two that bring their log sums, one that issues the MMAs.
// Every wait is bounded.
//
// 2 x 256 rows of 32 heads on 8 of 128 channels, 8k keys: 37 us, 0.62 PFLOP/s
// (a CTA a unit with its start in the open: 51; keys as legacy MMA fragments
// in every warp: 120).  The weights' warps bound it: without their work 26.
#include <algorithm>
#include <mutex>

#include "kv8_attn.h"
#include "kv8_tc.cuh"

namespace w4 {
namespace kv8 {
namespace {

using tc::kWaitCycles;
using tc::tc_fence_after;
using tc::tc_fence_before;
using tc::wait_bar;

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTile = 128;      // tokens of a key tile, rows of a query tile
constexpr int kLseRing = 8;
constexpr int kInfoRing = 4;

template <int D>
struct Shape {
  static constexpr int kTiles = D == 256 ? 1 : 2;      // key tiles of a unit
  static constexpr int kKeyBufs = D == 256 ? 1 : 2;    // units' keys in shared memory
  static constexpr int kBufs = 2;                      // query tiles in shared memory
  static constexpr int kKeyWarp = 8 * kTiles;   // weights: four warps a key tile and half of the columns
  static constexpr int kKeyWarps = 4;                // 24 warps in all with two key tiles
  static constexpr int kLoadWarp = kKeyWarp + kKeyWarps;
  static constexpr int kLseWarp = kLoadWarp + 1;       // one a query buffer
  static constexpr int kMmaWarp = kLseWarp + kBufs;
  static constexpr int kThreads = 32 * (kMmaWarp + 1);
  static constexpr int kBytes = kTile * D * 2;         // of a tile, keys or queries
  static constexpr int kQ = kKeyBufs * kTiles * kBytes;
  static constexpr int kLse = kQ + kBufs * kBytes;     // [kLseRing][kTile]
  static constexpr int kInfo = kLse + kLseRing * kTile * 4;   // [kInfoRing][kTiles][kTile] {page, factor}
  static constexpr int kSums = kInfo + kInfoRing * kTiles * kTile * 8;   // [2][kTiles][kTile]: second halves'
  static constexpr int kBars = kSums + 2 * kTiles * kTile * 4;
  static constexpr int kMisc = kBars + 20 * 8;
  static constexpr int kEnd = kMisc + 32 + 1024;
  // more than half an SM's: each CTA holds all of its tensor memory
  static constexpr int kSmem = kEnd > 117248 ? kEnd : 117248;
  static_assert(kSmem <= 232448 && 2 * kSmem > 232448, "shared memory");
};

// [2] [2] [2 x 2] [2 x 2] [2] [2] [2 x 2]
enum {
  kQFull = 0,
  kQFree = 2,
  kSFull = 4,
  kSFree = 8,
  kKFull = 12,
  kKFree = 14,
  kSumFull = 16,
  kBarCount = 20
};

// The units of a CTA: every gridDim.x-th block of tokens of all (sequence,
// head, block) that some row sees.  Every role walks them for itself.
struct Units {
  int blocks, x, h, b;          // of the next candidate
  int step_x, step_h, step_b;   // gridDim.x in those digits
  int per;                      // new tokens of a query tile
  Seq s;
  int head, seq, first, blk0, t_lo, t_hi, qtiles;   // of the unit
  __device__ __forceinline__ Units(const WeighParams& p, int tokens) {
    blocks = (p.bt.max_len + tokens - 1) / tokens;
    per = kTile / p.G;
    x = blockIdx.x % blocks;
    h = blockIdx.x / blocks;
    b = h / p.c.H;
    h %= p.c.H;
    step_x = gridDim.x % blocks;
    step_h = gridDim.x / blocks;
    step_b = step_h / p.c.H;
    step_h %= p.c.H;
  }
  __device__ __forceinline__ bool next(const WeighParams& p, int tokens, bool reports) {
    while (b < p.bt.B) {
      seq = b;
      head = h;
      blk0 = x * tokens;
      x += step_x;
      int up = x >= blocks ? 1 : 0;
      x -= up * blocks;
      h += step_h + up;
      up = h >= p.c.H ? 1 : 0;
      h -= up * p.c.H;
      b += step_b + up;
      s = sequence(p.bt, p.c.P, seq);
      if (!s.ok) {
        if (reports && blk0 == 0 && head == 0) report(p.status, W4_ERR_INDEX);
        continue;
      }
      if (blk0 >= s.len) continue;
      // rows that see some token of the block: positions from blk0 on, and within the window
      first = s.len - s.n;   // position of the first row
      t_lo = max(0, blk0 - first);
      t_hi = p.window > 0
                 ? (int)min((long long)s.n, (long long)blk0 + tokens - 1 + p.window - first)
                 : s.n;
      if (t_lo >= t_hi) continue;
      qtiles = (t_hi - t_lo + per - 1) / per;
      return true;
    }
    return false;
  }
};

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int x, int head,
                                       int row, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(head), "r"(row), "r"(bar)
      : "memory");
}

template <int D>
__global__ void __launch_bounds__(Shape<D>::kThreads, 1)
    weigh_many_kernel(const __grid_constant__ WeighParams p) {
  using S = Shape<D>;
  constexpr int kTiles = S::kTiles, kBufs = S::kBufs, kKeyBufs = S::kKeyBufs;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw;
  const uint32_t sb = smem_addr(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto bar = [&](int i) { return sb + S::kBars + 8 * i; };
  float* lse = reinterpret_cast<float*>(sm + S::kLse);   // minus log2(e) lse; -inf: adds nothing
  int2* info = reinterpret_cast<int2*>(sm + S::kInfo);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + S::kMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + S::kMisc + 4);

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kQFull + i), 2);
      mbar_init(bar(kQFree + i), 1);
      mbar_init(bar(kKFull + i), S::kKeyWarps);
      mbar_init(bar(kKFree + i), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(kSFull + i), 1);
      mbar_init(bar(kSFree + i), 8);
      mbar_init(bar(kSumFull + i), 4);
    }
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == S::kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // a query tile's rows: whole tokens; the rows after them stay zero
  const int rows = kTile / p.G * p.G;
  for (int x = tid; x < kBufs * (D / 64) * (kTile - rows) * 8; x += S::kThreads) {
    const int i = x / 8 / (kTile - rows), r = rows + x / 8 % (kTile - rows);
    sts128(sb + S::kQ + i * (kTile * 128) + r * 128 + (x & 7) * 16, 0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // only now that the tensor memory is held (as in kv8_chunk.cu)
  pdl_launch_dependents();
  pdl_wait();
  constexpr uint32_t tmem = 0;   // all 512 columns: they begin at 0
  bool ok = __syncthreads_and(*tmem_slot == 0 && (sb & 1023u) == 0) != 0;

  constexpr int kTokens = kTiles * kTile;
  Units u(p, kTokens);
  int T = 0, n = 0;   // query tiles and units before this one
  if (warp == S::kMmaWarp) {
    // -------------------------------------------------------- MMA issuer
    constexpr uint32_t kDesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kTile >> 3) << 17) |
                               ((uint32_t)(kTile >> 4) << 24);
    const uint64_t dk = desc_sw128(sb), dq = desc_sw128(sb + S::kQ);
    for (; ok && u.next(p, kTokens, false); ++n) {
      const int kb = n % kKeyBufs;
      ok = wait_bar(bar(kKFull + kb), (uint32_t)(n / kKeyBufs) & 1u, abort_flag);
      for (int t = 0; ok && t < u.qtiles; ++t, ++T) {
        const int buf = T % kBufs, par = T & 1;
        ok = wait_bar(bar(kQFull + buf), (uint32_t)(T / kBufs) & 1u, abort_flag);
        for (int z = 0; ok && z < kTiles; ++z) {
          ok = wait_bar(bar(kSFree + 2 * par + z), ((uint32_t)(T >> 1) & 1u) ^ 1u, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint64_t a0 = dk + (kb * kTiles + z) * (S::kBytes / 16),
                         b0 = dq + buf * (S::kBytes / 16);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_ss_f16(tmem + (2 * par + z) * kTile, a0 + (k >> 2) * (kTile * 128 / 16) + (k & 3) * 2,
                       b0 + (k >> 2) * (kTile * 128 / 16) + (k & 3) * 2, kDesc, k > 0);
          mma_commit(bar(kSFull + 2 * par + z));
        }
        if (ok) mma_commit(bar(kQFree + buf));
      }
      if (ok) mma_commit(bar(kKFree + kb));
    }
    if (ok) {   // the last commit lands before the CTA may leave
      if (n > 0)
        mbar_wait_bounded(bar(kKFree + (n - 1) % kKeyBufs), (uint32_t)((n - 1) / kKeyBufs) & 1u,
                          kWaitCycles);
    } else {
      const long long t0 = clock64();
      while (clock64() - t0 < (1 << 20)) {
      }
    }
  } else if (warp >= S::kLseWarp) {
    // --------------------------------------------- log sums of a query tile
    const int buf = warp - S::kLseWarp;
    for (; ok && u.next(p, kTokens, false); ++n) {
      for (int t = 0; ok && t < u.qtiles; ++t, ++T) {
        if (T % kBufs != buf) continue;
        const int end = min(rows, (u.t_hi - u.t_lo) * p.G - t * rows);
        const int row0 = u.s.row0 + u.t_lo + t * u.per;
        float v[kTile / 32];
#pragma unroll
        for (int i = 0; i < kTile / 32; ++i) {
          const int r = lane + 32 * i;
          v[i] = -INFINITY;
          if (r < end) v[i] = p.lse[(long long)(row0 + r / p.G) * p.Hq + u.head * p.G + r % p.G];
        }
        // (the ring is longer than the buffers': its reader may lag behind the MMAs)
        if (!wait_bar(bar(kQFree + buf), ((uint32_t)(T / kBufs) & 1u) ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int i = 0; i < kTile / 32; ++i)
          lse[(T % kLseRing) * kTile + lane + 32 * i] =
              v[i] == -INFINITY ? -INFINITY : -v[i] * kLog2e;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kQFull + buf));
      }
    }
  } else if (warp >= S::kLoadWarp) {
    // ------------------------------------------------------- query tiles
    for (; ok && u.next(p, kTokens, false); ++n) {
      for (int t = 0; ok && t < u.qtiles; ++t, ++T) {
        const int buf = T % kBufs;
        if (!wait_bar(bar(kQFree + buf), ((uint32_t)(T / kBufs) & 1u) ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        const int row0 = u.s.row0 + u.t_lo + t * u.per;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(kQFull + buf), rows * D * 2);
          for (int c = 0; c < D / 64; ++c)
            tma_3d(sb + S::kQ + buf * S::kBytes + c * (kTile * 128), &p.tm, c * 64, u.head * p.G, row0,
                   bar(kQFull + buf));
        }
      }
    }
  } else if (warp >= S::kKeyWarp) {
    // ------------------------------------------------------------- keys
    constexpr int kKeyThreads = 32 * S::kKeyWarps, kChunks = D / 16;   // 16-code chunks of a token
    constexpr int kEach = kTokens * kChunks / kKeyThreads, kBatch = 8;
    static_assert(kEach % kBatch == 0 && kTokens % kKeyThreads == 0, "whole shares");
    const int kt = tid - 32 * S::kKeyWarp, lg = __ffs(p.c.P) - 1;
    for (; ok && u.next(p, kTokens, kt == 0); ++n) {
      const int kb = n % kKeyBufs;
      const int32_t* table = p.bt.table + (long long)u.seq * p.bt.max_pages;
      auto page_of = [&](int t) {
        return u.blk0 + t < u.s.len ? __ldg(table + ((u.blk0 + t) >> lg)) : -1;
      };
      int pages[kEach], own[kTokens / kKeyThreads];
      float f[kTokens / kKeyThreads];
#pragma unroll
      for (int i = 0; i < kTokens / kKeyThreads; ++i) own[i] = page_of(kt + i * kKeyThreads);
#pragma unroll
      for (int i = 0; i < kEach; ++i) pages[i] = page_of((kt + i * kKeyThreads) / kChunks);
#pragma unroll
      for (int i = 0; i < kTokens / kKeyThreads; ++i) {
        f[i] = 0.0f;
        if ((unsigned)own[i] < (unsigned)p.c.num_pages)
          f[i] = __ldg(p.c.ks + p.c.pair(own[i], u.head));
      }
      const uint32_t keys = sb + kb * kTiles * S::kBytes;
#pragma unroll
      for (int i0 = 0; i0 < kEach; i0 += kBatch) {
        uint4 v[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int x = kt + (i0 + i) * kKeyThreads, tok = u.blk0 + x / kChunks;
          v[i] = make_uint4(0, 0, 0, 0);
          if ((unsigned)pages[i0 + i] < (unsigned)p.c.num_pages)
            v[i] = __ldg(reinterpret_cast<const uint4*>(p.c.kc + p.c.block(pages[i0 + i], u.head) +
                                                        (tok & (p.c.P - 1)) * D + x % kChunks * 16));
        }
        if (i0 == 0) {
          // the first loads are on their way before the keys' place is free.  A
          // unit's factors stay until its weights are done, which this does not
          // wait for: they lag by two query tiles at most, so by two units
          if (!wait_bar(bar(kKFree + kb), ((uint32_t)(n / kKeyBufs) & 1u) ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int k = 0; k < kTokens / kKeyThreads; ++k) {
            const int t = kt + k * kKeyThreads;
            const bool good = (unsigned)own[k] < (unsigned)p.c.num_pages;
            if (!good && u.blk0 + t < u.s.len) report(p.status, W4_ERR_INDEX);
            info[(n % kInfoRing) * kTokens + t] =
                make_int2(good ? own[k] : -1, __float_as_int(f[k] * (p.scale * kLog2e)));
          }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int x = kt + (i0 + i) * kKeyThreads, t = x / kChunks, c = x % kChunks,
                    r = t & (kTile - 1);
          const uint32_t to = keys + (t >> 7) * S::kBytes + (c >> 2) * (kTile * 128) + r * 128;
          const int e = 2 * (c & 3);
          sts128(to + ((e ^ (r & 7)) << 4), codes_bf16(v[i].x, 0x4140), codes_bf16(v[i].x, 0x4342),
                 codes_bf16(v[i].y, 0x4140), codes_bf16(v[i].y, 0x4342));
          sts128(to + (((e + 1) ^ (r & 7)) << 4), codes_bf16(v[i].z, 0x4140),
                 codes_bf16(v[i].z, 0x4342), codes_bf16(v[i].w, 0x4140), codes_bf16(v[i].w, 0x4342));
        }
      }
      if (!ok) break;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kKFull + kb));
    }
  } else {
    // -------------------------------------------------------- the weights
    const int z = (warp >> 2) % kTiles, half = warp / (4 * kTiles);
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int mine = z * kTile + (tid & 127);
    float* sums = reinterpret_cast<float*>(sm + S::kSums) + mine;
    for (; ok && u.next(p, kTokens, false); ++n) {
      const int tok = u.blk0 + mine;
      uint64_t ff = 0;
      float sum = 0.0f, old = 0.0f;
      float* to = nullptr;
      for (int t = 0; t < u.qtiles; ++t, ++T) {
        const int par = T & 1, r0 = u.t_lo * p.G + t * rows;
        if (!wait_bar(bar(kSFull + 2 * par + z), (uint32_t)(T >> 1) & 1u, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (t == 0) {
          const int2 v = info[(n % kInfoRing) * kTokens + mine];
          const float f = __int_as_float(v.y);
          ff = pack2(f, f);
          if (half == 0 && v.x >= 0) {
            to = p.c.weight + (p.c.pair(v.x, u.head) * p.c.P + tok % p.c.P);
            old = *to;
          }
        }
        // columns whose rows see the token
        const int lo = (int)max(-1LL, min(1LL << 20, ((long long)tok - u.first) * p.G - r0));
        int hi = min(rows, u.t_hi * p.G - r0) - 1;   // (then come other rows, or zeros)
        if (p.window > 0)
          hi = (int)max(-1LL, min((long long)hi, ((long long)tok + p.window - u.first) * p.G - 1 - r0));
        const bool cut = __any_sync(0xffffffffu, lo > 0 || hi < rows - 1);
        const float* nl = lse + (T % kLseRing) * kTile;
#pragma unroll 1
        for (int c0 = half * (kTile / 2); c0 < (half + 1) * (kTile / 2); c0 += 32) {
          float x[32];
          tc::tmem_ld<32>(tmem + lanes + (2 * par + z) * kTile + c0, x);
          float4 l4[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) l4[e] = *reinterpret_cast<const float4*>(nl + c0 + 4 * e);
          tc::tmem_wait_ld<32>(x);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            unpack2(fma2(pack2(x[4 * e], x[4 * e + 1]), ff, pack2(l4[e].x, l4[e].y)), x[4 * e],
                    x[4 * e + 1]);
            unpack2(fma2(pack2(x[4 * e + 2], x[4 * e + 3]), ff, pack2(l4[e].z, l4[e].w)),
                    x[4 * e + 2], x[4 * e + 3]);
          }
          if (cut) {
            const uint32_t seen = columns(lo - c0, hi - c0);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(seen >> e & 1u)) x[e] = -INFINITY;
          }
          uint64_t s0 = 0, s1 = 0;
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
#pragma unroll
            for (int k = 0; k < 4; ++k) x[e + k] = exp2_fast(x[e + k]);
            s0 = add2(s0, pack2(x[e], x[e + 1]));
            s1 = add2(s1, pack2(x[e + 2], x[e + 3]));
          }
          float a, b;
          unpack2(add2(s0, s1), a, b);
          sum += a + b;
        }
        if (t + 1 == u.qtiles) {
          // the halves meet before the first gives the scores' columns back, so
          // a sum is read before the second may reach the unit after next
          float* other = sums + (n & 1) * kTokens;
          if (half == 1) {
            *other = sum;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kSumFull + 2 * (n & 1) + z));
          } else {
            if (!wait_bar(bar(kSumFull + 2 * (n & 1) + z), (uint32_t)(n >> 1) & 1u, abort_flag)) {
              ok = false;
              break;
            }
            if (to != nullptr) *to = old + (sum + *other);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kSFree + 2 * par + z));
      }
    }
  }
  if (!ok) {
    if (*abort_flag == 0) report(p.status, W4_ERR_TIMEOUT);
    *abort_flag = 1;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == S::kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(*tmem_slot)
                 : "memory");
}

template <int D>
w4_status launch_many(WeighParams& p, int sms, int dev, w4_stream_t stream) {
  using S = Shape<D>;
  static std::mutex mu;
  static bool done[64] = {};
  if (dev < 0 || dev >= 64) return W4_ERR_DEVICE;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      const cudaError_t e = cudaFuncSetAttribute(
          weigh_many_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
      if (e != cudaSuccess) {
        note_cuda_error(e);
        (void)cudaGetLastError();
        return W4_ERR_LAUNCH;
      }
      done[dev] = true;
    }
  }
  // query tiles: 64 channels of the group's heads of some tokens, rows of 128 bytes
  PFN_cuTensorMapEncodeTiled_v12000 enc = tc::encoder();
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.Hq, (cuuint64_t)p.bt.rows};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)p.q_stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)(kTile / p.G)};
  const cuuint32_t ones[3] = {1, 1, 1};
  if (enc == nullptr ||
      enc(&p.tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16*>(p.q), dims, strides,
          box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS) {
    note_cuda_error(cudaErrorInvalidValue);
    return W4_ERR_LAUNCH;
  }
  const int tokens = kTile * S::kTiles;
  const long long units = (long long)((p.bt.max_len + tokens - 1) / tokens) * p.c.H * p.bt.B;
  return launch(weigh_many_kernel<D>, dim3((unsigned)std::min<long long>(units, sms)), S::kThreads,
                S::kSmem, stream, p);
}

}  // namespace

w4_status weigh_many(WeighParams& p, int sms, int dev, w4_stream_t stream) {
  switch (p.c.D) {
    case 64: return launch_many<64>(p, sms, dev, stream);
    case 128: return launch_many<128>(p, sms, dev, stream);
    default: return launch_many<256>(p, sms, dev, stream);
  }
}

}  // namespace kv8
}  // namespace w4
