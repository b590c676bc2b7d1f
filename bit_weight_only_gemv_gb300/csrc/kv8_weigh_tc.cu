// Accumulated attention weights (w4_kv8_weigh) for prompt chunks, on the
// 5th-generation tensor cores (tcgen05, sm_103a).
//
// S^T = K q^T with tokens as the MMA's 128 rows: a token's scores lie along
// one thread's columns of tensor memory, so that its weights
//   2^(scale log2(e) ks S - log2(e) lse)
// add up in that thread's registers, in a fixed order of rows, without any
// exchange.  A CTA expands the keys of 256 tokens (128 of 256-channel heads)
// to bf16 once and takes all query rows that see one of them past, 128 at a
// time: two row tiles' keys share each query tile, which halves what the
// queries cost in L2 traffic.
//
// 2 x 256 rows of 32 heads on 8 of 128 channels, 8k keys: 51 us, 0.45 PFLOP/s
// (keys as legacy MMA fragments in every warp: 120 us).  A CTA's start (page
// ids, keys, expansion: about 6 us, 3.4 times over on 152 SMs) and about 2200
// cycles a query tile against 1024 of MMAs make that up; smaller CTAs, two an SM, hide more
// of the start and lose more on the queries (59 us).
//
// Roles: eight warps per key tile that exponentiate and add (a thread has a
// token and half of the columns), six that bring the
// query tiles in (two per buffer, so that several are on their way), one that issues
// the MMAs.  Every wait is bounded.
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

template <int D>
struct Shape {
  static constexpr int kTiles = D == 256 ? 1 : 2;   // key tiles of a CTA
  static constexpr int kBufs = D == 256 ? 2 : 3;    // query tiles in shared memory
  static constexpr int kLoadWarp = 8 * kTiles;      // weights: four warps a key tile and half of the columns
  static constexpr int kLoadWarps = 6;
  static constexpr int kPerBuf = kLoadWarps / kBufs;
  static constexpr int kMmaWarp = kLoadWarp + kLoadWarps;
  static constexpr int kThreads = 32 * (kMmaWarp + 1);
  static constexpr int kBytes = kTile * D * 2;      // of a tile, keys or queries
  static constexpr int kQ = kTiles * kBytes;
  static constexpr int kLse = kQ + kBufs * kBytes;  // [kLseRing][kTile]
  static constexpr int kBars = kLse + kLseRing * kTile * 4;
  static constexpr int kMisc = kBars + 16 * 8;
  static constexpr int kSums = kMisc + 64;          // [kTiles][kTile]: the second halves' sums
  static constexpr int kEnd = kSums + kTiles * kTile * 4 + 1024;
  // more than half an SM's: each CTA holds all of its tensor memory
  static constexpr int kSmem = kEnd > 117248 ? kEnd : 117248;
  static_assert(kSmem <= 232448 && 2 * kSmem > 232448, "shared memory");
};

enum { kQFull = 0, kQFree = 3, kSFull = 6, kSFree = 10, kBarCount = 14 };   // [3] [3] [2 x 2] [2 x 2]

template <int D>
__global__ void __launch_bounds__(Shape<D>::kThreads, 1)
    weigh_many_kernel(const __grid_constant__ WeighParams p) {
  using S = Shape<D>;
  constexpr int kTiles = S::kTiles, kBufs = S::kBufs;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw;
  const uint32_t sb = smem_addr(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto bar = [&](int i) { return sb + S::kBars + 8 * i; };
  float* lse = reinterpret_cast<float*>(sm + S::kLse);   // minus log2(e) lse; -inf: adds nothing
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + S::kMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + S::kMisc + 4);

  if (tid == 0) {
    for (int i = 0; i < 3; ++i) {
      mbar_init(bar(kQFull + i), S::kPerBuf);
      mbar_init(bar(kQFree + i), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(kSFull + i), 1);
      mbar_init(bar(kSFree + i), 8);
    }
    *abort_flag = 0;
    mbar_init_fence();
  }
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.y, b = blockIdx.z;
  const Seq s = sequence(p.bt, p.c.P, b);
  const int first = s.len - s.n;   // position of the first row
  const int blk0 = blockIdx.x * (kTile * kTiles);
  // rows that see some token of the block: positions from blk0 on, and within the window
  const int t_lo = max(0, blk0 - first);
  const int t_hi = p.window > 0 ? min(s.n, blk0 + kTile * kTiles - 1 + p.window - first) : s.n;
  if (!s.ok || blk0 >= s.len || t_lo >= t_hi) {
    if (!s.ok && tid == 0 && blockIdx.x == 0 && h == 0) report(p.status, W4_ERR_INDEX);
    return;
  }
  const int r_lo = t_lo * p.G, r_hi = t_hi * p.G;
  const int qtiles = (r_hi - r_lo + kTile - 1) / kTile;

  if (warp == S::kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // ------------------------------------------------------------- the keys
  const int32_t* table = p.bt.table + (long long)b * p.bt.max_pages;
  constexpr int kChunks = D / 16;   // 16-code chunks of a token
#pragma unroll 4
  for (int x = tid; x < kTiles * kTile * kChunks; x += S::kThreads) {
    const int t = x / kChunks, c = x % kChunks, r = t & (kTile - 1);
    const int tok = blk0 + t;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (tok < s.len) {
      const int page = __ldg(table + tok / p.c.P);
      if (page >= 0 && page < p.c.num_pages)
        v = __ldg(reinterpret_cast<const uint4*>(p.c.kc + p.c.block(page, h) +
                                                 (long long)(tok % p.c.P) * D + c * 16));
    }
    const uint32_t to = sb + (t >> 7) * S::kBytes + (c >> 2) * (kTile * 128) + r * 128;
    const int e = 2 * (c & 3);
    sts128(to + ((e ^ (r & 7)) << 4), codes_bf16(v.x, 0x4140), codes_bf16(v.x, 0x4342),
           codes_bf16(v.y, 0x4140), codes_bf16(v.y, 0x4342));
    sts128(to + (((e + 1) ^ (r & 7)) << 4), codes_bf16(v.z, 0x4140), codes_bf16(v.z, 0x4342),
           codes_bf16(v.w, 0x4140), codes_bf16(v.w, 0x4342));
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;   // all 512 columns: they begin at 0
  bool ok = __syncthreads_and(*tmem_slot == 0 && (sb & 1023u) == 0) != 0;

  float* sums = reinterpret_cast<float*>(sm + S::kSums);
  // of a thread that adds a token's weight in the end: its first half, its place
  float sum = 0.0f;
  int page = -1, from = 0;
  long long at = 0;
  bool mine = false;
  if (warp == S::kMmaWarp) {
    // -------------------------------------------------------- MMA issuer
    constexpr uint32_t kDesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kTile >> 3) << 17) |
                               ((uint32_t)(kTile >> 4) << 24);
    const uint64_t dk = desc_sw128(sb), dq = desc_sw128(sb + S::kQ);
    for (int t = 0; ok && t < qtiles; ++t) {
      const int buf = t % kBufs, par = t & 1;
      ok = wait_bar(bar(kQFull + buf), (uint32_t)(t / kBufs) & 1u, abort_flag);
      for (int z = 0; ok && z < kTiles; ++z) {
        ok = wait_bar(bar(kSFree + 2 * par + z), ((uint32_t)(t >> 1) & 1u) ^ 1u, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint64_t a0 = dk + z * (S::kBytes / 16), b0 = dq + buf * (S::kBytes / 16);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ss_f16(tmem + (2 * par + z) * kTile, a0 + (k >> 2) * (kTile * 128 / 16) + (k & 3) * 2,
                     b0 + (k >> 2) * (kTile * 128 / 16) + (k & 3) * 2, kDesc, k > 0);
        mma_commit(bar(kSFull + 2 * par + z));
      }
      if (ok) mma_commit(bar(kQFree + buf));
    }
    if (ok) {   // the last commit lands before the CTA may leave
      mbar_wait_bounded(bar(kQFree + (qtiles - 1) % kBufs), (uint32_t)((qtiles - 1) / kBufs) & 1u,
                        kWaitCycles);
    } else {
      const long long t0 = clock64();
      while (clock64() - t0 < (1 << 20)) {
      }
    }
  } else if (warp >= S::kLoadWarp) {
    // ------------------------------------------------------- query tiles
    const int w = warp - S::kLoadWarp, buf = w / S::kPerBuf;
    const int lt = (w % S::kPerBuf) * 32 + lane;   // among the buffer's threads
    const int R = s.n * p.G;
    for (int t = buf; ok && t < qtiles; t += kBufs) {
      if (!wait_bar(bar(kQFree + buf), ((uint32_t)(t / kBufs) & 1u) ^ 1u, abort_flag)) {
        ok = false;
        break;
      }
      const int r0 = r_lo + t * kTile;
      for (int x = lt; x < kTile * (D / 8); x += 32 * S::kPerBuf) {
        const int r = x / (D / 8), ch = x % (D / 8);
        const int row = min(r0 + r, R - 1);
        const uint32_t dst = sb + S::kQ + buf * S::kBytes + (ch >> 3) * (kTile * 128) + r * 128 +
                             (((ch & 7) ^ (r & 7)) << 4);
        const __nv_bfloat16* src = p.q + (long long)(s.row0 + row / p.G) * p.q_stride +
                                   (long long)(h * p.G + row % p.G) * D + ch * 8;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                     "r"(r0 + r < r_hi ? 16 : 0)
                     : "memory");
      }
      // (the ring is longer than the buffers': its reader may lag behind the MMAs)
      for (int r = lt; r < kTile; r += 32 * S::kPerBuf) {
        float v = -INFINITY;
        if (r0 + r < r_hi) {
          const int row = r0 + r;
          const float l = p.lse[(long long)(s.row0 + row / p.G) * p.Hq + h * p.G + row % p.G];
          if (l != -INFINITY) v = -l * kLog2e;
        }
        lse[(t % kLseRing) * kTile + r] = v;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kQFull + buf));
    }
  } else {
    // -------------------------------------------------------- the weights
    const int z = (warp >> 2) % kTiles, half = warp / (4 * kTiles);
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int tok = blk0 + z * kTile + (tid & 127);
    float f = 0.0f;
    if (tok < s.len) {
      page = __ldg(table + tok / p.c.P);
      if (page < 0 || page >= p.c.num_pages) {
        page = -1;
        report(p.status, W4_ERR_INDEX);
      } else {
        f = __ldg(p.c.ks + p.c.pair(page, h)) * (p.scale * kLog2e);
      }
    }
    const uint64_t ff = pack2(f, f);
    for (int t = 0; t < qtiles; ++t) {
      const int par = t & 1, r0 = r_lo + t * kTile;
      if (!wait_bar(bar(kSFull + 2 * par + z), (uint32_t)(t >> 1) & 1u, abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // columns whose rows see the token
      const int lo = (int)max(-1LL, min(1LL << 20, (long long)(tok - first) * p.G - r0));
      const int hi = p.window > 0
                         ? (int)max(-1LL, min(1LL << 20, (long long)(tok + p.window - first) * p.G - 1 - r0))
                         : kTile - 1;
      const bool cut = __any_sync(0xffffffffu, lo > 0 || hi < kTile - 1);
      const float* nl = lse + (t % kLseRing) * kTile;
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
          unpack2(fma2(pack2(x[4 * e + 2], x[4 * e + 3]), ff, pack2(l4[e].z, l4[e].w)), x[4 * e + 2],
                  x[4 * e + 3]);
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
        float u, v;
        unpack2(add2(s0, s1), u, v);
        sum += u + v;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kSFree + 2 * par + z));
    }
    if (half == 1) sums[z * kTile + (tid & 127)] = sum;
    mine = ok && half == 0 && page >= 0;
    if (mine) at = p.c.pair(page, h) * p.c.P + tok % p.c.P;
    if (mine) from = z * kTile + (tid & 127);
  }
  if (!ok) {
    if (*abort_flag == 0) report(p.status, W4_ERR_TIMEOUT);
    *abort_flag = 1;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (mine && *abort_flag == 0) p.c.weight[at] += sum + sums[from];
  if (warp == S::kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(*tmem_slot)
                 : "memory");
}

template <int D>
w4_status launch_many(const WeighParams& p, int dev, w4_stream_t stream) {
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
  const int tokens = kTile * S::kTiles;
  return launch(weigh_many_kernel<D>,
                dim3((unsigned)((p.bt.max_len + tokens - 1) / tokens), (unsigned)p.c.H,
                     (unsigned)p.bt.B),
                S::kThreads, S::kSmem, stream, p);
}

}  // namespace

w4_status weigh_many(const WeighParams& p, int dev, w4_stream_t stream) {
  switch (p.c.D) {
    case 64: return launch_many<64>(p, dev, stream);
    case 128: return launch_many<128>(p, dev, stream);
    default: return launch_many<256>(p, dev, stream);
  }
}

}  // namespace kv8
}  // namespace w4
