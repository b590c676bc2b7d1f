// Accumulated attention weights of the cached tokens (w4_kv8_weigh):
//   weight[t] += sum over the rows r that see t of 2^(scale log2(e) q_r.k_t - log2(e) lse_r).
//
// Every token's sum belongs to one warp, in a fixed order of rows, and is added to
// its weight once: the same bits at every call.  Keys are read once (values not at all);
// S^T = K q^T on the tensor cores as in the attention kernels, tokens as rows.
//
// Few rows on a key head (single tokens): the bytes of the keys bound it;
// equal runs of 16-token slices over all sequences, each warp streaming its
// own through a ring of tiled copies, query fragments in registers; also over
// chosen pages.  8
// sequences of up to 16k tokens, 32 heads on 8 of 128 channels: 25.9 us, 3.8
// TB/s; about 10 us of that are the start (lengths, page ids, first copies), the
// rest runs at 6 TB/s.
// Up to 64 rows (48 but for 128 channels): a warp keeps its tokens' keys as fragments in registers,
// converted once, and walks all query rows, which the CTA brings into shared
// memory in fragment order; the legacy MMAs bound it (2 x 8k keys, 8 heads of
// 128 channels: 20 rows 12.7 us, 64 rows 16.3).  Beyond that kv8_weigh_tc.cu.
#include <algorithm>
#include <mutex>

#include "gemv_host.h"
#include "kv8_attn.h"
#include "kv8_mma.cuh"
#include "kv8_runs.cuh"

namespace w4 {
namespace kv8 {
namespace {

constexpr int kSlice = 16;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kRing = 64;
// Slices of a CTA's run, at least (two a warp): one token on 2k keys, 32 heads on
// 8 of 128 channels 6.4 us (8: 5.7, 32: 8.0), on 16k keys of one head 6.7 (8: 6.1,
// 32: 8.1), 8 on 1k 9.4 (8: 9.1, 32: 12.0).
constexpr int kMinSlices = 16;
constexpr long long kWait = 1LL << 31;   // about a second

// ------------------------------------------------------------ few rows
template <int D>
struct Shape {
  static constexpr int kStageBytes = kSlice * D;
  static constexpr int kStages = D == 256 ? 3 : 6;
  static constexpr int kMeta = kWarps * kStages * kStageBytes;   // [kWarps][kRing] Meta
  static constexpr int kBars = kMeta + kWarps * kRing * 16;
  static constexpr int kMisc = kBars + kWarps * kStages * 8;
  static constexpr int kSmem = kMisc + 8 * (2 * kWarps + 2) + 1024;
};

struct Meta {
  int page;   // -1: nothing to read
  int tok;
  float ks;
  int pad;
};

__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int x, int tok, int h,
                                       int page, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(tok), "r"(h), "r"(page), "r"(bar)
      : "memory");
}

// kSel: over the pages of p.sel, one row a sequence.  A run's entries are then
// (sequence, head) pairs, and groups of more query rows than a tile go through
// the same slices tile by tile, so that a token's additions keep their order.
// 16 sequences, 128 pages of 32 tokens each out of up to 1024, 32 heads on 8 of 128
// channels: 20.2 us (the whole cache 73.7).
template <int D, int NQ, bool kSel>
__global__ void __launch_bounds__(kThreads, 2)
    weigh_token_kernel(const __grid_constant__ WeighParams p) {
  using S = Shape<D>;
  constexpr int kRows = 8 * NQ, kStages = S::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_addr(smem_raw) & 1023u)) & 1023u;
  uint8_t* sm = smem_raw + pad;
  const uint32_t sbase = smem_addr(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, i = lane >> 2, j = lane & 3;
  Meta* meta = reinterpret_cast<Meta*>(sm + S::kMeta) + warp * kRing;
  const uint32_t bar0 = sbase + S::kBars + warp * kStages * 8;
  const uint32_t stage0 = sbase + warp * kStages * S::kStageBytes;
  long long* scan = reinterpret_cast<long long*>(sm + S::kMisc);
  pdl_launch_dependents();
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(bar0 + 8 * s, 1);
    mbar_init_fence();
  }
  pdl_wait();
  if (blockIdx.x == 0)
    for (int b = tid; b < p.bt.B; b += kThreads)
      if (!sequence(p.bt, p.c.P, b).ok) report(p.status, W4_ERR_INDEX);
  const int per = p.c.P / kSlice;
  auto weight = [&](int e, int* units) -> long long {
    const Seq s = sequence(p.bt, p.c.P, kSel ? e / p.c.H : e);
    if (!s.ok || s.n == 0) return 0;
    if (kSel) {
      const int n = load_in(p.n_sel + e);
      if (n <= 0 || n > p.max_sel) {
        if (n != 0 && blockIdx.x == 0) report(p.status, W4_ERR_INDEX);
        return 0;
      }
      *units += 1;
      return (long long)n * per;
    }
    *units += p.c.H;   // one row tile
    return head_slices(s, p.G, p.window, kRows, kSlice) * p.c.H;
  };
  Run run;
  const bool any = find_run<kWarps>(kSel ? p.bt.B * p.c.H : p.bt.B, kMinSlices, weight, scan, &run);
  __syncthreads();
  if (!any) return;

  int put = 0, got = 0;
  uint32_t got_phase = 0;
  bool dead = false;
  long long g = run.g0, off = run.off;
  int entry = run.entry;
  while (g < run.g1 && !dead) {
    const int b = kSel ? entry / p.c.H : entry;
    const Seq s = sequence(p.bt, p.c.P, b);
    Tile t = tile_of(s, p.G, p.window, 0, kRows, kSlice);   // one row tile
    if (kSel) t.slices = load_in(p.n_sel + entry) * per;
    const int h = kSel ? entry - b * p.c.H : quotient(off, t.slices);
    const int sl0 = kSel ? (int)off : (int)(off - (long long)h * t.slices);
    const int sl1 = (int)min((long long)t.slices, sl0 + (run.g1 - g));
    const int32_t* table = p.bt.table + (long long)b * p.bt.max_pages;
    const int R = s.n * p.G;
#pragma unroll 1
    for (int r0 = 0; r0 < (kSel ? R : 1) && !dead; r0 += kRows) {   // dense: one row tile
      uint2 raw[NQ][D / 16];   // query rows, on their way
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const int r = (kSel ? r0 : 0) + 8 * n + i;
        load_query<D>(r < R ? p.q + (long long)(s.row0 + r / p.G) * p.q_stride +
                                  (long long)(h * p.G + r % p.G) * D
                            : nullptr,
                      j, raw[n]);
      }
      const int count = (sl1 - sl0 - warp + kWarps - 1) / kWarps;
      // the steps' loads set out before the first copies (behind them they would
      // queue) and are waited for after them
      float ks = 0.0f;
      auto fill_steps = [&](int k0) {
        if (k0 + lane < count) meta[(k0 + lane) & (kRing - 1)].ks = ks;
        __syncwarp();
      };
      auto issue = [&](int k) {
        if (k >= count || dead) return;
        if ((k & 31) == 0) {   // descriptions of the next 32 slices
          __syncwarp();
          const int kk = k + lane;
          if (kk < count) {
            const int sl = sl0 + warp + kWarps * kk;
            Meta d = {-1, t.lo + sl * kSlice, 0.0f, 0};
            bool read = d.tok < t.hi;
            if (kSel) {
              const int lp = load_in(p.sel + (long long)entry * p.max_sel + sl / per);
              read = lp >= 0 && (long long)lp * p.c.P < s.len;
              if (!read) report(p.status, W4_ERR_INDEX);
              d.tok = read ? lp * p.c.P + sl % per * kSlice : 0;
              read &= d.tok < t.hi &&
                      !(p.window > 0 && d.tok + kSlice <= (long long)t.pmin + 1 - p.window);
            }
            if (read) {
              const int page = load_in(table + d.tok / p.c.P);
              if (page < 0 || page >= p.c.num_pages) {
                report(p.status, W4_ERR_INDEX);
              } else {
                d.page = page;
                ks = load_in(p.c.ks + p.c.pair(page, h));
              }
            }
            meta[kk & (kRing - 1)] = d;
          }
          __syncwarp();
        }
        if (lane == 0) {
          const Meta d = meta[k & (kRing - 1)];
          const uint32_t bar = bar0 + 8 * put, st = stage0 + put * S::kStageBytes;
          if (d.page < 0) {
            mbar_arrive(bar);
          } else {
            mbar_arrive_expect_tx(bar, S::kStageBytes);
#pragma unroll
            for (int x = 0; x < D; x += 128)
              tma_4d(st + x * kSlice, &p.tm, x, d.tok & (p.c.P - 1), h, d.page, bar);
          }
        }
        if (++put == kStages) put = 0;
        if (k > 0 && (k & 31) == 0) fill_steps(k);   // once its first copy is on its way
      };
#pragma unroll 1
      for (int k = 0; k < kStages; ++k) issue(k);
      fill_steps(0);
      uint32_t q[NQ][D / 16][2];
      float f[NQ][2], lse2[NQ][2];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const float down = scale_query<D>(raw[n], q[n]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          f[n][c] = __shfl_sync(0xffffffffu, down, 8 * j + 4 * c) * (p.scale * kLog2e);
          const int rc = (kSel ? r0 : 0) + 8 * n + 2 * j + c;
          float l = INFINITY;   // adds nothing
          if (rc < R) {
            l = p.lse[(long long)(s.row0 + rc / p.G) * p.Hq + h * p.G + rc % p.G] * kLog2e;
            if (l == -INFINITY) l = INFINITY;
          }
          lse2[n][c] = l;
        }
      }
#pragma unroll 1
      for (int k = 0; k < count; ++k) {
        if (!mbar_wait_bounded(bar0 + 8 * got, got_phase, kWait)) {
          dead = true;
          if (lane == 0) report(p.status, W4_ERR_TIMEOUT);
          break;
        }
        const Meta d = meta[k & (kRing - 1)];
        if (d.page >= 0) {
          float* w = p.c.weight + p.c.pair(d.page, h) * p.c.P + (d.tok & (p.c.P - 1)) + i;
          float x[NQ][4];
          key_scores<D, NQ>(stage0 + got * S::kStageBytes, i, j, q, x);
          const bool cut = d.tok + kSlice - 1 > t.pmin || (p.window > 0 && d.tok <= t.pmax - p.window);
          float a0 = 0.0f, a1 = 0.0f;
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float y = exp2_fast(fmaf(x[n][e], d.ks * f[n][e & 1], -lse2[n][e & 1]));
              if (cut) {
                // (chosen pages: one row a sequence, the last position)
                const int r = kSel ? 0 : min(R - 1, 8 * n + 2 * j + (e & 1));
                const int pos = s.len - s.n + r / p.G, tok = d.tok + i + 8 * (e >> 1);
                if (tok > pos || (p.window > 0 && tok <= pos - p.window)) y = 0.0f;
              }
              (e < 2 ? a0 : a1) += y;
            }
          a0 += __shfl_xor_sync(0xffffffffu, a0, 1);
          a1 += __shfl_xor_sync(0xffffffffu, a1, 1);
          a0 += __shfl_xor_sync(0xffffffffu, a0, 2);
          a1 += __shfl_xor_sync(0xffffffffu, a1, 2);
          if (j == 0) {
            // one addition to each weight, which nothing here waits for (when 8 x
            // 16k keys took 29.0 us, loading the old weight first cost 30.8)
            if (d.tok + i < s.len) atomicAdd(w, a0);
            if (d.tok + i + 8 < s.len) atomicAdd(w + 8, a1);
          }
        }
        __syncwarp();
        if (++got == kStages) {
          got = 0;
          got_phase ^= 1u;
        }
        issue(k + kStages);
      }
    }
    const long long step = sl1 - sl0;
    g += step;
    off += step;
    if (off == (long long)t.slices * (kSel ? 1 : p.c.H) && g < run.g1) {
      off = 0;
      int none = 0;
      do ++entry;
      while (weight(entry, &none) == 0);
    }
  }
  if (dead)   // copies still in flight land before the CTA leaves
    for (int s = 0; s < kStages; ++s) mbar_wait_bounded(bar0 + 8 * s, got_phase, kWait >> 4);
}

// ------------------------------------------------------------ many rows
// The most rows of this kernel, and of it at a head size; above, kv8_weigh_tc.cu.
// 2 x 8k keys, 8 heads of 64 and 128 channels, 4 of 256: 48 rows 12.4, 14.7 and
// 14.5 us here and 12.8, 18.7 and 15.1 there; 64 rows 13.5, 16.2 and 16.4 against
// 12.8, 18.6 and 15.2; 96 rows 16.2, 20.1 and 20.7 against 12.8, 18.7 and 15.2.
constexpr int kManyRows = 64;
constexpr int many_rows(int D) { return D == 128 ? kManyRows : 48; }

__device__ __forceinline__ void mma_bf16(float d[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// One CTA per (block of tokens, head, sequence); kSub 16-token slices a warp.
template <int D, int kSub>
__global__ void __launch_bounds__(kThreads, 2)
    weigh_chunk_kernel(const __grid_constant__ WeighParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // [tile of 8 rows][D / 32][lane] 16 bytes: the lane's four column registers
  // of two steps of 16 channels
  const uint32_t qs = smem_addr(smem_raw);
  float* lse2 = reinterpret_cast<float*>(smem_raw + kManyRows * D * 2);
  pdl_launch_dependents();
  pdl_wait();
  constexpr int kTokens = kWarps * kSub * kSlice;
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int i = lane >> 2, j = lane & 3;
  const Seq s = sequence(p.bt, p.c.P, b);
  if (!s.ok) {
    if (tid == 0 && blockIdx.x == 0 && h == 0) report(p.status, W4_ERR_INDEX);
    return;
  }
  const int first = s.len - s.n;   // position of the first row
  const int blk0 = blockIdx.x * kTokens;
  if (s.n == 0 || blk0 >= s.len) return;
  const int R = s.n * p.G;
  // rows that see some token of the block: positions from blk0 on, and within the window
  int t_lo = max(0, blk0 - first), t_hi = s.n;
  if (p.window > 0) t_hi = (int)min((long long)s.n, (long long)blk0 + kTokens - 1 + p.window - first);
  if (t_lo >= t_hi) return;
  const int r_lo = t_lo * p.G, r_hi = t_hi * p.G;

  // this warp's keys
  uint32_t a[kSub][D / 16][4];
  float f[kSub], sum[kSub][2];
  int page[kSub], tok[kSub];
#pragma unroll
  for (int z = 0; z < kSub; ++z) {
    tok[z] = blk0 + (warp * kSub + z) * kSlice;
    page[z] = -1;
    f[z] = sum[z][0] = sum[z][1] = 0.0f;
    if (tok[z] < s.len) {
      page[z] = load_in(p.bt.table + (long long)b * p.bt.max_pages + tok[z] / p.c.P);
      if (page[z] < 0 || page[z] >= p.c.num_pages) {
        page[z] = -1;
        if (lane == 0) report(p.status, W4_ERR_INDEX);
      }
    }
    const bool have = page[z] >= 0;
    if (have) f[z] = load_in(p.c.ks + p.c.pair(page[z], h)) * (p.scale * kLog2e);
    const uint8_t* blk = p.c.kc + (have ? p.c.block(page[z], h) + (long long)(tok[z] % p.c.P) * D : 0);
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      const int chunk = D == 64 ? j : 8 * (c / 2) + 2 * j + (c & 1);
      uint4 x = make_uint4(0, 0, 0, 0), y = x;
      if (have) {
        x = load_in(reinterpret_cast<const uint4*>(blk + i * D + chunk * 16));
        y = load_in(reinterpret_cast<const uint4*>(blk + (i + 8) * D + chunk * 16));
      }
      const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        a[z][4 * c + w][0] = codes_bf16(xw[w], 0x4140);
        a[z][4 * c + w][1] = codes_bf16(yw[w], 0x4140);
        a[z][4 * c + w][2] = codes_bf16(xw[w], 0x4342);
        a[z][4 * c + w][3] = codes_bf16(yw[w], 0x4342);
      }
    }
  }
  const int n = r_hi - r_lo, tiles = (n + 7) / 8;
  for (int x = tid; x < tiles * 8 * (D / 8); x += kThreads) {
    // 8 channels (16 bytes) of a row: two steps of one lane
    const int r = x / (D / 8), c8 = x % (D / 8), chunk = c8 >> 1;
    // the chunk's lane and its place among the lane's chunks
    const int jj = D == 64 ? chunk : (chunk & 7) >> 1;
    const int c = D == 64 ? 0 : 2 * (chunk >> 3) + (chunk & 1);
    const uint32_t dst =
        qs + (((r >> 3) * (D / 32) + 2 * c + (c8 & 1)) * 32 + (r & 7) * 4 + jj) * 16;
    const int row = min(r_lo + r, R - 1);
    const __nv_bfloat16* src = p.q + (long long)(s.row0 + row / p.G) * p.q_stride +
                               (long long)(h * p.G + row % p.G) * D + c8 * 8;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  }
  for (int r = tid; r < tiles * 8; r += kThreads) {
    float l = INFINITY;   // adds nothing
    if (r < n) {
      const int row = r_lo + r;
      l = p.lse[(long long)(s.row0 + row / p.G) * p.Hq + h * p.G + row % p.G] * kLog2e;
      if (l == -INFINITY) l = INFINITY;
    }
    lse2[r] = l;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
#pragma unroll 1
  for (int t = 0; t < tiles; ++t) {
    float x[kSub][4];
#pragma unroll
    for (int z = 0; z < kSub; ++z)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[z][e] = 0.0f;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {
      const uint4 q = lds128(qs + ((t * (D / 32) + k) * 32 + lane) * 16);
#pragma unroll
      for (int z = 0; z < kSub; ++z) {
        mma_bf16(x[z], a[z][2 * k], q.x, q.y);
        mma_bf16(x[z], a[z][2 * k + 1], q.z, q.w);
      }
    }
    const float2 l = *reinterpret_cast<const float2*>(lse2 + 8 * t + 2 * j);
    const int pmin = first + (r_lo + 8 * t) / p.G;
    const int pmax = first + min(R - 1, r_lo + 8 * t + 7) / p.G;
#pragma unroll
    for (int z = 0; z < kSub; ++z) {
      float y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = exp2_fast(fmaf(x[z][e], f[z], (e & 1) ? -l.y : -l.x));
      if (tok[z] + kSlice - 1 > pmin || (p.window > 0 && tok[z] <= pmax - p.window)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int pos = first + min(R - 1, r_lo + 8 * t + 2 * j + (e & 1)) / p.G;
          const int k = tok[z] + i + 8 * (e >> 1);
          if (k > pos || (p.window > 0 && k <= pos - p.window)) y[e] = 0.0f;
        }
      }
      sum[z][0] += y[0] + y[1];
      sum[z][1] += y[2] + y[3];
    }
  }
#pragma unroll
  for (int z = 0; z < kSub; ++z)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float v = sum[z][e];
      v += __shfl_xor_sync(0xffffffffu, v, 1);
      v += __shfl_xor_sync(0xffffffffu, v, 2);
      const int k = tok[z] + i + 8 * e;
      if (j == 0 && page[z] >= 0 && k < s.len)
        p.c.weight[p.c.pair(page[z], h) * p.c.P + k % p.c.P] += v;
    }
}

// ================================================================= host side
template <typename K>
w4_status allow_smem(K kern, int smem, int dev, bool* done) {
  static std::mutex mu;
  if (dev < 0 || dev >= 64) return W4_ERR_DEVICE;
  std::lock_guard<std::mutex> lock(mu);
  if (!done[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) {
      note_cuda_error(e);
      (void)cudaGetLastError();
      return W4_ERR_LAUNCH;
    }
    done[dev] = true;
  }
  return W4_OK;
}

template <int D, int NQ, bool kSel>
w4_status launch_token(WeighParams& p, int sms, w4_stream_t stream, int dev) {
  static bool done[64] = {};
  if (!tensor_map(&p.tm, p.c.kc, p.c, kSlice)) {
    note_cuda_error(cudaErrorInvalidValue);
    return W4_ERR_LAUNCH;
  }
  const w4_status st = allow_smem(weigh_token_kernel<D, NQ, kSel>, Shape<D>::kSmem, dev, done);
  if (st != W4_OK) return st;
  return launch(weigh_token_kernel<D, NQ, kSel>, dim3((unsigned)(2 * sms)), kThreads, Shape<D>::kSmem,
                stream, p);
}

template <int D>
w4_status launch_chunk(const WeighParams& p, w4_stream_t stream, int dev) {
  constexpr int kSub = D == 256 ? 1 : 2;   // 128 registers of fragments are too many
  constexpr int kSmem = kManyRows * D * 2 + kManyRows * 4;
  static bool done[64] = {};
  const w4_status st = allow_smem(weigh_chunk_kernel<D, kSub>, kSmem, dev, done);
  if (st != W4_OK) return st;
  const int tokens = kWarps * kSub * kSlice;
  return launch(weigh_chunk_kernel<D, kSub>,
                dim3((unsigned)((p.bt.max_len + tokens - 1) / tokens), (unsigned)p.c.H,
                     (unsigned)p.bt.B),
                kThreads, kSmem, stream, p);
}

}  // namespace
}  // namespace kv8
}  // namespace w4

using namespace w4;

extern "C" w4_status w4_kv8_weigh(const void* q, size_t q_row_stride, int q_heads,
                                  const float* lse, const w4_kv8_cache* cache,
                                  const w4_kv8_batch* batch, float scale, int window,
                                  int32_t* status_dev, unsigned flags, w4_stream_t stream) {
  return w4_kv8_weigh_pages(q, q_row_stride, q_heads, lse, cache, batch, scale, window, nullptr,
                            nullptr, 0, status_dev, flags, stream);
}

extern "C" w4_status w4_kv8_weigh_pages(const void* q, size_t q_row_stride, int q_heads,
                                        const float* lse, const w4_kv8_cache* cache,
                                        const w4_kv8_batch* batch, float scale, int window,
                                        const int32_t* sel, const int32_t* n_sel, int max_sel,
                                        int32_t* status_dev, unsigned flags, w4_stream_t stream) {
  kv8::WeighParams p = {};
  w4_status st = kv8::view(cache, batch, &p.c, &p.bt);
  if (st != W4_OK) return st;
  if (lse == nullptr || p.c.weight == nullptr || (flags & ~W4_FLAG_PDL) != 0 || window < 0 ||
      (sel == nullptr) != (n_sel == nullptr) || (sel != nullptr && max_sel < 1))
    return W4_ERR_ARG;
  if ((st = kv8::check_q(q, q_row_stride, q_heads, p.c)) != W4_OK) return st;
  if (sel != nullptr && (p.bt.max_new != 1 || max_sel > (1 << 24))) return W4_ERR_SHAPE;
  if (kv8::misaligned(lse, 4) || kv8::misaligned(sel, 4) || kv8::misaligned(n_sel, 4))
    return W4_ERR_ALIGN;
  int dev = -1;
  DeviceInfo di;
  if (!current_device(&dev, &di)) return W4_ERR_DEVICE;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride = (long long)q_row_stride;
  p.lse = lse;
  p.Hq = q_heads;
  p.G = q_heads / p.c.H;
  p.scale = scale;
  p.window = window;
  p.sel = sel;
  p.n_sel = n_sel;
  p.max_sel = max_sel;
  p.status = status_dev;
  if (p.bt.max_len == 0) return W4_OK;
  const long long rows = (long long)p.bt.max_new * p.G;
  const int one = rows <= 8 ? 1 : 0;
  if (sel != nullptr) {
    switch (p.c.D * 2 + one) {
      case 64 * 2 + 1: return kv8::launch_token<64, 1, true>(p, di.sms, stream, dev);
      case 64 * 2: return kv8::launch_token<64, 2, true>(p, di.sms, stream, dev);
      case 128 * 2 + 1: return kv8::launch_token<128, 1, true>(p, di.sms, stream, dev);
      case 128 * 2: return kv8::launch_token<128, 2, true>(p, di.sms, stream, dev);
      case 256 * 2 + 1: return kv8::launch_token<256, 1, true>(p, di.sms, stream, dev);
      default: return kv8::launch_token<256, 2, true>(p, di.sms, stream, dev);
    }
  }
  if (rows > kv8::many_rows(p.c.D)) return kv8::weigh_many(p, di.sms, dev, stream);
  if (rows > 16) {
    switch (p.c.D) {
      case 64: return kv8::launch_chunk<64>(p, stream, dev);
      case 128: return kv8::launch_chunk<128>(p, stream, dev);
      default: return kv8::launch_chunk<256>(p, stream, dev);
    }
  }
  switch (p.c.D * 2 + one) {
    case 64 * 2 + 1: return kv8::launch_token<64, 1, false>(p, di.sms, stream, dev);
    case 64 * 2: return kv8::launch_token<64, 2, false>(p, di.sms, stream, dev);
    case 128 * 2 + 1: return kv8::launch_token<128, 1, false>(p, di.sms, stream, dev);
    case 128 * 2: return kv8::launch_token<128, 2, false>(p, di.sms, stream, dev);
    case 256 * 2 + 1: return kv8::launch_token<256, 1, false>(p, di.sms, stream, dev);
    default: return kv8::launch_token<256, 2, false>(p, di.sms, stream, dev);
  }
}
