// Attention over the 8-bit cache for few query rows on a key head: single
// tokens of a batch, also over chosen pages (w4_kv8_attn), and the entry that
// picks between this kernel and the prompt-chunk kernel.
//
// One pass over the keys and values with a running maximum and sum:
//   x_t = scale log2(e) q.k_t,  m = max x_t,  l = sum 2^(x_t - m),
//   o = sum 2^(x_t - m) v_t / l.
// The bytes of the cache bound it (2 D bytes a token and head against
// 4 D G flops), so the work is cut into equal runs of 16-token slices over
// all sequences and heads, one run a CTA, whatever the lengths: a run that
// begins or ends inside a (sequence, head) leaves a partial result in the
// workspace, and the last of its CTAs to arrive joins the parts in order.
// Each warp streams its own slices: a ring of tiled copies (TMA, swizzled so
// that no read below meets a bank conflict), its own running m, l and o; the
// CTA's warps join through shared memory once per run and unit.
//
// Tensor cores take the products in fp16 (kv8_mma.cuh): codes are exact,
// query rows are scaled by a power of two, weights 2^(x - m) are scaled by
// 2^11 times the block's value step over the largest step met so far (so a
// block's step costs one multiplication per weight).  m moves only when a
// score passes it by kLag: then, and when a larger step comes, o and l are
// rescaled; so most slices need no exchange between lanes.  A slice with
// weights below fp16's normal range takes one more pass over its values for
// each 29 bits of range: a channel that the heavy tokens leave at zero shows
// the light ones, and they keep their 11 bits too.
//
// 24 sequences of 4k to 16k tokens, 64 heads on 8 of 128 channels: 96 us, 5.5
// TB/s (81% of a plain copy's rate), DRAM reads 1.000 of the bytes counted.
// One token on 700 (512-token window, 8 heads on 2 of 256 channels): 15.7 us, a chain
// of about ten memory latencies: lengths, query and page ids, copies, the
// join in shared memory, the parts, the arrival, the last CTA's join.
#include <algorithm>
#include <mutex>

#include "gemv_host.h"
#include "kv8_attn.h"
#include "kv8_mma.cuh"
#include "kv8_runs.cuh"

namespace w4 {
namespace kv8 {
namespace {

constexpr int kSlice = 16;               // tokens of a slice
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kRing = 64;                // slice descriptions kept per warp
constexpr float kLag = 4.0f;             // log2 of how far a score may pass m
constexpr float kWeightScale = 2048.0f;  // weights as fp16: at most 2^(4 + 11)
constexpr float kHalfNormal = 6.103515625e-05f;   // 2^-14, fp16's least normal value
constexpr float kLevel = 536870912.0f;            // 2^29: from there to 2^15, well in range
constexpr float kLeast = 7.5e-37f;                // above 2^-120: five ranges reach it
constexpr long long kWait = 1LL << 31;   // about a second
// Slices of a CTA's run, at least (two a warp): one token on 2k keys, 32 heads on
// 8 of 128 channels 11.5 us (4: 13.9, 8: 11.8, 32: 13.8), on 16k keys of one head
// 20.0 (8: 29.5, 32: 17.4), 8 on 1k 18.1 (8: 17.8, 32: 21.2).
constexpr int kMinSlices = 16;

template <int D, int NQ>
struct Shape {
  static constexpr int kRows = 8 * NQ;                        // query rows of a unit
  static constexpr int kStageBytes = 2 * kSlice * D;          // keys, then values
  static constexpr int kPerSm = D == 256 ? 1 : 2;             // resident CTAs
  static constexpr int kStages = D == 64 ? 6 : 3;
  static constexpr int kPitch = D + 4;                        // floats of a joined row
  static constexpr int kStageTotal = kWarps * kStages * kStageBytes;
  static_assert(kWarps * kRows * kPitch * 4 <= kStageTotal, "the join reuses the stages");
  static constexpr int kMeta = kStageTotal;                   // [kWarps][kRing] Meta
  static constexpr int kStats = kMeta + kWarps * kRing * 16;  // [kWarps][kRows] (m, l)
  static constexpr int kBars = kStats + kWarps * kRows * 8;
  static constexpr int kMisc = kBars + kWarps * kStages * 8;
  static constexpr int kSmem = kMisc + 16 + 8 * (2 * kWarps + 2) + 1024;   // and alignment
};

struct Meta {
  int page;   // -1: nothing to read
  int tok;    // position of the slice's first token
  float ks, vs;
};

struct AttnParams {
  CUtensorMap tm_k, tm_v;   // [page][head][token][channel] bytes, boxes of 16 tokens
  Cache c;
  Batch bt;
  __nv_bfloat16* out;
  float* lse;
  const __nv_bfloat16* q;
  long long q_stride;
  int Hq, G;
  float scale;
  int window;
  const int32_t* sel;
  const int32_t* n_sel;
  int max_sel;
  int32_t* arrived;   // [CTAs], zero between calls: of the unit whose first part the CTA has
  float* parts;       // [2 * CTAs][rows][D]
  float* part_stats;  // [2 * CTAs][rows][2]: m, l (l = -1: refused)
  int32_t* status;
};

// Pages chosen for a (sequence, head); a count that is none is 0 (refused later).
__device__ __forceinline__ int chosen(const AttnParams& p, long long bh, bool* bad) {
  const int n = __ldg(p.n_sel + bh);
  if (n < 0 || n > p.max_sel) {
    *bad = true;
    return 0;
  }
  return n;
}

// A row tile over the whole sequence (pages < 0) or over `pages` chosen ones.
__device__ __forceinline__ Tile unit_tile(const AttnParams& p, const Seq& s, int rt, int rows,
                                          int pages) {
  Tile t = tile_of(s, p.G, p.window, rt, rows, kSlice);
  if (pages >= 0) {
    t.lo = 0;
    t.slices = max(1, pages * (p.c.P / kSlice));
  }
  return t;
}

// Slices of an entry: a sequence (all heads), or with chosen pages a
// (sequence, head).
__device__ __forceinline__ long long entry_slices(const AttnParams& p, int e, int rows, int* units) {
  const int b = p.sel == nullptr ? e : e / p.c.H;
  const Seq s = sequence(p.bt, p.c.P, b);
  if (!s.ok || s.n == 0) return 0;
  const int rts = (s.n * p.G + rows - 1) / rows;
  *units += p.sel == nullptr ? rts * p.c.H : rts;
  if (p.sel == nullptr) return head_slices(s, p.G, p.window, rows, kSlice) * p.c.H;
  bool bad = false;
  return (long long)unit_tile(p, s, 0, rows, chosen(p, e, &bad)).slices * rts;
}

__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int x, int tok, int h,
                                       int page, uint32_t bar, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::"
      "cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(tok), "r"(h), "r"(page), "r"(bar), "l"(pol)
      : "memory");
}

template <int D, int NQ>
__global__ void __launch_bounds__(kThreads, Shape<D, NQ>::kPerSm)
    attn_token_kernel(const __grid_constant__ AttnParams p) {
  using S = Shape<D, NQ>;
  constexpr int kRows = S::kRows, kStages = S::kStages, kPitch = S::kPitch;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_addr(smem_raw) & 1023u)) & 1023u;
  uint8_t* sm = smem_raw + pad;
  const uint32_t sbase = smem_addr(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, i = lane >> 2, j = lane & 3;
  Meta* meta = reinterpret_cast<Meta*>(sm + S::kMeta) + warp * kRing;
  float2* stats = reinterpret_cast<float2*>(sm + S::kStats);
  float* join = reinterpret_cast<float*>(sm);
  const uint32_t bar0 = sbase + S::kBars + warp * kStages * 8;
  const uint32_t stage0 = sbase + warp * kStages * S::kStageBytes;
  volatile int* refused = reinterpret_cast<volatile int*>(sm + S::kMisc);   // [2]: even, odd units
  volatile int* flag = refused + 2;
  long long* scan = reinterpret_cast<long long*>(sm + S::kMisc + 16);

  pdl_launch_dependents();
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(bar0 + 8 * s, 1);
    mbar_init_fence();
  }
  if (tid < 2) refused[tid] = 0;
  pdl_wait();
  // sequences whose bounds are broken belong to no run: the first CTA says so
  if (blockIdx.x == 0)
    for (int b = tid; b < p.bt.B; b += kThreads)
      if (!sequence(p.bt, p.c.P, b).ok) report(p.status, W4_ERR_INDEX);
  Run run;
  const bool any = find_run<kWarps>(
      p.sel == nullptr ? p.bt.B : p.bt.B * p.c.H, kMinSlices,
      [&](int e, int* units) { return entry_slices(p, e, kRows, units); }, scan, &run);
  __syncthreads();
  if (!any) return;

  const uint64_t pol = policy_evict_first();
  int put = 0, got = 0;              // stages filled and read, modulo kStages
  uint32_t got_phase = 0;
  bool dead = false;                 // a wait ran out
  long long g = run.g0, off = run.off;
  int entry = run.entry;
  int odd = 0;                       // units walked, modulo 2
  while (g < run.g1) {
    // ---------------------------------------------------------- the unit
    const int b = p.sel == nullptr ? entry : entry / p.c.H;
    const Seq s = sequence(p.bt, p.c.P, b);
    const int rts = (s.n * p.G + kRows - 1) / kRows;
    int h, rt = 0, sl0, n_pages = -1;
    bool bad = false;
    Tile t;
    long long left;   // slices of the entry from this unit's slice sl0 on
    if (p.sel != nullptr) {
      h = entry - b * p.c.H;
      n_pages = chosen(p, entry, &bad);
      t = unit_tile(p, s, 0, kRows, n_pages);
      rt = quotient(off, t.slices);
      sl0 = (int)(off - (long long)rt * t.slices);
      t = unit_tile(p, s, rt, kRows, n_pages);
      left = (long long)t.slices * rts - off;
    } else {
      const long long per = head_slices(s, p.G, p.window, kRows, kSlice);
      h = quotient(off, per);
      long long rem = off - per * h;
      t = unit_tile(p, s, 0, kRows, -1);
      while (rem >= t.slices) {
        rem -= t.slices;
        t = unit_tile(p, s, ++rt, kRows, -1);
      }
      sl0 = (int)rem;
      left = per * p.c.H - off;
    }
    const int sl1 = (int)min((long long)t.slices, sl0 + (run.g1 - g));
    const long long bh = (long long)b * p.c.H + h;
    const int32_t* table = p.bt.table + (long long)b * p.bt.max_pages;
    const int R = s.n * p.G;

    uint2 raw[NQ][D / 16];   // query rows, on their way
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int r = rt * kRows + 8 * n + i;
      load_query<D>(r < R ? p.q + (long long)(s.row0 + r / p.G) * p.q_stride +
                                (long long)(h * p.G + r % p.G) * D
                          : nullptr,
                    j, raw[n]);
    }
    // ------------------------- this warp's slices, the first on their way
    const int count = (sl1 - sl0 - warp + kWarps - 1) / kWarps;   // may be <= 0
    // descriptions k0 .. k0 + 31; the steps' loads set out before the first
    // copies (behind them they would queue) and are waited for after them
    float ks = 0.0f, vs = 0.0f;
    auto fill = [&](int k0) {
      __syncwarp();
      const int k = k0 + lane;
      if (k < count) {
        const int sl = sl0 + warp + kWarps * k;
        Meta d = {-1, 0, 0.0f, 0.0f};
        int lp = 0;
        bool read = false;
        if (n_pages >= 0) {
          const int per = p.c.P / kSlice, e = sl / per;
          if (e < n_pages) {
            lp = __ldg(p.sel + bh * p.max_sel + e);
            if (lp < 0 || (long long)lp * p.c.P >= s.len) {
              bad = true;
            } else {
              d.tok = lp * p.c.P + (sl - e * per) * kSlice;
              read = d.tok < t.hi && !(p.window > 0 && d.tok + kSlice <= (long long)t.pmin + 1 - p.window);
            }
          }
        } else {
          d.tok = t.lo + sl * kSlice;
          lp = d.tok / p.c.P;
          read = d.tok < t.hi;
        }
        if (read) {
          const int page = __ldg(table + lp);
          if (page < 0 || page >= p.c.num_pages) {
            bad = true;
          } else {
            d.page = page;
            ks = __ldg(p.c.ks + p.c.pair(page, h));
            vs = __ldg(p.c.vs + p.c.pair(page, h));
          }
        }
        meta[k & (kRing - 1)] = d;
      }
      __syncwarp();
    };
    auto fill_steps = [&](int k0) {
      const int k = k0 + lane;
      if (k < count) {
        meta[k & (kRing - 1)].ks = ks;
        meta[k & (kRing - 1)].vs = vs;
      }
      __syncwarp();
    };
    auto issue = [&](int k) {
      if (k >= count || dead) return;
      if ((k & 31) == 0) fill(k);
      if (lane == 0) {
        const Meta d = meta[k & (kRing - 1)];
        const uint32_t bar = bar0 + 8 * put, st = stage0 + put * S::kStageBytes;
        if (d.page < 0) {
          mbar_arrive(bar);
        } else {
          mbar_arrive_expect_tx(bar, S::kStageBytes);
          const int row = d.tok & (p.c.P - 1);
#pragma unroll
          for (int x = 0; x < D; x += 128) {
            tma_4d(st + x * kSlice, &p.tm_k, x, row, h, d.page, bar, pol);
            tma_4d(st + kSlice * D + x * kSlice, &p.tm_v, x, row, h, d.page, bar, pol);
          }
        }
      }
      if (++put == kStages) put = 0;
      if (k > 0 && (k & 31) == 0) fill_steps(k);
    };
#pragma unroll 1
    for (int k = 0; k < kStages; ++k) issue(k);
    fill_steps(0);
    // --------------------------------------------------- query fragments
    uint32_t q[NQ][D / 16][2];
    float f[NQ][2];   // of this lane's two columns: scale log2(e) / the row's power of two
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const float down = scale_query<D>(raw[n], q[n]);
      f[n][0] = __shfl_sync(0xffffffffu, down, 8 * j) * (p.scale * kLog2e);
      f[n][1] = __shfl_sync(0xffffffffu, down, 8 * j + 4) * (p.scale * kLog2e);
    }
    float m[NQ][2], l[NQ][2], o[NQ][D / 16][4];
    float vref = 0.0f;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.0f;
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][c][e] = 0.0f;
    }

#pragma unroll 1
    for (int k = 0; k < count; ++k) {
      if (!dead && !mbar_wait_bounded(bar0 + 8 * got, got_phase, kWait)) {
        dead = true;
        if (lane == 0) report(p.status, W4_ERR_TIMEOUT);
      }
      if (dead) break;
      const Meta d = meta[k & (kRing - 1)];
      if (d.page >= 0) {
        const uint32_t st = stage0 + got * S::kStageBytes;
        float x[NQ][4];
        key_scores<D, NQ>(st, i, j, q, x);
        bool over = fabsf(d.vs) > vref;   // a larger step, or a score past m
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[n][e] *= d.ks * f[n][e & 1];
        if (d.tok + kSlice - 1 > t.pmin || (p.window > 0 && d.tok <= t.pmax - p.window)) {
          // some row does not see some token
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int r = min(R - 1, rt * kRows + 8 * n + 2 * j + (e & 1));
              const int pos = s.len - s.n + r / p.G, tok = d.tok + i + 8 * (e >> 1);
              if (tok > pos || (p.window > 0 && tok <= pos - p.window)) x[n][e] = -INFINITY;
            }
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) over |= x[n][e] > m[n][e & 1] + kLag;
        if (__any_sync(0xffffffffu, over)) {
          const float vnew = fmaxf(vref, fabsf(d.vs));
          const float keep_v = vnew > 0.0f ? __fdividef(vref, vnew) : 0.0f;
          vref = vnew;
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float mx = fmaxf(x[n][c], x[n][c + 2]);
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
              mx = fmaxf(mx, m[n][c]);
              const float keep = mx == -INFINITY ? 1.0f : exp2_fast(m[n][c] - mx);
              m[n][c] = mx;
              l[n][c] *= keep;
#pragma unroll
              for (int a = 0; a < D / 16; ++a) {
                o[n][a][c] *= keep * keep_v;
                o[n][a][c + 2] *= keep * keep_v;
              }
            }
        }
        const float r = vref > 0.0f ? __fdividef(d.vs, vref) * kWeightScale : 0.0f;
        bool small = false;   // a weight below fp16's normal range
        uint32_t w[NQ][2];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float mm = m[n][c & 1];
            const float e = exp2_fast(x[n][c] - (mm == -INFINITY ? 0.0f : mm));
            l[n][c & 1] += e;
            x[n][c] = e * r;
            small |= fabsf(x[n][c]) < kHalfNormal && x[n][c] != 0.0f;
          }
          w[n][0] = transpose8(pack_half2(x[n][0], x[n][1]));
          w[n][1] = transpose8(pack_half2(x[n][2], x[n][3]));
        }
        if (!__any_sync(0xffffffffu, small)) {
          value_sums<false, D, NQ>(st + kSlice * D, i, j, w, o);
        } else {
          // weights of every size keep fp16's bits: those of one 29-bit
          // range of exponents at a time, brought into fp16's
          float up = 1.0f, back = 1.0f;
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (fabsf(x[n][c]) < kLeast) x[n][c] = 0.0f;
          do {
            small = false;
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
              float y[4];
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const float z = x[n][c] * up;
                y[c] = z;
                if (fabsf(z) < kHalfNormal) {
                  y[c] = 0.0f;
                  small |= x[n][c] != 0.0f;
                } else {
                  x[n][c] = 0.0f;
                }
              }
              w[n][0] = transpose8(pack_half2(y[0], y[1]));
              w[n][1] = transpose8(pack_half2(y[2], y[3]));
            }
            value_sums<true, D, NQ>(st + kSlice * D, i, j, w, o, back);
            up *= kLevel;
            back *= 1.0f / kLevel;
          } while (__any_sync(0xffffffffu, small));
        }
      }
      __syncwarp();
      if (++got == kStages) {
        got = 0;
        got_phase ^= 1u;
      }
      issue(k + kStages);
    }
    if (bad || dead) refused[odd] = 1;

    // ------------------------------------------ join the warps (and CTAs)
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], 4);
        l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], 8);
        l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], 16);
        if (i == 0) stats[warp * kRows + 8 * n + 2 * j + c] = make_float2(m[n][c], l[n][c]);
      }
    __syncthreads();   // every stage has been read
    const float back = vref * (1.0f / kWeightScale);
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        float* to = join + (warp * kRows + 8 * n + 2 * j) * kPitch + value_channel<D>(i, c);
        *reinterpret_cast<float2*>(to) = make_float2(o[n][c][0] * back, o[n][c][2] * back);
        *reinterpret_cast<float2*>(to + kPitch) = make_float2(o[n][c][1] * back, o[n][c][3] * back);
      }
    __syncthreads();
    const bool no = refused[odd] != 0;
    if (tid == 0) refused[odd ^ 1] = 0;   // read by all before the last barrier, next set after it
    const bool whole = sl0 == 0 && sl1 == t.slices;
    if (no && tid == 0 && !dead) report(p.status, W4_ERR_INDEX);
    const int slot = 2 * blockIdx.x + (sl0 == 0 ? 1 : 0);
    for (int x = tid; x < kRows * (D / 4); x += kThreads) {
      const int r = x / (D / 4), c4 = x % (D / 4);
      const int row = rt * kRows + r;
      float M = -INFINITY, L = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, stats[w * kRows + r].x);
      float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 st = stats[w * kRows + r];
        const float k = st.x == -INFINITY ? (st.y == 0.0f ? 0.0f : 1.0f) : exp2_fast(st.x - M);
        const float4 v = *reinterpret_cast<const float4*>(join + (w * kRows + r) * kPitch + 4 * c4);
        L += k * st.y;
        a.x += k * v.x;
        a.y += k * v.y;
        a.z += k * v.z;
        a.w += k * v.w;
      }
      if (!whole) {
        *reinterpret_cast<float4*>(p.parts + ((long long)slot * kRows + r) * D + 4 * c4) = a;
        if (c4 == 0)
          *reinterpret_cast<float2*>(p.part_stats + ((long long)slot * kRows + r) * 2) =
              make_float2(M, no ? -1.0f : L);
      } else if (row < R && !no) {
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
        const __nv_bfloat162 u = __floats2bfloat162_rn(a.x * inv, a.y * inv);
        const __nv_bfloat162 v = __floats2bfloat162_rn(a.z * inv, a.w * inv);
        const long long at = (long long)(s.row0 + row / p.G) * p.Hq + h * p.G + row % p.G;
        *reinterpret_cast<uint2*>(p.out + at * D + 4 * c4) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&u), *reinterpret_cast<const uint32_t*>(&v));
        if (c4 == 0 && p.lse != nullptr)
          p.lse[at] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
      }
    }
    if (!whole) {
      // CTAs that hold a part of this unit: those of its first to its last slice
      const long long u0 = g - sl0, u1 = u0 + t.slices - 1;
      const int c0 = run.holder(u0), c1 = run.holder(u1);
      // a CTA has the first part of one cut unit at most: its last
      int32_t* arrived = p.arrived + c0;
      __syncthreads();
      if (tid == 0) {
        const int was = atomic_add_acq_rel_gpu(arrived, 1);
        *flag = was == c1 - c0;
        if (was == c1 - c0) *arrived = 0;
      }
      __syncthreads();
      if (*flag) {
        for (int x = tid; x < kRows * (D / 4); x += kThreads) {
          const int r = x / (D / 4), c4 = x % (D / 4);
          const int row = rt * kRows + r;
          if (row >= R) continue;
          float M = -INFINITY, L = 0.0f;
          bool none = false;
          // the first CTA's part began the unit, the others' run began inside it
#pragma unroll 8
          for (int c = c0; c <= c1; ++c) {
            const int sl = c == c0 ? 2 * c + 1 : 2 * c;
            const float2 st = __ldcg(reinterpret_cast<const float2*>(p.part_stats) +
                                     (long long)sl * kRows + r);
            M = fmaxf(M, st.x);
            none |= st.y < 0.0f;
          }
          if (none) continue;
          float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
          for (int c = c0; c <= c1; ++c) {
            const int sl = c == c0 ? 2 * c + 1 : 2 * c;
            const float2 st = __ldcg(reinterpret_cast<const float2*>(p.part_stats) +
                                     (long long)sl * kRows + r);
            const float4 v = __ldcg(reinterpret_cast<const float4*>(
                p.parts + ((long long)sl * kRows + r) * D + 4 * c4));
            const float k = st.x == -INFINITY ? (st.y == 0.0f ? 0.0f : 1.0f) : exp2_fast(st.x - M);
            L += k * st.y;
            a.x += k * v.x;
            a.y += k * v.y;
            a.z += k * v.z;
            a.w += k * v.w;
          }
          const float inv = L == 0.0f ? 0.0f : 1.0f / L;
          const __nv_bfloat162 u = __floats2bfloat162_rn(a.x * inv, a.y * inv);
          const __nv_bfloat162 v = __floats2bfloat162_rn(a.z * inv, a.w * inv);
          const long long at = (long long)(s.row0 + row / p.G) * p.Hq + h * p.G + row % p.G;
          *reinterpret_cast<uint2*>(p.out + at * D + 4 * c4) = make_uint2(
              *reinterpret_cast<const uint32_t*>(&u), *reinterpret_cast<const uint32_t*>(&v));
          if (c4 == 0 && p.lse != nullptr)
            p.lse[at] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
        }
      }
    }
    fence_proxy_async_smem();   // the joined rows, before copies into the same bytes
    __syncthreads();
    odd ^= 1;
    // --------------------------------------------------------- next unit
    const long long step = sl1 - sl0;
    g += step;
    off += step;
    if (step == left && g < run.g1) {
      off = 0;
      int none = 0;
      do ++entry;
      while (entry_slices(p, entry, kRows, &none) == 0);
    }
  }
  if (dead) {   // copies still in flight land before the CTA leaves
    for (int s = 0; s < kStages; ++s) mbar_wait_bounded(bar0 + 8 * s, got_phase, kWait >> 4);
  }
}

// ================================================================= host side
size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

struct Plan {
  int nq, ctas;
  size_t parts, stats, bytes;
};

Plan plan_token(const Cache& c, const Batch& b, int G, int sms) {
  Plan pl;
  const long long rows = (long long)b.max_new * G;
  // Two column tiles read the keys once for 16 rows, but from 128 channels on
  // their accumulators do not fit the registers of two CTAs an SM: 16 rows on
  // 16 x 16k keys of 128 channels 74 us against 64 with one, of 256 channels
  // 124 against 117; of 64 channels 39 against 47.
  pl.nq = c.D == 64 && rows > 8 ? 2 : 1;
  pl.ctas = std::min(sms * (c.D == 256 ? 1 : 2), kHeadCounters);
  pl.parts = up256((size_t)2 * pl.ctas * 8 * pl.nq * c.D * 4);
  pl.stats = up256((size_t)2 * pl.ctas * 8 * pl.nq * 8);
  pl.bytes = kHeadBytes + pl.parts + pl.stats;
  return pl;
}

template <int D, int NQ>
w4_status launch_token(const AttnParams& p, int ctas, w4_stream_t stream, int dev) {
  static std::mutex mu;
  static bool done[64] = {};
  if (dev < 0 || dev >= 64) return W4_ERR_DEVICE;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      const cudaError_t e = cudaFuncSetAttribute(attn_token_kernel<D, NQ>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 Shape<D, NQ>::kSmem);
      if (e != cudaSuccess) {
        note_cuda_error(e);
        (void)cudaGetLastError();
        return W4_ERR_LAUNCH;
      }
      done[dev] = true;
    }
  }
  return launch(attn_token_kernel<D, NQ>, dim3((unsigned)ctas), kThreads, Shape<D, NQ>::kSmem,
                stream, p);
}

}  // namespace

bool tensor_map(CUtensorMap* m, uint8_t* codes, const Cache& c, int rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tc::encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)c.D, (cuuint64_t)c.P, (cuuint64_t)c.H,
                              (cuuint64_t)c.num_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)c.D, (cuuint64_t)c.head_stride,
                                 (cuuint64_t)c.page_stride};
  const cuuint32_t box[4] = {(cuuint32_t)std::min(c.D, 128), (cuuint32_t)rows, 1, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, codes, dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             c.D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace kv8
}  // namespace w4

using namespace w4;

extern "C" size_t w4_kv8_attn_workspace_bytes(const w4_kv8_cache* cache, const w4_kv8_batch* batch,
                                              int q_heads, int max_sel) {
  kv8::Cache c;
  kv8::Batch b;
  if (kv8::view(cache, batch, &c, &b) != W4_OK || q_heads < 1 || q_heads % c.H != 0 ||
      q_heads / c.H > W4_KV8_MAX_GROUP || max_sel < 0)
    return 0;
  DeviceInfo di;
  planning_device(&di);
  if (max_sel == 0 && (long long)b.max_new * (q_heads / c.H) >= kv8::chunk_rows(c.D))
    return kv8::chunk_workspace_bytes(c, b, q_heads / c.H, di.sms);
  return kv8::plan_token(c, b, q_heads / c.H, di.sms).bytes;
}

extern "C" w4_status w4_kv8_attn(void* out, float* lse, const void* q, size_t q_row_stride,
                                 int q_heads, const w4_kv8_cache* cache,
                                 const w4_kv8_batch* batch, float scale, int window,
                                 const int32_t* sel, const int32_t* n_sel, int max_sel,
                                 void* workspace, size_t workspace_bytes, int32_t* status_dev,
                                 unsigned flags, w4_stream_t stream) {
  kv8::AttnParams p = {};
  w4_status st = kv8::view(cache, batch, &p.c, &p.bt);
  if (st != W4_OK) return st;
  if (out == nullptr || (flags & ~W4_FLAG_PDL) != 0 || window < 0 ||
      (sel == nullptr) != (n_sel == nullptr) || (sel != nullptr && max_sel < 1))
    return W4_ERR_ARG;
  if ((st = kv8::check_q(q, q_row_stride, q_heads, p.c)) != W4_OK) return st;
  if (sel != nullptr && (p.bt.max_new != 1 || max_sel > (1 << 24))) return W4_ERR_SHAPE;
  if (kv8::misaligned(out, 16) || kv8::misaligned(lse, 4) || kv8::misaligned(sel, 4) ||
      kv8::misaligned(n_sel, 4) || kv8::misaligned(workspace, 16))
    return W4_ERR_ALIGN;
  int dev = -1;
  DeviceInfo di;
  const bool have = current_device(&dev, &di);
  if (!have) planning_device(&di);
  if (sel == nullptr && (long long)p.bt.max_new * (q_heads / p.c.H) >= kv8::chunk_rows(p.c.D)) {
    if (workspace == nullptr ||
        workspace_bytes < kv8::chunk_workspace_bytes(p.c, p.bt, q_heads / p.c.H, di.sms))
      return W4_ERR_WORKSPACE;
    if (!have) return W4_ERR_DEVICE;
    const kv8::ChunkArgs a = {static_cast<__nv_bfloat16*>(out), lse,
                              static_cast<const __nv_bfloat16*>(q), (long long)q_row_stride,
                              q_heads, scale, window, status_dev};
    return kv8::chunk_attn(p.c, p.bt, a, workspace, di.sms, dev, stream);
  }
  const kv8::Plan pl = kv8::plan_token(p.c, p.bt, q_heads / p.c.H, di.sms);
  if (workspace == nullptr || workspace_bytes < pl.bytes) return W4_ERR_WORKSPACE;
  if (!have) return W4_ERR_DEVICE;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride = (long long)q_row_stride;
  p.Hq = q_heads;
  p.G = q_heads / p.c.H;
  p.scale = scale;
  p.window = window;
  p.sel = sel;
  p.n_sel = n_sel;
  p.max_sel = max_sel;
  p.status = status_dev;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.arrived = reinterpret_cast<int32_t*>(ws);
  p.parts = reinterpret_cast<float*>(ws + kv8::kHeadBytes);
  p.part_stats = reinterpret_cast<float*>(ws + kv8::kHeadBytes + pl.parts);
  if (!kv8::tensor_map(&p.tm_k, p.c.kc, p.c, kv8::kSlice) ||
      !kv8::tensor_map(&p.tm_v, p.c.vc, p.c, kv8::kSlice)) {
    note_cuda_error(cudaErrorInvalidValue);
    return W4_ERR_LAUNCH;
  }
  switch (p.c.D * 4 + pl.nq) {
    case 64 * 4 + 1: return kv8::launch_token<64, 1>(p, pl.ctas, stream, dev);
    case 64 * 4 + 2: return kv8::launch_token<64, 2>(p, pl.ctas, stream, dev);
    case 128 * 4 + 1: return kv8::launch_token<128, 1>(p, pl.ctas, stream, dev);
    default: return kv8::launch_token<256, 1>(p, pl.ctas, stream, dev);
  }
}
