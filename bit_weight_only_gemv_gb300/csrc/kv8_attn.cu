// Attention over the 8-bit cache (w4_kv8_attn) and the accumulation of
// attention weights (w4_kv8_weigh).
#include "kv8.cuh"

namespace w4 {
namespace kv8 {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxD = 256;

struct AttnParams {
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
  int32_t* status;
};

// The sequence of packed row `row` (-1: none holds it).
__device__ int sequence_of(const Batch& bt, int row) {
  if (bt.offsets == nullptr) return row < bt.B ? row : -1;
  int lo = 0, hi = bt.B;   // the last b with offsets[b] <= row
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (__ldg(bt.offsets + mid) <= row) lo = mid;
    else hi = mid;
  }
  return lo;
}

// One CTA per (row, query head): its warps share out the keys, each with its
// own running maximum and sum, joined at the end.
__global__ void __launch_bounds__(32 * kWarps) attn_simple_kernel(const AttnParams p) {
  __shared__ float part[kWarps][kMaxD + 2];
  pdl_launch_dependents();
  pdl_wait();
  const int row = blockIdx.x, i = blockIdx.y, h = i / p.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int P = p.c.P, D = p.c.D;
  const int b = sequence_of(p.bt, row);
  if (b < 0) return;
  const Seq s = sequence(p.bt, P, b);
  if (!s.ok) {
    if (threadIdx.x == 0) report(p.status, W4_ERR_INDEX);
    return;
  }
  if (row < s.row0 || row >= s.row0 + s.n) return;
  const int pos = s.len - s.n + row - s.row0;
  const __nv_bfloat16* q = p.q + row * p.q_stride + (long long)i * D;
  const int per = D / 32;
  float qv[kMaxD / 32], acc[kMaxD / 32];
  for (int d = 0; d < per; ++d) {
    qv[d] = __bfloat162float(q[lane + 32 * d]);
    acc[d] = 0.0f;
  }
  const int32_t* table = p.bt.table + (long long)b * p.bt.max_pages;
  const long long bh = (long long)b * p.c.H + h;
  const int32_t* sel = p.sel == nullptr ? nullptr : p.sel + bh * p.max_sel;
  const int from = p.window > 0 ? max(0, pos + 1 - p.window) : 0;
  const int np = (s.len + P - 1) / P;
  int entries = np;
  bool bad = false;
  if (sel != nullptr) {
    entries = __ldg(p.n_sel + bh);
    if (entries < 0 || entries > p.max_sel) bad = true, entries = 0;
  }
  float m = -INFINITY, l = 0.0f;
  for (int e = sel == nullptr ? from / P : 0; e < entries; ++e) {
    const int lp = sel == nullptr ? e : __ldg(sel + e);
    if (lp < 0 || lp >= np) {
      bad = true;
      break;
    }
    if (lp * P > pos) break;
    const int page = __ldg(table + lp);
    if (page < 0 || page >= p.c.num_pages) {
      bad = true;
      break;
    }
    const float ks = p.c.ks[p.c.pair(page, h)], vs = p.c.vs[p.c.pair(page, h)];
    const uint8_t* kc = p.c.kc + p.c.block(page, h);
    const uint8_t* vc = p.c.vc + p.c.block(page, h);
    for (int t = warp; t < P; t += kWarps) {
      const int kp = lp * P + t;
      if (kp > pos || kp < from) continue;
      float dot = 0.0f;
      for (int d = 0; d < per; ++d)
        dot += qv[d] * (float)((int)kc[(long long)t * D + lane + 32 * d] - 128);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      const float x = dot * ks * p.scale;
      const float mn = fmaxf(m, x);
      const float keep = mn == m ? 1.0f : expf(m - mn), w = expf(x - mn);
      m = mn;
      l = l * keep + w;
      for (int d = 0; d < per; ++d)
        acc[d] = acc[d] * keep + w * vs * (float)((int)vc[(long long)t * D + lane + 32 * d] - 128);
    }
  }
  if (bad) {   // the same in every warp
    if (threadIdx.x == 0) report(p.status, W4_ERR_INDEX);
    return;
  }
  for (int d = 0; d < per; ++d) part[warp][lane + 32 * d] = acc[d];
  if (lane == 0) {
    part[warp][kMaxD] = m;
    part[warp][kMaxD + 1] = l;
  }
  __syncthreads();
  float mm = -INFINITY, ll = 0.0f;
  for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, part[w][kMaxD]);
  float f[kWarps];
  for (int w = 0; w < kWarps; ++w) {
    f[w] = mm == -INFINITY ? 0.0f : expf(part[w][kMaxD] - mm);
    ll += f[w] * part[w][kMaxD + 1];
  }
  for (int d = threadIdx.x; d < D; d += 32 * kWarps) {
    float a = 0.0f;
    for (int w = 0; w < kWarps; ++w) a += f[w] * part[w][d];
    p.out[((long long)row * p.Hq + i) * D + d] = __float2bfloat16_rn(ll == 0.0f ? 0.0f : a / ll);
  }
  if (threadIdx.x == 0 && p.lse != nullptr)
    p.lse[(long long)row * p.Hq + i] = ll == 0.0f ? -INFINITY : mm + logf(ll);
}

struct WeighParams {
  Cache c;
  Batch bt;
  const __nv_bfloat16* q;
  long long q_stride;
  const float* lse;
  int Hq, G;
  float scale;
  int window;
  int32_t* status;
};

// One CTA per (page, head, sequence), one warp per token in turn.
__global__ void __launch_bounds__(32 * kWarps) weigh_simple_kernel(const WeighParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lp = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int P = p.c.P, D = p.c.D, per = D / 32;
  const Seq s = sequence(p.bt, P, b);
  if (!s.ok) {
    if (threadIdx.x == 0 && lp == 0) report(p.status, W4_ERR_INDEX);
    return;
  }
  if (lp * P >= s.len) return;
  const int page = __ldg(p.bt.table + (long long)b * p.bt.max_pages + lp);
  if (page < 0 || page >= p.c.num_pages) {
    if (threadIdx.x == 0) report(p.status, W4_ERR_INDEX);
    return;
  }
  const float ks = p.c.ks[p.c.pair(page, h)];
  const uint8_t* kc = p.c.kc + p.c.block(page, h);
  for (int t = warp; t < P && lp * P + t < s.len; t += kWarps) {
    const int kp = lp * P + t;
    float sum = 0.0f;
    for (int r = 0; r < s.n; ++r) {
      const int pos = s.len - s.n + r;
      if (kp > pos || (p.window > 0 && kp <= pos - p.window)) continue;
      for (int g = 0; g < p.G; ++g) {
        const __nv_bfloat16* q = p.q + (s.row0 + r) * p.q_stride + (long long)(h * p.G + g) * D;
        float dot = 0.0f;
        for (int d = 0; d < per; ++d)
          dot += __bfloat162float(q[lane + 32 * d]) *
                 (float)((int)kc[(long long)t * D + lane + 32 * d] - 128);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        const float l = p.lse[(long long)(s.row0 + r) * p.Hq + h * p.G + g];
        if (l != -INFINITY) sum += expf(dot * ks * p.scale - l);
      }
    }
    if (lane == 0) p.c.weight[p.c.pair(page, h) * P + t] += sum;
  }
}

}  // namespace
}  // namespace kv8
}  // namespace w4

using namespace w4;

extern "C" size_t w4_kv8_attn_workspace_bytes(const w4_kv8_cache* cache, const w4_kv8_batch* batch,
                                              int q_heads, int max_sel) {
  (void)cache, (void)batch, (void)q_heads, (void)max_sel;
  return 0;
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
  if (workspace_bytes < w4_kv8_attn_workspace_bytes(cache, batch, q_heads, max_sel))
    return W4_ERR_WORKSPACE;
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
  return kv8::launch(kv8::attn_simple_kernel, dim3((unsigned)p.bt.rows, (unsigned)q_heads),
                     32 * kv8::kWarps, 0, (flags & W4_FLAG_PDL) != 0, stream, p);
}

extern "C" w4_status w4_kv8_weigh(const void* q, size_t q_row_stride, int q_heads,
                                  const float* lse, const w4_kv8_cache* cache,
                                  const w4_kv8_batch* batch, float scale, int window,
                                  int32_t* status_dev, unsigned flags, w4_stream_t stream) {
  kv8::WeighParams p = {};
  w4_status st = kv8::view(cache, batch, &p.c, &p.bt);
  if (st != W4_OK) return st;
  if (lse == nullptr || p.c.weight == nullptr || (flags & ~W4_FLAG_PDL) != 0 || window < 0)
    return W4_ERR_ARG;
  if ((st = kv8::check_q(q, q_row_stride, q_heads, p.c)) != W4_OK) return st;
  if (kv8::misaligned(lse, 4)) return W4_ERR_ALIGN;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride = (long long)q_row_stride;
  p.lse = lse;
  p.Hq = q_heads;
  p.G = q_heads / p.c.H;
  p.scale = scale;
  p.window = window;
  p.status = status_dev;
  const int pages = (p.bt.max_len + p.c.P - 1) / p.c.P;
  if (pages == 0) return W4_OK;
  return kv8::launch(kv8::weigh_simple_kernel,
                     dim3((unsigned)pages, (unsigned)p.c.H, (unsigned)p.bt.B), 32 * kv8::kWarps, 0,
                     (flags & W4_FLAG_PDL) != 0, stream, p);
}
