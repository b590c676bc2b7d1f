// New tokens' keys and values into the 8-bit cache (w4_kv8_append), and the
// host's checks that every kv8 call shares.
//
// One CTA per (touched page, head, keys or values).  With m the largest new
// |value| of the block and s0 the step of the tokens already in it, the step
// becomes s = max(s0, least power of two >= m / 127): a power of two, so that
// the division value / s, the ratio s0 / s and code * step are exact and the
// only rounding is the one to a whole code.  One pass finds m (and refuses
// values that are not finite), a second one, from registers or L1, writes the
// codes; older codes are touched only when the step grows.  Latency bounds
// it: the chain is lengths, then rows and page together, then the old step.
// One token for each of 8 sequences: 3.4 us, of which the host's call is as
// much; 16 chunks of up to 256 tokens, 8 heads of 128 channels: 8.4 us, 1.5 TB/s.
#include "kv8.cuh"

namespace w4 {
namespace kv8 {
namespace {



constexpr int kHeld = 4;   // input vectors a thread keeps between its two passes

// Four codes times a ratio of steps.
__device__ __forceinline__ uint32_t rescale4(uint32_t x, float ratio) {
  uint32_t y = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    y |= to_code((float)((int)((x >> (8 * j)) & 0xFF) - 128) * ratio) << (8 * j);
  return y;
}

__device__ __forceinline__ void unpack8(const uint4& w, float f[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_bits_to_float(u[i] & 0xFFFFu);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

__global__ void __launch_bounds__(256) append_kernel(Cache c, Batch bt,
                                                     const __nv_bfloat16* __restrict__ k,
                                                     const __nv_bfloat16* __restrict__ v,
                                                     long long row_stride, int32_t* status) {
  __shared__ uint32_t red[8];
  __shared__ uint32_t lo_sm[256 / 2][4], hi_sm[256 / 2][4];   // [thread][2 words] halves
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.y, b = blockIdx.z >> 1;
  const bool is_v = blockIdx.z & 1;
  const Seq s = sequence(bt, c.P, b);
  if (!s.ok || s.len > (long long)bt.max_pages * c.P) {
    if (threadIdx.x == 0 && blockIdx.x == 0) report(status, W4_ERR_INDEX);
    return;
  }
  const int first = max(0, s.len - s.n);              // new tokens at negative positions: nowhere
  const int lp = first / c.P + (int)blockIdx.x;
  const int p0 = lp * c.P;
  const int lo = max(first, p0), hi = min(s.len, p0 + c.P);
  if (lo >= hi) return;
  const int tid = threadIdx.x, nth = blockDim.x;
  // rows lo .. hi - 1 of this head; 16-byte vectors of 8 values, the first
  // kHeld of a thread kept in registers, on their way before anything waits
  const int vecs = c.D / 8, col = tid % vecs, r0 = tid / vecs, rstep = nth / vecs;
  const __nv_bfloat16* src = (is_v ? v : k) +
                             (long long)(s.row0 + lo - (s.len - s.n)) * row_stride +
                             (long long)h * c.D + col * 8;
  const int rows = hi - lo;
  uint4 held[kHeld];
#pragma unroll
  for (int z = 0; z < kHeld; ++z)
    if (r0 + z * rstep < rows)
      held[z] = __ldg(reinterpret_cast<const uint4*>(src + (r0 + z * rstep) * row_stride));
  const int page = __ldg(bt.table + (long long)b * bt.max_pages + lp);
  if (page < 0 || page >= c.num_pages) {
    if (tid == 0) report(status, W4_ERR_INDEX);
    return;
  }
  const bool has_old = lo > p0;
  float* steps = is_v ? c.vs : c.ks;
  const float s0 = has_old ? steps[c.pair(page, h)] : 0.0f;
  // largest |value|; bf16 bits without the sign are in order, and those of
  // infinities and NaN come last
  uint32_t top = 0;
  auto look = [&](const uint4& w) {
    const uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
    top = max(top, max(m & 0xFFFFu, m >> 16));
  };
#pragma unroll
  for (int z = 0; z < kHeld; ++z)
    if (r0 + z * rstep < rows) look(held[z]);
  for (int r = r0 + kHeld * rstep; r < rows; r += rstep)
    look(__ldg(reinterpret_cast<const uint4*>(src + r * row_stride)));
  top = __reduce_max_sync(0xffffffffu, top);
  if ((tid & 31) == 0) red[tid >> 5] = top;
  __syncthreads();
  for (int i = 0; i < nth / 32; ++i) top = max(top, red[i]);
  if (top >= 0x7F80u) {
    if (tid == 0) report(status, W4_ERR_VALUE);
    return;
  }
  const float step = fmaxf(s0, pow2_step(__uint_as_float(top << 16)));
  // a power of two (as the library's own steps are) divides by a product
  const bool exact = (__float_as_uint(step) & 0x7FFFFFu) == 0;
  const float inv = __fdiv_rn(1.0f, step);
  uint8_t* blk = (is_v ? c.vc : c.kc) + c.block(page, h);
  uint32_t mn[2] = {~0u, ~0u}, mx[2] = {0, 0};   // by channel, four to a word
  auto store = [&](const uint4& w, int r) {
    float f[8];
    unpack8(w, f);
    uint32_t out[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      out[i >> 2] |= to_code(exact ? f[i] * inv : __fdiv_rn(f[i], step)) << (8 * (i & 3));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mn[i] = __vminu4(mn[i], out[i]);
      mx[i] = __vmaxu4(mx[i], out[i]);
    }
    *reinterpret_cast<uint2*>(blk + (long long)(lo - p0 + r) * c.D + col * 8) =
        make_uint2(out[0], out[1]);
  };
#pragma unroll
  for (int z = 0; z < kHeld; ++z)
    if (r0 + z * rstep < rows) store(held[z], r0 + z * rstep);
  for (int r = r0 + kHeld * rstep; r < rows; r += rstep)
    store(__ldg(reinterpret_cast<const uint4*>(src + r * row_stride)), r);
  const bool grow = has_old && step != s0;
  const float ratio = grow ? __fdiv_rn(s0, step) : 1.0f;
  if (grow) {
    const int words = (lo - p0) * c.D / 4;
    uint32_t* w = reinterpret_cast<uint32_t*>(blk);
    for (int i = tid; i < words; i += nth) w[i] = rescale4(w[i], ratio);
  }
  if (tid == 0) steps[c.pair(page, h)] = step;
  if (is_v) {
    if (c.weight != nullptr)
      for (int i = tid; i < rows; i += nth) c.weight[c.pair(page, h) * c.P + lo - p0 + i] = 0.0f;
    return;
  }
  if (c.ranges == nullptr) return;
  // lowest and highest code of each channel: the threads of one column in
  // turn, then what the block held before
  uint32_t* lp_sm = &lo_sm[0][0];
  uint32_t* hp_sm = &hi_sm[0][0];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    lp_sm[2 * tid + i] = mn[i];
    hp_sm[2 * tid + i] = mx[i];
  }
  __syncthreads();
  if (r0 != 0) return;
  for (int o = tid + vecs; o < nth; o += vecs)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mn[i] = __vminu4(mn[i], lp_sm[2 * o + i]);
      mx[i] = __vmaxu4(mx[i], hp_sm[2 * o + i]);
    }
  uint8_t* rg = c.ranges + c.pair(page, h) * 2 * c.D + col * 8;
  uint2* rlo = reinterpret_cast<uint2*>(rg);
  uint2* rhi = reinterpret_cast<uint2*>(rg + c.D);
  const uint2 olo = has_old ? *rlo : make_uint2(~0u, ~0u), ohi = has_old ? *rhi : make_uint2(0, 0);
  uint32_t l[2] = {olo.x, olo.y}, u[2] = {ohi.x, ohi.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (grow) {   // rescaling is monotone: the range of the rescaled codes
      l[i] = rescale4(l[i], ratio);
      u[i] = rescale4(u[i], ratio);
    }
    l[i] = __vminu4(l[i], mn[i]);
    u[i] = __vmaxu4(u[i], mx[i]);
  }
  *rlo = make_uint2(l[0], l[1]);
  *rhi = make_uint2(u[0], u[1]);
}

}  // namespace

w4_status view(const w4_kv8_cache* c, const w4_kv8_batch* b, Cache* cv, Batch* bv) {
  if (c == nullptr || b == nullptr || c->kc == nullptr || c->vc == nullptr || c->ks == nullptr ||
      c->vs == nullptr || b->table == nullptr || b->lens == nullptr)
    return W4_ERR_ARG;
  if (c->num_pages < 1 || c->kv_heads < 1 || b->batch < 1 || b->max_pages < 1 || b->rows < 1 ||
      b->max_new < 1 || b->max_len < 0)
    return W4_ERR_ARG;
  const int P = c->page_tokens, D = c->head_dim;
  if ((P != 16 && P != 32 && P != 64 && P != 128) || (D != 64 && D != 128 && D != 256) ||
      c->kv_heads > 4096 || b->batch > W4_KV8_MAX_BATCH || b->rows > (1 << 20) ||
      (long long)b->max_len > (long long)b->max_pages * P || b->max_len > (1 << 30))
    return W4_ERR_SHAPE;
  if (b->offsets == nullptr && (b->rows != b->batch || b->max_new != 1)) return W4_ERR_SHAPE;
  if (misaligned(c->kc, 16) || misaligned(c->vc, 16) || misaligned(c->ranges, 16) ||
      c->page_stride % 16 != 0 || c->head_stride % 16 != 0 || misaligned(c->ks, 4) ||
      misaligned(c->vs, 4) || misaligned(c->weight, 4) || misaligned(b->table, 4) ||
      misaligned(b->lens, 4) || misaligned(b->offsets, 4))
    return W4_ERR_ALIGN;
  if (c->head_stride < (size_t)P * D || c->page_stride < (size_t)P * D ||
      c->head_stride >= (1ull << 40) || c->page_stride >= (1ull << 40))
    return W4_ERR_ARG;
  cv->kc = static_cast<uint8_t*>(c->kc);
  cv->vc = static_cast<uint8_t*>(c->vc);
  cv->ks = c->ks;
  cv->vs = c->vs;
  cv->ranges = static_cast<uint8_t*>(c->ranges);
  cv->weight = c->weight;
  cv->num_pages = c->num_pages;
  cv->H = c->kv_heads;
  cv->P = P;
  cv->D = D;
  cv->page_stride = (long long)c->page_stride;
  cv->head_stride = (long long)c->head_stride;
  bv->table = b->table;
  bv->lens = b->lens;
  bv->offsets = b->offsets;
  bv->B = b->batch;
  bv->max_pages = b->max_pages;
  bv->rows = b->rows;
  bv->max_new = b->max_new;
  bv->max_len = b->max_len;
  return W4_OK;
}

w4_status check_q(const void* q, size_t q_row_stride, int q_heads, const Cache& c) {
  if (q == nullptr || q_heads < 1) return W4_ERR_ARG;
  if (q_heads % c.H != 0 || q_heads / c.H > W4_KV8_MAX_GROUP) return W4_ERR_SHAPE;
  if (misaligned(q, 16) || q_row_stride % 8 != 0) return W4_ERR_ALIGN;
  if (q_row_stride < (size_t)q_heads * c.D || q_row_stride >= (1ull << 32)) return W4_ERR_ARG;
  return W4_OK;
}

}  // namespace kv8
}  // namespace w4

using namespace w4;

extern "C" w4_status w4_kv8_append(const w4_kv8_cache* cache, const w4_kv8_batch* batch,
                                   const void* k, const void* v, size_t row_stride,
                                   int32_t* status_dev, unsigned flags, w4_stream_t stream) {
  kv8::Cache c;
  kv8::Batch b;
  const w4_status st = kv8::view(cache, batch, &c, &b);
  if (st != W4_OK) return st;
  if (k == nullptr || v == nullptr || (flags & ~W4_FLAG_PDL) != 0) return W4_ERR_ARG;
  if (kv8::misaligned(k, 16) || kv8::misaligned(v, 16) || row_stride % 8 != 0) return W4_ERR_ALIGN;
  if (row_stride < (size_t)c.H * c.D || row_stride >= (1ull << 32)) return W4_ERR_ARG;
  // pages that max_new tokens can touch, wherever they start
  const long long nt = (b.max_new + c.P - 2) / c.P + 1;
  const int threads = b.max_new == 1 ? 64 : 256;
  return kv8::launch(kv8::append_kernel, dim3((unsigned)nt, (unsigned)c.H, (unsigned)(2 * b.B)),
                     threads, 0, stream, c, b,
                     static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v),
                     (long long)row_stride, status_dev);
}
