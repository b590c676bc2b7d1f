// Penalties, biases and masks on the output product's logits (w4_logits_adjust).
//
// One CTA per (tile of the vocabulary, row), a 32-bit word for each token of
// the tile in shared memory:
//   bits 0..18   occurrences after the prompt
//   bit  19      occurs in the prompt
//   bits 20..31  1 + index of its last bias
// The CTA reads the row's bias list and history once, keeps what falls into its
// tile, and then walks the tile: a token that no rule names and the mask
// allows costs no global access, one that the mask forbids a store.  Every CTA
// of a row sees the whole lists, so all of them find the same errors.
#include "kv8.cuh"

namespace w4 {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kCount = (1u << 19) - 1, kPrompt = 1u << 19;
constexpr int kBiasShift = 20;

struct LogitParams {
  void* logits;
  long long stride;
  int V, tile;
  w4_logit_rules r;
  int32_t* status;
};

__device__ __forceinline__ float load(const float* p) { return *p; }
__device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store(float* p, float v) { *p = v; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <typename T>
__global__ void __launch_bounds__(kThreads) adjust_kernel(LogitParams p) {
  extern __shared__ uint32_t word[];
  pdl_launch_dependents();
  const int tid = threadIdx.x, row = blockIdx.y;
  const int v0 = blockIdx.x * p.tile, n = min(p.tile, p.V - v0);
  for (int i = tid; i < n; i += kThreads) word[i] = 0;
  pdl_wait();
  const w4_logit_rules& r = p.r;
  const int len = r.tokens != nullptr ? __ldg(r.lens + row) : 0;
  const int prompt = r.prompt != nullptr ? __ldg(r.prompt + row) : 0;
  const int nb = r.bias_ids == nullptr ? 0 : r.n_bias != nullptr ? __ldg(r.n_bias + row) : r.max_bias;
  const float rep = r.repetition != nullptr ? __ldg(r.repetition + row) : 1.0f;
  const float pres = r.presence != nullptr ? __ldg(r.presence + row) : 0.0f;
  const float freq = r.frequency != nullptr ? __ldg(r.frequency + row) : 0.0f;
  const int mrow = r.mask == nullptr ? -1 : r.mask_rows != nullptr ? __ldg(r.mask_rows + row) : row;
  int bad = 0;
  if (len < 0 || len > r.max_tokens || prompt < 0 || prompt > len || nb < 0 || nb > r.max_bias ||
      mrow < -1 || (mrow >= r.num_masks && r.mask != nullptr))
    bad = W4_ERR_INDEX;
  else if (!(rep > 0.0f) || isinf(rep) || !isfinite(pres) || !isfinite(freq))
    bad = W4_ERR_VALUE;
  if (bad != 0) {
    if (tid == 0 && blockIdx.x == 0) report(p.status, bad);
    return;
  }
  __syncthreads();
  bool out = false;
  const int32_t* bias_ids = r.bias_ids + (long long)row * r.bias_stride;
  for (int i = tid; i < nb; i += kThreads) {
    const int v = __ldg(bias_ids + i);
    out |= v < 0 || v >= p.V;
    if ((unsigned)(v - v0) < (unsigned)n) atomicMax(word + (v - v0), (uint32_t)(i + 1) << kBiasShift);
  }
  __syncthreads();
  const int32_t* tokens = r.tokens + (long long)row * r.token_stride;
  for (int i = tid; i < len; i += kThreads) {
    const int v = __ldg(tokens + i);
    out |= v < 0 || v >= p.V;
    if ((unsigned)(v - v0) < (unsigned)n) {
      if (i >= prompt)
        atomicAdd(word + (v - v0), 1u);
      else
        atomicOr(word + (v - v0), kPrompt);
    }
  }
  if (__syncthreads_or(out)) {
    if (tid == 0 && blockIdx.x == 0) report(p.status, W4_ERR_INDEX);
    return;
  }
  T* x = static_cast<T*>(p.logits) + (long long)row * p.stride + v0;
  const float* bias = r.bias + (long long)row * r.bias_stride;
  const uint32_t* mask = r.mask + (long long)max(mrow, 0) * r.mask_stride + v0 / 32;
  for (int i = tid; i < n; i += kThreads) {
    const bool allowed = mrow < 0 || ((__ldg(mask + i / 32) >> (i & 31)) & 1);
    const uint32_t w = word[i];
    if (!allowed) {
      store(x + i, -INFINITY);
    } else if (w != 0) {
      float f = load(x + i);
      const uint32_t c = w & kCount;
      if ((w & (kCount | kPrompt)) != 0) f = f > 0.0f ? __fdiv_rn(f, rep) : f * rep;
      if (c != 0) f = f - __fmul_rn(freq, (float)c) - pres;
      if ((w >> kBiasShift) != 0) f += __ldg(bias + (w >> kBiasShift) - 1);
      store(x + i, f);
    }
  }
}

}  // namespace
}  // namespace w4

using namespace w4;

extern "C" w4_status w4_logits_adjust(void* logits, int logits_type, size_t row_stride, int rows,
                                      int V, const w4_logit_rules* rules, int32_t* status_dev,
                                      unsigned flags, w4_stream_t stream) {
  if (logits == nullptr || rules == nullptr || rows < 1 || V < 1 ||
      (logits_type != W4_TYPE_BF16 && logits_type != W4_TYPE_F32) || (flags & ~W4_FLAG_PDL) != 0)
    return W4_ERR_ARG;
  LogitParams p = {};
  p.r = *rules;
  w4_logit_rules& r = p.r;
  if ((r.tokens == nullptr) != (r.lens == nullptr) || (r.bias_ids == nullptr) != (r.bias == nullptr) ||
      (r.prompt != nullptr && r.tokens == nullptr) || (r.n_bias != nullptr && r.bias == nullptr) ||
      (r.mask_rows != nullptr && r.mask == nullptr) || r.max_tokens < 0 || r.max_bias < 0 ||
      (r.mask != nullptr && r.num_masks < (r.mask_rows == nullptr ? rows : 1)))
    return W4_ERR_ARG;
  if (rows > W4_KV8_MAX_BATCH || V > (1 << 30) || r.max_tokens > W4_LOGITS_MAX_HISTORY ||
      r.max_bias > W4_LOGITS_MAX_BIAS)
    return W4_ERR_SHAPE;
  const void* words[] = {r.tokens, r.lens, r.prompt, r.repetition, r.presence, r.frequency,
                         r.bias_ids, r.bias, r.n_bias, r.mask, r.mask_rows};
  for (const void* w : words)
    if (kv8::misaligned(w, 4)) return W4_ERR_ALIGN;
  if (kv8::misaligned(logits, logits_type == W4_TYPE_F32 ? 4 : 2)) return W4_ERR_ALIGN;
  if (row_stride < (size_t)V || row_stride >= (1ull << 40) ||
      (r.tokens != nullptr && (r.token_stride < (size_t)r.max_tokens || r.token_stride >= (1ull << 40))) ||
      (r.bias != nullptr && (r.bias_stride < (size_t)r.max_bias || r.bias_stride >= (1ull << 40))) ||
      (r.mask != nullptr && (r.mask_stride < ((size_t)V + 31) / 32 || r.mask_stride >= (1ull << 40))))
    return W4_ERR_ARG;
  p.logits = logits;
  p.stride = (long long)row_stride;
  p.V = V;
  p.tile = 8192;
  p.status = status_dev;
  const dim3 grid((unsigned)((V - 1) / p.tile + 1), (unsigned)rows);
  const size_t smem = (size_t)p.tile * 4;
  return logits_type == W4_TYPE_F32
             ? kv8::launch(adjust_kernel<float>, grid, kThreads, smem, stream, p)
             : kv8::launch(adjust_kernel<__nv_bfloat16>, grid, kThreads, smem, stream, p);
}
