// Penalties, biases and masks on the output product's logits (w4_logits_adjust).
//
// One CTA per (tile of the vocabulary, row), a 32-bit word for each token of
// the tile in shared memory:
//   bits 0..18   occurrences after the prompt
//   bit  19      occurs in the prompt
//   bits 20..31  1 + index of its last bias
// The CTA reads the row's bias list and history once, keeps what falls into its
// tile, and then walks the tile, eight tokens a lane: tokens that no rule names
// and the mask allows cost no global access, eight that the mask forbids a store.
// Where few of a warp's eights have a token named, those go token by token, a
// token a lane; among the frequent ones all eights are worked through.  The warps
// take pieces of 256 tokens in turn, since the tokens that a history names are
// neighbours in most vocabularies (the frequent ones come first).  Tiles start
// on 16-byte boundaries of the row in memory, wherever the row does, so that
// a lane's eight logits are whole vectors but for a row's ends.
// Every CTA of a row sees the whole lists, so all of them find the same errors.
// Chains of loads bound it (counts, lists, logits), so each link has many in
// flight: a warp's mask words come before the lists, histories sixteen tokens a
// thread at a time.  Half of a warp's time is waiting for global loads (24 rows of 262144
// under masks: 1.8 of 4 instructions issued a cycle at 32 warps an SM).
#include <mutex>

#include "kv8.cuh"

namespace w4 {
namespace {

constexpr uint32_t kCount = (1u << 19) - 1, kPrompt = 1u << 19;
constexpr int kBiasShift = 20;
constexpr int kPiece = 256;   // tokens that a warp takes at a time, four times over
constexpr unsigned kFull = 0xffffffffu;
constexpr int kSparse = 4;    // eights of a piece with a token named that go token by token

struct LogitParams {
  void* logits;
  long long stride;
  int V;
  w4_logit_rules r;
  int32_t* status;
};

// What a row's rules are, and logits under them.  The quotient by the repetition is a product
// with its reciprocal: a logit has two roundings of 2^-24 there instead of one (a division is some ten
// instructions for each of a lane's eight); far from 1, where the reciprocal would be rounded harder, it
// is a division.  The product with the frequency is fused, one rounding less.
struct RowRules {
  float rep, inv, pres, freq;
  bool divide;
  const float* bias;

  __device__ __forceinline__ float apply(float f, uint32_t w) const {
    const uint32_t c = w & kCount;
    if ((w & (kCount | kPrompt)) != 0)
      f = f > 0.0f ? (divide ? __fdiv_rn(f, rep) : f * inv) : f * rep;
    if (c != 0) f = fmaf(-freq, (float)c, f) - pres;
    if ((w >> kBiasShift) != 0) f += load_in(bias + (w >> kBiasShift) - 1);
    return f;
  }
  // Eight at once, the same without branches but where one of them has a bias.
  __device__ __forceinline__ void apply8(float (&f)[8], const uint32_t (&w)[8], uint32_t any) const {
    if (divide) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = apply(f[i], w[i]);
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t c = w[i] & kCount;
      const float g = f[i] * (f[i] > 0.0f ? inv : rep);
      f[i] = (w[i] & (kCount | kPrompt)) != 0 ? g : f[i];
      const float h = fmaf(-freq, (float)c, f[i]) - pres;
      f[i] = c != 0 ? h : f[i];
    }
    if ((any >> kBiasShift) != 0)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if ((w[i] >> kBiasShift) != 0) f[i] += load_in(bias + (w[i] >> kBiasShift) - 1);
  }
};

// Eight neighbouring logits as they are stored.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void store(float* p) const {
    *reinterpret_cast<float4*>(p) = a;
    *reinterpret_cast<float4*>(p + 4) = b;
  }
  __device__ __forceinline__ void forbid() { a = b = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY); }
  __device__ __forceinline__ void adjust(const RowRules& r, const uint32_t (&w)[8], uint32_t any,
                                         uint32_t allowed) {
    float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (any != 0) r.apply8(f, w, any);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (allowed >> i) & 1 ? f[i] : -INFINITY;
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
  __device__ __forceinline__ void mask(uint32_t allowed) {
    a.x = allowed & 1 ? a.x : -INFINITY;
    a.y = allowed & 2 ? a.y : -INFINITY;
    a.z = allowed & 4 ? a.z : -INFINITY;
    a.w = allowed & 8 ? a.w : -INFINITY;
    b.x = allowed & 16 ? b.x : -INFINITY;
    b.y = allowed & 32 ? b.y : -INFINITY;
    b.z = allowed & 64 ? b.z : -INFINITY;
    b.w = allowed & 128 ? b.w : -INFINITY;
  }
};
template <>
struct Eight<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = v; }
  __device__ __forceinline__ void forbid() { v = make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u); }
  __device__ __forceinline__ void adjust(const RowRules& r, const uint32_t (&w)[8], uint32_t any,
                                         uint32_t allowed) {
    uint32_t u[4] = {v.x, v.y, v.z, v.w};
    if (any != 0) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      }
      r.apply8(f, w, any);
#pragma unroll
      for (int i = 0; i < 4; ++i) {   // logits that no rule names keep their bits
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        const uint32_t keep = (w[2 * i] != 0 ? 0u : 0xFFFFu) | (w[2 * i + 1] != 0 ? 0u : 0xFFFF0000u);
        u[i] = (u[i] & keep) | (*reinterpret_cast<const uint32_t*>(&b) & ~keep);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t off = (allowed >> (2 * i) & 1 ? 0u : 0xFFFFu) | (allowed >> (2 * i + 1) & 1 ? 0u : 0xFFFF0000u);
      u[i] = (u[i] & ~off) | (0xFF80FF80u & off);
    }
    v = make_uint4(u[0], u[1], u[2], u[3]);
  }
  __device__ __forceinline__ void mask(uint32_t allowed) {
    uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t off = (allowed >> (2 * i) & 1 ? 0u : 0xFFFFu) | (allowed >> (2 * i + 1) & 1 ? 0u : 0xFFFF0000u);
      u[i] = (u[i] & ~off) | (0xFF80FF80u & off);
    }
    v = make_uint4(u[0], u[1], u[2], u[3]);
  }
};

__device__ __forceinline__ float load(const float* p) { return *p; }
__device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store(float* p, float v) { *p = v; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// kThreads * 32 tokens a CTA; kAhead of a warp's four pieces have their logits loaded together.
template <typename T, int kThreads, int kAhead, int kResident>
__global__ void __launch_bounds__(kThreads, kResident) adjust_kernel(const __grid_constant__ LogitParams p) {
  extern __shared__ uint32_t word[];   // 32 for each thread
  constexpr int threads = kThreads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, row = blockIdx.y;
  T* const logits = static_cast<T*>(p.logits) + (long long)row * p.stride;
  // logits before the row since a 16-byte boundary; the tile's tokens v0 .. v0 + tile - 1, of which
  // some may lie outside the vocabulary
  const int before = (int)(reinterpret_cast<uintptr_t>(logits) % 16 / sizeof(T));
  const int tile = threads * 32, v0 = (int)blockIdx.x * tile - before;
#pragma unroll
  for (int i = 0; i < 8; ++i) reinterpret_cast<uint4*>(word)[tid + i * threads] = make_uint4(0, 0, 0, 0);
  pdl_wait();
  const w4_logit_rules& r = p.r;
  const int len = r.tokens != nullptr ? load_in(r.lens + row) : 0;
  const int prompt = r.prompt != nullptr ? load_in(r.prompt + row) : 0;
  const int nb = r.bias_ids == nullptr ? 0 : r.n_bias != nullptr ? load_in(r.n_bias + row) : r.max_bias;
  const int mrow = r.mask == nullptr ? -1 : r.mask_rows != nullptr ? load_in(r.mask_rows + row) : row;
  RowRules rules;
  rules.rep = r.repetition != nullptr ? load_in(r.repetition + row) : 1.0f;
  rules.pres = r.presence != nullptr ? load_in(r.presence + row) : 0.0f;
  rules.freq = r.frequency != nullptr ? load_in(r.frequency + row) : 0.0f;
  rules.inv = __frcp_rn(rules.rep);
  rules.divide = !(rules.rep > 0x1p-100f && rules.rep < 0x1p100f);
  rules.bias = r.bias + (long long)row * r.bias_stride;
  int bad = 0;
  if (len < 0 || len > r.max_tokens || prompt < 0 || prompt > len || nb < 0 || nb > r.max_bias ||
      mrow < -1 || (mrow >= r.num_masks && r.mask != nullptr))
    bad = W4_ERR_INDEX;
  else if (!(rules.rep > 0.0f) || isinf(rules.rep) || !isfinite(rules.pres) || !isfinite(rules.freq))
    bad = W4_ERR_VALUE;
  if (bad != 0) {
    if (tid == 0 && blockIdx.x == 0) report(p.status, bad);
    return;
  }
  // 32 tokens' bits of the mask for each lane: tokens from v0 + at on
  const int warps = threads >> 5;
  uint32_t allow = kFull;
  if (mrow >= 0) {
    const int at = ((lane >> 3) * warps + warp) * kPiece + (lane & 7) * 32;
    const uint32_t* mask = r.mask + (long long)mrow * r.mask_stride;
    const int words = (p.V + 31) / 32, w = (v0 + at + 32) / 32 - 1;   // rounded down, from -1 on
    const uint32_t lo = w >= 0 && w < words ? load_in(mask + w) : 0u;
    const uint32_t hi = before != 0 && w + 1 < words ? load_in(mask + w + 1) : 0u;
    allow = __funnelshift_r(lo, hi, v0 & 31);
  }
  __syncthreads();
  bool out = false;
  const int32_t* bias_ids = r.bias_ids + (long long)row * r.bias_stride;
  for (int i = tid; i < nb; i += threads) {
    const int v = load_in(bias_ids + i);
    out |= v < 0 || v >= p.V;
    if ((unsigned)(v - v0) < (unsigned)tile) atomicMax(word + (v - v0), (uint32_t)(i + 1) << kBiasShift);
  }
  __syncthreads();
  // the history, the prompt's tokens, then the others: vectors of four tokens between 16-byte
  // boundaries, each token a subtraction, two comparisons and an atomic under a predicate
  const int32_t* tokens = r.tokens + (long long)row * r.token_stride;
  uint32_t most = 0;   // a token below 0 is a large number
  const uint32_t words = smem_addr(word);
  auto walk = [&](int from, int to, auto note) {
    auto take = [&](int v) {
      most = max(most, (uint32_t)v);
      note((uint32_t)(v - v0));
    };
    const int32_t* t = tokens + from;
    const int n = to - from;
    const int head = min(n, (int)((16 - (reinterpret_cast<uintptr_t>(t) & 15)) & 15) / 4);
    const int vecs = (n - head) / 4, tail = head + 4 * vecs;
    if (tid < head) take(load_in(t + tid));
    if (tid < n - tail) take(load_in(t + tail + tid));
    const int4* body = reinterpret_cast<const int4*>(t + head);
    int i = tid;
    for (; i + 3 * threads < vecs; i += 4 * threads) {
      int4 v[4];
#pragma unroll
      for (int z = 0; z < 4; ++z) v[z] = load_in(body + i + z * threads);
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        take(v[z].x);
        take(v[z].y);
        take(v[z].z);
        take(v[z].w);
      }
    }
#pragma unroll 3
    for (; i < vecs; i += threads) {
      const int4 v = load_in(body + i);
      take(v.x);
      take(v.y);
      take(v.z);
      take(v.w);
    }
  };
  walk(0, prompt, [&](uint32_t i) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.lt.u32 q, %0, %1;\n\t@q red.shared.or.b32 [%2], %3;\n\t}" ::"r"(i),
                 "r"((uint32_t)tile), "r"(words + 4 * i), "r"(kPrompt)
                 : "memory");
  });
  walk(prompt, len, [&](uint32_t i) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.lt.u32 q, %0, %1;\n\t@q red.shared.add.u32 [%2], 1;\n\t}" ::"r"(i),
                 "r"((uint32_t)tile), "r"(words + 4 * i)
                 : "memory");
  });
  out |= most >= (uint32_t)p.V;
  if (__syncthreads_or(out)) {
    if (tid == 0 && blockIdx.x == 0) report(p.status, W4_ERR_INDEX);
    return;
  }
#pragma unroll 1
  for (int s0 = 0; s0 < 4; s0 += kAhead) {
    Eight<T> f[kAhead];
    uint32_t any[kAhead], may[kAhead];
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
      const int at = ((s0 + s) * warps + warp) * kPiece + lane * 8, v = v0 + at;
      may[s] = (__shfl_sync(kFull, allow, (s0 + s) * 8 + (lane >> 2)) >> (8 * (lane & 3))) & 0xFFu;
      const uint4 a = *reinterpret_cast<const uint4*>(word + at), b = *reinterpret_cast<const uint4*>(word + at + 4);
      any[s] = a.x | a.y | a.z | a.w | b.x | b.y | b.z | b.w;
      if (may[s] != 0 && (may[s] != 0xFFu || any[s] != 0) && v >= 0 && v + 8 <= p.V) f[s].load(logits + v);
    }
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
      const int first = ((s0 + s) * warps + warp) * kPiece, at = first + lane * 8, v = v0 + at;
      const bool ends = v < 0 || v + 8 > p.V;   // a row's ends
      const uint32_t named = __ballot_sync(kFull, any[s] != 0 && may[s] != 0 && !ends);
      const bool dense = __popc(named) > kSparse;
      if (ends) {
        if (may[s] != 0xFFu || any[s] != 0)
          for (int i = max(0, -v); i < min(8, p.V - v); ++i) {
            const uint32_t w = word[at + i];
            if (!((may[s] >> i) & 1))
              store(logits + v + i, -INFINITY);
            else if (w != 0)
              store(logits + v + i, rules.apply(load(logits + v + i), w));
          }
      } else if (may[s] == 0) {
        f[s].forbid();
        f[s].store(logits + v);
      } else if (dense && any[s] != 0) {
        const uint4 a = *reinterpret_cast<const uint4*>(word + at), b = *reinterpret_cast<const uint4*>(word + at + 4);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        f[s].adjust(rules, w, any[s], may[s]);
        f[s].store(logits + v);
      } else if (may[s] != 0xFFu) {
        f[s].mask(may[s]);
        f[s].store(logits + v);
      }
      if (!dense && named != 0) {
        // few of the warp's eights have a token named: four of them at a time, a token a lane
        __syncwarp();   // what the mask changed beside them is stored
        for (uint32_t left = named; left != 0;) {
          uint32_t mine = left;
          for (int q = lane >> 3; q > 0; --q) mine &= mine - 1;
          const int src = mine != 0 ? __ffs((int)mine) - 1 : 0, i = first + src * 8 + (lane & 7);
          const uint32_t ok = __shfl_sync(kFull, may[s], src);
          const uint32_t w = word[i];
          if (mine != 0 && w != 0 && ((ok >> (lane & 7)) & 1)) store(logits + v0 + i, rules.apply(load(logits + v0 + i), w));
          left &= left - 1;
          left &= left - 1;
          left &= left - 1;
          left &= left - 1;
        }
      }
    }
  }
}

template <typename T, int kThreads, int kAhead, int kResident>
w4_status run(const LogitParams& p, long long span, int rows, w4_stream_t stream) {
  constexpr size_t smem = (size_t)kThreads * 128;
  auto kern = adjust_kernel<T, kThreads, kAhead, kResident>;
  if (smem > 48 << 10) {   // once for each device: more shared memory than the default
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return W4_ERR_DEVICE;
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) {
        note_cuda_error(e);
        (void)cudaGetLastError();
        return W4_ERR_LAUNCH;
      }
      done[dev] = true;
    }
  }
  const dim3 grid((unsigned)((span - 1) / (32 * kThreads) + 1), (unsigned)rows);
  return kv8::launch(kern, grid, kThreads, smem, stream, p);
}

// While the CTAs of 256 threads and 8192 tokens are resident together (four an SM), each with all
// its logits on their way at once.  Of more work, as many as registers allow, one piece's
// logits at a time; with long histories CTAs of 512 threads and 16384 tokens, which read them half
// as often.  Measured, in this order of variants: one row of 262144 tokens 4.4, 5.0 and 5.4 us; 24
// rows under masks, histories to 4096, 13.5, 11.4 and 11.9 us; 64 rows of 100277 with histories to
// 30000 25, 20 and 17.6 us; 2000 rows of 4000 18.7, 18.4 and 28 us.
template <typename T>
w4_status run(const LogitParams& p, bool aligned, int rows, w4_stream_t stream) {
  const long long span = (long long)p.V + (aligned ? 0 : 16 / (int)sizeof(T) - 1);
  if (((span - 1) / 8192 + 1) * rows <= 4 * 152) return run<T, 256, 4, 4>(p, span, rows, stream);
  if (span > 8192 && p.r.tokens != nullptr && p.r.max_tokens > 8192)
    return run<T, 512, 1, 3>(p, span, rows, stream);
  return run<T, 256, 1, 6>(p, span, rows, stream);
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
  p.status = status_dev;
  const int el = logits_type == W4_TYPE_F32 ? 4 : 2;
  const bool aligned = !kv8::misaligned(logits, 16) && (rows == 1 || row_stride * el % 16 == 0);
  return logits_type == W4_TYPE_F32 ? run<float>(p, aligned, rows, stream)
                                    : run<__nv_bfloat16>(p, aligned, rows, stream);
}
