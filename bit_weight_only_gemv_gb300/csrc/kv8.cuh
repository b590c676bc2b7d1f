// Shared by the 8-bit key/value cache's kernels: the cache and batch as the
// kernels see them, a sequence's bounds, and the host's argument checks.
#pragma once

#include "common.cuh"

namespace w4 {
namespace kv8 {

// The start of every call's workspace: arrival counters of the token kernel,
// one a CTA, zero between calls.  Nothing else is ever written there, so one
// buffer serves calls of every kind and shape in turn.
constexpr size_t kHeadBytes = W4_WORKSPACE_HEAD;
constexpr int kHeadCounters = (int)(kHeadBytes / 4);

struct Cache {
  uint8_t* kc;
  uint8_t* vc;
  float* ks;
  float* vs;
  uint8_t* ranges;
  float* weight;
  int num_pages, H, P, D;
  long long page_stride, head_stride;

  __device__ __forceinline__ long long block(int page, int h) const {   // bytes into kc / vc
    return (long long)page * page_stride + (long long)h * head_stride;
  }
  __device__ __forceinline__ long long pair(int page, int h) const {    // index of (page, head)
    return (long long)page * H + h;
  }
};

struct Batch {
  const int32_t* table;
  const int32_t* lens;
  const int32_t* offsets;
  int B, max_pages, rows, max_new, max_len;
};

// One sequence: its new rows, how many, and its length.
struct Seq {
  int row0, n, len;
  bool ok;   // false: a bound is broken (W4_ERR_INDEX)
};

__device__ __forceinline__ Seq sequence(const Batch& bt, int P, int b) {
  Seq s;
  s.len = load_in(bt.lens + b);
  if (bt.offsets != nullptr) {
    s.row0 = load_in(bt.offsets + b);
    s.n = load_in(bt.offsets + b + 1) - s.row0;
  } else {
    s.row0 = b;
    s.n = 1;
  }
  s.ok = s.len >= 0 && s.len <= bt.max_len && s.n >= 0 && s.n <= bt.max_new && s.row0 >= 0 &&
         s.row0 <= bt.rows - s.n;
  return s;
}

// The least power of two s >= 2^-100 with m <= 127 s, for finite m >= 0: with
// m = 1.f * 2^e, 127 = 1.984375 * 2^6 holds it at 2^(e - 6) when 1.f <=
// 1.984375, else at 2^(e - 5).
__device__ __forceinline__ float pow2_step(float m) {
  const uint32_t b = __float_as_uint(m);
  int e = (int)(b >> 23) - 127 - ((b & 0x7FFFFFu) <= 0x7E0000u ? 6 : 5);
  e = max(e, -100);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// 128 + rint(v) as a code (|v| <= 127 by construction of the step; the clamp
// bounds it for steps that are no power of two).
__device__ __forceinline__ uint32_t to_code(float v) {
  return (uint32_t)(__float2int_rn(fminf(fmaxf(v, -128.0f), 127.0f)) + 128);
}

// Codes of a word as bf16 pairs u - 128: byte u under 0x43 reads 128 + its
// low seven bits once bit 7 is cleared; minus 128 where bit 7 was set, else minus 256.
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w, uint32_t sel) {
  const uint32_t t = __byte_perm(w, 0x43434343u, sel);
  const uint32_t a = t & 0xFF7FFF7Fu;
  const uint32_t b = (~t & 0x00800080u) | 0x43004300u;
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// host: W4_OK and the kernels' view, or the argument error.
w4_status view(const w4_kv8_cache* c, const w4_kv8_batch* b, Cache* cv, Batch* bv);

// host: checks of a call's query rows.
w4_status check_q(const void* q, size_t q_row_stride, int q_heads, const Cache& c);

inline bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

// host: launch as a programmatic dependent of the previous kernel in the
// stream.  Every kernel here waits for that one before it reads or writes
// anything, so this is always right, and hides the launch and the set-up.
template <typename... KArgs, typename... Args>
w4_status launch(void (*kern)(KArgs...), dim3 grid, int threads, size_t smem, w4_stream_t stream,
                 Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  if (e != cudaSuccess) {
    note_cuda_error(e);
    (void)cudaGetLastError();
    return W4_ERR_LAUNCH;
  }
  return W4_OK;
}

}  // namespace kv8
}  // namespace w4
