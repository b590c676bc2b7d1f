// Routing to experts (w4_route) and the sum of their outputs (w4_moe_combine).
//
// Page "Running a 26B MoE on an 8 GB Jetson by streaming experts from SSD",
// section "Streaming without touching a single GPU kernel": the router's top-k
// ids go to the slot pool and the routed product.
//
// route_kernel<V>: one warp a token, V neighbouring experts a lane.  Scores
// c = s + bias become 32-bit keys in the order of the floats; each of the
// top_k rounds is one warp maximum and one ballot, and the lane that held it
// looks for its next one.  Without a bias the key is the logit itself, whose
// order is the scores'.  With one, fp32 scores carry rounding errors: two that
// are compared and lie within `tol` of each other (bounded below) send the
// token through refine(), which chooses among doubles.
#include "kv8.cuh"

namespace w4 {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kRouteWarps = 4;

struct RouteParams {
  int32_t* ids;
  float* weights;
  const void* logits;
  const float* bias;
  long long stride;
  int rows, E, k, G, size, top_groups, best;   // size: experts of a group
  bool sigmoid, renorm, f32, vec;
  float scale;
  int32_t* status;
};

// In the order of the floats; -0 and +0 alike (their sum with +0 is +0).
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t b = __float_as_uint(f + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float logit(const RouteParams& p, long long row, int e) {
  const long long i = row * p.stride + e;
  return p.f32 ? __ldg(static_cast<const float*>(p.logits) + i)
               : bf16_bits_to_float(__ldg(static_cast<const uint16_t*>(p.logits) + i));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.0f, 1.0f + expf(-x)); }

// The choice of one token with scores in 64 bits; sm holds E doubles of this
// warp.  Lane j < k gets the j-th expert.
__device__ __noinline__ int refine(const RouteParams& p, long long row, double* sm) {
  const int lane = threadIdx.x & 31;
  const double kTaken = __longlong_as_double(0x7ff8000000000000ll);   // NaN
  double m = -INFINITY, z = 0.0;
  if (!p.sigmoid) {
    for (int e = lane; e < p.E; e += 32) m = fmax(m, (double)logit(p, row, e));
    for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(kFull, m, o));
    for (int e = lane; e < p.E; e += 32) {
      const double s = exp((double)logit(p, row, e) - m);
      sm[e] = s;
      z += s;
    }
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
  }
  for (int e = lane; e < p.E; e += 32) {
    const double s = p.sigmoid ? 1.0 / (1.0 + exp(-(double)logit(p, row, e))) : sm[e] / z;
    sm[e] = s + (p.bias != nullptr ? (double)__ldg(p.bias + e) : 0.0);
  }
  __syncwarp();
  uint32_t in = kFull;   // chosen groups
  if (p.G > 1) {
    double gs = -INFINITY;
    if (lane < p.G) {
      double a = -INFINITY, b = -INFINITY;
      for (int i = 0; i < p.size; ++i) {
        const double c = sm[lane * p.size + i];
        b = fmax(b, fmin(a, c));
        a = fmax(a, c);
      }
      gs = p.best == 2 ? a + b : a;
    }
    int better = 0;
    for (int g = 0; g < p.G; ++g) {
      const double o = __shfl_sync(kFull, gs, g);
      better += o > gs || (o == gs && g < lane);
    }
    in = __ballot_sync(kFull, lane < p.G && better < p.top_groups);
  }
  __syncwarp();
  for (int e = lane; e < p.E; e += 32) {
    if (p.G > 1 && !((in >> (e / p.size)) & 1))
      sm[e] = kTaken;
    else if (p.bias == nullptr)
      sm[e] = (double)logit(p, row, e);   // the scores' order is the logits'
  }
  int mine = 0;
  for (int j = 0; j < p.k; ++j) {
    double c = kTaken;
    int at = p.E;
    for (int e = lane; e < p.E; e += 32)
      if (!isnan(sm[e]) && (isnan(c) || sm[e] > c)) {
        c = sm[e];
        at = e;
      }
    for (int o = 16; o > 0; o >>= 1) {
      const double oc = __shfl_xor_sync(kFull, c, o);
      const int oat = __shfl_xor_sync(kFull, at, o);
      if (!isnan(oc) && (isnan(c) || oc > c || (oc == c && oat < at))) {
        c = oc;
        at = oat;
      }
    }
    if (lane == (at & 31)) sm[at] = kTaken;
    if (lane == j) mine = at;
  }
  return mine;
}

template <int V>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(RouteParams p) {
  extern __shared__ double refine_sm[];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long row = (long long)blockIdx.x * kRouteWarps + warp;
  if (row >= p.rows) return;
  const int e0 = lane * V;
  float x[V];
  if (p.vec) {   // E = 32 V and every row on a 16-byte boundary
    if (p.f32) {
      const float4* src = reinterpret_cast<const float4*>(
          static_cast<const float*>(p.logits) + row * p.stride + e0);
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        const float4 w = __ldg(src + i);
        x[4 * i] = w.x;
        x[4 * i + 1] = w.y;
        x[4 * i + 2] = w.z;
        x[4 * i + 3] = w.w;
      }
    } else {
      const uint2* src = reinterpret_cast<const uint2*>(
          static_cast<const uint16_t*>(p.logits) + row * p.stride + e0);
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        const uint2 w = __ldg(src + i);
        x[4 * i] = bf16_bits_to_float(w.x & 0xFFFFu);
        x[4 * i + 1] = __uint_as_float(w.x & 0xFFFF0000u);
        x[4 * i + 2] = bf16_bits_to_float(w.y & 0xFFFFu);
        x[4 * i + 3] = __uint_as_float(w.y & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = e0 + i < p.E ? logit(p, row, e0 + i) : -INFINITY;
  }
  float top = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    bad |= isnan(x[i]);
    top = fmaxf(top, x[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
  if (!p.sigmoid && isinf(top)) bad = true;
  uint32_t key[V];
  const bool groups = p.G > 1;
  const bool sums = p.bias != nullptr || (groups && p.best == 2);   // scores themselves compared
  float z = 1.0f, tol = 0.0f;
  float c[V];
  if (sums || (!p.renorm && !p.sigmoid)) {
    // Errors of a score s: the exponential's 2 units and the division's and sum's few for a
    // sigmoid, 2^-21 s in all; a softmax's sum adds (V + 5) / 2 units and x - top its own half.
    if (p.sigmoid) {
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = sigmoid(x[i]);
      tol = 0x1p-20f * sigmoid(top);
    } else {
      z = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        c[i] = expf(x[i] - top);
        z += c[i];
      }
      z = warp_sum(z);
      const float r = __fdividef(1.0f, z);
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] *= r;
      tol = 0x1p-17f * r;
    }
    if (p.bias != nullptr) {
      float most = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float b = e0 + i < p.E ? __ldg(p.bias + e0 + i) : 0.0f;
        bad |= !isfinite(b);
        c[i] += b;
        most = fmaxf(most, fabsf(c[i]));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(kFull, most, o));
      tol += 0x1p-22f * most;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = 0.0f;
  }
  if (__any_sync(kFull, bad)) {
    if (lane == 0) report(p.status, W4_ERR_VALUE);
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    key[i] = e0 + i < p.E ? order_key(p.bias != nullptr ? c[i] : x[i]) : 0u;
  bool close = false;   // two compared scores nearer than fp32 can tell
  if (groups) {
    const bool by_sum = p.best == 2;
    float gs = 0.0f;       // lane g: the score of group g (its key where one logit decides)
    uint32_t gk = 0;
    for (int g = 0; g < p.G; ++g) {
      const int lo = g * p.size, hi = lo + p.size;
      uint32_t a = 0;
      float f1 = -INFINITY, f2 = -INFINITY;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (e0 + i >= lo && e0 + i < hi) {
          a = max(a, key[i]);
          f2 = fmaxf(f2, fminf(f1, c[i]));
          f1 = fmaxf(f1, c[i]);
        }
      if (by_sum) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const float o1 = __shfl_xor_sync(kFull, f1, o), o2 = __shfl_xor_sync(kFull, f2, o);
          f2 = fmaxf(fmaxf(f2, o2), fminf(f1, o1));
          f1 = fmaxf(f1, o1);
        }
        if (lane == g) gs = f1 + f2;
      } else {
        a = __reduce_max_sync(kFull, a);
        if (lane == g) gk = a;
      }
    }
    if (by_sum) gk = lane < p.G ? order_key(gs) : 0u;
    uint32_t in = 0, last = 0;
    for (int j = 0; j <= p.top_groups && j < p.G; ++j) {
      const uint32_t m = __reduce_max_sync(kFull, gk);
      if (j == p.top_groups) {   // the best of those left out
        if (sums) close |= key_value(last) - key_value(m) < 3.0f * tol;
        break;
      }
      last = m;
      const uint32_t who = __ballot_sync(kFull, gk == m);
      in |= who & (0u - who);
      if (lane == __ffs(who) - 1) gk = 0;
    }
    int g = e0 / p.size, left = (g + 1) * p.size - e0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (left == 0) {
        ++g;
        left = p.size;
      }
      --left;
      if (!((in >> (g & 31)) & 1)) key[i] = 0;
    }
  }
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) mine = max(mine, key[i]);
  int my_id = 0, prev_id = 0;
  uint32_t prev = 0;
  const bool check = p.bias != nullptr;
  const int rounds = p.k + (check ? 1 : 0);
  for (int j = 0; j < rounds; ++j) {
    const uint32_t m = __reduce_max_sync(kFull, mine);
    if (m == 0) break;   // as many experts as there are: none left to compare with
    const int src = __ffs(__ballot_sync(kFull, mine == m)) - 1;
    int at = 0;
    if (lane == src) {
#pragma unroll
      for (int i = V - 1; i >= 0; --i) at = key[i] == m ? i : at;
      mine = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (i == at) key[i] = 0;
        mine = max(mine, key[i]);
      }
      at += e0;
    }
    at = __shfl_sync(kFull, at, src);
    if (check && j > 0 && key_value(prev) - key_value(m) < tol) {
      // equal inputs are equal scores at any width, and in order already
      const bool same = logit(p, row, at) == logit(p, row, prev_id) &&
                        __ldg(p.bias + at) == __ldg(p.bias + prev_id);
      close |= !same;
    }
    prev = m;
    prev_id = at;
    if (lane == j && j < p.k) my_id = at;
  }
  if (close) my_id = refine(p, row, refine_sm + warp * p.E);
  // weights: relative to the largest chosen logit where they are divided by their sum, so that
  // small scores do not vanish
  const bool has = lane < p.k;
  const float xl = has ? logit(p, row, my_id) : -INFINITY;
  float w;
  if (p.renorm) {
    float m = xl;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    if (p.sigmoid) m = fminf(m, 0.0f);
    w = has && xl > -INFINITY ? (p.sigmoid && m == 0.0f ? sigmoid(xl) : expf(xl - m)) : 0.0f;
    if (p.sigmoid && m < 0.0f) w = __fdividef(w, 1.0f + expf(xl));
    const float sum = warp_sum(w);
    w = sum > 0.0f ? p.scale * __fdividef(w, sum) : 0.0f;
  } else {
    w = p.scale * (p.sigmoid ? sigmoid(xl) : __fdividef(expf(xl - top), z));
  }
  if (has) {
    p.ids[row * p.k + lane] = my_id;
    p.weights[row * p.k + lane] = w;
  }
}

// ---------------------------------------------------------------- combine
constexpr int kCombineThreads = 128;

struct CombineParams {
  __nv_bfloat16* out;
  const __nv_bfloat16* y;
  const float* weights;
  const int32_t* ids;
  const __nv_bfloat16* add;
  int num_experts, k, N, chunks;   // chunks: CTAs along a row
  int32_t* status;
};

template <int VEC>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(CombineParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const long long row = blockIdx.x / p.chunks;
  const int chunk = blockIdx.x % p.chunks;
  const int n = (chunk * kCombineThreads + threadIdx.x) * VEC;
  const float* wt = p.weights + row * p.k;
  if (p.ids != nullptr) {
    bool ok = true;
    for (int j = 0; j < p.k; ++j) {
      const int id = __ldg(p.ids + row * p.k + j);
      ok = ok && id >= 0 && id < p.num_experts;
    }
    if (!ok) {
      if (chunk == 0 && threadIdx.x == 0) report(p.status, W4_ERR_INDEX);
      return;
    }
  }
  if (n >= p.N) return;
  const __nv_bfloat16* y = p.y + row * p.k * (long long)p.N + n;
  float acc[VEC];
  if constexpr (VEC == 8) {
    auto spread = [](const uint4& w, float f[8]) {
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_bits_to_float(u[i] & 0xFFFFu);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      }
    };
    if (p.add != nullptr) {
      spread(*reinterpret_cast<const uint4*>(p.add + row * p.N + n), acc);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
    }
    int j = 0;
    for (; j + 8 <= p.k; j += 8) {
      uint4 v[8];
#pragma unroll
      for (int z = 0; z < 8; ++z)
        v[z] = __ldg(reinterpret_cast<const uint4*>(y + (long long)(j + z) * p.N));
#pragma unroll
      for (int z = 0; z < 8; ++z) {
        float f[8];
        spread(v[z], f);
        const float w = __ldg(wt + j + z);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, f[i], acc[i]);
      }
    }
#pragma unroll 2
    for (; j < p.k; ++j) {
      float f[8];
      spread(__ldg(reinterpret_cast<const uint4*>(y + (long long)j * p.N)), f);
      const float w = __ldg(wt + j);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, f[i], acc[i]);
    }
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(acc[2 * i], acc[2 * i + 1]);
      o[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p.out + row * p.N + n) = make_uint4(o[0], o[1], o[2], o[3]);
  } else {
    acc[0] = p.add != nullptr ? __bfloat162float(p.add[row * p.N + n]) : 0.0f;
#pragma unroll 8
    for (int j = 0; j < p.k; ++j)
      acc[0] = fmaf(__ldg(wt + j), __bfloat162float(__ldg(y + (long long)j * p.N)), acc[0]);
    p.out[row * p.N + n] = __float2bfloat16_rn(acc[0]);
  }
}

}  // namespace
}  // namespace w4

using namespace w4;

extern "C" w4_status w4_route(int32_t* ids, float* weights, const w4_router* router,
                              const void* logits, int logits_type, size_t row_stride,
                              const float* bias, int rows, int32_t* status_dev, unsigned flags,
                              w4_stream_t stream) {
  if (ids == nullptr || weights == nullptr || router == nullptr || logits == nullptr)
    return W4_ERR_ARG;
  const w4_router& r = *router;
  if (rows < 1 || r.experts < 1 || r.top_k < 1 || r.groups < 1 || r.top_groups < 1 ||
      (r.group_best != 1 && r.group_best != 2) ||
      (r.score != W4_ROUTE_SOFTMAX && r.score != W4_ROUTE_SIGMOID) || (r.renorm & ~1) != 0 ||
      !(r.scale - r.scale == 0.0f) || (flags & ~W4_FLAG_PDL) != 0 ||
      (logits_type != W4_TYPE_BF16 && logits_type != W4_TYPE_F32))
    return W4_ERR_ARG;
  if (r.experts > W4_ROUTE_MAX_EXPERTS || r.top_k > W4_ROUTE_MAX_TOP_K ||
      r.groups > W4_ROUTE_MAX_GROUPS || r.experts % r.groups != 0 || r.top_groups > r.groups ||
      r.top_k > r.top_groups * (r.experts / r.groups))
    return W4_ERR_SHAPE;
  const int el = logits_type == W4_TYPE_F32 ? 4 : 2;
  if (kv8::misaligned(ids, 4) || kv8::misaligned(weights, 4) || kv8::misaligned(bias, 4) ||
      kv8::misaligned(logits, el))
    return W4_ERR_ALIGN;
  if (row_stride < (size_t)r.experts || row_stride >= (1ull << 32)) return W4_ERR_ARG;
  RouteParams p = {};
  p.ids = ids;
  p.weights = weights;
  p.logits = logits;
  p.bias = bias;
  p.stride = (long long)row_stride;
  p.rows = rows;
  p.E = r.experts;
  p.k = r.top_k;
  p.size = r.experts / r.groups;
  p.G = r.top_groups == r.groups ? 1 : r.groups;   // every group in: as without groups
  p.top_groups = r.top_groups;
  p.best = p.size == 1 ? 1 : r.group_best;
  p.sigmoid = r.score == W4_ROUTE_SIGMOID;
  p.renorm = r.renorm != 0;
  p.f32 = logits_type == W4_TYPE_F32;
  p.scale = r.scale;
  p.status = status_dev;
  const bool sums = bias != nullptr || (p.G > 1 && p.best == 2);
  const size_t smem = sums ? (size_t)kRouteWarps * p.E * sizeof(double) : 0;
  const unsigned grid = (unsigned)((rows + kRouteWarps - 1) / kRouteWarps);
  auto go = [&](auto kern, int v) {
    p.vec = v >= 4 && p.E == 32 * v && !kv8::misaligned(logits, 16) && row_stride * el % 16 == 0;
    return kv8::launch(kern, dim3(grid), 32 * kRouteWarps, smem, stream, p);
  };
  if (p.E <= 32) return go(route_kernel<1>, 1);
  if (p.E <= 64) return go(route_kernel<2>, 2);
  if (p.E <= 128) return go(route_kernel<4>, 4);
  if (p.E <= 256) return go(route_kernel<8>, 8);
  if (p.E <= 512) return go(route_kernel<16>, 16);
  return go(route_kernel<32>, 32);
}

extern "C" w4_status w4_moe_combine(void* out, const void* y, const float* weights,
                                    const int32_t* ids, int num_experts, const void* add, int rows,
                                    int top_k, int N, int32_t* status_dev, unsigned flags,
                                    w4_stream_t stream) {
  if (out == nullptr || y == nullptr || weights == nullptr || rows < 1 || top_k < 1 || N < 1 ||
      (ids != nullptr && num_experts < 1) || (flags & ~W4_FLAG_PDL) != 0)
    return W4_ERR_ARG;
  if (top_k > W4_ROUTE_MAX_TOP_K) return W4_ERR_SHAPE;
  if (kv8::misaligned(out, 2) || kv8::misaligned(y, 2) || kv8::misaligned(add, 2) ||
      kv8::misaligned(weights, 4) || kv8::misaligned(ids, 4))
    return W4_ERR_ALIGN;
  CombineParams p = {};
  p.out = static_cast<__nv_bfloat16*>(out);
  p.y = static_cast<const __nv_bfloat16*>(y);
  p.weights = weights;
  p.ids = ids;
  p.add = static_cast<const __nv_bfloat16*>(add);
  p.num_experts = num_experts;
  p.k = top_k;
  p.N = N;
  p.status = status_dev;
  const bool vec = N % 8 == 0 && !kv8::misaligned(out, 16) && !kv8::misaligned(y, 16) &&
                   !kv8::misaligned(add, 16);
  const int per = kCombineThreads * (vec ? 8 : 1);
  p.chunks = (N - 1) / per + 1;
  if ((long long)p.chunks * rows > 0x7fffffffll) return W4_ERR_SHAPE;
  const dim3 grid((unsigned)((long long)p.chunks * rows));
  return vec ? kv8::launch(combine_kernel<8>, grid, kCombineThreads, 0, stream, p)
             : kv8::launch(combine_kernel<1>, grid, kCombineThreads, 0, stream, p);
}
