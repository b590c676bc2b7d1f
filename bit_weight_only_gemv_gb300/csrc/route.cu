// Routing to experts (w4_route) and the sum of their outputs (w4_moe_combine).
//
// Page "Running a 26B MoE on an 8 GB Jetson by streaming experts from SSD",
// section "Streaming without touching a single GPU kernel": the router's top-k
// ids go to the slot pool and the routed product.
//
// route_kernel<V, F32>: one warp a token.  Every group has as many lanes (a power
// of two; without groups all 32), each with up to V neighbouring experts, so
// that a group's best scores are a butterfly away.  The chain of a token's instructions
// bounds it (at 16384 tokens 1.65 of 4 issued a cycle and SM), so a candidate is one word: its score as a fixed-point number above its place,
// places counted down.  One integer maximum over the warp then gives value,
// expert and the lowest number among equals, and a lane's candidates, sorted once
// by a network of minima and maxima, only move up.  What the word says of the
// score:
//   bf16 logits, no bias   the logit itself, exactly
//   fp32 logits, no bias   (logit - largest) in 2^-18, as far as 32 below
//   with a bias            score + (bias - least bias) in about 2^-23 of their range
// Of candidates, or groups, that are nearer than this (and the scores' fp32
// errors) can tell, the order is found from 64-bit scores of those few alone; of
// more than 32 such candidates by refine() over all experts.  Such tokens are slow: 16384 random
// ones over 256 experts in 8 groups take 15 us, with a spread that saturates the scores up to 1260.
// One token takes 1.9 us in a graph, 192 tokens over 256 experts in 8 groups with
// biases 3.3 us (latency: about 800 instructions a warp); for many tokens
// route_many_kernel takes a quarter of the warps.
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
  int shift, each;   // lanes of a group: 1 << shift; experts of a lane
  int shift8;        // the same of eight lanes
  bool sigmoid, renorm, f32, vec;
  float scale;
  int32_t* status;
};

// In the order of the floats; -0 and +0 alike (their sum with +0 is +0).
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t b = __float_as_uint(f + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// Largest of the warp's values, NaN if one of them is.
__device__ __forceinline__ float warp_max_nan(float v) {
  float m;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}
__device__ __forceinline__ float warp_min_f(float v) {
  float m;
  asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}
__device__ __forceinline__ float warp_max_f(float v) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

__device__ __forceinline__ float logit(const RouteParams& p, long long row, int e) {
  const long long i = row * p.stride + e;
  return p.f32 ? load_in(static_cast<const float*>(p.logits) + i)
               : bf16_bits_to_float(load_in(static_cast<const uint16_t*>(p.logits) + i));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// (A quick quotient, two units of the last place off where a rounded one is half of one: weights stay
// within the bound that w4_route states, and the choice does not hang on them.)
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.0f, 1.0f + expf(-x)); }

// exp(a - b), a <= b, b finite, with what the difference loses by its rounding: |a - b| 2^-24 of the
// result, which would be most of a small weight's error.  That rest is a number of its own (the
// error of a sum, by six additions), and exp(d + rest) = exp(d) (1 + rest) to 2^-34.  Off by 5 2^-24
// of the result: expf two units in the last place, the product half of one.
__device__ __forceinline__ float exp_of_difference(float a, float b) {
  const float d = a - b, back = d - a;
  const float rest = (a - (d - back)) - (b + back);
  const float f = expf(d);
  return d > -110.0f ? fmaf(f, rest, f) : f;   // (0 from there on; the rest of an infinite d is none)
}

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
    sm[e] = s + (p.bias != nullptr ? (double)load_in(p.bias + e) : 0.0);
  }
  __syncwarp();
  uint32_t in = kFull;   // chosen groups
  if (p.G > 1) {
    // by one logit alone where no sum is taken, as everywhere: scores that are 1 or 0 in 64 bits are
    // equal where their logits are not
    const bool by_logit = p.bias == nullptr && p.best == 1;
    double gs = -INFINITY;
    if (lane < p.G) {
      double a = -INFINITY, b = -INFINITY;
      for (int i = 0; i < p.size; ++i) {
        const int e = lane * p.size + i;
        const double c = by_logit ? (double)logit(p, row, e) : sm[e];
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

// 64-bit sum of a softmax's exponentials; 1 where no score needs it: a sigmoid, or scores that are
// compared without a bias (all have the same divisor).
__device__ __noinline__ double divisor(const RouteParams& p, long long row, float top) {
  if (p.sigmoid || p.bias == nullptr) return 1.0;
  double z = 0.0;
  for (int e = threadIdx.x & 31; e < p.E; e += 32) z += exp((double)logit(p, row, e) - (double)top);
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
  return z;
}

__device__ __forceinline__ double exact_score(const RouteParams& p, long long row, int e, float top,
                                              double z) {
  const double x = (double)logit(p, row, e);
  const double s = p.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - (double)top) / z;
  return p.bias != nullptr ? s + (double)load_in(p.bias + e) : s;
}

// Order of the first `cnt` candidates by 64-bit scores (without a bias by the logits), equal ones
// by number: lane j gives the expert e_j and gets the j-th.
__device__ __noinline__ int exact_order(const RouteParams& p, long long row, int e, int cnt, float top,
                                        int* sm) {
  const int lane = threadIdx.x & 31;
  const double z = divisor(p, row, top);
  double c = 0.0;
  if (lane < cnt)
    c = p.bias != nullptr ? exact_score(p, row, e, top, z) : (double)logit(p, row, e);
  int rank = 0;
  for (int j = 0; j < cnt; ++j) {
    const double o = __shfl_sync(kFull, c, j);
    const int oe = __shfl_sync(kFull, e, j);
    rank += o > c || (o == c && oe < e);
  }
  __syncwarp();
  if (lane < cnt) sm[rank] = e;
  __syncwarp();
  return lane < cnt ? sm[lane] : 0;
}

// Whether this lane's group is chosen, of groups whose 32-bit scores leave it open: those within
// `slack` of the border have their best experts' scores (`mine`: bits of this lane's that can be
// among them) added up in 64 bits, the others stand as they are.
__device__ __noinline__ bool exact_group(const RouteParams& p, long long row, int e0, uint32_t mine_lo,
                                         uint32_t mine_hi, float gs, bool in, float least, float next,
                                         float slack, float top) {
  const int lane = threadIdx.x & 31, g = lane >> p.shift;
  const bool open = g < p.G && gs < next + slack && gs > least - slack;
  const bool first = (lane & ((1 << p.shift) - 1)) == 0;
  const int left = p.top_groups - __popc(__ballot_sync(kFull, first && in && !open));
  const double z = divisor(p, row, top);
  double a = -INFINITY, b = -INFINITY;
  unsigned long long mask = open ? ((unsigned long long)mine_hi << 32) | mine_lo : 0ull;
  while (mask != 0) {
    const int i = __ffsll((long long)mask) - 1;
    mask &= mask - 1;
    const double c = exact_score(p, row, e0 + i, top, z);
    b = fmax(b, fmin(a, c));
    a = fmax(a, c);
  }
  for (int o = 1; o < (1 << p.shift); o <<= 1) {
    const double oa = __shfl_xor_sync(kFull, a, o), ob = __shfl_xor_sync(kFull, b, o);
    b = fmax(fmax(b, ob), fmin(a, oa));
    a = fmax(a, oa);
  }
  const double sum = p.best == 2 ? a + b : a;
  int rank = 0;
  for (int i = 0; i < p.G; ++i) {
    const double o = __shfl_sync(kFull, sum, i << p.shift);
    const bool there = __shfl_sync(kFull, (int)open, i << p.shift);
    rank += there && (o > sum || (o == sum && i < g));
  }
  return open ? rank < left : in;
}

template <int V>
struct Log2 {
  static constexpr int value = 1 + Log2<V / 2>::value;
};
template <>
struct Log2<1> {
  static constexpr int value = 0;
};

// Descending order of V words by a network (odd-even merges).
template <int V>
__device__ __forceinline__ void sort_down(uint32_t (&k)[V]) {
#pragma unroll
  for (int lp = 0; lp < Log2<V>::value; ++lp)
#pragma unroll
    for (int lq = lp; lq >= 0; --lq) {
      const int p = 1 << lp, q = 1 << lq, j = q % p;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i >= j && (i - j) % (2 * q) < q && i + q < V && i / (2 * p) == (i + q) / (2 * p)) {
          const uint32_t a = k[i], b = k[i + q];
          k[i] = max(a, b);
          k[i + q] = min(a, b);
        }
    }
}

// Rows first, first + step, ... below end, one after another; sm: this warp's room for 64-bit scores.
template <int V, bool F32>
__device__ __forceinline__ void route_rows(const RouteParams& p, long long first, long long step,
                                           long long end, double* sm) {
  constexpr int kPlace = V <= 8 ? 8 : 5 + Log2<V>::value;       // bits of a place
  constexpr int kBits = 32 - kPlace < 23 ? 32 - kPlace : 23;    // bits of a fixed-point score
  constexpr float kOne = (float)(1 << kBits), kBase = 8388608.0f;   // 2^23: the unit is 1
  constexpr bool kSorted = V <= 16;
  const int lane = threadIdx.x & 31;
  const int g = lane >> p.shift, l = lane & ((1 << p.shift) - 1);
  const int e0 = g * p.size + l * p.each;
  const int n = g < p.G ? min(max(p.size - l * p.each, 0), p.each) : 0;   // experts of this lane
  const bool biased = p.bias != nullptr, groups = p.G > 1;
  const bool sums = biased || (groups && p.best == 2);   // scores themselves are compared
  const bool fixed = biased || F32;                      // not the logits' own order
  const uint32_t places = (1u << kPlace) - 1;
  // biases above the least of them
  float b[V], range = 1.0f;
  bool bad_bias = false;
  if (biased) {
    float lo = INFINITY, hi = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      b[i] = i < n ? load_in(p.bias + e0 + i) : 0.0f;
      if (i < n) {
        bad_bias |= !isfinite(b[i]);
        lo = fminf(lo, b[i]);
        hi = fmaxf(hi, b[i]);
      }
    }
    bad_bias = __any_sync(kFull, bad_bias);
    lo = warp_min_f(lo);
    hi = warp_max_f(hi);
    range = 1.0f + (hi - lo);
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] -= lo;
  }
  const bool wide = !(range < 1e30f);   // no fixed point holds it
  const float unit = __fdividef(kOne - 8.0f, range);
  for (long long row = first; row < end; row += step) {
    float x[V];
    if (p.vec) {   // whole aligned vectors of four experts
      if constexpr (V >= 4) {
        if constexpr (F32) {
          const float4* src = reinterpret_cast<const float4*>(
              static_cast<const float*>(p.logits) + row * p.stride + e0);
#pragma unroll
          for (int i = 0; i < V / 4; ++i) {
            const float4 w = n > 0 ? load_in(src + i) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
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
            const uint2 w = n > 0 ? load_in(src + i) : make_uint2(0xFF80FF80u, 0xFF80FF80u);
            x[4 * i] = __uint_as_float(w.x << 16);
            x[4 * i + 1] = __uint_as_float(w.x & 0xFFFF0000u);
            x[4 * i + 2] = __uint_as_float(w.y << 16);
            x[4 * i + 3] = __uint_as_float(w.y & 0xFFFF0000u);
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = i < n ? logit(p, row, e0 + i) : -INFINITY;
    }
    float top = x[0];
#pragma unroll
    for (int i = 1; i < V; ++i) top = max_nan(top, x[i]);
    top = warp_max_nan(top);
    if (isnan(top) || (!p.sigmoid && isinf(top)) || bad_bias) {
      if (lane == 0) report(p.status, W4_ERR_VALUE);
      continue;
    }
    // Scores.  A sigmoid's error is below 2^-21 whatever its size (the exponential's argument
    // is off by |x| 2^-24, which s (1 - s) |x| < 0.23 holds down; quotient and sum add 2^-22); a
    // softmax's below 2^-18 of the largest (its sum adds (V + 5) 2^-24).  c: with the bias;
    // two of them differ by 2^-20 (or 2^-17 of the largest) and four roundings of 2^-24 of the
    // range more or less than they should.
    float z = 1.0f, tol = 0.0f, f1 = -INFINITY, f2 = -INFINITY;   // a lane's two best
    uint32_t key[V];
    float c[V];
    if (sums || (!p.renorm && !p.sigmoid)) {
      if (p.sigmoid) {
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = __fdividef(1.0f, 1.0f + __expf(-x[i]));
        tol = 0x1p-20f + 0x1p-22f * range;
      } else {
        z = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          c[i] = __expf(x[i] - top);
          z += c[i];
        }
        z = warp_sum(z);
        const float r = __fdividef(1.0f, z);
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] *= r;
        tol = 0x1p-17f * r + 0x1p-22f * range;
      }
      if (biased) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          c[i] += b[i];
          const float f = fmaf(c[i], unit, kBase + 4.0f);
          key[i] = (__float_as_uint(f) << kPlace) | (places - (lane * V + i));
        }
      }
      if (groups) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float v = i < n ? c[i] : -INFINITY;
          f2 = fmaxf(f2, fminf(f1, v));
          f1 = fmaxf(f1, v);
        }
      }
    }
    if (!biased) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (F32) {
          const float f = fmaxf(fmaf(x[i] - top, kOne / 32.0f, kBase + (kOne - 2.0f)), kBase + 1.0f);
          key[i] = (__float_as_uint(f) << kPlace) | (places - (lane * V + i));
        } else {
          key[i] = (order_key(x[i]) & 0xFFFF0000u) | (0xFFFFu - (lane * V + i));
        }
      }
    }
    bool close = wide;   // too many compared scores nearer than fp32 can tell
    bool in = true;      // whether this lane's group is chosen
    if (groups) {
      // the group's score in each of its lanes; one logit alone decides where no sum is taken
      float gs;
      if (sums) {
        for (int o = 1; o < (1 << p.shift); o <<= 1) {
          const float o1 = __shfl_xor_sync(kFull, f1, o), o2 = __shfl_xor_sync(kFull, f2, o);
          f2 = fmaxf(fmaxf(f2, o2), fminf(f1, o1));
          f1 = fmaxf(f1, o1);
        }
        gs = p.best == 2 ? f1 + f2 : f1;
      } else {
        gs = x[0];
#pragma unroll
        for (int i = 1; i < V; ++i) gs = fmaxf(gs, x[i]);
        for (int o = 1; o < (1 << p.shift); o <<= 1)
          gs = fmaxf(gs, __shfl_xor_sync(kFull, gs, o));
      }
      int rank = 0;
      for (int i = 0; i < p.G; ++i) {
        const float o = __shfl_sync(kFull, gs, i << p.shift);
        rank += o > gs || (o == gs && i < g);
      }
      in = g < p.G && rank < p.top_groups;
      if (sums) {
        const float least = warp_min_f(in ? gs : INFINITY);
        const float next = warp_max_f(in || g >= p.G ? -INFINITY : gs);
        if (least - next < 3.0f * tol && !wide) {
          uint32_t can[2] = {0, 0};
          const float from = (p.best == 2 ? f2 : f1) - tol;
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (i < n && c[i] >= from) can[i / 32] |= 1u << (i % 32);
          in = exact_group(p, row, e0, can[0], can[1], gs, in, least, next, 3.0f * tol, top);
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = in && i < n ? key[i] : 0u;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = i < n ? key[i] : 0u;
    }
    uint32_t mine = 0, my = 0, m = 0, kth = 0;
    if constexpr (kSorted) {
      sort_down<V>(key);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) mine = max(mine, key[i]);
    }
    auto pop = [&]() {   // the largest word of the warp, which is then gone
      if constexpr (kSorted) {
        m = __reduce_max_sync(kFull, key[0]);
        const bool hit = key[0] == m;
#pragma unroll
        for (int i = 0; i + 1 < V; ++i) key[i] = hit ? key[i + 1] : key[i];
        key[V - 1] = hit ? 0u : key[V - 1];
      } else {
        m = __reduce_max_sync(kFull, mine);
        if (mine == m) {
          mine = 0;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            key[i] = key[i] == m ? 0u : key[i];
            mine = max(mine, key[i]);
          }
        }
      }
    };
    int cnt = 0;
    for (; cnt < p.k; ++cnt) {
      pop();
      if (lane == cnt) my = m;
    }
    kth = m;
    uint32_t near = 0;
    if (fixed) {
      // Units that two scores can be apart and still be in the wrong order: their errors and the
      // rounding of the word.  Candidates are taken as far as the last one is clear of the k-th.
      near = 3 + (biased ? (uint32_t)fminf(tol * unit, kOne) : 1u);
      while (true) {
        pop();
        if (m == 0 || (kth >> kPlace) - (m >> kPlace) >= near) break;
        if (cnt == 32) {
          // still none: experts of the k-th one's own inputs have its score, and are in order already
          const uint32_t kp = places - (kth & places);
          const int kl = (int)(kp / V);
          const int ek = (kl >> p.shift) * p.size + (kl & ((1 << p.shift) - 1)) * p.each + (int)(kp % V);
          const float xk = logit(p, row, ek), bk = biased ? load_in(p.bias + ek) : 0.0f;
          bool other = false;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float f = biased ? fmaf(c[i], unit, kBase + 4.0f)
                                   : fmaxf(fmaf(x[i] - top, kOne / 32.0f, kBase + (kOne - 2.0f)), kBase + 1.0f);
            const int far = (int)((__float_as_uint(f) << kPlace) >> kPlace) - (int)(kth >> kPlace);
            if (in && i < n && (uint32_t)abs(far) < near && !(x[i] == xk && (!biased || load_in(p.bias + e0 + i) == bk)))
              other = true;
          }
          close |= __any_sync(kFull, other);
          break;
        }
        if (lane == cnt) my = m;
        ++cnt;
      }
    }
    // lane j's candidate
    const uint32_t place = (fixed ? places : 0xFFFFu) - (my & (fixed ? places : 0xFFFFu));
    const int pl = (int)(place / V), pi = (int)(place % V);
    int e = (pl >> p.shift) * p.size + (pl & ((1 << p.shift) - 1)) * p.each + pi;
    float xl = lane < cnt ? logit(p, row, e) : -INFINITY;
    if (fixed) {
      // equal inputs are equal scores at any width, and in order already
      const float bl = biased && lane < cnt ? load_in(p.bias + e) : 0.0f;
      const uint32_t up = __shfl_up_sync(kFull, my, 1);
      const float xu = __shfl_up_sync(kFull, xl, 1), bu = __shfl_up_sync(kFull, bl, 1);
      const bool unsure = lane > 0 && lane < cnt && (up >> kPlace) - (my >> kPlace) < near &&
                          !(xu == xl && bu == bl);
      if (close || __any_sync(kFull, unsure)) {
        e = close ? refine(p, row, sm) : exact_order(p, row, e, cnt, top, reinterpret_cast<int*>(sm));
        xl = lane < p.k ? logit(p, row, e) : -INFINITY;
      }
    }
    // weights: relative to the largest chosen logit where they are divided by their sum, so that
    // small scores do not vanish
    const bool has = lane < p.k;
    if (!has) xl = -INFINITY;
    float w;
    if (p.renorm) {
      float t = warp_max_f(xl);
      if (p.sigmoid) t = fminf(t, 0.0f);
      w = xl > -INFINITY ? (p.sigmoid && t == 0.0f ? sigmoid(xl) : exp_of_difference(xl, t)) : 0.0f;
      if (p.sigmoid && t < 0.0f) w = __fdividef(w, 1.0f + expf(xl));
      const float sum = warp_sum(w);
      w = sum > 0.0f ? p.scale * __fdividef(w, sum) : 0.0f;
    } else {
      w = p.scale * (p.sigmoid ? sigmoid(xl) : __fdividef(exp_of_difference(xl, top), z));
    }
    if (has) {
      p.ids[row * p.k + lane] = e;
      p.weights[row * p.k + lane] = w;
    }
  }
}

template <int V, bool F32>
__global__ void __launch_bounds__(32 * kRouteWarps, V <= 8 ? 8 : 1) route_kernel(const __grid_constant__ RouteParams p) {
  extern __shared__ double refine_sm[];
  pdl_wait();
  const int warp = threadIdx.x >> 5;
  route_rows<V, F32>(p, (long long)blockIdx.x * kRouteWarps + warp, (long long)gridDim.x * kRouteWarps, p.rows,
                     refine_sm + warp * (p.E > 32 ? p.E : 32));
}

template <int V, bool F32>
__device__ __noinline__ void route_again(const RouteParams& p, long long row, double* sm) {
  route_rows<V, F32>(p, row, 1, row + 1, sm);
}

// A 64-bit score that needs no other expert's: with a sigmoid, or without a bias, where a softmax's
// common divisor changes no comparison.  One copy of the code, which few calls run.
__device__ __noinline__ double exact_alone(const RouteParams& p, long long row, int e, float top) {
  return exact_score(p, row, e, top, 1.0);
}

// Four tokens a warp, eight lanes each with V neighbouring experts: what a warp does for one token
// it does here for four.  A lane keeps its best eight words, sorted.  Scores too near each other are
// compared in 64 bits by the lanes that have them, all at once, since a token that takes long is what
// the call's end waits for; whatever this cannot settle (a NaN, a softmax with a bias, too many of
// them, a lane whose eight were all taken) is left to route_rows.
constexpr int kManyWarps = 4;
constexpr int kManyRows = 4096;   // tokens from which on it is the faster one, for any experts and groups

template <int V, bool F32>
__global__ void __launch_bounds__(32 * kManyWarps) route_many_kernel(const __grid_constant__ RouteParams p) {
  extern __shared__ double refine_sm[];
  __shared__ float4 bias_sm[8 * V / 4];   // biases above the least: vector i of lane l at 8 i + l
  __shared__ float ends_sm[2 * kManyWarps];
  constexpr float kOne = 8388608.0f, kBase = 8388608.0f;   // 23 bits of a score, 8 of a place
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & 7;
  const int g = l >> p.shift8;
  const bool biased = p.bias != nullptr, groups = p.G > 1;
  const bool sums = biased || (groups && p.best == 2);
  const bool fixed = biased || F32;
  float range = 1.0f;
  bool again = false;
  if (biased) {
    float lo = INFINITY, hi = -INFINITY;
    bool bad = false;
    for (int e = threadIdx.x; e < 8 * V; e += 32 * kManyWarps) {
      const float v = load_in(p.bias + e);
      bad |= !isfinite(v);
      lo = fminf(lo, v);
      hi = fmaxf(hi, v);
    }
    lo = warp_min_f(lo);
    hi = warp_max_f(hi);
    if (lane == 0) {
      ends_sm[warp] = lo;
      ends_sm[kManyWarps + warp] = hi;
    }
    again = __syncthreads_or(bad);
    for (int i = 0; i < kManyWarps; ++i) {
      lo = fminf(lo, ends_sm[i]);
      hi = fmaxf(hi, ends_sm[kManyWarps + i]);
    }
    for (int e = threadIdx.x; e < 8 * V; e += 32 * kManyWarps)
      reinterpret_cast<float*>(bias_sm + (e % V / 4 * 8 + e / V))[e % 4] = load_in(p.bias + e) - lo;
    __syncthreads();
    range = 1.0f + (hi - lo);
    again |= !(range < 1e30f);
  }
  const float unit = __fdividef(kOne - 8.0f, range);
  const long long steps = ((long long)p.rows + 3) / 4;
  for (long long r4 = (long long)blockIdx.x * kManyWarps + warp; r4 < steps; r4 += (long long)gridDim.x * kManyWarps) {
    const long long row = min(4 * r4 + (lane >> 3), (long long)p.rows - 1);
    float x[V];
    if constexpr (F32) {
      const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(p.logits) + row * p.stride + l * V);
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        const float4 w = load_in(src + i);
        x[4 * i] = w.x;
        x[4 * i + 1] = w.y;
        x[4 * i + 2] = w.z;
        x[4 * i + 3] = w.w;
      }
    } else {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.logits) + row * p.stride + l * V);
#pragma unroll
      for (int i = 0; i < V / 8; ++i) {
        const uint4 w = load_in(src + i);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          x[8 * i + 2 * z] = __uint_as_float(u[z] << 16);
          x[8 * i + 2 * z + 1] = __uint_as_float(u[z] & 0xFFFF0000u);
        }
      }
    }
    float top = x[0];
#pragma unroll
    for (int i = 1; i < V; ++i) top = max_nan(top, x[i]);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = max_nan(top, __shfl_xor_sync(kFull, top, o));
    bool redo = again || isnan(top) || (!p.sigmoid && isinf(top));
    const bool alone = p.sigmoid || !biased;
    float z = 1.0f, tol = 0.0f, f1 = -INFINITY, f2 = -INFINITY;
    uint32_t key[V];
    if (sums || (!p.renorm && !p.sigmoid)) {   // errors as in route_rows
      float scale = 1.0f;
      if (p.sigmoid) {
        tol = 0x1p-20f + 0x1p-22f * range;
      } else {
        float part[4] = {};   // summed in the order of 32 lanes, a quarter of this one's experts each
#pragma unroll
        for (int i = 0; i < V; ++i) part[i / (V / 4)] += __expf(x[i] - top);
#pragma unroll
        for (int o = 4; o >= 1; o >>= 1)
#pragma unroll
          for (int q = 0; q < 4; ++q) part[q] += __shfl_xor_sync(kFull, part[q], o);
        z = (part[0] + part[2]) + (part[1] + part[3]);
        scale = __fdividef(1.0f, z);
        tol = 0x1p-17f * scale + 0x1p-22f * range;
      }
      if (sums) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
          float4 b = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (biased) b = bias_sm[8 * i + l];
          const float add[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int at = 4 * i + y;
            const float s = p.sigmoid ? __fdividef(1.0f, 1.0f + __expf(-x[at])) : __expf(x[at] - top) * scale;
            const float c = s + add[y];
            f2 = fmaxf(f2, fminf(f1, c));
            f1 = fmaxf(f1, c);
            key[at] = (__float_as_uint(fmaf(c, unit, kBase + 4.0f)) << 8) | (255 - (l * V + at));
          }
        }
      }
    }
    if (!biased) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (F32) {
          const float f = fmaxf(fmaf(x[i] - top, kOne / 32.0f, kBase + (kOne - 2.0f)), kBase + 1.0f);
          key[i] = (__float_as_uint(f) << 8) | (255 - (l * V + i));
        } else {
          key[i] = (order_key(x[i]) & 0xFFFF0000u) | (0xFFFFu - (l * V + i));
        }
      }
    }
    // the lane's best eight, sorted: eights sorted, and of two the better half sorted again
#pragma unroll
    for (int q = 0; q < V / 8; ++q) sort_down<8>(reinterpret_cast<uint32_t(&)[8]>(key[8 * q]));
#pragma unroll
    for (int q = 1; q < V / 8; ++q) {
#pragma unroll
      for (int i = 0; i < 8; ++i) key[i] = max(key[i], key[8 * q + 7 - i]);
#pragma unroll
      for (int d = 4; d >= 1; d >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if ((i & d) == 0) {
            const uint32_t a = key[i], c = key[i + d];
            key[i] = max(a, c);
            key[i + d] = min(a, c);
          }
    }
    const uint32_t near = 3 + (biased ? (uint32_t)fminf(tol * unit, kOne) : 1u);
    const uint32_t low = fixed ? 255u : 0xFFFFu;   // bits of a place
    if (groups) {
      float gs;
      if (sums) {
        for (int o = 1; o < (1 << p.shift8); o <<= 1) {
          const float o1 = __shfl_xor_sync(kFull, f1, o), o2 = __shfl_xor_sync(kFull, f2, o);
          f2 = fmaxf(fmaxf(f2, o2), fminf(f1, o1));
          f1 = fmaxf(f1, o1);
        }
        gs = p.best == 2 ? f1 + f2 : f1;
      } else {
        gs = x[0];
#pragma unroll
        for (int i = 1; i < V; ++i) gs = fmaxf(gs, x[i]);
        for (int o = 1; o < (1 << p.shift8); o <<= 1) gs = fmaxf(gs, __shfl_xor_sync(kFull, gs, o));
      }
      int rank = 0;
      float nearest = INFINITY;
      for (int i = 0; i < p.G; ++i) {
        const float o = __shfl_sync(kFull, gs, (lane & 24) | (i << p.shift8));
        rank += o > gs || (o == gs && i < g);
        nearest = i == g ? nearest : fminf(nearest, fabsf(o - gs));
      }
      // a group at the border and another too near it: all groups again, by the 64-bit scores of each
      // lane's three best words, among which its two best experts are
      const bool open = sums && (rank == p.top_groups || rank == p.top_groups - 1) && nearest < 3.0f * tol;
      const uint32_t rows_open = __ballot_sync(kFull, open && !redo);
      if (rows_open != 0) {
        const bool mine = ((rows_open >> (lane & 24)) & 255u) != 0;
        redo |= mine && (!alone || (fixed && key[3] != 0 && (key[1] >> 8) - (key[3] >> 8) < near));
        double a = -INFINITY, b = -INFINITY;
        for (int i = 0; i < 3; ++i) {
          const uint32_t word = i == 0 ? key[0] : i == 1 ? key[1] : key[2];
          const double c = exact_alone(p, row, min((int)(low - (word & low)), p.E - 1), top);
          b = fmax(b, fmin(a, c));
          a = fmax(a, c);
        }
        for (int o = 1; o < (1 << p.shift8); o <<= 1) {
          const double oa = __shfl_xor_sync(kFull, a, o), ob = __shfl_xor_sync(kFull, b, o);
          b = fmax(fmax(b, ob), fmin(a, oa));
          a = fmax(a, oa);
        }
        const double sum = p.best == 2 ? a + b : a;
        int exact_rank = 0;
        for (int i = 0; i < p.G; ++i) {
          const double o = __shfl_sync(kFull, sum, (lane & 24) | (i << p.shift8));
          exact_rank += o > sum || (o == sum && i < g);
        }
        rank = mine ? exact_rank : rank;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) key[i] = rank < p.top_groups ? key[i] : 0u;
    }
    uint32_t my = 0, m = 0;
    int taken = 0;
    auto pop = [&]() {
      m = key[0];
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
      const bool hit = key[0] == m;
      taken += hit;
#pragma unroll
      for (int i = 0; i < 7; ++i) key[i] = hit ? key[i + 1] : key[i];
      key[7] = hit ? 0u : key[7];
    };
    for (int j = 0; j < p.k; ++j) {
      pop();
      my = l == j ? m : my;
    }
    int e = min((int)(low - (my & low)), p.E - 1);   // (none left: redone)
    const bool has = l < p.k;
    float xl = has ? logit(p, row, e) : -INFINITY;
    if (fixed) {
      const uint32_t kth = m;
      pop();
      redo |= m != 0 && (kth >> 8) - (m >> 8) < near;   // the best left out is too near the last chosen
      const float bl = biased && has ? load_in(p.bias + e) : 0.0f;
      const uint32_t up = __shfl_up_sync(kFull, my, 1, 8);
      const float xu = __shfl_up_sync(kFull, xl, 1, 8), bu = __shfl_up_sync(kFull, bl, 1, 8);
      const bool unsure = l > 0 && has && (up >> 8) - (my >> 8) < near && !(xu == xl && bu == bl);
      redo |= unsure && !alone;
      // a row's chosen experts in the order of their 64-bit scores (without a bias of the logits)
      const uint32_t who = __ballot_sync(kFull, unsure && !redo);
      if (who != 0) {
        const bool mine = ((who >> (lane & 24)) & 255u) != 0;
        const double c = biased ? exact_alone(p, row, e, top) : (double)xl;
        int rank = 0;
        for (int i = 0; i < p.k; ++i) {
          const double o = __shfl_sync(kFull, c, (lane & 24) | i);
          const int oe = __shfl_sync(kFull, e, (lane & 24) | i);
          rank += o > c || (o == c && oe < e);
        }
        int to = e;
        float xto = xl;
        for (int i = 0; i < p.k; ++i) {
          const int place = __shfl_sync(kFull, rank, (lane & 24) | i);
          const int oe = __shfl_sync(kFull, e, (lane & 24) | i);
          const float ox = __shfl_sync(kFull, xl, (lane & 24) | i);
          if (mine && has && place == l) {
            to = oe;
            xto = ox;
          }
        }
        e = to;
        xl = xto;
      }
    }
    redo |= V > 8 && taken >= 8;   // its ninth may belong among them
    float w;
    if (p.renorm) {
      float t = xl;
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) t = fmaxf(t, __shfl_xor_sync(kFull, t, o));
      if (p.sigmoid) t = fminf(t, 0.0f);
      w = xl > -INFINITY ? (p.sigmoid && t == 0.0f ? sigmoid(xl) : exp_of_difference(xl, t)) : 0.0f;
      if (p.sigmoid && t < 0.0f) w = __fdividef(w, 1.0f + expf(xl));
      float sum = w;
#pragma unroll
      for (int o = 4; o >= 1; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);   // as 32 lanes do
      w = sum > 0.0f ? p.scale * __fdividef(w, sum) : 0.0f;
    } else {
      w = p.scale * (p.sigmoid ? sigmoid(xl) : __fdividef(exp_of_difference(xl, top), z));
    }
    const uint32_t undone = __ballot_sync(kFull, redo && 4 * r4 + (lane >> 3) < p.rows);
    if (has && 4 * r4 + (lane >> 3) < p.rows && ((undone >> (lane & 24)) & 255u) == 0) {
      p.ids[row * p.k + l] = e;
      p.weights[row * p.k + l] = w;
    }
    if (undone != 0)
      for (int q = 0; q < 4; ++q)
        if (((undone >> (8 * q)) & 255u) != 0)
          route_again<V / 4, F32>(p, 4 * r4 + q, refine_sm + warp * p.E);
  }
}

// ---------------------------------------------------------------- combine
// Eight columns a thread, its token's k rows all on their way at once: HBM bounds it.  4001 tokens'
// 8 rows of 2816 and one added: 34.5 us, 6.55 TB/s (a copy: 6.65).
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
  pdl_wait();
  const long long row = blockIdx.x / p.chunks;
  const int chunk = blockIdx.x % p.chunks;
  const long long n = ((long long)chunk * kCombineThreads + threadIdx.x) * VEC;
  const float* wt = p.weights + row * p.k;
  if (p.ids != nullptr) {
    bool ok = true;
    for (int j = 0; j < p.k; ++j) {
      const int id = load_in(p.ids + row * p.k + j);
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
        v[z] = load_in(reinterpret_cast<const uint4*>(y + (long long)(j + z) * p.N));
#pragma unroll
      for (int z = 0; z < 8; ++z) {
        float f[8];
        spread(v[z], f);
        const float w = load_in(wt + j + z);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, f[i], acc[i]);
      }
    }
#pragma unroll 2
    for (; j < p.k; ++j) {
      float f[8];
      spread(load_in(reinterpret_cast<const uint4*>(y + (long long)j * p.N)), f);
      const float w = load_in(wt + j);
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
      acc[0] = fmaf(load_in(wt + j), __bfloat162float(load_in(y + (long long)j * p.N)), acc[0]);
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
  p.G = r.top_groups == r.groups ? 1 : r.groups;   // every group in: as without groups
  p.size = r.experts / p.G;
  p.top_groups = r.top_groups;
  p.best = p.size == 1 ? 1 : r.group_best;
  p.sigmoid = r.score == W4_ROUTE_SIGMOID;
  p.renorm = r.renorm != 0;
  p.f32 = logits_type == W4_TYPE_F32;
  p.scale = r.scale;
  p.status = status_dev;
  while ((32 >> p.shift) > p.G && p.shift < 5) ++p.shift;
  if ((32 >> p.shift) < p.G) --p.shift;
  p.each = (p.size + (1 << p.shift) - 1) >> p.shift;
  // room for the 64-bit scores, where such may be needed
  const bool fixed = bias != nullptr || p.f32;
  const size_t smem = fixed ? (size_t)kRouteWarps * (p.E > 32 ? p.E : 32) * sizeof(double) : 0;
  // a warp's rows share what it makes of the biases: at most the CTAs that are resident together
  // (8 an SM by their registers; 6 or 12 an SM with theirs, or a CTA for every four rows, were
  // 18 to 22 us where this is 18.5: 16384 tokens, 256 experts in 8 groups, biases)
  const long long ctas = ((long long)rows + kRouteWarps - 1) / kRouteWarps;
  const unsigned grid = (unsigned)(ctas < 152 * 8 ? ctas : 152 * 8);
  auto go = [&](auto bf16, auto f32, int v) {
    p.vec = v >= 4 && p.each == v && p.size == v << p.shift && !kv8::misaligned(logits, 16) &&
            row_stride * el % 16 == 0;
    return p.f32 ? kv8::launch(f32, dim3(grid), 32 * kRouteWarps, smem, stream, p)
                 : kv8::launch(bf16, dim3(grid), 32 * kRouteWarps, smem, stream, p);
  };
  // Many tokens over experts that eight lanes hold in whole vectors: half the instructions a token,
  // a quarter of the warps (16384 tokens 20 -> 16 us over 256 experts in groups with biases,
  // 7.9 -> 5.6 us over 128 without; 4096 tokens 8.4 to 9.9 -> 7.6 to 8.8 and 3.2 -> 2.75; 3000 of them
  // 7.0 -> 8.8 and 2.65 -> 2.7; 500 of them 3.1 -> 8.5 and 2.1 -> 2.5).
  if (rows >= kManyRows && p.k <= 8 && (p.E == 256 || p.E == 128 || p.E == 64) && (p.G & (p.G - 1)) == 0 && p.G <= 8 &&
      !kv8::misaligned(logits, 16) && row_stride * el % 16 == 0) {
    while ((8 >> p.shift8) > p.G) ++p.shift8;
    // a lane's eight words are too few where one lane holds all that can be chosen
    if (p.k < 8 || p.G == 1 || p.top_groups << p.shift8 > 1) {
      p.vec = p.each % 4 == 0;   // for the rows that are left to route_rows
      const long long steps = ((long long)rows + 3) / 4, most = ((steps + kManyWarps - 1) / kManyWarps);
      const unsigned many = (unsigned)(most < 152 * 6 ? most : 152 * 6);
      const size_t room = (size_t)kManyWarps * p.E * sizeof(double);
      auto run = [&](auto bf16, auto f32) {
        return p.f32 ? kv8::launch(f32, dim3(many), 32 * kManyWarps, room, stream, p)
                     : kv8::launch(bf16, dim3(many), 32 * kManyWarps, room, stream, p);
      };
      if (p.E == 64) return run(route_many_kernel<8, false>, route_many_kernel<8, true>);
      if (p.E == 128) return run(route_many_kernel<16, false>, route_many_kernel<16, true>);
      return run(route_many_kernel<32, false>, route_many_kernel<32, true>);
    }
  }
  if (p.each <= 1) return go(route_kernel<1, false>, route_kernel<1, true>, 1);
  if (p.each <= 2) return go(route_kernel<2, false>, route_kernel<2, true>, 2);
  if (p.each <= 4) return go(route_kernel<4, false>, route_kernel<4, true>, 4);
  if (p.each <= 8) return go(route_kernel<8, false>, route_kernel<8, true>, 8);
  if (p.each <= 16) return go(route_kernel<16, false>, route_kernel<16, true>, 16);
  if (p.each <= 32) return go(route_kernel<32, false>, route_kernel<32, true>, 32);
  return go(route_kernel<64, false>, route_kernel<64, true>, 64);
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
