// The clipped policy loss of a token, or of two at once, and sums over tokens.
#pragma once
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/seqsum.h"
#include "places.h"
#include "row_slice.cuh"

namespace sq {
namespace loss {

// ---- arithmetic on one float or on two (an instruction for both, each rounded as by itself)

struct Two {
  uint64_t v;
};
__device__ __forceinline__ Two two(float a, float b) { return {row::pair(a, b)}; }
// The assembler joins a packed product and a packed sum of it into one operation,
// rounded once, whatever the flags say (1 + 2^-12 squared less 1 + 2^-11 gave 2^-24).
// A product is a sum with -0 here, which it cannot know to be that.
static __constant__ float2 kMinusZero = {-0.0f, -0.0f};
template <typename V>
__device__ __forceinline__ V splat(float a);
template <>
__device__ __forceinline__ float splat<float>(float a) { return a; }
template <>
__device__ __forceinline__ Two splat<Two>(float a) { return two(a, a); }
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float sub(float a, float b) { return a - b; }
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ float fma(float a, float b, float c) { return __fmaf_rn(a, b, c); }
__device__ __forceinline__ Two add(Two a, Two b) { return {row::add2(a.v, b.v)}; }
__device__ __forceinline__ Two sub(Two a, Two b) {
  Two r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two fma(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ Two mul(Two a, Two b) { return fma(a, b, two(kMinusZero.x, kMinusZero.y)); }
// f of each
template <typename F>
__device__ __forceinline__ float each(float a, F f) { return f(a); }
template <typename F>
__device__ __forceinline__ Two each(Two a, F f) {
  float x, y;
  row::split(a.v, x, y);
  return two(f(x), f(y));
}
// conditions on each
struct Both {
  bool x, y;
};
template <typename F>
__device__ __forceinline__ bool test(float a, F f) { return f(a); }
template <typename F>
__device__ __forceinline__ Both test(Two a, F f) {
  float x, y;
  row::split(a.v, x, y);
  return {f(x), f(y)};
}
__device__ __forceinline__ bool either(bool a, bool b) { return a || b; }
__device__ __forceinline__ Both either(Both a, Both b) { return {a.x || b.x, a.y || b.y}; }
__device__ __forceinline__ bool unless(bool a, bool b) { return a && !b; }
__device__ __forceinline__ Both unless(Both a, Both b) { return {a.x && !b.x, a.y && !b.y}; }
__device__ __forceinline__ bool all(bool a) { return a; }
__device__ __forceinline__ bool all(Both a) { return a.x && a.y; }
__device__ __forceinline__ float pick(bool c, float a, float b) { return c ? a : b; }
__device__ __forceinline__ Two pick(Both c, Two a, Two b) {
  float ax, ay, bx, by;
  row::split(a.v, ax, ay);
  row::split(b.v, bx, by);
  return two(c.x ? ax : bx, c.y ? ay : by);
}

// A sum in two floats: each addition's rounding error is found exactly (Knuth,
// The Art of Computer Programming 2, 4.2.2) and kept in lo, so the sum of n
// numbers is off by some n 2^-48 of the sum of their magnitudes.  (fp64
// additions would do, but this GPU has one fp64 lane for 64 of fp32: six sums
// over 2 M tokens take the whole GPU 20 us.)  While hi is finite so is lo.
struct Sum {
  float hi = 0.0f, lo = 0.0f;
  __device__ __forceinline__ void add(float x) {
    const float s = hi + x, b = s - hi;
    lo += (hi - (s - b)) + (x - b);
    hi = s;
  }
  __device__ __forceinline__ void add(Sum o) {
    add(o.hi);
    lo += o.lo;
  }
  __device__ __forceinline__ float nearest() const { return fabsf(hi) < INFINITY ? hi + lo : hi; }
};
// Two of them.
struct TwoSums {
  Two hi = {0}, lo = {0};
  __device__ __forceinline__ void add(Two x) {
    const Two s = loss::add(hi, x), b = sub(s, hi);
    lo = loss::add(lo, loss::add(sub(hi, sub(s, b)), sub(x, b)));
    hi = s;
  }
  __device__ __forceinline__ void get(Sum &a, Sum &b) const {
    row::split(hi.v, a.hi, b.hi);
    row::split(lo.v, a.lo, b.lo);
  }
};
// of N neighbouring lanes, the same tree in every one
template <int N = 32>
__device__ __forceinline__ Sum warp_add(Sum v) {
#pragma unroll
  for (int o = N / 2; o; o >>= 1) {
    Sum w;
    w.hi = __shfl_xor_sync(~0u, v.hi, o), w.lo = __shfl_xor_sync(~0u, v.lo, o);
    // (the smaller lane's first: x + y and y + x differ in their errors' roundings)
    const bool up = threadIdx.x & o;
    Sum a = up ? w : v;
    a.add(up ? v : w);
    v = a;
  }
  return v;
}

// A bound on ln(ratio) in two floats: near = the nearest float, rest = what is left.
struct Bound {
  float near, rest;
};
struct Policy {
  const float *old_logps, *advantages, *weights, *ref_logps;
  float up, down, top;              // bounds of the ratio, and what these floats leave of them
  float up_rest, down_rest, top_rest;
  Bound ln_up, ln_down, ln_top;     // their logarithms
  float kl_coef, entropy_coef, inv_temperature;
};

// e^x - 1 - x, m = e^x - 1 and r = e^x.  For |x| < 1 by its series (the first term
// left out is 2 / 13! of the sum), where none loses digits to a difference, and r
// comes with what its rounding and m's left out; elsewhere without inf - inf, and r
// is far(r).
template <typename V, typename F>
__device__ __forceinline__ V excess(V x, V &m, V &r, V &r_rest, F far) {
  V p = splat<V>(1.0f / 479001600.0f);
  p = fma(p, x, splat<V>(1.0f / 39916800.0f));
  p = fma(p, x, splat<V>(1.0f / 3628800.0f));
  p = fma(p, x, splat<V>(1.0f / 362880.0f));
  p = fma(p, x, splat<V>(1.0f / 40320.0f));
  p = fma(p, x, splat<V>(1.0f / 5040.0f));
  p = fma(p, x, splat<V>(1.0f / 720.0f));
  p = fma(p, x, splat<V>(1.0f / 120.0f));
  p = fma(p, x, splat<V>(1.0f / 24.0f));
  p = fma(p, x, splat<V>(1.0f / 6.0f));
  p = fma(p, x, splat<V>(0.5f));
  const V one = splat<V>(1.0f);
  V k = mul(mul(x, x), p);
  m = add(x, k), r = add(one, m);
  r_rest = add(add(sub(one, r), m), add(sub(x, m), k));   // (|k| < |x|, |m| < 2)
  const auto near = test(x, [](float v) { return fabsf(v) < 1.0f; });
  if (!all(near)) {
    m = pick(near, m, each(x, [](float v) { return expm1f(v); }));
    r = pick(near, r, far(each(x, [](float v) { return expf(v); })));
    r_rest = pick(near, r_rest, splat<V>(0.0f));
    k = pick(near, k, sub(m, each(x, [](float v) { return fminf(v, 3.40282347e38f); })));
  }
  return k;
}

// A used token's terms, each before its weight.
template <typename V>
struct Terms {
  V policy, policy_rest;        // the term's nearest float, and what it leaves
  V kl, past, old_kl;           // past: 1 where the ratio is past its bound
  V slope;                      // of policy + kl_coef * kl by logp
};

// The ratio's side of a bound is that of the exact difference of the two
// log-probabilities, which its nearest float d and the error of that, e, are: the
// difference of d and a float within twice of it is exact, and elsewhere e and the
// bound's rest are too small to matter.
template <typename V>
__device__ __forceinline__ Terms<V> policy_terms(const Policy &p, V logp, V old, V advantage, V ref) {
  const V zero = splat<V>(0.0f), d = sub(logp, old), b = sub(d, logp),
          e = pick(test(d, [](float v) { return fabsf(v) < INFINITY; }), sub(sub(logp, sub(d, b)), add(old, b)), zero);
  const auto gain = test(advantage, [](float v) { return v >= 0.0f; });
  const auto positive = [](float v) { return v > 0.0f; };
  auto of = [&](float with_gain, float without) { return pick(gain, splat<V>(with_gain), splat<V>(without)); };
  const auto above = test(add(sub(d, of(p.ln_up.near, p.ln_top.near)), sub(e, of(p.ln_up.rest, p.ln_top.rest))), positive);
  const auto below = unless(test(add(sub(splat<V>(p.ln_down.near), d), sub(splat<V>(p.ln_down.rest), e)), positive), gain);
  const auto past = either(above, below);
  Terms<V> t;
  V m, ratio, ratio_rest;
  t.old_kl = excess(d, m, ratio, ratio_rest, [&](V r) {
    // an advantage of 0 leaves nothing of a ratio beyond fp32 either, where no bound has met that
    return pick(unless(test(r, [](float v) { return v == INFINITY; }), test(advantage, [](float v) { return v != 0.0f; })),
                splat<V>(3.40282347e38f), r);
  });
  const V f = pick(past, pick(below, splat<V>(p.down), of(p.up, p.top)), ratio),
          f_rest = pick(past, pick(below, splat<V>(p.down_rest), of(p.up_rest, p.top_rest)), fma(ratio, e, ratio_rest));
  const V loss = sub(zero, advantage);
  t.policy = mul(loss, f);
  t.policy_rest = add(fma(loss, f, sub(zero, t.policy)), mul(loss, f_rest));
  t.slope = pick(past, zero, mul(loss, ratio));
  t.past = pick(past, splat<V>(1.0f), zero);
  t.kl = zero;
  if (p.ref_logps) {
    V unused;
    t.kl = excess(sub(ref, logp), m, unused, unused, [](V r) { return r; });
    if (p.kl_coef != 0.0f) t.slope = sub(t.slope, mul(splat<V>(p.kl_coef), m));
  }
  return t;
}

// A kernel that may begin while the one before it ends (it waits for that with
// griddepcontrol.wait before it reads anything).
template <typename Args>
inline cudaError_t launch_after(void (*kernel)(Args), const Args &args, int64_t ctas, int threads, int cluster, bool after,
                                cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  if (cluster > 1) {
    at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    at[cfg.numAttrs].val.clusterDim.x = cluster;
    at[cfg.numAttrs].val.clusterDim.y = at[cfg.numAttrs].val.clusterDim.z = 1;
    cfg.numAttrs++;
  }
  if (after) {
    at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs++;
  }
  cfg.attrs = at;
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

constexpr int64_t kClusterTokens = 65536;   // whose sums one cluster takes, without scratch
// The settings, checked; false: refused.
bool take_policy(const seqsum_policy *from, int64_t n, bool rows, Policy *to);
// The loss and its statistics over n tokens from their log-probabilities, after the kernel that writes those.  tokens:
// null, or the tokens of rows of `vocab` logits.
int sum_policy(const Policy &policy, const float *logps, const float *entropies, const int64_t *tokens, int64_t vocab,
               int64_t n, float *loss, float *stats, void *scratch, bool after, cudaStream_t stream);

}  // namespace loss
}  // namespace sq
