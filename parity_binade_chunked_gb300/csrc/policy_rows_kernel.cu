// The clipped policy loss from rows of logits, and the logits' gradient
// (seqsum_token_policy_grad): the rows in one read, then the loss over tokens.
//
// For a row, with c = log2(e) / T, m its maximum, d_i = (x_i - m) c:
//   s = sum 2^d_i,  q = sum 2^d_i d_i
//   logp = (x_t - m) / T - ln s,  H = ln s - ln 2 q / s
//   g = w (slope of the token's loss by logp),  b = w entropy_coef
//   d logits_i = 2^d_i (c0 + c1 d_i) + [i = t] g / T
//     c0 = (b (H - ln s) - g) / (s T),  c1 = b ln 2 / (s T)
// A row's vectors are cut into segments as those of the log-probabilities are:
// its results go by its numbers and its address modulo 16 alone.
#include <atomic>
#include <type_traits>

#include "policy_terms.cuh"
#include "row_exp.cuh"

namespace sq {
namespace {

using namespace row;

constexpr float kLn2 = 0.693147181f;
// Octaves below the maximum at which 2^d is 0 whatever it is multiplied with; a masked place (d = -inf) counts as there.
constexpr float kFar = -200.0f;
constexpr float kMost = 1e38f;   // well inside fp32

struct RowsArgs {
  const void *logits;
  int64_t rows, stride;
  int32_t vocab;
  const int64_t *tokens;
  loss::Policy policy;
  float *logps, *entropies;
  void *dlogits;
  int64_t dstride;
  int32_t steps;       // that a CTA takes of a row at most
  Waits waits;
};

// x - base of a vector's numbers in pairs, each rounded once.
template <typename T>
struct Differences;
template <>
struct Differences<float> {
  __device__ __forceinline__ static void of(uint4 w, float base, uint64_t *d) {
    const uint64_t b = pair(-base, -base);
    d[0] = add2(pair(__uint_as_float(w.x), __uint_as_float(w.y)), b);
    d[1] = add2(pair(__uint_as_float(w.z), __uint_as_float(w.w)), b);
  }
};
// 16-bit numbers go into the subtraction as they are (that saves the
// instructions that would unpack them: a third of these for fp16).
template <>
struct Differences<__nv_bfloat16> {
  __device__ __forceinline__ static float one(uint32_t h, float base) {
    float d;
    asm("sub.rn.f32.bf16 %0, %1, %2;" : "=f"(d) : "h"((uint16_t)h), "f"(base));
    return d;
  }
  __device__ __forceinline__ static void of(uint4 w, float base, uint64_t *d) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; k++) d[k] = pair(one(u[k], base), one(u[k] >> 16, base));
  }
};
template <>
struct Differences<__half> {
  __device__ __forceinline__ static float one(uint32_t h, float base) {
    float d;
    asm("sub.rn.f32.f16 %0, %1, %2;" : "=f"(d) : "h"((uint16_t)h), "f"(base));
    return d;
  }
  __device__ __forceinline__ static void of(uint4 w, float base, uint64_t *d) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; k++) d[k] = pair(one(u[k], base), one(u[k] >> 16, base));
  }
};

// d of a vector's numbers, and 2^d, in pairs
template <typename T>
__device__ __forceinline__ void powers(uint4 w, float base, float c, uint64_t *d, uint64_t *e) {
  const uint64_t cc = pair(c, c);
  Differences<T>::of(w, base, d);
#pragma unroll
  for (int k = 0; k < Elem<T>::kPerVec / 2; k++) {
    float x, y;
    d[k] = mul2(d[k], cc);
    split(d[k], x, y);
    e[k] = pair(ex2(x), ex2(y));
  }
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// A masked place has d = -inf, and 0 * -inf is NaN: it is brought within reach,
// to where 2^d still is 0.  In 16 bits that is done to two numbers at once before
// anything else, where the largest number lies far enough above the type's Low,
// but not so far that d or its product with a factor passes fp32's range
// (near_low: not so); elsewhere to d.  Neither changes a bit of what other places give.
// (A part without a number above -inf counts as one whose largest is 0: its
// places, brought to Low, have to be far from that too, or their sum is not 0.)
template <typename T>
struct Low {
  static constexpr float value = 0.0f;
};
template <>
struct Low<__half> {
  static constexpr float value = -65504.0f;
  static constexpr uint32_t two = 0xfbfffbffu;
};
template <>
struct Low<__nv_bfloat16> {
  static constexpr float value = -0x1.92p99f;   // (some -1e30: c times the type's lowest is -inf from c = 1 on)
  static constexpr uint32_t two = 0xf149f149u;
};
template <typename T>
__device__ __forceinline__ bool near_low(float base, float c, float factor = 1.0f) {
  if constexpr (sizeof(T) == 4) return true;
  const float d = (base - Low<T>::value) * c;
  return !(d > -kFar && d < kMost && fabsf(factor) * d < kMost);
}
template <typename T, bool kNearLow>
__device__ __forceinline__ uint4 within_reach(uint4 w) {
  if constexpr (sizeof(T) == 4 || kNearLow) {
    return w;
  } else {
    using T2 = std::conditional_t<std::is_same<T, __half>::value, __half2, __nv_bfloat162>;
    const uint32_t low = Low<T>::two;
    auto one = [&](uint32_t x) {
      const T2 y = __hmax2_nan(*reinterpret_cast<const T2 *>(&x), *reinterpret_cast<const T2 *>(&low));
      return *reinterpret_cast<const uint32_t *>(&y);
    };
    return make_uint4(one(w.x), one(w.y), one(w.z), one(w.w));
  }
}
template <typename T, bool kNearLow>
__device__ __forceinline__ uint64_t within_reach(uint64_t d) {
  if constexpr (sizeof(T) != 4 && !kNearLow) return d;
  float x, y;
  split(d, x, y);
  return pair(fmaxf(x, kFar), fmaxf(y, kFar));
}

// The sums of a vector, in one order.
template <typename T, bool kNearLow>
__device__ __forceinline__ void vec_sums(uint4 w, float base, float c, float &s, float &q) {
  constexpr int kE = Elem<T>::kPerVec;
  uint64_t d[kE / 2], e[kE / 2], u = pair(0.0f, 0.0f);
  powers<T>(within_reach<T, kNearLow>(w), base, c, d, e);
#pragma unroll
  for (int k = 0; k < kE / 2; k++) u = fma2(e[k], within_reach<T, kNearLow>(d[k]), u);
#pragma unroll
  for (int o = kE / 4; o; o >>= 1)
#pragma unroll
    for (int k = 0; k < o; k++) e[k] = add2(e[k], e[k + o]);
  float x, y;
  split(e[0], x, y);
  s = x + y;
  split(u, x, y);
  q = x + y;
}

// The largest number of a part of a row and its sums relative to that.  While
// all is -inf they are 0 (with NaN beside it: the largest is -inf, but s is NaN).
struct Part {
  float m = -INFINITY, s = 0.0f, q = 0.0f;
  // relative to `to` >= m instead
  __device__ __forceinline__ void move(float to, float c) {
    const float base = to == -INFINITY ? 0.0f : to, d = (m - base) * c, f = ex2(d);
    q = f * __fmaf_rn(fmaxf(d, kFar), s, q);
    s *= f;
    m = to;
  }
  template <typename T, int N, bool kNearLow>
  __device__ __forceinline__ static void sums_of(const uint4 *v, float base, float c, float &s, float &q) {
    float t[N], u[N];
#pragma unroll
    for (int k = 0; k < N; k++) vec_sums<T, kNearLow>(v[k], base, c, t[k], u[k]);
#pragma unroll
    for (int o = N / 2; o; o >>= 1)
#pragma unroll
      for (int k = 0; k < o; k++) t[k] += t[k + o], u[k] += u[k + o];
    s = t[0], q = u[0];
  }
  // N vectors, by a whole warp
  template <typename T, int N>
  __device__ __forceinline__ void add(const uint4 *v, float c) {
    float to = m;
#pragma unroll
    for (int k = 0; k < N; k++) to = Elem<T>::vec_max(v[k], to);
    const float base = to == -INFINITY ? 0.0f : to;
    float t, u;
    if (__any_sync(~0u, near_low<T>(base, c))) sums_of<T, N, true>(v, base, c, t, u);
    else sums_of<T, N, false>(v, base, c, t, u);
    move(to, c);
    s += t, q += u;
  }
  // the lanes' parts, the same in every lane
  __device__ __forceinline__ void of_warp(float c) {
    move(warp_max_all(m), c);
    s = warp_add(s), q = warp_add(q);
  }
};

// What a warp tells of its segment: m, s, q, and the token's logit where it has that.
__device__ __forceinline__ uint4 word(const Part &p, float xt) {
  return make_uint4(__float_as_uint(p.m), __float_as_uint(p.s), __float_as_uint(p.q), __float_as_uint(xt));
}
// Several (at most 32 N) parts joined, in every thread: lane l joins parts l, l + 32 and so on, then the lanes.
template <int N>
__device__ __forceinline__ Part join(const uint4 *box, int n, float c) {
  const int lane = threadIdx.x & 31;
  Part p[N];
  float to = -INFINITY;
#pragma unroll
  for (int k = 0; k < N; k++)
    if (lane + 32 * k < n) {
      const uint4 w = box[lane + 32 * k];
      p[k].m = __uint_as_float(w.x), p[k].s = __uint_as_float(w.y), p[k].q = __uint_as_float(w.z);
      to = fmaxf(to, p[k].m);
    }
  to = warp_max_all(to);
#pragma unroll
  for (int k = 0; k < N; k++) p[k].move(to, c);
#pragma unroll
  for (int k = 1; k < N; k++) p[0].s += p[k].s, p[0].q += p[k].q;
  p[0].s = warp_add(p[0].s), p[0].q = warp_add(p[0].q);
  return p[0];
}

// What a used row's loss has beside its logits.
struct Token {
  int32_t token;
  float weight, old, advantage, ref;
};
__device__ __forceinline__ bool used_row(const RowsArgs &a, int64_t row, Token &t) {
  const int64_t token = a.tokens[row];
  t.weight = a.policy.weights[row];
  t.token = (int32_t)token;
  return t.weight != 0.0f && token >= 0 && token < a.vocab;
}
__device__ __forceinline__ void rest_of(const RowsArgs &a, int64_t row, Token &t) {
  t.old = a.policy.old_logps[row], t.advantage = a.policy.advantages[row];
  t.ref = a.policy.ref_logps ? a.policy.ref_logps[row] : 0.0f;
}

// Of 32 of a cluster's rows at a time a lane each: what stands beside them, so
// that no row waits for loads of its own, and which of them are used.
struct Ahead {
  Token mine;
  uint32_t used;
  template <bool kRest, typename F>
  __device__ __forceinline__ void load(const RowsArgs &a, uint32_t from, uint32_t turns, F row_of) {
    const uint32_t it = from + (threadIdx.x & 31);
    mine = {};
    const bool is = it < turns && used_row(a, row_of(it), mine);
    if (kRest && is) rest_of(a, row_of(it), mine);
    used = __ballot_sync(~0u, is);
  }
  __device__ __forceinline__ bool is_used(uint32_t it) const { return used >> (it & 31) & 1; }
  __device__ __forceinline__ int32_t token_of(uint32_t it) const { return __shfl_sync(~0u, mine.token, it & 31); }
  __device__ __forceinline__ Token of(uint32_t it) const {
    const int l = it & 31;
    return {__shfl_sync(~0u, mine.token, l), __shfl_sync(~0u, mine.weight, l), __shfl_sync(~0u, mine.old, l),
            __shfl_sync(~0u, mine.advantage, l), __shfl_sync(~0u, mine.ref, l)};
  }
};

// What a row's sums give, and the factors of its gradient.
struct Result {
  float base, logp, entropy, c0, c1, g;
  bool nothing;   // above -inf: the gradient is 0
};
__device__ __forceinline__ Result result_of(const RowsArgs &a, const Token &t, const Part &p, float xt) {
  const float inv = a.policy.inv_temperature, ln = logf(p.s);
  Result r;
  r.base = p.m == -INFINITY ? 0.0f : p.m;
  r.nothing = p.s == 0.0f;
  r.logp = r.nothing ? -INFINITY : (xt - r.base) * inv - ln;
  r.entropy = r.nothing ? 0.0f : ln - kLn2 * __fdiv_rn(p.q, p.s);
  const float slope = loss::policy_terms(a.policy, r.logp, t.old, t.advantage, t.ref).slope;
  const float g = t.weight * slope, b = t.weight * a.policy.entropy_coef, f = __fdiv_rn(inv, p.s);
  r.c0 = -g * f, r.c1 = 0.0f, r.g = g * inv;
  if (a.policy.entropy_coef != 0.0f) r.c0 = (b * (r.entropy - ln) - g) * f, r.c1 = b * kLn2 * f;
  return r;
}

// A vector's gradient, but for what its token adds.
template <typename T, bool kBonus, bool kNearLow>
__device__ __forceinline__ void vec_gradient(uint4 w, const Result &r, float c, float *y) {
  constexpr int kE = Elem<T>::kPerVec;
  uint64_t d[kE / 2], e[kE / 2];
  powers<T>(kBonus ? within_reach<T, kNearLow>(w) : w, r.base, c, d, e);
  const uint64_t c0 = pair(r.c0, r.c0), c1 = pair(r.c1, r.c1);
#pragma unroll
  for (int k = 0; k < kE / 2; k++)
    split(mul2(e[k], kBonus ? fma2(c1, within_reach<T, kNearLow>(d[k]), c0) : c0), y[2 * k], y[2 * k + 1]);
}
// `g` more where `at`, the token's place from the vector's start, is in it
template <int kE>
__device__ __forceinline__ void vec_token(int32_t at, float g, float *y) {
  if ((uint32_t)at < (uint32_t)kE) {
#pragma unroll
    for (int k = 0; k < kE; k++)
      if (k == at) y[k] += g;
  }
}
// The token's own place: as a vector's number, and g more.
__device__ __forceinline__ float token_gradient(const Result &r, float xt, float c, bool bonus) {
  const float d = (xt - r.base) * c;
  return ex2(d) * (bonus ? __fmaf_rn(r.c1, fmaxf(d, kFar), r.c0) : r.c0) + r.g;
}
// f(whether there is a bonus, whether the largest number is near the lowest), as constants
template <typename T, typename F>
__device__ __forceinline__ void by_kind(bool bonus, bool near, F f) {
  if (!bonus) f(std::false_type{}, std::false_type{});
  else if (sizeof(T) == 4 || near) f(std::true_type{}, std::true_type{});
  else f(std::true_type{}, std::false_type{});
}

// kLag: the next row is summed before a row's gradient is written, so that the
// exchange and what follows it are not waited for.
template <bool kLag>
constexpr int kBuffers = kLag ? 3 : 2;      // one row coming, the others at work
template <bool kLag>
constexpr int kRowBoxes = kLag ? 4 : 2;     // exchanges under way
template <int kWarps>
constexpr int kThreads = kWarps * 32 + 32;  // and one warp that brings rows in and joins their sums

// A cluster's rows one after another (see Stream).  All warps but one of each CTA sum
// their segments of a used row and tell every CTA of the cluster; the last one,
// which also brings rows in, joins the sums and works out what the row's gradient
// takes, which the others then write.  (Where each of them joined and worked out
// for itself, that was a third of their instructions.)  An unused row is not read;
// zeros are written for it.
//
// A warp's word of row n + 2 comes after every CTA's last warp has read the words
// of row n (each CTA's words of n + 1 come after its own last warp has), so there
// are two boxes in turn, and one place for a row's result; twice as many where the
// next row is summed first.
//
// A wait that gave up makes its row's sum NaN in every CTA (a word of NaN), or in
// the CTA whose last warp missed the words; what a warp has yet to write of used
// rows is marked NaN after that, each place by the thread that would have written
// it.
template <typename T, int kWarps, bool kLag>
__global__ __launch_bounds__(kThreads<kWarps>) void rows_kernel(const RowsArgs a) {
  extern __shared__ uint4 buffers[];   // kB of a.steps steps
  constexpr int kE = Elem<T>::kPerVec, kB = kBuffers<kLag>, kX = kRowBoxes<kLag>, kR = kLag ? 2 : 1,
                kLog2Warps = kWarps == 8 ? 3 : 2;
  __shared__ uint4 box[kX][kMaxCluster * kWarps];
  __shared__ uint64_t full[kB], empty[kB], told[kX], ready[kR];
  __shared__ Result result[kR];
  __shared__ bool stop[kR];
  const uint32_t size = cluster_size(), rank = cluster_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t first = blockIdx.x / size, step = gridDim.x / size;
  const uint32_t turns = ((uint32_t)a.rows - first + step - 1) / step;   // (at most one cluster a row)
  const int log2_size = __ffs(size) - 1, log2_segments = log2_size + kLog2Warps, segments = (int)size * kWarps;
  const float c = kLog2e * a.policy.inv_temperature;
  if (threadIdx.x == 0) {
    for (int b = 0; b < kB; b++) bar_init(&full[b], 2), bar_init(&empty[b], kWarps);
    for (int b = 0; b < kX; b++) {
      bar_init(&told[b], 1);
      bar_expect(&told[b], segments * 16);
    }
    for (int b = 0; b < kR; b++) bar_init(&ready[b], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  cluster_sync();   // every CTA's barriers are ready
  // (the sums over tokens may come onto the SMs, and wait for the end of this kernel)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  auto row_of = [&](uint32_t it) { return (int64_t)(first + it * step); };
  auto stream = [&](uint32_t it, uint32_t b) {
    Stream<T> x;
    x.set(static_cast<const T *>(a.logits) + row_of(it) * a.stride, a.vocab, rank, log2_size, buffers + b * a.steps * 32);
    return x;
  };
  // the segment of the token's vector: the last that begins at or before its step
  auto segment_of = [&](const Stream<T> &x, int32_t token) {
    return (((uint32_t)((token + x.off) / kE / 32 + 1) << log2_segments) - 1) / (uint32_t)x.steps;
  };
  bool ok = true;
  if (warp == kWarps) {
    Ahead coming, rows;   // of the rows that are brought in, and of those that are finished
    uint32_t next = 0, brought = 0;
    auto bring = [&] {    // the next used row
      for (; next < turns; next++) {
        if (next % 32 == 0) coming.load<false>(a, next, turns, row_of);
        if (coming.is_used(next)) {
          const uint32_t b = brought % kB;
          stream(next, b).bring(static_cast<const T *>(a.logits) + row_of(next) * a.stride, &full[b]);
          brought++, next++;
          return;
        }
      }
    };
    for (int b = 0; b < kB; b++) bring();
    uint32_t n = 0;
    for (uint32_t it = 0; it < turns && ok; it++) {
      if (it % 32 == 0) rows.load<true>(a, it, turns, row_of);
      if (!rows.is_used(it)) continue;
      const Token t = rows.of(it);
      const uint4 *boxes = box[n % kX];
      uint64_t *bar = &told[n % kX];
      ok = __all_sync(~0u, bar_wait(bar, n / kX & 1, a.waits.limit));
      if (ok && lane == 0) bar_expect(bar, segments * 16);   // for a later row
      Part all = join<kMaxCluster * kWarps / 32>(boxes, segments, c);
      const float xt = __uint_as_float(boxes[segment_of(stream(it, 0), t.token)].w);
      if (!ok) all.s = NAN;
      const Result r = result_of(a, t, all, xt);
      if (lane == 0) {
        result[n % kR] = r;
        stop[n % kR] = !ok;
        bar_arrive(&ready[n % kR]);
        if (rank == 0) a.logps[row_of(it)] = r.logp, a.entropies[row_of(it)] = r.entropy;
      }
      if (!ok) break;
      // another row into this one's buffer
      if (next < turns) ok = __all_sync(~0u, bar_wait(&empty[n % kB], n / kB & 1, a.waits.limit));
      if (ok) bring();
      n++;
    }
    // copies in flight land before the CTA goes
    for (uint32_t i = brought > kB ? brought - kB : 0; i < brought; i++) bar_wait(&full[i % kB], i / kB & 1);
  } else {
    const uint32_t segment = rank * kWarps + warp;
    struct Own {   // this warp's steps of a row's slice
      int32_t from, to;
    };
    auto own = [&](const Stream<T> &x) {
      return Own{x.step_of(segment, log2_segments) - x.begin / 32, x.step_of(segment + 1, log2_segments) - x.begin / 32};
    };
    // f(vector's place in the buffer, numbers) gives what is written, for each of the warp's steps
    auto write = [&](const Stream<T> &x, Own o, int64_t row, auto f) {
      T *d = static_cast<T *>(a.dlogits) + row * a.dstride;
      const bool aligned = same_alignment(d, x.off);
      // steps at the row's ends, or all where its gradient lies between 16-byte places
      const int32_t head = o.from < o.to && !(aligned && x.inside(o.from)) ? o.from++ : -1;
      const int32_t tail = o.from < o.to && !(aligned && x.inside(o.to - 1)) ? --o.to : -1;
      if (aligned) {
        const int32_t vec = o.from * 32 + lane, steps = o.to - o.from;
        uint4 *out = reinterpret_cast<uint4 *>(d + x.index(vec, 0));
#pragma unroll 2
        for (int32_t k = 0; k < steps; k++) {
          float y[kE];
          f(vec + 32 * k, y);
          out[32 * k] = Elem<T>::pack(y);
        }
        o.from = o.to;
      }
#pragma unroll 1
      for (int32_t k = o.from; k < o.to + 2; k++) {
        const int32_t st = k < o.to ? k : k == o.to ? head : tail;
        if (st < 0) continue;
        const int32_t vec = st * 32 + lane, at = x.index(vec, 0);
        float y[kE];
        f(vec, y);
        if (aligned && at >= 0 && at + kE <= a.vocab) *reinterpret_cast<uint4 *>(d + at) = Elem<T>::pack(y);
        else x.write_edge(d, vec, y);
      }
    };
    auto zeros = [&](const Stream<T> &x, int64_t row) {
      write(x, own(x), row, [](int32_t, float *y) {
#pragma unroll
        for (int e = 0; e < kE; e++) y[e] = 0.0f;
      });
    };
    auto write_row = [&](int64_t row, float v) {
      if (rank == 0 && threadIdx.x == 0) a.logps[row] = a.entropies[row] = v;
    };
    const bool bonus = a.policy.entropy_coef != 0.0f;
    // a row that was summed: its turn, its number among the used ones, the token's place in the slice (-1: another
    // warp's) and its logit
    struct Summed {
      uint32_t it, n;
      int32_t at;
      float xt;
    };
    auto buffer = [&](uint32_t n) { return n % kB; };
    auto sum_row = [&](uint32_t it, uint32_t n, int32_t token) {
      const Stream<T> x = stream(it, buffer(n));
      const Own o = own(x);
      ok &= bar_wait(&full[buffer(n)], n / kB & 1, a.waits.limit) & !a.waits.fails(n, segment);
      Part part;
      int32_t st = o.from;
      const uint4 *p = x.buf + st * 32 + lane;
      for (; st + 4 <= o.to; st += 4, p += 128) {
        const uint4 v[4] = {p[0], p[32], p[64], p[96]};
        part.add<T, 4>(v, c);
      }
      if (st + 2 <= o.to) {
        const uint4 v[2] = {p[0], p[32]};
        part.add<T, 2>(v, c);
        st += 2, p += 64;
      }
      if (st < o.to) part.add<T, 1>(p, c);
      if (!ok) part.s = NAN;   // the wait gave up: so is the row's sum, in every CTA
      part.of_warp(c);
      Summed r = {it, n, token - x.index(0, 0), 0.0f};
      if (r.at >= 0 && r.at / kE / 32 >= o.from && r.at / kE / 32 < o.to) r.xt = Elem<T>::load(reinterpret_cast<const T *>(x.buf) + r.at);
      else r.at = -1;
      if (lane < (int)size) send(&box[n % kX][segment], &told[n % kX], lane, word(part, r.xt));
      return r;
    };
    auto write_gradient = [&](const Summed &w) {
      const int64_t row = row_of(w.it);
      const Stream<T> x = stream(w.it, buffer(w.n));
      ok &= bar_wait(&ready[w.n % kR], w.n / kR & 1, a.waits.limit);
      Result r = result[w.n % kR];
      ok = __all_sync(~0u, ok & !stop[w.n % kR]);
      if (!ok) {
        r.c0 = r.g = NAN, r.nothing = false;
        write_row(row, NAN);   // (the last warp may have given up before this row)
      }
      if (r.nothing) {
        zeros(x, row);
      } else {
        by_kind<T>(bonus, near_low<T>(r.base, c, r.c1), [&](auto bonus, auto near) {
          write(x, own(x), row, [&](int32_t vec, float *y) {
            vec_gradient<T, decltype(bonus)::value, decltype(near)::value>(x.buf[vec], r, c, y);
          });
        });
        // the thread that wrote the token's place writes it again
        if (w.at >= 0 && lane == w.at / kE % 32)
          Elem<T>::store(static_cast<T *>(a.dlogits) + row * a.dstride + x.index(0, 0) + w.at, token_gradient(r, w.xt, c, bonus));
      }
      __syncwarp();
      if (ok && lane == 0) bar_arrive(&empty[buffer(w.n)]);
    };
    uint32_t it = 0, n = 0;   // n: used rows
    Ahead rows;
    Summed was = {};
    for (; it < turns && ok; it++) {
      if (it % 32 == 0) rows.load<false>(a, it, turns, row_of);
      if (!rows.is_used(it)) {
        zeros(stream(it, 0), row_of(it));
        write_row(row_of(it), 0.0f);
        continue;
      }
      const Summed now = sum_row(it, n, rows.token_of(it));
      if (!kLag) write_gradient(now);
      else if (n > 0) write_gradient(was);
      was = now;
      n++;
      ok = __all_sync(~0u, ok);
    }
    if (kLag && n > 0) write_gradient(was);
    if (!ok) {
      // what this warp has yet to write is marked, each place by the thread that would have written it
      for (uint32_t i = it; i < turns; i++) {
        const int64_t row = row_of(i);
        const Stream<T> x = stream(i, 0);
        Token t;
        if (!used_row(a, row, t)) {
          zeros(x, row);
          write_row(row, 0.0f);
          continue;
        }
        write_row(row, NAN);
        const int32_t from = x.index((x.step_of(segment, log2_segments) - x.begin / 32) * 32, 0),
                      to = x.index((x.step_of(segment + 1, log2_segments) - x.begin / 32) * 32, 0);
        write_nan(static_cast<T *>(a.dlogits) + row * a.dstride, max(from, 0), min(to, a.vocab));
      }
    }
  }
  __syncwarp();
  cluster_sync();
  if (!ok) stay();
}

// Short rows, in registers: G lanes a row, 32 / G rows a warp; no barrier, and
// what is worked out once a row is worked out for a warp's rows together.
template <typename T, int KV, int G>
__global__ __launch_bounds__(128, KV <= 8 ? 8 : 5) void short_rows_kernel(const RowsArgs a) {
  constexpr int kE = Elem<T>::kPerVec;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x % G;
  const int64_t row = ((int64_t)blockIdx.x * 128 + threadIdx.x) / G;
  const bool there = row < a.rows;
  Token t = {};
  const bool used = there && used_row(a, row, t);
  const T *p = static_cast<const T *>(a.logits) + row * a.stride;
  const int32_t off = (int32_t)((uint32_t)reinterpret_cast<uintptr_t>(p) & 15u) / (int)sizeof(T);
  // vector k of this lane begins with the row's number first + k * G * kE; the whole of it is the row's below `whole`
  const int32_t first = lane * kE - off;
  const uint32_t whole = there && a.vocab >= kE ? (uint32_t)(a.vocab - kE + 1) : 0u;
  constexpr uint32_t ninf = Elem<T>::kNegInf;
  uint4 v[KV];
  float xt = 0.0f;
#pragma unroll
  for (int k = 0; k < KV; k++) {
    const int32_t i = first + k * G * kE;
    v[k] = make_uint4(ninf, ninf, ninf, ninf);
    if (used && (uint32_t)i < whole) {
      v[k] = *reinterpret_cast<const uint4 *>(p + i);
    } else if (used && i + kE > 0 && i < a.vocab) {
      float x[kE];
#pragma unroll
      for (int e = 0; e < kE; e++) x[e] = i + e >= 0 && i + e < a.vocab ? Elem<T>::load(p + i + e) : -INFINITY;
      v[k] = Elem<T>::pack(x);
    }
  }
  if (used) {
    rest_of(a, row, t);
    xt = Elem<T>::load(p + t.token);   // before a gradient in place overwrites it
  }
  const float c = kLog2e * a.policy.inv_temperature;
  Part part;
#pragma unroll
  for (int k = 0; k < KV; k++) part.m = Elem<T>::vec_max(v[k], part.m);
#pragma unroll
  for (int o = G / 2; o; o >>= 1) part.m = fmaxf(part.m, __shfl_xor_sync(~0u, part.m, o));
  const float base = part.m == -INFINITY ? 0.0f : part.m;
  const bool near = __any_sync(~0u, near_low<T>(base, c));
  auto add = [&](auto near) {
#pragma unroll
    for (int k = 0; k < KV; k++) {
      float s, q;
      vec_sums<T, decltype(near)::value>(v[k], base, c, s, q);
      part.s += s, part.q += q;
    }
  };
  if (near) add(std::true_type{});
  else add(std::false_type{});
#pragma unroll
  for (int o = G / 2; o; o >>= 1) {
    part.s += __shfl_xor_sync(~0u, part.s, o);
    part.q += __shfl_xor_sync(~0u, part.q, o);
  }
  Result r = result_of(a, t, part, xt);
  if (!used) r.logp = r.entropy = 0.0f;
  if (there && lane == 0) a.logps[row] = r.logp, a.entropies[row] = r.entropy;
  const bool bonus = a.policy.entropy_coef != 0.0f;
  if (!used || r.nothing) r.c0 = r.c1 = r.g = 0.0f;   // (2^-inf times that)
  const bool clamp = bonus && __any_sync(~0u, near_low<T>(base, c, r.c1));
  __syncwarp();   // every lane of the row has its numbers: they may be overwritten
  if (!there) return;
  // (the exponentials are taken again: kept, they would cost the registers of the warps that hide the loads)
  asm volatile("" : "+f"(r.base));
  T *d = static_cast<T *>(a.dlogits) + row * a.dstride;
  const bool aligned = same_alignment(d, off);
  by_kind<T>(bonus, clamp, [&](auto bonus, auto near) {
#pragma unroll
    for (int k = 0; k < KV; k++) {
      const int32_t i = first + k * G * kE;
      if (i + kE > 0 && i < a.vocab) {
        float y[kE];
        vec_gradient<T, decltype(bonus)::value, decltype(near)::value>(v[k], r, c, y);
        if (aligned && (uint32_t)i < whole) {
          *reinterpret_cast<uint4 *>(d + i) = Elem<T>::pack(y);
        } else {
#pragma unroll
          for (int e = 0; e < kE; e++)
            if (i + e >= 0 && i + e < a.vocab) Elem<T>::store(d + i + e, y[e]);
        }
      }
    }
  });
  // the thread that wrote the token's place writes it again
  if (used && !r.nothing && lane == (t.token + off) / kE % G) Elem<T>::store(d + t.token, token_gradient(r, xt, c, bonus));
}

// Rows too large for the buffers: one CTA a part of a row, its passes read
// global memory again (L2).
template <typename T, int NT>
__global__ __launch_bounds__(NT) void reread_rows_kernel(const RowsArgs a) {
  __shared__ uint4 box[kMaxCluster];
  __shared__ uint4 part[NT / 32];
  const uint32_t size = cluster_size(), rank = cluster_rank();
  cluster_begun();
  const int64_t row = blockIdx.x / size;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T *p = static_cast<const T *>(a.logits) + row * a.stride;
  T *d = static_cast<T *>(a.dlogits) + row * a.dstride;
  Slice<T, 0, NT> x;
  x.set(p, a.vocab, rank, size);
  const bool aligned = same_alignment(d, x.off);
  Token t;
  if (!used_row(a, row, t)) {   // (the whole cluster)
    cluster_wait_begun();
    write_zeros(x, d, aligned);
    if (rank == 0 && threadIdx.x == 0) a.logps[row] = a.entropies[row] = 0.0f;
    return;
  }
  rest_of(a, row, t);
  const float xt = Elem<T>::load(p + t.token);   // before a gradient in place overwrites it
  const float c = kLog2e * a.policy.inv_temperature;
  Part mine;
  for (int k = 0; k < x.steps; k += 4) {
    const uint4 v[4] = {x.read(k), x.read(k + 1), x.read(k + 2), x.read(k + 3)};
    mine.add<T, 4>(v, c);
  }
  mine.of_warp(c);
  if (lane == 0) part[warp] = word(mine, 0.0f);
  __syncthreads();
  mine = join<1>(part, NT / 32, c);
  __syncwarp();
  cluster_wait_begun();
  if (threadIdx.x < size) {
    const uint32_t to = remote(&box[rank], threadIdx.x);
    st_remote(to, pair(mine.m, mine.s));
    st_remote(to + 8, pair(mine.q, xt));
  }
  __syncwarp();
  cluster_sync();   // no CTA reads or writes another's memory after this
  mine = join<1>(box, (int)size, c);
  const Result r = result_of(a, t, mine, xt);
  if (rank == 0 && threadIdx.x == 0) a.logps[row] = r.logp, a.entropies[row] = r.entropy;
  if (r.nothing) {
    write_zeros(x, d, aligned);
    return;
  }
  by_kind<T>(a.policy.entropy_coef != 0.0f, near_low<T>(r.base, c, r.c1), [&](auto bonus, auto near) {
    for (int k = 0; k < x.steps; k++) {
      float y[x.kE];
      vec_gradient<T, decltype(bonus)::value, decltype(near)::value>(x.read(k), r, c, y);
      vec_token<x.kE>(t.token - x.index(k, 0), r.g, y);
      x.write(d, aligned, k, y);
    }
  });
}

constexpr int kDevices = 16;           // whose occupancy is kept
constexpr int kShort = 12;             // steps of the rows that a warp takes by itself

constexpr size_t shared_bytes(int64_t steps, int buffers) { return (size_t)steps * buffers * 32 * 16; }
// of a row that a CTA has room for beside its boxes
constexpr int most_steps(int buffers) { return (220 << 10) / (buffers * 32 * 16); }

template <typename T, int kWarps, bool kLag>
cudaError_t launch_streamed(RowsArgs a, int log2_size, cudaStream_t stream) {
  constexpr int kB = kBuffers<kLag>, kMost = most_steps(kB);
  static std::atomic<int> fits[kDevices][4][kMost + 1];   // clusters at once, by size and steps (0: not known)
  auto kernel = rows_kernel<T, kWarps, kLag>;
  const size_t shared = shared_bytes(a.steps, kB);
  int device = 0, most = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  if (device < kDevices) most = fits[device][log2_size][a.steps].load(std::memory_order_relaxed);
  if (most == 0) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)shared_bytes(kMost, kB));
    if (e == cudaSuccess) e = launch_rows(kernel, a, 1, 1 << log2_size, kThreads<kWarps>, shared, stream, &most);
    if (e != cudaSuccess) return e;
    if (most < 1) return cudaErrorLaunchOutOfResources;
    if (device < kDevices) fits[device][log2_size][a.steps].store(most, std::memory_order_relaxed);
  }
  return launch_rows(kernel, a, a.rows < most ? a.rows : most, 1 << log2_size, kThreads<kWarps>, shared, stream);
}

template <typename T>
cudaError_t launch_policy_rows(RowsArgs a, cudaStream_t stream) {
  constexpr int kE = Elem<T>::kPerVec;
  const int64_t vecs = ((int64_t)a.vocab + kE - 1) / kE + 1;   // whatever the alignment
  const int64_t steps = (vecs + 31) / 32;
  if (steps <= kShort) {
    // lanes a row by its length alone; vectors a lane that the rows at hand have (more of them change no bit)
    const bool at16 = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && (a.rows == 1 || a.stride % kE == 0);
    const int64_t most = vecs - (at16 ? 1 : 0);
    const int group = vecs <= 64 ? 8 : vecs <= 128 ? 16 : 32;
    const int64_t ctas = (a.rows * group + 127) / 128;
    if (group == 8)
      return most <= 16   ? launch_rows(short_rows_kernel<T, 2, 8>, a, ctas, 1, 128, 0, stream)
             : most <= 32 ? launch_rows(short_rows_kernel<T, 4, 8>, a, ctas, 1, 128, 0, stream)
                          : launch_rows(short_rows_kernel<T, 8, 8>, a, ctas, 1, 128, 0, stream);
    if (group == 16) return launch_rows(short_rows_kernel<T, 8, 16>, a, ctas, 1, 128, 0, stream);
    return most <= 256 ? launch_rows(short_rows_kernel<T, 8, 32>, a, ctas, 1, 128, 0, stream)
                       : launch_rows(short_rows_kernel<T, kShort, 32>, a, ctas, 1, 128, 0, stream);
  }
  int log2_size = 0;
  // As few CTAs a row as leave three of them room on an SM, four warps each (4096 x 50001 bf16: two of eight warps 145 us,
  // four of four 139; 16384 x 20000: 257 and 221; of half that size 174 and 299).  Beyond eight such, eight warps each
  // (4096 x 131072 fp32: 918 us, four 1058), and where one CTA has an SM to itself, the next row summed first (827).
  while (1 << log2_size < kMaxCluster && steps > (int64_t)66 << log2_size) log2_size++;
  a.steps = (int32_t)((steps + (1 << log2_size) - 1) >> log2_size);
  if (a.steps > most_steps(2)) return launch_rows(reread_rows_kernel<T, 512>, a, a.rows, kMaxCluster, 512, 0, stream);
  if (a.steps <= 66) return launch_streamed<T, 4, false>(a, log2_size, stream);
  if (a.steps > 104 && a.steps <= most_steps(3)) return launch_streamed<T, 8, true>(a, log2_size, stream);
  return launch_streamed<T, 8, false>(a, log2_size, stream);
}

bool bad_rows(const void *logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t stride) {
  if (rows < 0 || rows > SEQSUM_MAX_ROWS || vocab < 0 || vocab > kMaxVocab || stride < 0) return true;
  if (dtype != SEQSUM_FP32 && dtype != SEQSUM_FP16 && dtype != SEQSUM_BF16) return true;
  return rows > 0 && vocab > 0 && (!logits || reinterpret_cast<uintptr_t>(logits) % (dtype == SEQSUM_FP32 ? 4 : 2));
}

}  // namespace
}  // namespace sq

extern "C" int seqsum_token_policy_grad(const void *logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                                        const int64_t *tokens, const seqsum_policy *policy, void *dlogits,
                                        int64_t drow_stride, float *logps, float *entropies, float *loss, float *stats,
                                        void *scratch, cudaStream_t stream) {
  using namespace sq;
  if (bad_rows(logits, dtype, rows, vocab, row_stride) || bad_rows(dlogits, dtype, rows, vocab, drow_stride))
    return SEQSUM_EINVAL;
  RowsArgs a = {logits, rows, row_stride, (int32_t)vocab, tokens, {}, logps, entropies, dlogits, drow_stride, 0, row::waits()};
  if (!loss::take_policy(policy, rows, true, &a.policy) || !loss || !stats) return SEQSUM_EINVAL;
  for (const float *out : {(const float *)loss, (const float *)stats, (const float *)logps, (const float *)entropies})
    if (reinterpret_cast<uintptr_t>(out) % sizeof(float)) return SEQSUM_EINVAL;
  if (reinterpret_cast<uintptr_t>(scratch) % sizeof(float2)) return SEQSUM_EINVAL;
  if (rows > 0) {
    if (!tokens || !logps || !entropies || (rows > 1 && drow_stride < vocab)) return SEQSUM_EINVAL;
    if (!scratch && rows > loss::kClusterTokens) return SEQSUM_EINVAL;
    // the loss is taken from the log-probabilities and the tokens' numbers once these and the gradient are written
    const loss::Policy &p = a.policy;
    const int64_t size = dtype == SEQSUM_FP32 ? 4 : 2, bytes = rows * (int64_t)sizeof(float);
    const bool in_place = dlogits == logits && (rows == 1 || drow_stride == row_stride);
    using loss::place;
    if (!loss::apart({place(dlogits, rows, (__int128)drow_stride * size, vocab * size), place(logps, bytes), place(entropies, bytes),
                      place(loss, sizeof(float)), place(stats, 6 * sizeof(float)),
                      place(scratch, rows > loss::kClusterTokens ? SEQSUM_POLICY_SCRATCH : 0)},
                     {place(in_place ? nullptr : logits, rows, (__int128)row_stride * size, vocab * size),
                      place(tokens, rows * (int64_t)sizeof(int64_t)), place(p.old_logps, bytes), place(p.advantages, bytes),
                      place(p.weights, bytes), place(p.ref_logps, bytes)}))
      return SEQSUM_EINVAL;
    const cudaError_t e = dtype == SEQSUM_FP32   ? launch_policy_rows<float>(a, stream)
                          : dtype == SEQSUM_FP16 ? launch_policy_rows<__half>(a, stream)
                                                 : launch_policy_rows<__nv_bfloat16>(a, stream);
    if (e != cudaSuccess) return note_cuda(e);
  }
  return loss::sum_policy(a.policy, logps, entropies, tokens, vocab, rows, loss, stats, scratch, rows > 0, stream);
}
