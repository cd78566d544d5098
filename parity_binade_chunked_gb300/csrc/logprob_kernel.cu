// Log-probabilities of given tokens and their gradient with respect to the
// logits (seqsum_token_logprob, _grad, _backward).
//
//   lse = m + ln sum exp(x_i - m),  logp = x_t - lse,
//   d logits_i = dlogp * ([i = t] - exp(x_i - lse))
//
// A row's 16-byte vectors, counted from the aligned address at or below its
// first number, are cut into segments, one for each warp that works on it.  A
// segment's maximum and the sum of its exponentials relative to that are formed
// by one warp in one order, and the segments' sums are joined in one order.  So
// a row's results go by its numbers and its address modulo 16 alone, not by the
// other rows of the call; at another place within 16 bytes other numbers share
// a vector, and last bits may differ.  (Vectors counted from the row's first
// number would end that, at the cost of a shift of every vector.)
#include <math.h>

#include <atomic>

#include "../../include/seqsum.h"
#include "row_slice.cuh"

namespace sq {
namespace {

using namespace row;

constexpr float kLog2e = 1.44269504f;

struct LogprobArgs {
  const void *logits;
  int64_t rows, stride;
  int32_t vocab;
  const int64_t *tokens;
  float *logps, *lses;
  const float *dlogps, *lses_in;
  void *dlogits;
  int64_t dstride;
  int32_t parts;                                     // backward: CTAs a row
  int32_t steps;                                     // that a CTA takes of a row at most
  Waits waits;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// exp(v - base) of a vector's numbers: the largest one's is exactly 1 where base is it.
template <int kE>
__device__ __forceinline__ void exps(const float *v, float base, float *y) {
  const uint64_t b = pair(-base, -base), l = pair(kLog2e, kLog2e);
#pragma unroll
  for (int e = 0; e < kE; e += 2) {
    float p, q;
    split(mul2(add2(pair(v[e], v[e + 1]), b), l), p, q);
    y[e] = ex2(p), y[e + 1] = ex2(q);
  }
}

// The sum of a vector's exponentials, in one order.
template <typename T>
__device__ __forceinline__ float vec_sum(uint4 w, float base) {
  constexpr int kE = Elem<T>::kPerVec;
  float v[kE], s[kE];
  Elem<T>::unpack(w, v);
  exps<kE>(v, base, s);
  uint64_t t[kE / 2];
#pragma unroll
  for (int e = 0; e < kE / 2; e++) t[e] = pair(s[e], s[e + kE / 2]);
#pragma unroll
  for (int o = kE / 4; o; o >>= 1)
#pragma unroll
    for (int e = 0; e < o; e++) t[e] = add2(t[e], t[e + o]);
  float p, q;
  split(t[0], p, q);
  return p + q;
}

// A thread's part of a segment: the largest number so far and the sum of
// exp(x - largest), four vectors at a time.  While all is -inf the sum is 0
// (with NaN beside it: the largest is -inf, but the sum is NaN).
struct Part {
  float m = -INFINITY, s = 0.0f;
  template <typename T, int N>
  __device__ __forceinline__ void add(const uint4 *v) {
    float to = m;
#pragma unroll
    for (int k = 0; k < N; k++) to = Elem<T>::vec_max(v[k], to);
    const float base = to == -INFINITY ? 0.0f : to;
    float t[N];
#pragma unroll
    for (int k = 0; k < N; k++) t[k] = vec_sum<T>(v[k], base);
#pragma unroll
    for (int o = N / 2; o; o >>= 1)
#pragma unroll
      for (int k = 0; k < o; k++) t[k] += t[k + o];
    s = s * ex2((m - base) * kLog2e) + t[0];
    m = to;
  }
  // the warp's, as (largest, sum)
  __device__ __forceinline__ uint64_t of_warp() const {
    const float to = warp_max_all(m), base = to == -INFINITY ? 0.0f : to;
    return pair(to, warp_add(s * ex2((m - base) * kLog2e)));
  }
};

// The largest number and the sum of several (at most 64) parts, in every
// thread: lane l joins parts l and l + 32, then the lanes.
__device__ __forceinline__ void join(const uint64_t *box, int n, float &m, float &sum) {
  const int lane = threadIdx.x & 31;
  float m0 = -INFINITY, s0 = 0.0f, m1 = -INFINITY, s1 = 0.0f;
  if (lane < n) split(box[lane], m0, s0);
  if (lane + 32 < n) split(box[lane + 32], m1, s1);
  m = warp_max_all(fmaxf(m0, m1));
  const float base = m == -INFINITY ? 0.0f : m;
  sum = warp_add(s0 * ex2((m0 - base) * kLog2e) + s1 * ex2((m1 - base) * kLog2e));
}

// exp(x - base) * coef of a vector
template <typename T>
__device__ __forceinline__ void vec_scaled(uint4 w, float base, float coef, float *y) {
  constexpr int kE = Elem<T>::kPerVec;
  float v[kE];
  Elem<T>::unpack(w, v);
  exps<kE>(v, base, y);
  const uint64_t c = pair(coef, coef);
#pragma unroll
  for (int e = 0; e < kE; e += 2) split(mul2(pair(y[e], y[e + 1]), c), y[e], y[e + 1]);
}
// `g` more where `at`, the token's place from the vector's start, is in it
template <int kE>
__device__ __forceinline__ void vec_token(int32_t at, float g, float *y) {
  if ((uint32_t)at < (uint32_t)kE) {
#pragma unroll
    for (int e = 0; e < kE; e++)
      if (e == at) y[e] += g;
  }
}

template <typename S, typename T>
__device__ __forceinline__ void write_zeros(const S &x, T *d, bool aligned) {
  const float y[S::kE] = {};
  for (int k = 0; k < x.steps; k++) x.write(d, aligned, k, y);
}

// NaN to elements [from, to) of a row, by one warp
template <typename T>
__device__ __noinline__ void write_nan(T *d, int32_t from, int32_t to) {
#pragma unroll 1
  for (int32_t i = from + (int32_t)(threadIdx.x & 31); i < to; i += 32) Elem<T>::store(d + i, NAN);
}

template <typename T>
__device__ __forceinline__ bool same_alignment(const T *d, int32_t off) {
  return (reinterpret_cast<uintptr_t>(d) & 15) / sizeof(T) == (uintptr_t)off;
}

constexpr int kBoxes = 4;   // exchanges under way, a power of two

constexpr int kWarps = 8, kLog2Warps = 3;   // and one that brings rows in
constexpr int kBuffers = 2;                 // one row coming, one at work
// Whether the next row is summed before a row is finished, so that the words of
// one travel while the other is worked on.  Not where a gradient is due: that
// takes a third buffer, so one CTA an SM less (779 us for 8192 x 131072 bf16
// rows instead of 695).
template <bool kGrad>
constexpr int kLag = kGrad ? 0 : 1;

// A cluster's rows one after another (see Stream): a row's segments, and the
// sum and gradient of that row or the one before.  An element is one subtraction
// and one multiplication (two of each in an instruction), one ex2 and half an
// addition; the gradient takes the exponentials again from the buffer rather
// than room for them.  Bound by HBM with gradient: 8192 x 131072 bf16 695 us
// (6.2 of 6.8 TB/s), 4000 x 50000 133 us (6.0).  Without: 4096 x 50001 70 us
// (5.9 TB/s), 4096 x 131072 200 us (5.4), where issue slots are two thirds full.
// A wait that gave up makes its row's sum NaN in every CTA (a word of NaN), or
// in the warp that missed the words; what the warp has yet to write is marked
// NaN after that, each place by the thread that would have written it.
template <typename T, bool kGrad>
__global__ __launch_bounds__(kWarps * 32 + 32) void logprob_kernel(const LogprobArgs a) {
  extern __shared__ uint4 buffers[];   // kB buffers of a.steps steps
  constexpr int kE = Elem<T>::kPerVec, kB = kBuffers, kL = kLag<kGrad>;
  __shared__ uint64_t full[kB], empty[kB], told[kBoxes], box[kBoxes][kMaxCluster * kWarps];
  const uint32_t size = cluster_size(), rank = cluster_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t first = blockIdx.x / size, step = gridDim.x / size;
  const uint32_t turns = ((uint32_t)a.rows - first + step - 1) / step;   // (at most one cluster a row)
  const int log2_size = __ffs(size) - 1, log2_segments = log2_size + kLog2Warps, segments = (int)size * kWarps;
  if (threadIdx.x == 0) {
    for (int b = 0; b < kB; b++) bar_init(&full[b], 2), bar_init(&empty[b], kWarps);
    for (int b = 0; b < kBoxes; b++) {
      bar_init(&told[b], 1);
      bar_expect(&told[b], segments * 8);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  cluster_sync();   // every CTA's barriers are ready

  auto row_of = [&](uint32_t it) { return (int64_t)(first + it * step); };
  auto stream = [&](uint32_t it, uint32_t b) {
    Stream<T> x;
    x.set(static_cast<const T *>(a.logits) + row_of(it) * a.stride, a.vocab, rank, log2_size, buffers + b * a.steps * 32);
    return x;
  };
  bool ok = true;
  if (warp == kWarps) {
    uint32_t it = 0;
    for (uint32_t b = 0, use = 0; it < turns; it++) {
      if (use > 0) ok = __all_sync(~0u, bar_wait(&empty[b], (use - 1) & 1, a.waits.limit));
      if (!ok) break;
      stream(it, b).bring(static_cast<const T *>(a.logits) + row_of(it) * a.stride, &full[b]);
      if (++b == kB) b = 0, use++;
    }
    // copies in flight land before the CTA goes
    for (uint32_t i = it > kB ? it - kB : 0; i < it; i++) bar_wait(&full[i % kB], i / kB & 1);
  } else {
    const uint32_t segment = rank * kWarps + warp;
    // the thread that has vector `vec` of the slice, and the token's vector
    auto has = [&](int32_t vec) { return (int)threadIdx.x == vec % (kWarps * 32); };
    auto vec_of = [&](const Stream<T> &x, int64_t token) { return (int32_t)(token + x.off) / kE - x.begin; };
    Stream<T> was;
    int64_t was_token = 0;
    float was_xt = 0.0f, was_dlogp = 0.0f;   // the logit of the token, in the thread that has it
    bool was_mine = false;
    uint32_t was_b = 0;
    uint32_t it = 0;
    for (uint32_t b = 0, parity = 0; it < turns + kL && ok; it++) {
      Stream<T> x;
      int64_t token = 0;
      float xt = 0.0f, dlogp = 0.0f;
      bool have = false;
      if (!kL || it < turns) {
        x = stream(it, b);
        token = a.tokens[row_of(it)];
        if (kGrad) dlogp = a.dlogps[row_of(it)];
        ok &= bar_wait(&full[b], parity, a.waits.limit) & !a.waits.fails(it, segment);
        const Exchange tell = {box[it % kBoxes], &told[it % kBoxes]};
        int32_t st = x.step_of(segment, log2_segments) - x.begin / 32;
        const int32_t end = x.step_of(segment + 1, log2_segments) - x.begin / 32;
        Part part;
        const uint4 *p = x.buf + st * 32 + lane;
        for (; st + 4 <= end; st += 4, p += 128) {
          const uint4 v[4] = {p[0], p[32], p[64], p[96]};
          part.add<T, 4>(v);
        }
        if (st + 2 <= end) {
          const uint4 v[2] = {p[0], p[32]};
          part.add<T, 2>(v);
          st += 2, p += 64;
        }
        if (st < end) part.add<T, 1>(p);
        if (!ok) part.s = NAN;   // the wait gave up: so is the row's sum, in every CTA
        tell.post(segment, part.of_warp(), size);
        const int32_t vec = vec_of(x, token);
        if (token >= 0 && token < a.vocab && vec >= 0 && vec < x.n && has(vec)) {
          xt = Elem<T>::load(reinterpret_cast<const T *>(x.buf + vec) + (token - x.index(vec, 0)));
          have = true;
        }
        if (!kGrad) {
          __syncwarp();
          if (ok && lane == 0) bar_arrive(&empty[b]);
        }
      }
      if (!kL) was = x, was_token = token, was_xt = xt, was_dlogp = dlogp, was_mine = have, was_b = b;
      if (it >= kL) {
        const int64_t row = row_of(it - kL);
        const uint32_t t = (it - kL) % kBoxes;
        ok &= bar_wait(&told[t], ((it - kL) / kBoxes) & 1, a.waits.limit);
        if (ok && threadIdx.x == 0) bar_expect(&told[t], segments * 8);   // for its next row
        float m, s;
        join(box[t], segments, m, s);
        if (!__all_sync(~0u, ok)) s = NAN;
        const float base = m == -INFINITY ? 0.0f : m;
        const bool used = was_token >= 0 && was_token < a.vocab, nothing = s == 0.0f;
        if (rank == 0 && threadIdx.x == 0) {
          a.lses[row] = base + logf(s);
          if (!used) a.logps[row] = 0.0f;
        }
        if (was_mine) a.logps[row] = nothing ? -INFINITY : (was_xt - base) - logf(s);
        if constexpr (kGrad) {
          T *d = static_cast<T *>(a.dlogits) + row * a.dstride;
          const bool aligned = same_alignment(d, was.off);
          const float coef = -__fdiv_rn(was_dlogp, s);
          const bool zero = !used || nothing;
          const int32_t begin = was.step_of(segment, log2_segments) - was.begin / 32,
                        end = was.step_of(segment + 1, log2_segments) - was.begin / 32;
#pragma unroll 4
          for (int32_t st = begin; st < end; st++) {
            const int32_t vec = st * 32 + lane, at = was.index(vec, 0);
            float y[kE];
            if (zero) {
#pragma unroll
              for (int e = 0; e < kE; e++) y[e] = 0.0f;
            } else {
              vec_scaled<T>(was.buf[vec], base, coef, y);
              vec_token<kE>((int32_t)was_token - at, was_dlogp, y);
            }
            if (aligned && was.inside(st)) *reinterpret_cast<uint4 *>(d + at) = Elem<T>::pack(y);
            else was.write_edge(d, vec, y);
          }
          __syncwarp();
          if (ok && lane == 0) bar_arrive(&empty[was_b]);
        }
      }
      if (kL) was = x, was_token = token, was_xt = xt, was_dlogp = dlogp, was_mine = have, was_b = b;
      if (++b == kB) b = 0, parity ^= 1;
      ok = __all_sync(~0u, ok);
    }
    if (!ok) {
      // what this warp has yet to write is marked, each place by the thread that would have written it
      for (uint32_t i = it > kL ? it - kL : 0; i < turns; i++) {
        const int64_t row = row_of(i), token = a.tokens[row];
        const Stream<T> x = stream(i, 0);
        const bool used = token >= 0 && token < a.vocab;
        const int32_t vec = vec_of(x, token);
        if (rank == 0 && threadIdx.x == 0) a.lses[row] = NAN;
        if (used ? vec >= 0 && vec < x.n && has(vec) : rank == 0 && threadIdx.x == 0) a.logps[row] = NAN;
        if constexpr (kGrad) {
          const int32_t from = x.index((x.step_of(segment, log2_segments) - x.begin / 32) * 32, 0),
                        to = x.index((x.step_of(segment + 1, log2_segments) - x.begin / 32) * 32, 0);
          write_nan(static_cast<T *>(a.dlogits) + row * a.dstride, max(from, 0), min(to, a.vocab));
        }
      }
    }
  }
  __syncwarp();
  cluster_sync();
  if (!ok) stay();
}

// Short rows: a warp each, in registers; no barrier, no exchange.  Bound by HBM,
// where L2 does not hold the rows already: 8192 x 3001 bf16 27 us with gradient
// (floor 14.5) and 17 without (7.3), L2 flushed; streamed 45 and 35.  With room
// for 16 steps instead of 12 it takes 30 and 18.  (8192 x 4090, of 17 steps, is
// streamed: 48 and 37.)
template <typename T, int KV, bool kGrad>
__global__ __launch_bounds__(128) void logprob_short_kernel(const LogprobArgs a) {
  constexpr int kE = Elem<T>::kPerVec;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= a.rows) return;
  const int lane = threadIdx.x & 31;
  const T *p = static_cast<const T *>(a.logits) + row * a.stride;
  Slice<T, KV, 32> x;
  x.set(p, a.vocab, 0, 1);
  x.load();
  const int64_t token = a.tokens[row];
  const bool used = token >= 0 && token < a.vocab;
  const float xt = used ? Elem<T>::load(p + token) : 0.0f;   // before a gradient in place overwrites it
  Part part;
#pragma unroll
  for (int k = 0; k < KV; k += 4)
    if (k < x.steps) part.add<T, 4>(x.keep + k);
  float m, s;
  split(part.of_warp(), m, s);
  const float base = m == -INFINITY ? 0.0f : m;
  const bool nothing = s == 0.0f;
  if (lane == 0) {
    const float ln = logf(s);
    a.lses[row] = base + ln;
    a.logps[row] = used ? (nothing ? -INFINITY : (xt - base) - ln) : 0.0f;
  }
  if constexpr (kGrad) {
    T *d = static_cast<T *>(a.dlogits) + row * a.dstride;
    const bool aligned = same_alignment(d, x.off);
    if (!used || nothing) {
      write_zeros(x, d, aligned);
    } else {
      const float dlogp = a.dlogps[row], coef = -__fdiv_rn(dlogp, s);
#pragma unroll
      for (int k = 0; k < KV; k++)
        if (k < x.steps) {
          float y[kE];
          vec_scaled<T>(x.keep[k], base, coef, y);
          vec_token<kE>((int32_t)token - x.index(k, 0), dlogp, y);
          x.write(d, aligned, k, y);
        }
    }
  }
}

// Rows too large for the buffers (beyond 8 x 112 KB): one CTA a part of a row,
// its passes read global memory again (L2).
template <typename T, int NT, bool kGrad>
__global__ __launch_bounds__(NT) void logprob_reread_kernel(const LogprobArgs a) {
  __shared__ uint64_t box[kMaxCluster];
  __shared__ uint64_t part[NT / 32];
  const uint32_t size = cluster_size(), rank = cluster_rank();
  cluster_begun();
  const int64_t row = blockIdx.x / size;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T *p = static_cast<const T *>(a.logits) + row * a.stride;
  Slice<T, 0, NT> x;
  x.set(p, a.vocab, rank, size);
  const int64_t token = a.tokens[row];
  const bool used = token >= 0 && token < a.vocab;
  const float xt = used ? Elem<T>::load(p + token) : 0.0f;   // before a gradient in place overwrites it
  const float dlogp = kGrad ? a.dlogps[row] : 0.0f;

  Part mine;
  for (int k = 0; k < x.steps; k += 4) {
    const uint4 v[4] = {x.read(k), x.read(k + 1), x.read(k + 2), x.read(k + 3)};
    mine.add<T, 4>(v);
  }
  const uint64_t of_warp = mine.of_warp();
  if (lane == 0) part[warp] = of_warp;
  __syncthreads();
  float m, s;
  join(part, NT / 32, m, s);
  cluster_wait_begun();
  cluster_post(pair(m, s), box, rank, size);   // no CTA reads or writes another's memory after this
  join(box, (int32_t)size, m, s);
  const float base = m == -INFINITY ? 0.0f : m;
  const bool nothing = s == 0.0f;
  if (rank == 0 && threadIdx.x == 0) {
    const float ln = logf(s);
    a.lses[row] = base + ln;
    a.logps[row] = used ? (nothing ? -INFINITY : (xt - base) - ln) : 0.0f;
  }
  if constexpr (kGrad) {
    T *d = static_cast<T *>(a.dlogits) + row * a.dstride;
    const bool aligned = same_alignment(d, x.off);
    const float coef = -__fdiv_rn(dlogp, s);
    if (!used || nothing) {
      write_zeros(x, d, aligned);
    } else {
      for (int k = 0; k < x.steps; k++) {
        float y[x.kE];
        vec_scaled<T>(x.read(k), base, coef, y);
        vec_token<x.kE>((int32_t)token - x.index(k, 0), dlogp, y);
        x.write(d, aligned, k, y);
      }
    }
  }
}

// With the row's lse given every element stands for itself: one read, one
// write, 64 bytes a thread on the way.  Bound by HBM: 2048 x 32768 fp32 80 us
// (6.7 of 6.8 TB/s).
template <typename T, int KV, int NT>
__global__ __launch_bounds__(NT) void backward_kernel(const LogprobArgs a) {
  const int64_t row = blockIdx.x / a.parts;
  Slice<T, KV, NT> x;
  x.set(static_cast<const T *>(a.logits) + row * a.stride, a.vocab, blockIdx.x % a.parts, a.parts);
  x.load();
  const int64_t token = a.tokens[row];
  const bool used = token >= 0 && token < a.vocab;
  const float lse = a.lses_in[row], g = used ? a.dlogps[row] : 0.0f;
  T *d = static_cast<T *>(a.dlogits) + row * a.dstride;
  const bool aligned = same_alignment(d, x.off);
  if (!used || lse == -INFINITY) {
    write_zeros(x, d, aligned);
  } else {
#pragma unroll
    for (int k = 0; k < KV; k++)
      if (k < x.steps) {
        float y[x.kE];
        vec_scaled<T>(x.keep[k], lse, -g, y);
        vec_token<x.kE>((int32_t)token - x.index(k, 0), g, y);
        x.write(d, aligned, k, y);
      }
  }
}

constexpr int kDevices = 16;           // whose occupancy is kept
constexpr int kShort = 12;             // steps of the rows that a warp takes by itself

constexpr size_t shared_bytes(int64_t steps) { return (size_t)steps * kBuffers * 32 * 16; }
constexpr int kMostSteps = (224 << 10) / (kBuffers * 32 * 16);   // of a row that a CTA has room for

// CTAs a row, and how many such clusters run at once.  Two buffers of up to 52
// KB let two CTAs share an SM (three up to 37 KB), so that some compute while
// copies for others are in flight; fewer CTAs a row are better than more.
// (8192 x 131072 bf16, gradient: 64 steps a CTA 695 us, 128 steps 957; 4000 x
// 50000: 98 steps 133 us, 49 steps 155.)
template <typename T, bool kGrad>
int choose_logprob(LogprobArgs a, cudaStream_t stream) {
  static std::atomic<int> fits[kDevices][4][kMostSteps + 1];   // clusters at once, by size and steps (0: not known)
  constexpr int kE = Elem<T>::kPerVec;
  const int64_t vecs = ((int64_t)a.vocab + kE - 1) / kE + 1;   // whatever the alignment
  const int64_t steps = (vecs + 31) / 32;
  if (steps <= kShort) {
    const int64_t ctas = (a.rows + 3) / 4;
    const cudaError_t e = steps <= 4   ? launch_rows(logprob_short_kernel<T, 4, kGrad>, a, ctas, 1, 128, 0, stream)
                          : steps <= 8 ? launch_rows(logprob_short_kernel<T, 8, kGrad>, a, ctas, 1, 128, 0, stream)
                                       : launch_rows(logprob_short_kernel<T, kShort, kGrad>, a, ctas, 1, 128, 0, stream);
    return e == cudaSuccess ? SEQSUM_OK : note_cuda(e);
  }
  int size = 1, log2 = 0;
  while (size < kMaxCluster && steps > (int64_t)size * 104) size *= 2, log2++;
  a.steps = (int32_t)((steps + size - 1) / size);
  cudaError_t e;
  if (a.steps > kMostSteps) {
    e = launch_rows(logprob_reread_kernel<T, 512, kGrad>, a, a.rows, kMaxCluster, 512, 0, stream);
    return e == cudaSuccess ? SEQSUM_OK : note_cuda(e);
  }
  auto kernel = logprob_kernel<T, kGrad>;
  constexpr int kThreads = kWarps * 32 + 32;
  const size_t shared = shared_bytes(a.steps);
  int device = 0, most = 0;
  if ((e = cudaGetDevice(&device)) != cudaSuccess) return note_cuda(e);
  if (device < kDevices) most = fits[device][log2][a.steps].load(std::memory_order_relaxed);
  if (most == 0) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)shared_bytes(kMostSteps));
    if (e == cudaSuccess) e = launch_rows(kernel, a, 1, size, kThreads, shared, stream, &most);
    if (e != cudaSuccess) return note_cuda(e);
    if (most < 1) return SEQSUM_ECUDA;
    if (device < kDevices) fits[device][log2][a.steps].store(most, std::memory_order_relaxed);
  }
  e = launch_rows(kernel, a, a.rows < most ? a.rows : most, size, kThreads, shared, stream);
  return e == cudaSuccess ? SEQSUM_OK : note_cuda(e);
}

template <typename T>
int run_backward(LogprobArgs &a, cudaStream_t stream) {
  constexpr int NT = 256, KV = 4;
  const int64_t vecs = ((int64_t)a.vocab + Elem<T>::kPerVec - 1) / Elem<T>::kPerVec + 1;
  a.parts = (int32_t)((vecs + NT * KV - 1) / (NT * KV));
  if (a.parts < 1) a.parts = 1;
  if (a.rows * a.parts > 0x7fffffff) return SEQSUM_EINVAL;
  const cudaError_t e = launch_rows(backward_kernel<T, KV, NT>, a, a.rows * a.parts, 1, NT, 0, stream);
  return e == cudaSuccess ? SEQSUM_OK : note_cuda(e);
}

bool bad_rows(const void *logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t stride) {
  if (rows < 0 || rows > SEQSUM_MAX_ROWS || vocab < 0 || vocab > kMaxVocab || stride < 0) return true;
  if (dtype != SEQSUM_FP32 && dtype != SEQSUM_FP16 && dtype != SEQSUM_BF16) return true;
  return rows > 0 && vocab > 0 && (!logits || reinterpret_cast<uintptr_t>(logits) % (dtype == SEQSUM_FP32 ? 4 : 2));
}

}  // namespace
}  // namespace sq

extern "C" {

int seqsum_token_logprob(const void *logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                         const int64_t *tokens, float *logps, float *lses, cudaStream_t stream) {
  if (sq::bad_rows(logits, dtype, rows, vocab, row_stride)) return SEQSUM_EINVAL;
  if (rows == 0) return SEQSUM_OK;
  if (!tokens || !logps || !lses) return SEQSUM_EINVAL;
  sq::LogprobArgs a = {logits, rows, row_stride, (int32_t)vocab, tokens, logps, lses, nullptr, nullptr, nullptr, 0, 1, 0, sq::row::waits()};
  if (dtype == SEQSUM_FP32) return sq::choose_logprob<float, false>(a, stream);
  if (dtype == SEQSUM_FP16) return sq::choose_logprob<__half, false>(a, stream);
  return sq::choose_logprob<__nv_bfloat16, false>(a, stream);
}

int seqsum_token_logprob_grad(const void *logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                              const int64_t *tokens, const float *dlogps, void *dlogits, int64_t drow_stride,
                              float *logps, float *lses, cudaStream_t stream) {
  if (sq::bad_rows(logits, dtype, rows, vocab, row_stride) || sq::bad_rows(dlogits, dtype, rows, vocab, drow_stride))
    return SEQSUM_EINVAL;
  if (rows == 0) return SEQSUM_OK;
  if (!tokens || !dlogps || !logps || !lses || (rows > 1 && drow_stride < vocab)) return SEQSUM_EINVAL;
  sq::LogprobArgs a = {logits, rows, row_stride, (int32_t)vocab, tokens, logps, lses, dlogps, nullptr, dlogits, drow_stride, 1, 0, sq::row::waits()};
  if (dtype == SEQSUM_FP32) return sq::choose_logprob<float, true>(a, stream);
  if (dtype == SEQSUM_FP16) return sq::choose_logprob<__half, true>(a, stream);
  return sq::choose_logprob<__nv_bfloat16, true>(a, stream);
}

int seqsum_token_logprob_backward(const void *logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                                  const int64_t *tokens, const float *dlogps, const float *lses, void *dlogits,
                                  int64_t drow_stride, cudaStream_t stream) {
  if (sq::bad_rows(logits, dtype, rows, vocab, row_stride) || sq::bad_rows(dlogits, dtype, rows, vocab, drow_stride))
    return SEQSUM_EINVAL;
  if (rows == 0 || vocab == 0) return SEQSUM_OK;
  if (!tokens || !dlogps || !lses || (rows > 1 && drow_stride < vocab)) return SEQSUM_EINVAL;
  sq::LogprobArgs a = {logits, rows, row_stride, (int32_t)vocab, tokens, nullptr, nullptr, dlogps, lses, dlogits, drow_stride, 1, 0, sq::row::waits()};
  if (dtype == SEQSUM_FP32) return sq::run_backward<float>(a, stream);
  if (dtype == SEQSUM_FP16) return sq::run_backward<__half>(a, stream);
  return sq::run_backward<__nv_bfloat16>(a, stream);
}

}  // extern "C"
