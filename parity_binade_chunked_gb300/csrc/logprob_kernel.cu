// Log-probabilities of given tokens and their gradient with respect to the
// logits (seqsum_token_logprob, _grad, _backward).
//
//   lse = m + ln sum exp(x_i - m),  logp = x_t - lse,
//   d logits_i = dlogp * ([i = t] - exp(x_i - lse))
//
// The exponentials of a 16-byte vector are added in fp32, the vectors' sums
// as integers (2^-38 a unit): the row's sum does not depend on how it is
// split over threads and CTAs, so a row's results do not depend on the other
// rows of the call.
#include <math.h>

#include <atomic>

#include "../../include/seqsum.h"
#include "row_slice.cuh"

namespace sq {
namespace {

using namespace row;

constexpr float kLog2e = 1.44269504f;
constexpr float kUnit = 274877906944.0f;             // 2^38: at most 2^22 vectors of at most 4, or 2^21 of 8
constexpr uint64_t kBad = 1ull << 63;                // marks a sum with something in it that is no number

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
  int32_t blocks;                                    // blocks of 128 vectors a CTA takes of a row
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

// x, at most 32, in units of 2^-38: two halves, each rounded to an integer by
// adding a number whose last place is 1 (a conversion to 64 bits goes through
// the fp64 pipe, of which this GPU has little).
__device__ __forceinline__ uint64_t fixed38(float x) {
  const float big = x * 131072.0f, h = big + 8388608.0f, rest = __fmaf_rn(x, 131072.0f, -(h - 8388608.0f));
  const float l = __fmaf_rn(rest, 2097152.0f, 12582912.0f);
  return (uint64_t)((int64_t)(__float_as_int(h) - 0x4b000000) * 2097152 + (__float_as_int(l) - 0x4b400000));
}

// Writes a vector's gradient: coef * exponential, and `g` more at the token.
template <typename T, typename S>
__device__ __forceinline__ void vec_gradient(const S &x, int32_t vec, uint4 w, float base, T *d, bool aligned, float coef,
                                             float g, int32_t token) {
  constexpr int kE = Elem<T>::kPerVec;
  float v[kE], y[kE];
  Elem<T>::unpack(w, v);
  exps<kE>(v, base, y);
  const uint64_t c = pair(coef, coef);
#pragma unroll
  for (int e = 0; e < kE; e += 2) split(mul2(pair(y[e], y[e + 1]), c), y[e], y[e + 1]);
  const int32_t at = token - x.index(vec, 0);
  if (at >= 0 && at < kE) {
#pragma unroll
    for (int e = 0; e < kE; e++)
      if (e == at) y[e] += g;
  }
  x.write(d, aligned, vec, y);
}

template <typename S, typename T>
__device__ __forceinline__ void write_zeros(const S &x, T *d, bool aligned) {
  const float y[S::kE] = {};
  for (int k = 0; k < x.steps; k++) x.write(d, aligned, k, y);
}

template <typename T>
__device__ __forceinline__ bool same_alignment(const T *d, int32_t off) {
  return (reinterpret_cast<uintptr_t>(d) & 15) / sizeof(T) == (uintptr_t)off;
}

template <int NT>
struct LogprobShared {
  Exchange<NT> top, sum;
  uint64_t full[2];
};

// A cluster's rows one after another (see Stream): the maximum, the sum, the
// gradient, each a pass over the row's buffer.
template <typename T, int NT, bool kGrad>
__global__ __launch_bounds__(NT) void logprob_kernel(const LogprobArgs a) {
  extern __shared__ uint4 buffers[];
  __shared__ LogprobShared<NT> sh;
  constexpr int kE = Elem<T>::kPerVec, kBoxes = kMaxCluster * (NT / 32);
  const uint32_t size = cluster_size(), rank = cluster_rank();
  const int lane = threadIdx.x & 31;
  const int64_t first = blockIdx.x / size, step = gridDim.x / size;
  if (threadIdx.x == 0) {
    sh.top.init(size);
    sh.sum.init(size);
    bar_init(&sh.full[0], 1);
    bar_init(&sh.full[1], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  auto stream = [&](int64_t row, int b) {
    Stream<T, NT> x;
    x.set(static_cast<const T *>(a.logits) + row * a.stride, a.vocab, a.blocks, rank, buffers + b * a.blocks * 128);
    return x;
  };
  uint4 head, tail;
  if (threadIdx.x == 0) {
    stream(first, 0).copy(&sh.full[0]);
    if (first + step < a.rows) stream(first + step, 1).copy(&sh.full[1]);
  }
  stream(first, 0).read_edges(head, tail);
  cluster_sync();   // every CTA's barriers are ready

  bool ok = true;
  uint32_t it = 0;
  for (int64_t row = first; row < a.rows && ok; row += step, it++) {
    const Stream<T, NT> x = stream(row, it & 1);
    const int64_t token = a.tokens[row];
    const bool used = token >= 0 && token < a.vocab;
    const float dlogp = kGrad ? a.dlogps[row] : 0.0f;
    x.put_edges(head, tail);
    if (row + step < a.rows) stream(row + step, 0).read_edges(head, tail);
    ok &= bar_wait(&sh.full[it & 1], (it >> 1) & 1);

    float m = -INFINITY;
    x.blocks([&](int32_t, const uint4 *v) {
#pragma unroll
      for (int s = 0; s < 4; s++) m = Elem<T>::vec_max(v[s], m);
    });
    sh.top.post(__float_as_uint(warp_max_all(m)), rank, size);
    ok &= sh.top.wait(it & 1, size);
    // every warp has left the row before: its buffer is free
    if (threadIdx.x == 0 && it > 0 && row + step < a.rows) stream(row + step, (it + 1) & 1).copy(&sh.full[(it + 1) & 1]);
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kBoxes; i += 32)
      if (i + lane < (int)size * (NT / 32)) m = fmaxf(m, __uint_as_float((uint32_t)sh.top.box[i + lane]));
    m = warp_max_all(m);
    // a row of nothing but -inf: every exponential is 0 (with NaN beside them: m is -inf, but the sum is NaN)
    const float base = m == -INFINITY ? 0.0f : m;

    uint64_t sum = 0;
    float check = 0.0f;
    x.blocks([&](int32_t, const uint4 *v) {
      float t[4];
#pragma unroll
      for (int s = 0; s < 4; s++) t[s] = vec_sum<T>(v[s], base);
      const float q = (t[0] + t[1]) + (t[2] + t[3]);
      check += q;
      sum += fixed38(q);
    });
    const bool none = __any_sync(~0u, !(check < INFINITY));   // some exponential is no number
    sh.sum.post(none ? kBad : warp_sum_62(sum), rank, size);
    ok &= sh.sum.wait(it & 1, size);
    bool bad = false;
    sum = 0;
#pragma unroll
    for (int i = 0; i < kBoxes; i += 32)
      if (i + lane < (int)size * (NT / 32)) {
        const uint64_t v = sh.sum.box[i + lane];
        bad |= (v & kBad) != 0;
        sum += v & ~kBad;
      }
    bad = __any_sync(~0u, bad) || !ok;
    sum = warp_sum_62(sum);
    const float s = bad ? NAN : (float)sum * (1.0f / kUnit);
    const bool nothing = m == -INFINITY && !bad;
    const float ln = logf(s);
    if (rank == 0 && threadIdx.x == 0) {
      a.lses[row] = base + ln;
      if (!used) a.logps[row] = 0.0f;
    }
    const int32_t vec = (int32_t)(token + x.off) / kE - x.begin;   // the token's
    if (used && vec >= 0 && vec < x.n && x.owns(vec)) {
      float v[kE], xt = 0.0f;
      Elem<T>::unpack(x.buf[vec], v);
#pragma unroll
      for (int e = 0; e < kE; e++)
        if (x.index(vec, e) == token) xt = v[e];
      a.logps[row] = nothing ? -INFINITY : (xt - base) - ln;
    }
    if constexpr (kGrad) {
      T *d = static_cast<T *>(a.dlogits) + row * a.dstride;
      const bool aligned = same_alignment(d, x.off);
      const float coef = -__fdiv_rn(dlogp, s);
      const bool zero = !used || nothing;
      x.blocks([&](int32_t vec, const uint4 *v) {
#pragma unroll
        for (int s = 0; s < 4; s++) {
          if (zero) {
            const float y[kE] = {};
            x.write(d, aligned, vec + 32 * s, y);
          } else {
            vec_gradient<T>(x, vec + 32 * s, v[s], base, d, aligned, coef, dlogp, (int32_t)token);
          }
        }
      });
    }
    ok = __all_sync(~0u, ok);
  }
  if (!ok) {
    // a wait gave up: what is not done is marked, copies in flight may land before the CTA goes
    for (int64_t row = first; row < a.rows; row += step)
      if (rank == 0 && threadIdx.x == 0 && (row - first) / step >= (int64_t)it - 1) a.lses[row] = a.logps[row] = NAN;
    bar_wait(&sh.full[it & 1], (it >> 1) & 1);
    bar_wait(&sh.full[(it - 1) & 1], ((it - 1) >> 1) & 1);
  }
  cluster_sync();
}

// Rows too large for the buffers: one CTA a part of a row, its passes read
// global memory (L2).
template <typename T, int NT, bool kGrad>
__global__ __launch_bounds__(NT) void logprob_reread_kernel(const LogprobArgs a) {
  __shared__ uint64_t box[2][kMaxCluster];
  __shared__ uint64_t part[NT / 32];
  const uint32_t size = cluster_size(), rank = cluster_rank();
  const int64_t row = blockIdx.x / size;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T *p = static_cast<const T *>(a.logits) + row * a.stride;
  Slice<T, 0, NT> x;
  x.set(p, a.vocab, rank, size);
  const int64_t token = a.tokens[row];
  const bool used = token >= 0 && token < a.vocab;
  const float xt = used ? Elem<T>::load(p + token) : 0.0f;   // before a gradient in place overwrites it
  const float dlogp = kGrad ? a.dlogps[row] : 0.0f;

  float m = warp_max_all(x.largest());
  if (lane == 0) part[warp] = __float_as_uint(m);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NT / 32; i++) m = fmaxf(m, __uint_as_float((uint32_t)part[i]));
  cluster_post(__float_as_uint(m), box[0], rank, size);
  for (uint32_t r = 0; r < size; r++) m = fmaxf(m, __uint_as_float((uint32_t)box[0][r]));
  const float base = m == -INFINITY ? 0.0f : m;

  uint64_t sum = 0;
  float check = 0.0f;
  for (int k = 0; k < x.steps; k++) {
    const float q = vec_sum<T>(x.read(k), base);
    check += q;
    sum += fixed38(q);
  }
  const bool bad = __any_sync(~0u, !(check < INFINITY));
  sum = warp_sum_62(sum);
  __syncthreads();
  if (lane == 0) part[warp] = bad ? kBad : sum;
  __syncthreads();
  uint64_t all = 0, flag = 0;
#pragma unroll
  for (int i = 0; i < NT / 32; i++) all += part[i] & ~kBad, flag |= part[i] & kBad;
  cluster_post(all | flag, box[1], rank, size);   // no CTA reads or writes another's memory after this
  all = flag = 0;
  for (uint32_t r = 0; r < size; r++) all += box[1][r] & ~kBad, flag |= box[1][r] & kBad;
  const float s = flag ? NAN : (float)all * (1.0f / kUnit);
  const bool nothing = m == -INFINITY && !flag;
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
      for (int k = 0; k < x.steps; k++) vec_gradient<T>(x, k, x.read(k), base, d, aligned, coef, dlogp, (int32_t)token);
    }
  }
}

// With the row's lse given every element stands for itself.
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
      if (k < x.steps) vec_gradient<T>(x, k, x.keep[k], lse, d, aligned, -g, g, (int32_t)token);
  }
}

constexpr int kThreads = 256;
constexpr int kDevices = 16;                           // whose occupancy is kept
constexpr int kMostBlocks = 54;                        // two buffers of 108 KB

// CTAs a row, and how many such clusters run at once.  Three CTAs with two
// buffers of 32 KB keep an SM's share of copies in flight while others
// compute; where the rows are few, more and smaller CTAs shorten each row.
template <typename T, bool kGrad>
int choose_logprob(LogprobArgs a, cudaStream_t stream) {
  static std::atomic<int> fits[kDevices][4][kMostBlocks + 1];   // clusters at once, by their size and blocks (0: not known)
  const int64_t vecs = ((int64_t)a.vocab + Elem<T>::kPerVec - 1) / Elem<T>::kPerVec + 1;   // whatever the alignment
  const int64_t blocks = (vecs + 127) / 128;
  const int sms = multiprocessors();
  int size = 1, log2 = 0;
  while (size < kMaxCluster && (blocks > (int64_t)size * 16 || a.rows * size * 2 <= sms)) size *= 2, log2++;
  a.blocks = (int32_t)((blocks + size - 1) / size);
  cudaError_t e;
  if (a.blocks > kMostBlocks) {
    e = launch_rows(logprob_reread_kernel<T, 512, kGrad>, a, a.rows, size, 512, 0, stream);
    return e == cudaSuccess ? SEQSUM_OK : note_cuda(e);
  }
  auto kernel = logprob_kernel<T, kThreads, kGrad>;
  const size_t shared = (size_t)a.blocks * 2 * 128 * 16;
  int device = 0, most = 0;
  if ((e = cudaGetDevice(&device)) != cudaSuccess) return note_cuda(e);
  if (device < kDevices) most = fits[device][log2][a.blocks].load(std::memory_order_relaxed);
  if (most == 0) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostBlocks * 2 * 128 * 16);
    if (e == cudaSuccess) e = launch_rows(kernel, a, 1, size, kThreads, shared, stream, &most);
    if (e != cudaSuccess) return note_cuda(e);
    if (most < 1) return SEQSUM_ECUDA;
    if (device < kDevices) fits[device][log2][a.blocks].store(most, std::memory_order_relaxed);
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
  sq::LogprobArgs a = {logits, rows, row_stride, (int32_t)vocab, tokens, logps, lses, nullptr, nullptr, nullptr, 0, 1, 0};
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
  sq::LogprobArgs a = {logits, rows, row_stride, (int32_t)vocab, tokens, logps, lses, dlogps, nullptr, dlogits, drow_stride, 1, 0};
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
  sq::LogprobArgs a = {logits, rows, row_stride, (int32_t)vocab, tokens, nullptr, nullptr, dlogps, lses, dlogits, drow_stride, 1, 0};
  if (dtype == SEQSUM_FP32) return sq::run_backward<float>(a, stream);
  if (dtype == SEQSUM_FP16) return sq::run_backward<__half>(a, stream);
  return sq::run_backward<__nv_bfloat16>(a, stream);
}

}  // extern "C"
