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

#include "../../include/seqsum.h"
#include "row_slice.cuh"

namespace sq {
namespace {

using namespace row;

constexpr float kLog2e = 1.44269504f;
constexpr float kLn2 = 0.69314718f;
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
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T, int KV, int NT, bool kGrad>
__global__ __launch_bounds__(NT) void logprob_kernel(const LogprobArgs a) {
  __shared__ uint64_t box[2][kMaxCluster];
  __shared__ uint64_t part[NT / 32];
  __shared__ float pmax[NT / 32];
  const uint32_t size = cluster_size(), rank = cluster_rank();
  const int64_t row = blockIdx.x / size;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T *p = static_cast<const T *>(a.logits) + row * a.stride;
  Slice<T, KV, NT> x;
  x.set(p, a.vocab, rank, size);
  x.load();
  const int64_t token = a.tokens[row];
  const bool used = token >= 0 && token < a.vocab;
  const float xt = used ? Elem<T>::load(p + token) : 0.0f;   // before a gradient in place overwrites it

  float m = -INFINITY;
  x.each([&](int, const float *v) {
#pragma unroll
    for (int e = 0; e < x.kE; e++) m = fmaxf(m, v[e]);
  });
  m = warp_max(m);
  if (lane == 0) pmax[warp] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NT / 32; i++) m = fmaxf(m, pmax[i]);
  cluster_post(__float_as_uint(m), box[0], rank, size);
  for (uint32_t r = 0; r < size; r++) m = fmaxf(m, __uint_as_float((uint32_t)box[0][r]));
  // a row of nothing but -inf: every exponential is 0 (of NaN: m is -inf, but the sum is NaN)
  const float base = m == -INFINITY ? 0.0f : m;

  uint64_t sum = 0;
  bool bad = false;   // some exponential is no number
  x.each([&](int, const float *v) {
    float s[x.kE];
#pragma unroll
    for (int e = 0; e < x.kE; e++) s[e] = ex2((v[e] - base) * kLog2e);
#pragma unroll
    for (int o = x.kE / 2; o; o >>= 1)
#pragma unroll
      for (int e = 0; e < o; e++) s[e] += s[e + o];
    bad |= !(s[0] < INFINITY);
    sum += __float2ull_rn(s[0] * kUnit);   // (0 for NaN)
  });
  bad = __any_sync(~0u, bad);
  sum = warp_sum(sum);
  if (lane == 0) part[warp] = sum | (bad ? kBad : 0);
  __syncthreads();
  uint64_t all = 0, flag = 0;
#pragma unroll
  for (int i = 0; i < NT / 32; i++) all += part[i] & ~kBad, flag |= part[i] & kBad;
  cluster_post(all | flag, box[1], rank, size);   // no CTA reads or writes another's memory after this
  all = flag = 0;
  for (uint32_t r = 0; r < size; r++) all += box[1][r] & ~kBad, flag |= box[1][r] & kBad;
  const float s = flag ? NAN : (float)all * (1.0f / kUnit);
  const float ln = logf(s);
  if (rank == 0 && threadIdx.x == 0) {
    a.lses[row] = base + ln;
    a.logps[row] = used ? (m == -INFINITY && !flag ? -INFINITY : (xt - base) - ln) : 0.0f;
  }
  if constexpr (kGrad) {
    T *d = static_cast<T *>(a.dlogits) + row * a.dstride;
    const bool aligned = (reinterpret_cast<uintptr_t>(d) & 15) / sizeof(T) == (uintptr_t)x.off;
    const bool zero = !used || (m == -INFINITY && !flag);
    const float g = zero ? 0.0f : a.dlogps[row];
    const float coef = -__fdiv_rn(g, s);
    x.each([&](int k, const float *v) {
      float y[x.kE];
#pragma unroll
      for (int e = 0; e < x.kE; e++) {
        y[e] = ex2((v[e] - base) * kLog2e) * coef;
        if (x.index(k, e) == token) y[e] += g;
        if (zero) y[e] = 0.0f;
      }
      x.write(d, aligned, k, y);
    });
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
  const bool zero = !used || lse == -INFINITY;
  T *d = static_cast<T *>(a.dlogits) + row * a.dstride;
  const bool aligned = (reinterpret_cast<uintptr_t>(d) & 15) / sizeof(T) == (uintptr_t)x.off;
  x.each([&](int k, const float *v) {
    float y[x.kE];
#pragma unroll
    for (int e = 0; e < x.kE; e++) {
      y[e] = ex2((v[e] - lse) * kLog2e) * -g;
      if (x.index(k, e) == token) y[e] += g;
      if (zero) y[e] = 0.0f;
    }
    x.write(d, aligned, k, y);
  });
}

template <typename T, int KV, int NT, bool kGrad>
int run_logprob(const LogprobArgs &a, int size, cudaStream_t stream) {
  const cudaError_t e = launch_rows(logprob_kernel<T, KV, NT, kGrad>, a, a.rows, size, NT, stream);
  return e == cudaSuccess ? SEQSUM_OK : note_cuda(e);
}

// The smallest cluster and vectors a thread that hold a row, more CTAs where
// the rows are few.
template <typename T, bool kGrad>
int choose_logprob(const LogprobArgs &a, cudaStream_t stream) {
  constexpr int NT = 512;
  const int64_t vecs = ((int64_t)a.vocab + 2 * Elem<T>::kPerVec - 2) / Elem<T>::kPerVec;   // whatever the alignment
  const int sms = multiprocessors();
  int size = 1;
  while (size < kMaxCluster && (vecs > (int64_t)size * NT * 8 || a.rows * size * 2 <= sms)) size *= 2;
  const int64_t per = ((vecs + size - 1) / size + NT - 1) / NT;
  if (per <= 1) return run_logprob<T, 1, NT, kGrad>(a, size, stream);
  if (per <= 2) return run_logprob<T, 2, NT, kGrad>(a, size, stream);
  if (per <= 4) return run_logprob<T, 4, NT, kGrad>(a, size, stream);
  if (per <= 8) return run_logprob<T, 8, NT, kGrad>(a, size, stream);
  return run_logprob<T, 0, NT, kGrad>(a, size, stream);
}

template <typename T>
int run_backward(LogprobArgs &a, cudaStream_t stream) {
  constexpr int NT = 256, KV = 4;
  const int64_t vecs = ((int64_t)a.vocab + 2 * Elem<T>::kPerVec - 2) / Elem<T>::kPerVec;
  a.parts = (int32_t)((vecs + NT * KV - 1) / (NT * KV));
  if (a.parts < 1) a.parts = 1;
  if (a.rows * a.parts > 0x7fffffff) return SEQSUM_EINVAL;
  const cudaError_t e = launch_rows(backward_kernel<T, KV, NT>, a, a.rows * a.parts, 1, NT, stream);
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
  sq::LogprobArgs a = {logits, rows, row_stride, (int32_t)vocab, tokens, logps, lses, nullptr, nullptr, nullptr, 0, 1};
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
  sq::LogprobArgs a = {logits, rows, row_stride, (int32_t)vocab, tokens, logps, lses, dlogps, nullptr, dlogits, drow_stride, 1};
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
  sq::LogprobArgs a = {logits, rows, row_stride, (int32_t)vocab, tokens, nullptr, nullptr, dlogps, lses, dlogits, drow_stride, 1};
  if (dtype == SEQSUM_FP32) return sq::run_backward<float>(a, stream);
  if (dtype == SEQSUM_FP16) return sq::run_backward<__half>(a, stream);
  return sq::run_backward<__nv_bfloat16>(a, stream);
}

}  // extern "C"
