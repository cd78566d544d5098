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

// The sum of a slice's exponentials in units of 2^-38; `bad` where one is no number.
template <typename S>
__device__ __forceinline__ uint64_t sum_exps(const S &x, float base, bool &bad) {
  uint64_t sum = 0;
  float check = 0.0f;
  x.each([&](int, const float *v) {
    float s[S::kE];
    exps<S::kE>(v, base, s);
    uint64_t t[S::kE / 2];
#pragma unroll
    for (int e = 0; e < S::kE / 2; e++) t[e] = pair(s[e], s[e + S::kE / 2]);
#pragma unroll
    for (int o = S::kE / 4; o; o >>= 1)
#pragma unroll
      for (int e = 0; e < o; e++) t[e] = add2(t[e], t[e + o]);
    float p, q;
    split(t[0], p, q);
    p += q;
    check += p;
    sum += __float2ull_rn(p * kUnit);   // (0 for NaN)
  });
  bad = !(check < INFINITY);
  return sum;
}

// Writes a slice's gradient: coef * exponential, and `g` more at the token.
template <typename S, typename T>
__device__ __forceinline__ void write_gradient(const S &x, float base, T *d, bool aligned, float coef, float g,
                                               int64_t token) {
  const int32_t token_vec = (int32_t)((token + x.off) / S::kE);
  const uint64_t c = pair(coef, coef);
  x.each([&](int k, const float *v) {
    float y[S::kE];
    exps<S::kE>(v, base, y);
#pragma unroll
    for (int e = 0; e < S::kE; e += 2) split(mul2(pair(y[e], y[e + 1]), c), y[e], y[e + 1]);
    if (x.first + 32 * k == token_vec) {
#pragma unroll
      for (int e = 0; e < S::kE; e++)
        if (x.index(k, e) == token) y[e] += g;
    }
    x.write(d, aligned, k, y);
  });
}

template <typename S, typename T>
__device__ __forceinline__ void write_zeros(const S &x, T *d, bool aligned) {
  float y[S::kE] = {};
  for (int k = 0; k < x.steps; k++) x.write(d, aligned, k, y);
}

template <typename T>
__device__ __forceinline__ bool same_alignment(const T *d, int32_t off) {
  return (reinterpret_cast<uintptr_t>(d) & 15) / sizeof(T) == (uintptr_t)off;
}

template <typename T, int KV, int NT, int kCtas, bool kGrad>
__global__ __launch_bounds__(NT, kCtas) void logprob_kernel(const LogprobArgs a) {
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
  const float dlogp = kGrad ? a.dlogps[row] : 0.0f;

  float m = warp_max(x.largest());
  if (lane == 0) pmax[warp] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NT / 32; i++) m = fmaxf(m, pmax[i]);
  cluster_post(__float_as_uint(m), box[0], rank, size);
  for (uint32_t r = 0; r < size; r++) m = fmaxf(m, __uint_as_float((uint32_t)box[0][r]));
  // a row of nothing but -inf: every exponential is 0 (with NaN beside them: m is -inf, but the sum is NaN)
  const float base = m == -INFINITY ? 0.0f : m;

  bool bad;
  uint64_t sum = sum_exps(x, base, bad);
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
    if (!used || nothing) write_zeros(x, d, aligned);
    else write_gradient(x, base, d, aligned, coef, dlogp, token);
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
  if (!used || lse == -INFINITY) write_zeros(x, d, aligned);
  else write_gradient(x, lse, d, aligned, -g, g, token);
}

template <typename T, int KV, int NT, int kCtas, bool kGrad>
int run_logprob(const LogprobArgs &a, int size, cudaStream_t stream) {
  const cudaError_t e = launch_rows(logprob_kernel<T, KV, NT, kCtas, kGrad>, a, a.rows, size, NT, stream);
  return e == cudaSuccess ? SEQSUM_OK : note_cuda(e);
}

// The smallest cluster and vectors a thread that hold a row, more CTAs where
// the rows are few.
template <typename T, bool kGrad>
int choose_logprob(const LogprobArgs &a, cudaStream_t stream) {
  const int64_t vecs = ((int64_t)a.vocab + Elem<T>::kPerVec - 1) / Elem<T>::kPerVec + 1;   // whatever the alignment
  const int sms = multiprocessors();
  int size = 1;
  while (size < kMaxCluster && (vecs > (int64_t)size * 256 * 8 || a.rows * size * 2 <= sms)) size *= 2;
  const int64_t mine = (vecs + size - 1) / size;
  if (mine <= 256) return run_logprob<T, 1, 256, 8, kGrad>(a, size, stream);
  if (mine <= 512) return run_logprob<T, 2, 256, 6, kGrad>(a, size, stream);
  if (mine <= 1024) return run_logprob<T, 4, 256, 5, kGrad>(a, size, stream);
  if (mine <= 2304) return run_logprob<T, 9, 256, 4, kGrad>(a, size, stream);
  if (mine <= 4608) return run_logprob<T, 9, 512, 2, kGrad>(a, size, stream);
  return run_logprob<T, 0, 512, 3, kGrad>(a, size, stream);
}

template <typename T>
int run_backward(LogprobArgs &a, cudaStream_t stream) {
  constexpr int NT = 256, KV = 4;
  const int64_t vecs = ((int64_t)a.vocab + Elem<T>::kPerVec - 1) / Elem<T>::kPerVec + 1;
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
