// The norm of all numbers of many tensors, and the tensors scaled to a
// largest norm (seqsum_tensors_norm, seqsum_tensors_clip).
//
// The order of the sum is fixed: a tensor is cut into chunks of 16384
// elements, a chunk's squares are added in fp32 in one shape (a thread's
// chains, then trees), the chunks' sums in double in one shape.  Which CTA
// takes which chunk does not matter, so the norm's bits depend on the numbers
// and the tensors' sizes alone.
#include <math.h>

#include <new>
#include <vector>

#include "../../include/seqsum.h"
#include "row_slice.cuh"

namespace sq {
namespace {

using row::Elem;

constexpr int kChunk = 16384;
constexpr int kThreads = 256;

struct Chunk {
  const void *in;
  void *out;
  int32_t n;
  int8_t type, out_type;
  int8_t aligned;      // both 16-byte aligned
  int8_t in_place;
};

struct TensorsArgs {
  const Chunk *chunks;
  int64_t nchunks;
  double *parts;
  uint32_t *ticket;
  float *factor;
  float *norm;
  float scale, max_norm;
};

template <typename T>
__device__ __forceinline__ void add_squares(uint4 v, float *acc) {
  float x[Elem<T>::kPerVec];
  Elem<T>::unpack(v, x);
#pragma unroll
  for (int e = 0; e < Elem<T>::kPerVec; e++) acc[e] = __fmaf_rn(x[e], x[e], acc[e]);
}

__device__ __forceinline__ float warp_add(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
__device__ __forceinline__ double warp_add(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
// the same tree in every thread
template <typename S>
__device__ __forceinline__ S block_add(S v, S *sh) {
  v = warp_add(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  v = sh[threadIdx.x & (kThreads / 32 - 1)];
#pragma unroll
  for (int o = kThreads / 64; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// Vector j of a chunk, 0 past its end; element by element where the chunk is
// not aligned or ends inside the vector.
template <typename T>
__device__ __forceinline__ uint4 chunk_vec(const T *p, int n, bool aligned, int j) {
  constexpr int E = Elem<T>::kPerVec;
  const int i = j * E;
  if (aligned && i + E <= n) return *reinterpret_cast<const uint4 *>(p + i);
  if (i >= n) return make_uint4(0, 0, 0, 0);
  float x[E];
#pragma unroll
  for (int e = 0; e < E; e++) x[e] = i + e < n ? Elem<T>::load(p + i + e) : 0.0f;
  return Elem<T>::pack(x);
}

template <typename T>
__device__ __forceinline__ float chunk_squares(const Chunk &c, float *sh) {
  constexpr int E = Elem<T>::kPerVec;
  constexpr int kSteps = kChunk / E / kThreads;
  const T *p = static_cast<const T *>(c.in);
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; e++) acc[e] = 0.0f;
#pragma unroll
  for (int h = 0; h < kSteps; h += 8) {
    uint4 v[8];
#pragma unroll
    for (int k = 0; k < 8; k++) v[k] = chunk_vec(p, c.n, c.aligned, (h + k) * kThreads + threadIdx.x);
#pragma unroll
    for (int k = 0; k < 8; k++) add_squares<T>(v[k], acc);
  }
#pragma unroll
  for (int o = E / 2; o; o >>= 1)
#pragma unroll
    for (int e = 0; e < o; e++) acc[e] += acc[e + o];
  return block_add(acc[0], sh);
}

// A chunk whose fp32 sum left the range in which it can be trusted: its
// squares in double, where those of every fp32 number are normal numbers.
template <typename T>
__device__ __noinline__ double chunk_squares_wide(const Chunk &c, double *sh) {
  const T *p = static_cast<const T *>(c.in);
  bool any = false;
  for (int i = threadIdx.x; i < c.n; i += kThreads) any |= Elem<T>::load(p + i) != 0.0f;
  if (!__syncthreads_or(any)) return 0.0;
  double s = 0.0;
  for (int i = threadIdx.x; i < c.n; i += kThreads) {
    const double x = Elem<T>::load(p + i);
    s += x * x;
  }
  return block_add(s, sh);
}

template <typename T>
__device__ __forceinline__ void chunk_part(const Chunk &c, double *part, float *sh, double *shd) {
  const float s = chunk_squares<T>(c, sh);
  double total = s;
  // below 2^-80 squares that left fp32's range could count; above all of it, the sum did
  if (!(s >= 8.2718061e-25f && s < INFINITY)) total = chunk_squares_wide<T>(c, shd);
  if (threadIdx.x == 0) *part = total;
}

__global__ __launch_bounds__(kThreads) void norm_kernel(const TensorsArgs a) {
  __shared__ float sh[kThreads / 32];
  __shared__ double shd[kThreads / 32];
  __shared__ bool last;
  for (int64_t i = blockIdx.x; i < a.nchunks; i += gridDim.x) {
    const Chunk c = a.chunks[i];
    if (c.type == SEQSUM_FP32) chunk_part<float>(c, &a.parts[i], sh, shd);
    else if (c.type == SEQSUM_FP16) chunk_part<__half>(c, &a.parts[i], sh, shd);
    else chunk_part<__nv_bfloat16>(c, &a.parts[i], sh, shd);
  }
  // the CTA that is done last adds the chunks' sums
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < a.nchunks; i += kThreads) s += __ldcg(&a.parts[i]);
  s = block_add(s, shd);
  if (threadIdx.x == 0) {
    *a.ticket = 0;
    const float norm = (float)(sqrt(s) * (double)a.scale);
    *a.norm = norm;
    const float q = __fdiv_rn(a.max_norm, norm + 1e-6f);
    *a.factor = (q > 1.0f ? 1.0f : q) * a.scale;   // NaN stays
  }
}

template <typename T, typename O>
__device__ __forceinline__ void chunk_scale(const Chunk &c, float f) {
  constexpr int E = Elem<T>::kPerVec, F = Elem<O>::kPerVec;
  constexpr int kSteps = kChunk / E / kThreads;
  const T *p = static_cast<const T *>(c.in);
  O *q = static_cast<O *>(c.out);
#pragma unroll
  for (int h = 0; h < kSteps; h += 4) {
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; k++) v[k] = chunk_vec(p, c.n, c.aligned, (h + k) * kThreads + threadIdx.x);
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const int i = ((h + k) * kThreads + threadIdx.x) * E;
      float x[E];
      Elem<T>::unpack(v[k], x);
#pragma unroll
      for (int e = 0; e < E; e++) x[e] *= f;
      if (c.aligned && i + E <= c.n) {
        if constexpr (F > E) {   // fp32 to 16 bits: half a vector
          float y[F] = {};
#pragma unroll
          for (int e = 0; e < E; e++) y[e] = x[e];
          const uint4 w = Elem<O>::pack(y);
          *reinterpret_cast<uint2 *>(q + i) = make_uint2(w.x, w.y);
        } else {
#pragma unroll
          for (int e = 0; e < E; e += F) *reinterpret_cast<uint4 *>(q + i + e) = Elem<O>::pack(x + e);
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; e++)
          if (i + e < c.n) Elem<O>::store(q + i + e, x[e]);
      }
    }
  }
}

template <typename T>
__device__ __forceinline__ void chunk_scale_to(const Chunk &c, float f) {
  if (c.out_type == SEQSUM_FP32) chunk_scale<T, float>(c, f);
  else if (c.out_type == SEQSUM_FP16) chunk_scale<T, __half>(c, f);
  else chunk_scale<T, __nv_bfloat16>(c, f);
}

__global__ __launch_bounds__(kThreads) void clip_kernel(const TensorsArgs a) {
  const float f = *a.factor;
  for (int64_t i = blockIdx.x; i < a.nchunks; i += gridDim.x) {
    const Chunk c = a.chunks[a.nchunks - 1 - i];   // the last ones read are still in L2
    if (c.in_place && f == 1.0f) continue;         // x * 1 is x
    if (c.type == SEQSUM_FP32) chunk_scale_to<float>(c, f);
    else if (c.type == SEQSUM_FP16) chunk_scale_to<__half>(c, f);
    else chunk_scale_to<__nv_bfloat16>(c, f);
  }
}

int bytes_of(int32_t dtype) { return dtype == SEQSUM_FP32 ? 4 : dtype == SEQSUM_FP16 || dtype == SEQSUM_BF16 ? 2 : 0; }

}  // namespace
}  // namespace sq

struct seqsum_tensors {
  int device = -1;
  int64_t nchunks = 0;
  sq::Chunk *chunks = nullptr;
  double *parts = nullptr;
  uint32_t *ticket = nullptr;   // and, after it, the factor
  int sms = 0;
};

namespace {

int run_tensors(seqsum_tensors *t, float max_norm, float scale, float *norm, bool clip, cudaStream_t stream) {
  if (!t || !norm) return SEQSUM_EINVAL;
  sq::TensorsArgs a = {t->chunks, t->nchunks, t->parts, t->ticket, reinterpret_cast<float *>(t->ticket + 1), norm,
                       scale, max_norm};
  const int64_t most = (int64_t)t->sms * 8;
  int64_t grid = t->nchunks < most ? t->nchunks : most;
  if (grid < 1) grid = 1;
  sq::norm_kernel<<<(unsigned)grid, sq::kThreads, 0, stream>>>(a);
  if (clip && t->nchunks > 0) sq::clip_kernel<<<(unsigned)grid, sq::kThreads, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SEQSUM_OK : sq::note_cuda(e);
}

}  // namespace

extern "C" {

int seqsum_tensors_create(const seqsum_tensor *tensors, int32_t n, seqsum_tensors **out) {
  if (!out || n < 0 || (n > 0 && !tensors)) return SEQSUM_EINVAL;
  *out = nullptr;
  int64_t nchunks = 0;
  for (int32_t i = 0; i < n; i++) {
    const seqsum_tensor &t = tensors[i];
    const int s = sq::bytes_of(t.dtype), so = t.out ? sq::bytes_of(t.out_dtype) : s;
    if (!s || !so || t.count < 0 || (t.count > 0 && !t.data)) return SEQSUM_EINVAL;
    if (reinterpret_cast<uintptr_t>(t.data) % s || reinterpret_cast<uintptr_t>(t.out) % so) return SEQSUM_EINVAL;
    if (t.count > (int64_t)1 << 46) return SEQSUM_EINVAL;
    nchunks += (t.count + sq::kChunk - 1) / sq::kChunk;
  }
  if (nchunks > 0x7fffffff) return SEQSUM_EINVAL;
  try {
    std::vector<sq::Chunk> chunks;
    chunks.reserve(nchunks);
    for (int32_t i = 0; i < n; i++) {
      const seqsum_tensor &t = tensors[i];
      void *to = t.out ? t.out : const_cast<void *>(t.data);
      const int32_t out_type = t.out ? t.out_dtype : t.dtype;
      const int s = sq::bytes_of(t.dtype), so = sq::bytes_of(out_type);
      const bool aligned = ((reinterpret_cast<uintptr_t>(t.data) | reinterpret_cast<uintptr_t>(to)) & 15) == 0;
      for (int64_t at = 0; at < t.count; at += sq::kChunk) {
        sq::Chunk c = {};
        c.in = static_cast<const char *>(t.data) + at * s;
        c.out = static_cast<char *>(to) + at * so;
        c.n = (int32_t)(t.count - at < sq::kChunk ? t.count - at : sq::kChunk);
        c.type = (int8_t)t.dtype;
        c.out_type = (int8_t)out_type;
        c.aligned = aligned;
        c.in_place = to == t.data && out_type == t.dtype;
        chunks.push_back(c);
      }
    }
    seqsum_tensors *h = new seqsum_tensors();
    h->nchunks = nchunks;
    h->sms = sq::multiprocessors();
    cudaError_t e = cudaGetDevice(&h->device);
    const int64_t room = nchunks > 0 ? nchunks : 1;
    if (e == cudaSuccess) e = cudaMalloc(&h->chunks, room * sizeof(sq::Chunk));
    if (e == cudaSuccess) e = cudaMalloc(&h->parts, room * sizeof(double));
    if (e == cudaSuccess) e = cudaMalloc(&h->ticket, 2 * sizeof(uint32_t));
    if (e == cudaSuccess) e = cudaMemset(h->ticket, 0, 2 * sizeof(uint32_t));
    if (e == cudaSuccess && nchunks > 0)
      e = cudaMemcpy(h->chunks, chunks.data(), nchunks * sizeof(sq::Chunk), cudaMemcpyHostToDevice);
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
    if (e != cudaSuccess) {
      cudaFree(h->chunks);
      cudaFree(h->parts);
      cudaFree(h->ticket);
      delete h;
      sq::note_cuda(e);
      return e == cudaErrorMemoryAllocation ? SEQSUM_ENOMEM : SEQSUM_ECUDA;
    }
    *out = h;
    return SEQSUM_OK;
  } catch (const std::bad_alloc &) {
    return SEQSUM_ENOMEM;
  }
}

void seqsum_tensors_destroy(seqsum_tensors *t) {
  if (!t) return;
  int prev = 0;
  cudaGetDevice(&prev);
  cudaSetDevice(t->device);
  cudaDeviceSynchronize();   // calls still in flight may read the table
  cudaFree(t->chunks);
  cudaFree(t->parts);
  cudaFree(t->ticket);
  cudaSetDevice(prev);
  delete t;
}

int seqsum_tensors_norm(seqsum_tensors *tensors, float scale, float *norm, cudaStream_t stream) {
  return run_tensors(tensors, INFINITY, scale, norm, false, stream);
}

int seqsum_tensors_clip(seqsum_tensors *tensors, float max_norm, float scale, float *norm, cudaStream_t stream) {
  return run_tensors(tensors, max_norm, scale, norm, true, stream);
}

}  // extern "C"
