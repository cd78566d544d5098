// The norm of all numbers of many tensors, and the tensors scaled to a
// largest norm (seqsum_tensors_norm, seqsum_tensors_clip).
//
// The order of the sum is fixed: a tensor is cut into chunks of 32768
// elements, a chunk's squares are added in fp32 in one shape (a thread's
// chains, then trees), the chunks' sums in double: those of a group one after
// another, the groups' in one shape.  Which CTA takes which group does not
// matter, so the norm's bits depend on the numbers and the tensors' sizes
// alone.
#include <math.h>

#include <new>
#include <vector>

#include "../../include/seqsum.h"
#include "row_slice.cuh"

namespace sq {
namespace {

using row::Elem;

constexpr int kChunk = 32768;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kCtas = 3;             // of an SM
constexpr int kGroups = 16384;       // at most
constexpr int kShortChunks = 8;      // lists that one cluster takes, a chunk a CTA

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
  int32_t nchunks, group, ngroups;   // chunks a group
  double *parts;                     // the groups' sums
  uint32_t *done;                    // CTAs that are done with the norm, tickets of clipping, CTAs done with it; 0 between calls
  float *factor;
  float *norm;
  float scale, max_norm;
};

template <int N>
struct Bytes;
template <>
struct Bytes<8> {
  using type = uint2;
};
template <>
struct Bytes<16> {
  using type = uint4;
};
__device__ __forceinline__ uint4 widen(uint4 v) { return v; }
__device__ __forceinline__ uint4 widen(uint2 v) { return make_uint4(v.x, v.y, 0, 0); }
template <typename V>
__device__ __forceinline__ V narrow(uint4 v) {
  if constexpr (sizeof(V) == 16) return v;
  else return make_uint2(v.x, v.y);
}

__device__ __forceinline__ double warp_add(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// Sums over the CTA, the same in every thread, with one barrier each: two
// rows of the table in turn.
template <typename S>
struct BlockSum {
  S *table;   // [2][kWarps]
  int turn = 0;
  __device__ __forceinline__ S operator()(S v) {
    v = warp_add(v);
    S *row = table + turn * kWarps;
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) row[threadIdx.x >> 5] = v;
    __syncthreads();
    v = row[threadIdx.x & (kWarps - 1)];
#pragma unroll
    for (int o = kWarps / 2; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
  }
};

// Vector j of a chunk by elements, 0 past its end.
__device__ __noinline__ uint4 vec_by_elements(const float *p, int n, int j) {
  float x[4];
  for (int e = 0; e < 4; e++) x[e] = j * 4 + e < n ? p[j * 4 + e] : 0.0f;
  return Elem<float>::pack(x);
}
__device__ __noinline__ uint4 vec_by_elements(const uint16_t *p, int n, int j) {   // either 16-bit type
  uint32_t w[4];
  for (int e = 0; e < 4; e++) {
    const int i = j * 8 + 2 * e;
    w[e] = (i < n ? p[i] : 0u) | (i + 1 < n ? (uint32_t)p[i + 1] << 16 : 0u);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight vectors a thread from the h-th on, each of `kThreads` in turn.
__device__ __forceinline__ void load_eight(const Chunk &c, int h, uint4 *v) {
  if (c.aligned && c.n == kChunk) {
    const uint4 *q = static_cast<const uint4 *>(c.in) + h * kThreads + threadIdx.x;
#pragma unroll
    for (int k = 0; k < 8; k++) v[k] = q[k * kThreads];
  } else {
    const int per = c.type == SEQSUM_FP32 ? 4 : 8;
#pragma unroll
    for (int k = 0; k < 8; k++) {
      const int j = (h + k) * kThreads + threadIdx.x;
      v[k] = make_uint4(0, 0, 0, 0);
      if (c.aligned && j * per + per <= c.n) v[k] = static_cast<const uint4 *>(c.in)[j];
      else if (j * per < c.n)
        v[k] = c.type == SEQSUM_FP32 ? vec_by_elements(static_cast<const float *>(c.in), c.n, j)
                                     : vec_by_elements(static_cast<const uint16_t *>(c.in), c.n, j);
    }
  }
}

// The squares of a thread's vectors of a chunk, whose first eight are in v;
// `next` loads what comes after the chunk.
template <typename T, typename F>
__device__ __forceinline__ float thread_squares(const Chunk &c, uint4 *v, F next) {
  constexpr int E = Elem<T>::kPerVec, kVecs = kChunk / E / kThreads;
  static_assert(kChunk % (8 * E * kThreads) == 0, "a chunk is a whole number of eight vectors a thread");
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; e++) acc[e] = 0.0f;
#pragma unroll
  for (int h = 0; h < kVecs; h += 8) {
#pragma unroll
    for (int k = 0; k < 8; k++) {
      float x[E];
      Elem<T>::unpack(v[k], x);
#pragma unroll
      for (int e = 0; e < E; e++) acc[e] = __fmaf_rn(x[e], x[e], acc[e]);
    }
    if (h + 8 < kVecs) load_eight(c, h + 8, v);
    else next();
  }
#pragma unroll
  for (int o = E / 2; o; o >>= 1)
#pragma unroll
    for (int e = 0; e < o; e++) acc[e] += acc[e + o];
  return acc[0];
}

// A thread's share of a chunk's squares in double, where those of every fp32
// number are normal numbers.
template <typename T>
__device__ __noinline__ double thread_squares_wide(const Chunk &c) {
  const T *p = static_cast<const T *>(c.in);
  double s = 0.0;
  for (int i = threadIdx.x; i < c.n; i += kThreads) {
    const float x = Elem<T>::load(p + i);
    if (x != 0.0f) s += (double)x * (double)x;   // (fp64 is slow here, and gradients are often zeros)
  }
  return s;
}

// Adds a chunk's squares to `to`, in thread 0.  (Only there anything is
// converted to double: with all threads' conversions the fp64 pipe was 70%
// busy, and the norm of 658 MB took 123 us.)
template <typename F>
__device__ __forceinline__ void add_squares(double &to, const Chunk &c, uint4 *v, BlockSum<float> &sum, BlockSum<double> &wide, F next) {
  const float s = sum(c.type == SEQSUM_FP32   ? thread_squares<float>(c, v, next)
                      : c.type == SEQSUM_FP16 ? thread_squares<__half>(c, v, next)
                                              : thread_squares<__nv_bfloat16>(c, v, next));
  // below 2^-80 squares that left fp32's range could count; above all of it, the sum did
  if (s >= 8.2718061e-25f && s < INFINITY) {
    if (threadIdx.x == 0) to += (double)s;
    return;
  }
  const double w = wide(c.type == SEQSUM_FP32   ? thread_squares_wide<float>(c)
                        : c.type == SEQSUM_FP16 ? thread_squares_wide<__half>(c)
                                                : thread_squares_wide<__nv_bfloat16>(c));
  if (threadIdx.x == 0) to += w;
}

// The norm, and the factor of the clipped numbers (NaN stays).
__device__ __forceinline__ float norm_of(const TensorsArgs &a, double squares) {
  return (float)(sqrt(squares) * (double)a.scale);
}
__device__ __forceinline__ float factor_of(const TensorsArgs &a, float norm) {
  const float q = __fdiv_rn(a.max_norm, norm + 1e-6f);
  return (q > 1.0f ? 1.0f : q) * a.scale;
}

// Bound by HBM: 101 us for 658 MB of bf16 in 244 tensors (95% of the measured
// copy rate), 348 us for 2.46 GB.  Chunks of zeros are not: they are read again
// number by number (64 x 2^20 bf16 26 us, zeros 416).  Three CTAs of 256 threads with 128 bytes a
// thread on the way hold 96 KB of loads an SM; the loads of the next chunk are
// out before the sum of this one goes through the CTA (without that 119 us).
// Chunks of 16384 numbers: 114 us.
__global__ __launch_bounds__(kThreads, kCtas) void norm_kernel(const TensorsArgs a) {
  __shared__ float table[2 * kWarps];
  __shared__ double wide_table[2 * kWarps];
  __shared__ bool last;
  BlockSum<float> sum{table};
  BlockSum<double> wide{wide_table};
  int g = blockIdx.x, i = g * a.group;
  Chunk c = a.chunks[i];
  uint4 v[8];
  load_eight(c, 0, v);
  double s = 0.0;
  while (g < a.ngroups) {
    const int of = g;
    if (++i == min((g + 1) * a.group, a.nchunks)) {
      g += gridDim.x;
      i = g * a.group;
    }
    Chunk after = c;
    if (g < a.ngroups) after = a.chunks[i];
    // the next chunk's numbers are on their way while this one's sum goes through the CTA
    add_squares(s, c, v, sum, wide, [&] {
      if (g < a.ngroups) load_eight(after, 0, v);
    });
    c = after;
    if (g != of && threadIdx.x == 0) {
      a.parts[of] = s;
      s = 0.0;
    }
  }
  // (a kernel that depends on this one, and waits for its end, may come onto the SM)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // the CTA that is done last adds the groups' sums
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(a.done, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  s = 0.0;
  for (int i = threadIdx.x; i < a.ngroups; i += 16 * kThreads) {
    double v[16];
#pragma unroll
    for (int k = 0; k < 16; k++) v[k] = i + k * kThreads < a.ngroups ? __ldcg(&a.parts[i + k * kThreads]) : 0.0;
#pragma unroll
    for (int o = 8; o; o >>= 1)
#pragma unroll
      for (int k = 0; k < o; k++) v[k] += v[k + o];
    s += v[0];
  }
  s = wide(s);
  if (threadIdx.x == 0) {
    *a.done = 0;
    const float norm = norm_of(a, s);
    *a.norm = norm;
    *a.factor = factor_of(a, norm);
  }
}

// Units of 16 bytes of the wider type, so that a warp's loads and stores are
// each without gaps.
template <typename T, typename O>
struct Scale {
  static constexpr int U = Elem<T>::kPerVec < Elem<O>::kPerVec ? Elem<T>::kPerVec : Elem<O>::kPerVec;
  using In = typename Bytes<U * sizeof(T)>::type;
  using Out = typename Bytes<U * sizeof(O)>::type;

  __device__ __forceinline__ static Out unit(In v, float f) {
    float x[8] = {}, y[8] = {};
    Elem<T>::unpack(widen(v), x);
#pragma unroll
    for (int e = 0; e < U; e++) y[e] = x[e] * f;
    return narrow<Out>(Elem<O>::pack(y));
  }
  // a whole chunk, 128 bytes a thread under way
  __device__ __forceinline__ static void whole(const Chunk &c, float f) {
    constexpr int kBatch = 128 / (U * (int)sizeof(T));
    static_assert(kChunk % (U * kBatch * kThreads) == 0, "a whole chunk is a number of whole batches");
    const In *p = static_cast<const In *>(c.in) + threadIdx.x;
    Out *q = static_cast<Out *>(c.out) + threadIdx.x;
#pragma unroll 1
    for (int h = 0; h < kChunk / U; h += kBatch * kThreads) {
      In v[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; k++) v[k] = p[h + k * kThreads];
#pragma unroll
      for (int k = 0; k < kBatch; k++) __stcs(q + h + k * kThreads, unit(v[k], f));
    }
  }
  // a part of one, or one that is not aligned: whole units where it is, then element by element
  __device__ __noinline__ static void part(const Chunk &c, float f) {
    const int units = c.aligned ? c.n / U : 0;
    const In *p = static_cast<const In *>(c.in);
    Out *q = static_cast<Out *>(c.out);
#pragma unroll 1
    for (int h = threadIdx.x; h < units; h += 4 * kThreads) {
      In v[4] = {};
#pragma unroll
      for (int k = 0; k < 4; k++)
        if (h + k * kThreads < units) v[k] = p[h + k * kThreads];
#pragma unroll
      for (int k = 0; k < 4; k++)
        if (h + k * kThreads < units) q[h + k * kThreads] = unit(v[k], f);
    }
    const T *pe = static_cast<const T *>(c.in);
    O *qe = static_cast<O *>(c.out);
#pragma unroll 1
    for (int h = units * U + threadIdx.x; h < c.n; h += 4 * kThreads) {
      float x[4] = {};
#pragma unroll
      for (int k = 0; k < 4; k++)
        if (h + k * kThreads < c.n) x[k] = Elem<T>::load(pe + h + k * kThreads);
#pragma unroll
      for (int k = 0; k < 4; k++)
        if (h + k * kThreads < c.n) Elem<O>::store(qe + h + k * kThreads, x[k] * f);
    }
  }
};

template <typename T, typename O>
__device__ __forceinline__ void chunk_scale(const Chunk &c, float f) {
  if (c.aligned && c.n == kChunk) Scale<T, O>::whole(c, f);
  else Scale<T, O>::part(c, f);
}

template <typename T>
__device__ __forceinline__ void chunk_scale_to(const Chunk &c, float f) {
  if (c.out_type == SEQSUM_FP32) chunk_scale<T, float>(c, f);
  else if (c.out_type == SEQSUM_FP16) chunk_scale<T, __half>(c, f);
  else chunk_scale<T, __nv_bfloat16>(c, f);
}

__device__ __forceinline__ void scale_chunk(const Chunk &c, float f) {
  if (c.in_place && f == 1.0f) return;   // x * 1 is x
  if (c.type == SEQSUM_FP32) chunk_scale_to<float>(c, f);
  else if (c.type == SEQSUM_FP16) chunk_scale_to<__half>(c, f);
  else chunk_scale_to<__nv_bfloat16>(c, f);
}

// Chunks by ticket, from the end: the last ones that the norm read are still
// in L2.  Bound by HBM: the numbers are read a second time, for which there is
// no room on chip.  (1.07 G fp16 numbers to fp32, norm included: 1250 us;
// 1375 where the chunks were taken in fixed turns and CTAs with slower paths
// to memory ended late.  In place: 293 us for 658 MB of bf16.)
__global__ __launch_bounds__(kThreads, kCtas) void clip_kernel(const TensorsArgs a) {
  __shared__ int slot[2];
  int i = (int)blockIdx.x, turn = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");   // launched while the norm is being taken
  const float f = *a.factor;
  while (i < a.nchunks) {
    int after = 0;
    if (threadIdx.x == 0) after = (int)(atomicAdd(&a.done[1], 1u) + gridDim.x);   // used once this chunk is done
    scale_chunk(a.chunks[a.nchunks - 1 - i], f);
    if (threadIdx.x == 0) slot[turn] = after;
    __syncthreads();
    i = slot[turn];
    turn ^= 1;
  }
  if (threadIdx.x == 0 && atomicAdd(&a.done[2], 1u) == gridDim.x - 1) a.done[1] = a.done[2] = 0;
}

// Short lists: one cluster takes the norm and scales, in one launch.
template <bool kClip>
__global__ __launch_bounds__(kThreads, 1) void short_kernel(const TensorsArgs a) {
  __shared__ float table[2 * kWarps];
  __shared__ double wide_table[2 * kWarps];
  __shared__ uint64_t parts[kShortChunks];
  BlockSum<float> sum{table};
  BlockSum<double> wide{wide_table};
  const uint32_t size = row::cluster_size(), rank = row::cluster_rank();
  row::cluster_begun();
  const bool any = (int)rank < a.nchunks;   // a chunk a CTA
  Chunk c = {};
  double s = 0.0;
  if (any) {
    c = a.chunks[rank];
    uint4 v[8];
    load_eight(c, 0, v);
    add_squares(s, c, v, sum, wide, [] {});
  }
  row::cluster_wait_begun();
  if (any && threadIdx.x == 0)
    for (uint32_t r = 0; r < size; r++) row::st_remote(row::remote(&parts[rank], r), __double_as_longlong(s));
  row::cluster_sync();
  s = 0.0;
  if ((int)(threadIdx.x & 31) < a.nchunks) s = __longlong_as_double(parts[threadIdx.x & 31]);
  s = warp_add(s);
  const float norm = norm_of(a, s);
  if (rank == 0 && threadIdx.x == 0) *a.norm = norm;
  if (kClip) {
    const float f = factor_of(a, norm);
    if (any) scale_chunk(c, f);
  }
}

int bytes_of(int32_t dtype) { return dtype == SEQSUM_FP32 ? 4 : dtype == SEQSUM_FP16 || dtype == SEQSUM_BF16 ? 2 : 0; }

}  // namespace
}  // namespace sq

struct seqsum_tensors {
  int device = -1;
  int32_t nchunks = 0, group = 1, ngroups = 0;
  sq::Chunk *chunks = nullptr;
  double *parts = nullptr;
  uint32_t *done = nullptr;   // three counters, and the factor
  int sms = 0;
};

namespace {

int run_tensors(seqsum_tensors *t, float max_norm, float scale, float *norm, bool clip, cudaStream_t stream) {
  if (!t || !norm) return SEQSUM_EINVAL;
  sq::TensorsArgs a = {t->chunks, t->nchunks, t->group, t->ngroups, t->parts, t->done,
                       reinterpret_cast<float *>(t->done + 3), norm, scale, max_norm};
  cudaError_t e;
  if (t->nchunks <= sq::kShortChunks) {
    const int size = t->nchunks > 4 ? 8 : t->nchunks > 1 ? 4 : 1;
    e = sq::row::launch_rows(clip ? sq::short_kernel<true> : sq::short_kernel<false>, a, 1, size, sq::kThreads, 0, stream);
    return e == cudaSuccess ? SEQSUM_OK : sq::note_cuda(e);
  }
  const int most = t->sms * sq::kCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(t->ngroups < most ? t->ngroups : most));
  cfg.blockDim = dim3(sq::kThreads);
  cfg.stream = stream;
  e = cudaLaunchKernelEx(&cfg, sq::norm_kernel, a);
  if (e == cudaSuccess && clip) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(t->nchunks < most ? t->nchunks : most));
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, sq::clip_kernel, a);
  }
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
  if (nchunks > 0x7fffffff - 65536) return SEQSUM_EINVAL;
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
    h->nchunks = (int32_t)nchunks;
    h->group = (int32_t)((nchunks + sq::kGroups - 1) / sq::kGroups);
    if (h->group < 1) h->group = 1;
    h->ngroups = (int32_t)((nchunks + h->group - 1) / h->group);
    h->sms = sq::multiprocessors();
    cudaError_t e = cudaGetDevice(&h->device);
    const int64_t room = nchunks > 0 ? nchunks : 1;
    if (e == cudaSuccess) e = cudaMalloc(&h->chunks, room * sizeof(sq::Chunk));
    if (e == cudaSuccess) e = cudaMalloc(&h->parts, (h->ngroups > 0 ? h->ngroups : 1) * sizeof(double));
    if (e == cudaSuccess) e = cudaMalloc(&h->done, 4 * sizeof(uint32_t));
    if (e == cudaSuccess) e = cudaMemset(h->done, 0, 4 * sizeof(uint32_t));
    if (e == cudaSuccess && nchunks > 0)
      e = cudaMemcpy(h->chunks, chunks.data(), nchunks * sizeof(sq::Chunk), cudaMemcpyHostToDevice);
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
    if (e != cudaSuccess) {
      cudaFree(h->chunks);
      cudaFree(h->parts);
      cudaFree(h->done);
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
  cudaFree(t->done);
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
