// Rows of logits on chip: a row is read once, in 16-byte vectors, by the
// CTAs of one thread-block cluster, and stays in their registers while it is
// reduced.  What the kernels on rows share: element types, the slice of a
// row that a thread holds, sums over a cluster.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace sq {

// Records the CUDA error of a failed call for seqsum_last_cuda_error() and
// returns SEQSUM_ECUDA.
int note_cuda(cudaError_t e);
// Multiprocessors of the current device (0 if it cannot be asked).
int multiprocessors();

namespace row {

constexpr int kMaxCluster = 8;           // the portable cluster size
constexpr int64_t kMaxVocab = 1 << 24;   // element indices fit 32 bits, 2^24 weights of 2^31 fit 64

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kPerVec = 4;
  static constexpr uint32_t kNegInf = 0xff800000u;
  __device__ static void unpack(uint4 v, float *x) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
  __device__ static uint4 pack(const float *x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
  // the maximum of a vector's numbers and m; NaN is passed over
  __device__ static float vec_max(uint4 v, float m) {
    const float a = fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), b = fmaxf(__uint_as_float(v.z), __uint_as_float(v.w));
    return fmaxf(m, fmaxf(a, b));
  }
  __device__ static float load(const float *p) { return *p; }
  __device__ static void store(float *p, float x) { *p = x; }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kPerVec = 8;
  static constexpr uint32_t kNegInf = 0xff80ff80u;
  __device__ static void unpack(uint4 v, float *x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; i++) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  __device__ static uint4 pack(const float *x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ static float vec_max(uint4 v, float m) {
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&v);
    const __nv_bfloat162 a = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(m, fmaxf(__low2float(a), __high2float(a)));
  }
  __device__ static float load(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
  __device__ static void store(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }
};
template <>
struct Elem<__half> {
  static constexpr int kPerVec = 8;
  static constexpr uint32_t kNegInf = 0xfc00fc00u;
  __device__ static void unpack(uint4 v, float *x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
  __device__ static uint4 pack(const float *x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ static float vec_max(uint4 v, float m) {
    const __half2 *h = reinterpret_cast<const __half2 *>(&v);
    const __half2 a = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(m, fmaxf(__low2float(a), __high2float(a)));
  }
  __device__ static float load(const __half *p) { return __half2float(*p); }
  __device__ static void store(__half *p, float x) { *p = __float2half_rn(x); }
};

// ---- two fp32 operations in one instruction, each rounded as by itself

__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split(uint64_t r, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// ---- clusters

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// Every thread of every CTA of the cluster; what was written to shared memory
// before it (its own or another CTA's) is seen after it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(const void *p, uint32_t rank) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(p), r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_remote(uint32_t a, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ uint64_t ld_remote64(uint32_t a) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_remote32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Puts `v` of this CTA (the same in every thread) at box[rank] of every CTA
// of the cluster and waits for theirs.
__device__ __forceinline__ void cluster_post(uint64_t v, uint64_t *box, uint32_t rank, uint32_t size) {
  if (size == 1) {
    if (threadIdx.x == 0) box[0] = v;
    __syncthreads();
  } else {
    if (threadIdx.x < size) st_remote(remote(&box[rank], threadIdx.x), v);
    cluster_sync();
  }
}

// ---- reductions

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
  return v;
}
__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
__device__ __forceinline__ uint64_t warp_scan(uint64_t v, int lane) {   // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t u = __shfl_up_sync(~0u, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// ---- the slice of a row that a thread holds
//
// The row's elements lie in 16-byte vectors counted from the aligned address
// at or below its first element; element e of vector j is index
// j * kPerVec + e - off of the row.  The cluster's CTAs take consecutive
// runs of vectors, a CTA's warps consecutive runs of those, a warp's vectors
// go to its lanes in turn: (CTA, warp, step, lane) is index order.  Vectors
// that stick out of the row are read element by element, so nothing outside
// the row is touched; what is not in the row is -inf.
//
// KV > 0: at most KV steps, kept in registers.  KV = 0: any number of steps,
// read again from global memory (L2) by every pass.
template <typename T, int KV, int NT>
struct Slice {
  static constexpr int kE = Elem<T>::kPerVec;
  static constexpr int kWarps = NT / 32;
  const T *p;
  int32_t vocab, off, steps, first, limit;   // this thread's vectors: first + 32 k < limit, k < steps
  uint4 keep[KV > 0 ? KV : 1];

  __device__ __forceinline__ void set(const T *row, int32_t v, uint32_t rank, uint32_t size) {
    p = row;
    vocab = v;
    off = (int32_t)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    const int32_t vecs = (off + v + kE - 1) / kE;
    const int32_t mine = (vecs + (int32_t)size - 1) / (int32_t)size;
    steps = (mine + NT - 1) / NT;
    const int32_t begin = mine * (int32_t)rank;
    limit = min(begin + mine, vecs);
    first = begin + (int32_t)(threadIdx.x >> 5) * steps * 32 + (int32_t)(threadIdx.x & 31);
  }
  __device__ __forceinline__ int32_t index(int k, int e) const { return (first + 32 * k) * kE + e - off; }
  __device__ __forceinline__ uint4 read(int k) const {
    const int32_t j = first + 32 * k;
    constexpr uint32_t ninf = Elem<T>::kNegInf;
    uint4 v = make_uint4(ninf, ninf, ninf, ninf);
    if (k < steps && j < limit) {
      const int32_t i = j * kE - off;
      if (i >= 0 && i + kE <= vocab) {
        v = *reinterpret_cast<const uint4 *>(p + i);
      } else {
        float x[kE];
#pragma unroll
        for (int e = 0; e < kE; e++) x[e] = i + e >= 0 && i + e < vocab ? Elem<T>::load(p + i + e) : -INFINITY;
        v = Elem<T>::pack(x);
      }
    }
    return v;
  }
  __device__ __forceinline__ void load() {
    if constexpr (KV > 0) {
#pragma unroll
      for (int k = 0; k < KV; k++) keep[k] = read(k);
    }
  }
  // the largest number of the slice; NaN is passed over
  __device__ __forceinline__ float largest() const {
    float m = -INFINITY;
    if constexpr (KV > 0) {
#pragma unroll
      for (int k = 0; k < KV; k++)
        if (k < steps) m = Elem<T>::vec_max(keep[k], m);
    } else {
      for (int k = 0; k < steps; k++) m = Elem<T>::vec_max(read(k), m);
    }
    return m;
  }
  // f(step, its elements as floats) for every step in index order
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    if constexpr (KV > 0) {
#pragma unroll
      for (int k = 0; k < KV; k++) {
        if (k < steps) {
          float x[kE];
          Elem<T>::unpack(keep[k], x);
          f(k, x);
        }
      }
    } else {
      for (int k = 0; k < steps; k++) {
        float x[kE];
        Elem<T>::unpack(read(k), x);
        f(k, x);
      }
    }
  }
  // writes a vector of the slice's place to another row of the same alignment or not
  __device__ __forceinline__ void write(T *row, bool aligned, int k, const float *x) const {
    const int32_t j = first + 32 * k;
    if (j >= limit) return;
    const int32_t i = j * kE - off;
    if (aligned && i >= 0 && i + kE <= vocab) {
      *reinterpret_cast<uint4 *>(row + i) = Elem<T>::pack(x);
    } else {
#pragma unroll
      for (int e = 0; e < kE; e++)
        if (i + e >= 0 && i + e < vocab) Elem<T>::store(row + i + e, x[e]);
    }
  }
};

// A launch of `rows` clusters of `size` CTAs.
template <typename Args>
inline cudaError_t launch_rows(void (*kernel)(Args), const Args &args, int64_t rows, int size, int threads,
                               cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * size));
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = size;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = size > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

}  // namespace row
}  // namespace sq
