// What the kernels on rows of logits share: element types, the parts of a row
// that a CTA or a thread has, what the CTAs of a cluster tell each other, sums
// over warps.  Rows are read in 16-byte vectors: once, into registers (short
// rows) or the shared memory of a cluster's CTAs, where they stay while they are
// reduced; or, where many long rows are sampled and beyond what eight CTAs
// hold, again from L2 for each pass.
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

struct Waits;
// What the next call's waits are given (seqsum_debug_set_fault).
Waits waits();

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
// In two parts, before the first access to another CTA's shared memory: every
// CTA of the cluster has begun (its memory is there) once the wait is over.
__device__ __forceinline__ void cluster_begun() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait_begun() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
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
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t ld_remote32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

// Puts `v` of this CTA (the same in every thread) at box[rank] of every CTA
// of the cluster and waits for theirs.
__device__ __forceinline__ void cluster_post(uint64_t v, uint64_t *box, uint32_t rank, uint32_t size) {
  if (threadIdx.x < size) st_remote(remote(&box[rank], threadIdx.x), v);
  cluster_sync();
}

// ---- reductions

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
  return v;
}
__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {   // of values below 2^58
  const uint32_t lo = __reduce_add_sync(~0u, (uint32_t)v & 0x3ffffffu), mid = __reduce_add_sync(~0u, (uint32_t)(v >> 26) & 0x3ffffffu),
                 hi = __reduce_add_sync(~0u, (uint32_t)(v >> 52));
  return lo + ((uint64_t)mid << 26) + ((uint64_t)hi << 52);
}
__device__ __forceinline__ uint32_t warp_scan(uint32_t v, int lane) {   // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(~0u, v, o);
    if (lane >= o) v += u;
  }
  return v;
}
__device__ __forceinline__ uint64_t warp_scan(uint64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t u = __shfl_up_sync(~0u, v, o);
    if (lane >= o) v += u;
  }
  return v;
}
// floats as unsigned integers of the same order, and back
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }
__device__ __forceinline__ float warp_max_all(float v) { return from_ordered(__reduce_max_sync(~0u, ordered(v))); }
__device__ __forceinline__ float warp_add(float v) {   // the same tree in every lane
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
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
// KV > 0: at most KV steps, kept in registers (for passes over elements each by
// itself, and for short rows, one a warp: NT = 32).  KV = 0: any number of
// steps, read again from global memory (L2) by every pass.
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
    first = begin + (NT == 32 ? 0 : (int32_t)(threadIdx.x >> 5) * steps * 32) + (int32_t)(threadIdx.x & 31);
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
  // f(step, its elements as floats) for every step in index order, read again
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    for (int k = 0; k < steps; k++) {
      float x[kE];
      Elem<T>::unpack(read(k), x);
      f(k, x);
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

// ---- rows streamed through shared memory
//
// A cluster takes row after row.  In each of its CTAs one warp brings the CTA's
// slice of each row into the next of a few buffers in shared memory, ahead of
// the work; all make passes over the buffers and leave them one by one.  So the
// next row's copy is on its way while this one is summed, and a pass costs no
// registers: as many CTAs as their buffers allow share an SM and fill each
// other's waits.
//
// A row's 16-byte vectors, counted from the aligned address at or below its
// first element, go to the lanes of a warp in steps of 32, and the steps are
// cut into segments as even as can be, one for each warp of the cluster.
// Where the cluster's size goes by the row's length alone, the same vectors
// meet in one thread in the same order whatever else a call holds.  (Which
// numbers share a vector goes by the row's address modulo 16.)
//
// What lies inside the row comes by one bulk copy; vectors that stick out of
// it are put together from elements read one by one, with -inf beside them and
// after them up to the end of the last step.
//
// The warps tell each other 8-byte words: each is written to every CTA of the
// cluster with an asynchronous store, and the stores count down a barrier
// there, so that neither a fence nor a barrier of the whole cluster is needed.
// A warp may post a word before it waits for the last one; a post then comes
// after every warp has left the exchange three before, so there are four boxes
// in turn.

// Waits for copies and for other CTAs are bounded.  A warp whose wait gave up
// has nothing computed from what it did not have: the word that it owes says
// so, or is not sent; later ones are not, so that the others' waits run out too;
// and each marks what it had yet to write.

constexpr uint32_t kWaitNs = 2000000000u;   // the limit of a wait

// A call's limit, and, for tests, a wait that is taken to have given up: that
// of warp `warp` of each cluster for its row `turn` (-1: none).
struct Waits {
  uint32_t limit;
  int32_t turn, warp;
  __device__ __forceinline__ bool fails(uint32_t it, uint32_t of) const { return it == (uint32_t)turn && of == (uint32_t)warp; }
};

__device__ __forceinline__ uint32_t smem(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint64_t *bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem(bar)) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t *bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t *bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem(bar)), "r"(parity)
      : "memory");
  return done;
}
static __device__ __noinline__ bool bar_wait_long(uint64_t *bar, uint32_t parity, uint32_t limit) {
  uint64_t t0, t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  do {
    for (int i = 0; i < 64; i++)
      if (bar_try(bar, parity)) return true;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  } while (t - t0 < limit);
  return false;
}
// false: gave up (of a warp's lanes, some may have)
__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity, uint32_t limit = kWaitNs) {
  return bar_try(bar, parity) || bar_wait_long(bar, parity, limit);
}
// A CTA whose waits gave up stays a millisecond past the cluster's last barrier:
// words that others had sent it by then, and that it did not wait for, land in
// its memory.
static __device__ __noinline__ void stay() {
  uint64_t t0, t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  do asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  while (t - t0 < 1000000);
}

// 16 bytes to shared memory of CTA `rank`, counted down at its `bar`.
__device__ __forceinline__ void send(uint4 *to, uint64_t *bar, uint32_t rank, uint4 v) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                   remote(to, rank)),
               "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"(remote(bar, rank))
               : "memory");
}
__device__ __forceinline__ void send(uint2 *to, uint64_t *bar, uint32_t rank, uint2 v) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(
                   remote(to, rank)),
               "r"(v.x), "r"(v.y), "r"(remote(bar, rank))
               : "memory");
}

struct Exchange {
  uint64_t *box;   // one for each warp of the cluster
  uint64_t *bar;

  // v (the same in every lane) to box `at` of every CTA
  __device__ __forceinline__ void post(int32_t at, uint64_t v, uint32_t size) const {
    const uint32_t lane = threadIdx.x & 31;
    if (lane < size)
      asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.u64 [%0], %1, [%2];" ::"r"(
                       remote(&box[at], lane)),
                   "l"(v), "r"(remote(bar, lane))
                   : "memory");
  }
};

// Where a CTA's slice of a row lies.
template <typename T>
struct Stream {
  static constexpr int kE = Elem<T>::kPerVec;
  int32_t vocab, off;
  int32_t steps;       // of the row
  int32_t begin, n;    // the first vector, and how many there are (whole steps, but for the row's end)
  uint4 *buf;

  // where a share of 2^log2 equal ones of the row's steps begins
  __device__ __forceinline__ int32_t step_of(uint32_t share, int log2) const {
    return (int32_t)(((uint64_t)steps * share) >> log2);
  }
  __device__ __forceinline__ void set(const T *row, int32_t v, uint32_t rank, int log2_size, uint4 *b) {
    vocab = v;
    off = (int32_t)((uint32_t)reinterpret_cast<uintptr_t>(row) & 15u) / (int)sizeof(T);
    const int32_t vecs = (off + v + kE - 1) / kE;
    steps = (vecs + 31) / 32;
    begin = step_of(rank, log2_size) * 32;
    n = min(step_of(rank + 1, log2_size) * 32, vecs) - begin;
    buf = b;
  }
  __device__ __forceinline__ int32_t index(int32_t vec, int e) const { return (begin + vec) * kE + e - off; }
  // this lane's vector of a step of the slice
  __device__ __forceinline__ uint4 vec(int32_t st) const { return buf[st * 32 + (threadIdx.x & 31)]; }

  __device__ __forceinline__ bool cut_head() const { return off > 0 && begin == 0 && n > 0; }
  __device__ __forceinline__ bool cut_tail() const { return n > 0 && index(n, 0) > vocab; }
  // One warp brings `row` in; `full` counts two arrivals.  First what lies inside ...
  __device__ __forceinline__ void bring_inner(const T *row, uint64_t *full) const {
    if ((threadIdx.x & 31) == 0) {
      const int32_t from = cut_head() ? 1 : 0, to = n - (cut_tail() ? 1 : 0);
      // (what was written to the buffer element by element, some rows ago, comes before the copy)
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      const uint32_t bytes = to > from ? (uint32_t)(to - from) * 16 : 0;
      bar_expect(full, bytes);
      if (bytes)
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                         smem(buf + from)),
                     "l"(row + index(from, 0)), "r"(bytes), "r"(smem(full))
                     : "memory");
    }
  }
  // ... then the elements of the vectors that stick out: lane e has element e
  // of the first vector, lane 16 + e that of the last ...
  __device__ __forceinline__ float edge(const T *row) const {
    const int lane = threadIdx.x & 31, e = lane & 15;
    if (e < kE && (lane < 16 ? cut_head() : cut_tail())) {
      const int32_t i = index(lane < 16 ? 0 : n - 1, e);
      if (i >= 0 && i < vocab) return Elem<T>::load(row + i);
    }
    return -INFINITY;
  }
  // ... which go into the buffer, with -inf up to the end of the last step.
  __device__ __forceinline__ void bring_edges(float v, uint64_t *full) const {
    const int lane = threadIdx.x & 31, e = lane & 15;
    constexpr uint32_t ninf = Elem<T>::kNegInf;
    if (lane >= (n & 31) && (n & 31)) buf[(n & ~31) + lane] = make_uint4(ninf, ninf, ninf, ninf);
    if (e < kE && (lane < 16 ? cut_head() : cut_tail()))
      Elem<T>::store(reinterpret_cast<T *>(buf + (lane < 16 ? 0 : n - 1)) + e, v);
    __syncwarp();
    if (lane == 0) bar_arrive(full);
  }
  __device__ __forceinline__ void bring(const T *row, uint64_t *full) const {
    bring_inner(row, full);
    bring_edges(edge(row), full);
  }
  // whether step `st` of the slice lies inside the row, all of it
  __device__ __forceinline__ bool inside(int32_t st) const {
    return index(st * 32, 0) >= 0 && index(st * 32 + 32, 0) <= vocab;
  }
  // writes the elements of vector `vec` that are in the row
  __device__ __forceinline__ void write_edge(T *row, int32_t vec, const float *x) const {
    const int32_t i = index(vec, 0);
#pragma unroll
    for (int e = 0; e < kE; e++)
      if (vec < n && i + e >= 0 && i + e < vocab) Elem<T>::store(row + i + e, x[e]);
  }
};

// A whole row in global memory, seen as a slice: what a CTA that has a row to
// itself reads again from L2 in every pass.
template <typename T>
struct FarRow {
  static constexpr int kE = Elem<T>::kPerVec;
  static constexpr int32_t begin = 0;
  const T *p;
  int32_t vocab, off, steps;
  __device__ __forceinline__ void set(const T *row, int32_t v) {
    p = row;
    vocab = v;
    off = (int32_t)((uint32_t)reinterpret_cast<uintptr_t>(row) & 15u) / (int)sizeof(T);
    steps = (off + v + 32 * kE - 1) / (32 * kE);
  }
  __device__ __forceinline__ int32_t step_of(uint32_t share, int log2) const {
    return (int32_t)(((uint64_t)steps * share) >> log2);
  }
  __device__ __forceinline__ int32_t index(int32_t vec, int e) const { return vec * kE + e - off; }
  __device__ __forceinline__ uint4 vec(int32_t st) const {
    const int32_t i = index(st * 32 + (int32_t)(threadIdx.x & 31), 0);
    if (i >= 0 && i + kE <= vocab) return __ldg(reinterpret_cast<const uint4 *>(p + i));
    float x[kE];
#pragma unroll
    for (int e = 0; e < kE; e++) x[e] = i + e >= 0 && i + e < vocab ? Elem<T>::load(p + i + e) : -INFINITY;
    return Elem<T>::pack(x);
  }
};

// A launch of `rows` clusters of `size` CTAs.
template <typename Args>
inline cudaError_t launch_rows(void (*kernel)(Args), const Args &args, int64_t rows, int size, int threads,
                               size_t shared, cudaStream_t stream, int *most = nullptr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * size));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = size;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (most) return cudaOccupancyMaxActiveClusters(most, (const void *)kernel, &cfg);
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

}  // namespace row
}  // namespace sq
