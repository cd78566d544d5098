// One token a row of logits (seqsum_sample_tokens).
//
// The weights are integers: w = rn(2^31 * 2^d), d the logit's distance to the
// row's maximum in octaves.  Sums of integers do not depend on their order, so
// the mass of a top-k set, the cut of top-p and the draw are exact, however
// the row is split over threads and CTAs; only 2^d itself is rounded.
//
// Every filter keeps a prefix of one order: larger d first, ties by lower
// index.  So the kept set is known by its last element, and that is found by
// counting: the entries' places in that order, as (bits of -d, index), are
// split into 256 bins, counts and masses are summed over the cluster, the bin
// in which the count passes k (or the mass passes the cut) is split again.
// Entries with d <= -32 have w = 0 and can be left out everywhere.
#include <math.h>

#include "../../include/seqsum.h"
#include "row_slice.cuh"

namespace sq {
namespace {

using namespace row;

constexpr int kBins = 256;
constexpr float kFloor = -32.0f;   // 2^31 * 2^d rounds to 0 from here on

struct SampleArgs {
  const void *logits;
  int64_t rows, stride;
  int32_t vocab;
  const float *u;
  seqsum_sampling s;
  int64_t *tokens;
  float *logps;
};

// A place in the order: an entry is before it where its key (the bits of -d)
// is smaller, or the same and its index is smaller.
struct Place {
  uint32_t key;
  int32_t index;
};

struct Shared {
  uint64_t box[4][kMaxCluster];   // what the cluster's CTAs tell each other
  uint64_t warp[32];
  uint32_t count[2][kBins];       // [0]: the first split, kept for the second search; [1]: later splits
  uint64_t mass[2][kBins];
  uint32_t tcount[kBins];         // ... summed over the cluster
  uint64_t tmass[kBins];
  int bin;                        // the bin that a search goes on in
  uint32_t bin_count, count_before;
  uint64_t bin_mass, mass_before;
  uint32_t best;                  // lowest index of the maximum
};

// floor(part * whole / 2^32), part <= 2^32, whole < 2^56
__device__ __forceinline__ uint64_t share(uint64_t part, uint64_t whole) {
  return (__umul64hi(part, whole) << 32) | ((part * whole) >> 32);
}

// Sum over the CTA's threads, in every thread.  sh.warp is free again after the next barrier.
template <int NT>
__device__ __forceinline__ uint64_t block_sum(uint64_t v, Shared &sh) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) sh.warp[threadIdx.x >> 5] = v;
  __syncthreads();
  uint64_t t = 0;
#pragma unroll
  for (int i = 0; i < NT / 32; i++) t += sh.warp[i];
  return t;
}

template <typename T, int KV, int NT>
struct Sampler {
  Slice<T, KV, NT> x;
  Shared &sh;
  float m, c;
  uint32_t rank, size;

  __device__ Sampler(Shared &s) : sh(s) {}

  // octaves below the maximum; NaN (a masked logit where c is 0, a NaN logit) counts as masked
  __device__ __forceinline__ float octaves(float v) const { return v == m ? 0.0f : (v - m) * c; }
  __device__ __forceinline__ static uint32_t weight(float d) { return __float2uint_rn(exp2f(d) * 2147483648.0f); }
  __device__ __forceinline__ static uint32_t key(float d) { return __float_as_uint(d) & 0x7fffffffu; }

  // f(d, index) for every entry whose weight may be above 0
  template <typename F>
  __device__ __forceinline__ void entries(F f) const {
    x.each([&](int k, const float *v) {
#pragma unroll
      for (int e = 0; e < x.kE; e++) {
        const float d = octaves(v[e]);
        if (d > kFloor) f(d, x.index(k, e));
      }
    });
  }

  // Sums the bins over the cluster and finds the first one at which the count
  // (or mass) reaches `need`; sh.bin = -1 where none does.
  __device__ void search(int level, bool by_mass, uint64_t need) {
    if (size > 1) cluster_sync(); else __syncthreads();
    if (threadIdx.x < kBins) {
      uint32_t n = 0;
      uint64_t w = 0;
      for (uint32_t r = 0; r < size; r++) {
        n += ld_remote32(remote(&sh.count[level][threadIdx.x], r));
        w += ld_remote64(remote(&sh.mass[level][threadIdx.x], r));
      }
      sh.tcount[threadIdx.x] = n;
      sh.tmass[threadIdx.x] = w;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      const int lane = threadIdx.x;
      uint64_t n = 0, w = 0;
#pragma unroll
      for (int i = 0; i < kBins / 32; i++) n += sh.tcount[lane * (kBins / 32) + i], w += sh.tmass[lane * (kBins / 32) + i];
      uint64_t nb = warp_scan(n, lane) - n, wb = warp_scan(w, lane) - w;
      const bool here = by_mass ? wb < need && need <= wb + w : nb < need && need <= nb + n;
      if (lane == 0) sh.bin = -1;
      __syncwarp();
      if (here) {
        int b = lane * (kBins / 32);
        for (;; b++) {
          const uint32_t bn = sh.tcount[b];
          const uint64_t bw = sh.tmass[b];
          if ((by_mass ? wb + bw : nb + bn) >= need) break;
          nb += bn, wb += bw;
        }
        sh.bin = b;
        sh.bin_count = sh.tcount[b], sh.bin_mass = sh.tmass[b];
        sh.count_before = (uint32_t)nb, sh.mass_before = wb;
      }
    }
    __syncthreads();
  }

  __device__ void clear(int level) {
    if (threadIdx.x < kBins) sh.count[level][threadIdx.x] = 0, sh.mass[level][threadIdx.x] = 0;
    __syncthreads();
  }
  __device__ __forceinline__ void put(int level, int bin, float d) {
    atomicAdd(&sh.count[level][bin], 1u);
    atomicAdd(reinterpret_cast<unsigned long long *>(&sh.mass[level][bin]), (unsigned long long)weight(d));
  }

  // The first split: an eighth of an octave a bin.
  __device__ void split_first() {
    clear(0);
    entries([&](float d, int32_t) { put(0, (int)(-d * 8.0f), d); });
  }

  // The end of the shortest prefix of the order that has `need` entries (or
  // `need` of mass), and the mass of that prefix.  Without one: the end of all.
  __device__ Place prefix(bool by_mass, uint64_t need, uint64_t *mass) {
    search(0, by_mass, need);
    if (sh.bin < 0) {
      uint64_t all = 0;
      for (int b = 0; b < kBins; b++) all += sh.tmass[b];
      *mass = all;
      return Place{0x7fffffffu, 0};
    }
    uint32_t lo = __float_as_uint(sh.bin * 0.125f), hi = __float_as_uint((sh.bin + 1) * 0.125f);
    int32_t ilo = 0, ihi = x.vocab;
    uint64_t before = 0;
    for (;;) {
      need -= by_mass ? sh.mass_before : (uint64_t)sh.count_before;
      before += sh.mass_before;
      const bool whole = sh.bin_count == 1 || (by_mass ? need == sh.bin_mass : need == sh.bin_count);
      const uint64_t bin_mass = sh.bin_mass;
      if (whole) {
        *mass = before + bin_mass;
        return hi - lo == 1 ? Place{lo, ihi} : Place{hi, 0};
      }
      // split keys [lo, hi), or, where that is one key, its indices [ilo, ihi)
      const bool ties = hi - lo == 1;
      const uint32_t width = ties ? (uint32_t)(ihi - ilo) : hi - lo;
      const int shift = max(0, 32 - __clz(width - 1) - 8);
      if (size > 1) cluster_sync(); else __syncthreads();   // everyone has read the bins of the split before
      clear(1);
      if (!ties) {
        entries([&](float d, int32_t) {
          const uint32_t q = key(d);
          if (q >= lo && q < hi) put(1, (q - lo) >> shift, d);
        });
      } else {
        entries([&](float d, int32_t i) {
          if (key(d) == lo && i >= ilo && i < ihi) put(1, (i - ilo) >> shift, d);
        });
      }
      search(1, by_mass, need);
      if (ties) {
        ilo += sh.bin << shift;
        ihi = min(ihi, ilo + (1 << shift));
      } else {
        lo += (uint32_t)sh.bin << shift;
        hi = min(hi, lo + (1u << shift));
      }
    }
  }
};

template <typename T, int KV, int NT>
__global__ __launch_bounds__(NT) void sample_kernel(const SampleArgs a) {
  __shared__ Shared sh;
  const uint32_t size = cluster_size(), rank = cluster_rank();
  const int64_t row = blockIdx.x / size;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sampler<T, KV, NT> s(sh);
  s.rank = rank, s.size = size;
  s.x.set(static_cast<const T *>(a.logits) + row * a.stride, a.vocab, rank, size);
  s.x.load();

  const float temperature = a.s.temperatures ? a.s.temperatures[row] : a.s.temperature;
  const int32_t top_k = a.s.top_ks ? a.s.top_ks[row] : a.s.top_k;
  const float top_p = a.s.top_ps ? a.s.top_ps[row] : a.s.top_p;
  const float min_p = a.s.min_ps ? a.s.min_ps[row] : a.s.min_p;

  // the maximum (fmaxf passes NaN over)
  float m = -INFINITY;
  s.x.each([&](int, const float *v) {
#pragma unroll
    for (int e = 0; e < s.x.kE; e++) m = fmaxf(m, v[e]);
  });
  m = warp_max(m);
  if (threadIdx.x == 0) sh.best = 0xffffffffu;
  if (lane == 0) sh.warp[warp] = __float_as_uint(m);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NT / 32; i++) m = fmaxf(m, __uint_as_float((uint32_t)sh.warp[i]));
  cluster_post(__float_as_uint(m), sh.box[0], rank, size);
  for (uint32_t r = 0; r < size; r++) m = fmaxf(m, __uint_as_float((uint32_t)sh.box[0][r]));

  if (m == -INFINITY) {   // nothing left to choose from
    if (rank == 0 && threadIdx.x == 0) a.tokens[row] = -1, a.logps[row] = -INFINITY;
    return;
  }
  if (!(temperature > 0.0f)) {   // the lowest index of the maximum
    uint32_t best = 0xffffffffu;
    s.x.each([&](int k, const float *v) {
#pragma unroll
      for (int e = 0; e < s.x.kE; e++)
        if (v[e] == m) best = min(best, (uint32_t)s.x.index(k, e));
    });
    best = __reduce_min_sync(~0u, best);
    if (lane == 0) atomicMin(&sh.best, best);
    __syncthreads();
    cluster_post(sh.best, sh.box[1], rank, size);
    for (uint32_t r = 0; r < size; r++) best = min(best, (uint32_t)sh.box[1][r]);
    if (rank == 0 && threadIdx.x == 0) a.tokens[row] = best, a.logps[row] = 0.0f;
    return;
  }
  s.m = m;
  s.c = __fdiv_rn(1.44269504f, temperature);

  // where the kept prefix ends
  Place end = {0x7fffffffu, 0};
  const bool by_k = top_k > 0 && top_k < a.vocab, by_p = top_p < 1.0f;
  if (by_k || by_p) {
    s.split_first();
    uint64_t mass = 0;
    if (by_k) {
      end = s.prefix(false, top_k, &mass);
    } else {
      s.search(0, false, 1);
      for (int b = 0; b < kBins; b++) mass += sh.tmass[b];
    }
    if (by_p) {
      const uint64_t part = top_p > 0.0f ? (uint64_t)(top_p * 4294967296.0f) : 0;
      const uint64_t cut = max((uint64_t)1, share(part, mass));
      uint64_t unused;
      end = s.prefix(true, cut, &unused);
    }
  }
  const uint32_t least = min_p > 0.0f ? __float2uint_rn(fminf(min_p, 1.0f) * 2147483648.0f) : 0;

  // the kept mass: of this thread, its warp, its CTA, the row
  auto kept = [&](float d, int32_t i) -> uint32_t {
    const uint32_t w = s.weight(d), q = s.key(d);
    return w >= least && (q < end.key || (q == end.key && i < end.index)) ? w : 0;
  };
  uint64_t mine = 0;
  s.entries([&](float d, int32_t i) { mine += kept(d, i); });
  const uint64_t of_warp = warp_sum(mine);
  __syncthreads();
  if (lane == 0) sh.warp[warp] = of_warp;
  __syncthreads();
  uint64_t of_cta = 0, before = 0;
#pragma unroll
  for (int i = 0; i < NT / 32; i++) {
    if (i < warp) before += sh.warp[i];
    of_cta += sh.warp[i];
  }
  cluster_post(of_cta, sh.box[2], rank, size);   // also: no CTA reads another's memory after this
  uint64_t z = 0;
  for (uint32_t r = 0; r < size; r++) {
    if (r < rank) before += sh.box[2][r];
    z += sh.box[2][r];
  }

  // the entry at which the running sum passes the target
  const float u = a.u[row];
  const uint64_t part = u > 0.0f ? (u < 1.0f ? (uint64_t)(u * 4294967296.0f) : 0xffffffffull) : 0;
  const uint64_t target = share(part, z);
  if (target < before || target >= before + of_warp) return;
  bool found = false;
  s.x.each([&](int k, const float *v) {
    if (found) return;
    uint64_t of_vec = 0;
#pragma unroll
    for (int e = 0; e < s.x.kE; e++) {
      const float d = s.octaves(v[e]);
      if (d > kFloor) of_vec += kept(d, s.x.index(k, e));
    }
    const uint64_t up_to = before + warp_scan(of_vec, lane);
    if (target >= up_to - of_vec && target < up_to) {
      uint64_t sum = up_to - of_vec;
#pragma unroll
      for (int e = 0; e < s.x.kE; e++) {
        const float d = s.octaves(v[e]);
        const uint32_t w = d > kFloor ? kept(d, s.x.index(k, e)) : 0;
        if (target >= sum && target < sum + w) {
          a.tokens[row] = s.x.index(k, e);
          a.logps[row] = (d - log2f((float)z * 4.6566128730773926e-10f)) * 0.69314718f;
        }
        sum += w;
      }
    }
    before = __shfl_sync(~0u, up_to, 31);
    found = target < before;
  });
}

template <typename T, int KV, int NT>
int run_sample(const SampleArgs &a, int size, cudaStream_t stream) {
  const cudaError_t e = launch_rows(sample_kernel<T, KV, NT>, a, a.rows, size, NT, 0, stream);
  return e == cudaSuccess ? SEQSUM_OK : note_cuda(e);
}

// The smallest cluster and vectors a thread that hold a row, more CTAs where
// the rows are few.
template <typename T>
int choose_sample(const SampleArgs &a, cudaStream_t stream) {
  constexpr int NT = 512;
  const int64_t vecs = ((int64_t)a.vocab + 2 * Elem<T>::kPerVec - 2) / Elem<T>::kPerVec;   // whatever the alignment
  const int sms = multiprocessors();
  int size = 1;
  while (size < kMaxCluster && (vecs > (int64_t)size * NT * 8 || a.rows * size * 2 <= sms)) size *= 2;
  const int64_t per = ((vecs + size - 1) / size + NT - 1) / NT;
  if (per <= 1) return run_sample<T, 1, NT>(a, size, stream);
  if (per <= 2) return run_sample<T, 2, NT>(a, size, stream);
  if (per <= 4) return run_sample<T, 4, NT>(a, size, stream);
  if (per <= 8) return run_sample<T, 8, NT>(a, size, stream);
  return run_sample<T, 0, NT>(a, size, stream);
}

}  // namespace
}  // namespace sq

extern "C" int seqsum_sample_tokens(const void *logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                                    const float *u, const seqsum_sampling *sampling, int64_t *tokens, float *logps,
                                    cudaStream_t stream) {
  if (rows < 0 || vocab < 0 || vocab > sq::row::kMaxVocab || rows > SEQSUM_MAX_ROWS || !sampling) return SEQSUM_EINVAL;
  if (dtype != SEQSUM_FP32 && dtype != SEQSUM_FP16 && dtype != SEQSUM_BF16) return SEQSUM_EINVAL;
  if (rows == 0) return SEQSUM_OK;
  if (!u || !tokens || !logps || (vocab > 0 && !logits) || row_stride < 0) return SEQSUM_EINVAL;
  if (reinterpret_cast<uintptr_t>(logits) % (dtype == SEQSUM_FP32 ? 4 : 2)) return SEQSUM_EINVAL;
  sq::SampleArgs a = {logits, rows, row_stride, (int32_t)vocab, u, *sampling, tokens, logps};
  if (dtype == SEQSUM_FP32) return sq::choose_sample<float>(a, stream);
  if (dtype == SEQSUM_FP16) return sq::choose_sample<__half>(a, stream);
  return sq::choose_sample<__nv_bfloat16>(a, stream);
}
