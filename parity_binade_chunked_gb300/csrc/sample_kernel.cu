// One token a row of logits (seqsum_sample_tokens).
//
// The weights are integers: w = rn(2^31 * 2^d), d the logit's distance to the
// row's maximum in octaves.  Sums of integers do not depend on their order, so
// the mass of a top-k set, the cut of top-p and the draw are exact, however
// the row is split over threads and CTAs; only 2^d itself is rounded.
//
// Every filter keeps a prefix of one order: larger d first, ties by lower
// index.  So the kept set is known by its last element, and that is found by
// counting: entries, by their place in that order (bits of -d, index), are
// split into 256 bins, the bin in which the count passes k (or the mass passes
// the cut) is split again, until at most 32 entries are left, which are placed
// by counting those before each.  Entries with d <= -32 have w = 0 and can be
// left out everywhere.
//
// Most of a row is kept out of the searches.  Top-k: j threads' maxima each in
// half of the cluster's warps are k entries, so the k-th is not below the least
// of those; what is not below is listed (some hundred entries) and searched in
// each CTA.  Top-p: the tail's mass by eighths of an octave, estimated from
// every fourth or eighth entry, says which eighths the cut is in; their entries
// are split, with the exact mass before them, which confirms the estimate.
//
// What bounds it is not HBM but, where the rows are few, the chain of a row's
// parts: some 8 without filters, 20 with, each a pass over a warp's steps or a
// wait for the cluster of about 1000 cycles (one row of 32000 bf16 numbers 6 and
// 13 us); where they are many, issue slots and the latency of L2: an element
// costs some 10 instructions a pass and there are two passes without filters,
// four with.  256 x 131072 bf16 (floor 9.9 us): plain 24 us, greedy 15, min-p
// 0.02 28, top-k 50 42, top-k 5000 175, top-p 0.9 95 us, and 193 us at
// temperature 1.5, where the kept are 40000 of a row and pass the lists; 512 x
// 131072 fp32 plain 80 us (floor 40).  The searches over rows in L2 run in 64
// registers, two CTAs an SM, and spill some 400 bytes a thread.  (GPU time of
// calls one after another in a graph.)
#include <math.h>

#include <atomic>
#include <type_traits>

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
  int32_t steps;   // that a CTA takes of a row at most
  Waits waits;
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

// floor(2^32 * x) for x in [0, 1]
__device__ __forceinline__ uint64_t part_of(float x) { return x > 0.0f ? (uint64_t)(x * 4294967296.0f) : 0; }

// 2^31 * 2^d as an integer: 0 for d <= kFloor, and for NaN
__device__ __forceinline__ uint32_t weight(float d) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(d));
  return __float2uint_rn(y * 2147483648.0f);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t key_of(float d) { return __float_as_uint(d) & 0x7fffffffu; }

// ---- rows too large for the buffers: one CTA a part of a row, every pass reads
// global memory (L2), and every search goes over the whole row.

template <typename T, int NT>
struct Sampler {
  Slice<T, 0, NT> x;
  Shared &sh;
  float m, c;
  uint32_t rank, size;

  __device__ Sampler(Shared &s) : sh(s) {}

  // octaves below the maximum; NaN (a masked logit where c is 0, a NaN logit) counts as masked
  __device__ __forceinline__ float octaves(float v) const { return v == m ? 0.0f : (v - m) * c; }

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
    cluster_sync();
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
      cluster_sync();   // everyone has read the bins of the split before
      clear(1);
      if (!ties) {
        entries([&](float d, int32_t) {
          const uint32_t q = key_of(d);
          if (q >= lo && q < hi) put(1, (q - lo) >> shift, d);
        });
      } else {
        entries([&](float d, int32_t i) {
          if (key_of(d) == lo && i >= ilo && i < ihi) put(1, (i - ilo) >> shift, d);
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

template <typename T, int NT>
__global__ __launch_bounds__(NT) void sample_reread_kernel(const SampleArgs a) {
  __shared__ Shared sh;
  const uint32_t size = cluster_size(), rank = cluster_rank();
  cluster_begun();
  const int64_t row = blockIdx.x / size;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sampler<T, NT> s(sh);
  s.rank = rank, s.size = size;
  s.x.set(static_cast<const T *>(a.logits) + row * a.stride, a.vocab, rank, size);

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
  cluster_wait_begun();
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
    const uint32_t w = weight(d), q = key_of(d);
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

// ---- rows streamed through shared memory (see Stream)
//
// A row has three parts: its maximum; what is kept of it and the mass of that
// by segments; the place of the token.  The words of a part travel while the
// next row's first part is worked on.
//
// Where the rows are many, a CTA takes a row to itself: it reads the row from
// HBM once and from L2 in the later passes, and tells no one anything.  Twice
// the SMs' number of rows is under way then, instead of a quarter (256 x 131072
// bf16 with top-p 0.9: 95 us, by clusters 180; 64 rows 52 by clusters).

// without top-k and top-p, and with them; rows on chip, and in L2
enum Kind { kPlain, kSearch, kFarPlain, kFarSearch };
__host__ __device__ constexpr bool is_far(Kind k) { return k >= kFarPlain; }
__host__ __device__ constexpr bool searches(Kind k) { return k == kSearch || k == kFarSearch; }

constexpr int kList = 1280;   // entries that a search can take out of the row
constexpr int kFarSteps = 8192;   // of a row that a CTA takes to itself, at most
template <Kind K>
constexpr int kOwn = is_far(K) ? 384 : 192;   // ... that a warp can of its segment
template <Kind K>
constexpr int kMost = is_far(K) ? 1 : kMaxCluster;   // CTAs a row at most

// What the CTA's warps share, and what others of the cluster write to.  Calls
// without top-k and top-p have no use for lists; they get a third buffer.
template <int W, Kind K>
struct Picks {
  static constexpr int kBinsHere = searches(K) ? kBins : 1, kPartHere = K == kSearch ? kBins : 1,
                       kListHere = searches(K) ? kList : 1, kOwnHere = searches(K) ? kOwn<K> : 1, kBoxes = kMost<K> * W;
  uint64_t full[3], empty[3], told[4], parts, totals, entries;
  uint32_t begun, whole;          // rows whose copy is on its way, whose edges are too (for the warp that brings them)
  uint64_t box[4][kBoxes];        // a word of every warp of the cluster
  uint64_t step_mass[is_far(K) ? kFarSteps / W : 32];   // of the segment that the token is in
  uint4 bins[kBinsHere];          // a split of the CTA's entries: count, and mass in three parts
  uint64_t part[2][kPartHere];    // this CTA's share of the bins, of every CTA: count and mass; rounds take turns
  uint4 total[kBinsHere];         // the bins summed over the cluster: count, mass
  uint32_t listed, small_listed;
  uint4 small[32];                // the last few entries of a search: key, index, weight
  uint2 list[kListHere], all[kListHere];  // (key, index): this CTA's entries, the row's
  uint2 own[W][kOwnHere];         // a warp's
};

template <Kind K>
constexpr int kBuffers = is_far(K) ? 0 : searches(K) ? 2 : 3;

__device__ __forceinline__ uint64_t mass_of(uint4 bin) { return bin.y + ((uint64_t)bin.z << 11) + ((uint64_t)bin.w << 22); }

struct Found {
  int bin;                        // -1: the need is not reached
  uint32_t count, count_before;
  uint64_t mass, mass_before;
};

template <typename T, int W, Kind K>
struct Picker {
  static constexpr int kE = Elem<T>::kPerVec, kThreads = W * 32;
  static constexpr int kAhead = 4;   // steps of far rows whose vectors are loaded side by side
  Picks<W, K> &sh;
  std::conditional_t<is_far(K), FarRow<T>, Stream<T>> x;
  uint32_t rank, size, posted = 0, heard = 0, totalled = 0, shared_lists = 0;
  int32_t st0, st1;     // this warp's steps
  float m, c;
  bool special;         // (v - m) * c needs care
  uint32_t limit;       // of a wait
  bool came = true;     // no wait of this warp gave up
  bool ok = true;       // ... none of the CTA's, as of the last agreement
  int own = -1;         // entries that this warp took out of its segment, from own_from octaves on
  float own_from = 0.0f;
  int32_t listed = -1;  // entries of sh.all, once a search goes over those; -1: over the row

  __device__ Picker(Picks<W, K> &s) : sh(s) {}

  // ---- the CTA's working warps, and the cluster's

  __device__ __forceinline__ void team() const { asm volatile("barrier.cta.sync 1, %0;" ::"n"(kThreads) : "memory"); }
  // Once a wait gave up the warp waits no more and tells no one anything, so
  // that no CTA goes on with what it did not have.
  __device__ __forceinline__ void wait(uint64_t *bar, uint32_t parity) {
    came = came && __all_sync(~0u, bar_wait(bar, parity, limit));
  }
  // All of the CTA's working warps go on together or give up together: after
  // every wait for another CTA, before a warp takes its way by what came.
  __device__ __forceinline__ void agree() {
    if (is_far(K)) return;   // (no waits that could give up)
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"((uint32_t)came), "n"(kThreads)
        : "memory");
    ok &= all != 0;
  }
  // A word of every warp to every warp.  Two may be on their way: a warp posts
  // its word after next only once it has waited for this one, so that of four
  // boxes the one that is written is never one that is still read.
  __device__ __forceinline__ void post(uint64_t v) {
    if (is_far(K)) {
      if ((threadIdx.x & 31) == 0) sh.box[posted & 3][threadIdx.x >> 5] = v;
      posted++;
      return;
    }
    const Exchange e = {sh.box[posted & 3], &sh.told[posted & 3]};
    posted++;
    if (came) e.post((int32_t)(rank * W + (threadIdx.x >> 5)), v, size);
  }
  __device__ __forceinline__ const uint64_t *hear() {
    const uint32_t b = heard & 3, parity = (heard >> 2) & 1;
    heard++;
    if (is_far(K)) return team(), sh.box[b];
    wait(&sh.told[b], parity);
    if (came && threadIdx.x == 0) bar_expect(&sh.told[b], size * W * 8);
    return sh.box[b];
  }
  // The sum of the words heard.
  __device__ __forceinline__ uint64_t sum_of(const uint64_t *box) const {
    constexpr int kPer = (kMost<K> * W + 31) / 32;
    uint64_t sum = 0;
#pragma unroll
    for (int k = 0; k < kPer; k++) {
      const uint32_t i = (threadIdx.x & 31) + 32 * k;
      if (i < size * W) sum += box[i];
    }
    return warp_sum(sum);
  }
  // sh.bins of every CTA, once all its warps are through, summed into sh.total
  // of each: every CTA sums its share of the bins and sends the sums around.
  // (Sent with asynchronous stores: a release of plain ones to the cluster
  // took 1300 to 5000 cycles, reading 256 bins of 8 CTAs 2000.)
  // What says that no one still reads what is written here: another CTA has
  // its sums, and so goes on, once those of this CTA's threads that sum for it
  // have sent theirs; the threads that sum for others may still be reading
  // `part`.  So rounds take two of them in turn: a round's words come after the
  // sums of the round before, which come after all of this CTA's warps began
  // that round, so after their reads two rounds back.  `total` needs one: its
  // words come after the sender had this CTA's words of the same round.
  // Returns the words posted before it, where there are some to hear.
  __device__ __forceinline__ const uint64_t *total_bins(bool posted_words) {
    const uint64_t *box = nullptr;
    team();
    if (is_far(K) || size == 1) {
      if (threadIdx.x < kBins) {
        const uint4 v = sh.bins[threadIdx.x];
        const uint64_t w = mass_of(v);
        sh.total[threadIdx.x] = make_uint4(v.x, (uint32_t)w, (uint32_t)(w >> 32), 0);
      }
      if (posted_words) box = hear();
      if (!is_far(K)) agree();
      else if (!posted_words) team();
      return box;
    }
    const uint32_t share = kBins / size, to = threadIdx.x / share, bin = threadIdx.x % share, parity = totalled++ & 1;
    uint64_t *part = sh.part[parity];
    if (came && threadIdx.x < kBins) {
      const uint4 v = sh.bins[threadIdx.x];
      const uint64_t w = mass_of(v);
      send(reinterpret_cast<uint2 *>(&part[rank * share + bin]), &sh.parts, to, make_uint2((uint32_t)w, (uint32_t)(w >> 32) | v.x << 16));
    }
    wait(&sh.parts, parity);
    if (came && threadIdx.x == 0) bar_expect(&sh.parts, kBins * 8);
    if (came && threadIdx.x < kBins) {
      uint32_t n = 0;
      uint64_t w = 0;
#pragma unroll
      for (uint32_t c = 0; c < kMaxCluster; c++)
        if (c < size) {
          const uint64_t v = part[c * share + bin];   // a slice's count fits 16 bits, its mass 48
          n += (uint32_t)(v >> 48), w += v & ((1ull << 48) - 1);
        }
      send(&sh.total[rank * share + bin], &sh.totals, to, make_uint4(n, (uint32_t)w, (uint32_t)(w >> 32), 0));
    }
    wait(&sh.totals, parity);
    if (came && threadIdx.x == 0) bar_expect(&sh.totals, kBins * 16);
    if (posted_words) box = hear();
    agree();
    return box;
  }
  __device__ __forceinline__ void clear_bins() {
    if (threadIdx.x < kBins) sh.bins[threadIdx.x] = make_uint4(0, 0, 0, 0);
    team();
  }

  // ---- entries

  __device__ __forceinline__ void octaves(uint4 w, float *d) const {
    Elem<T>::unpack(w, d);
    if (special) {
#pragma unroll
      for (int e = 0; e < kE; e++) d[e] = d[e] == m ? 0.0f : (d[e] - m) * c;
    } else {
      const uint64_t mm = pair(-m, -m), cc = pair(c, c);
#pragma unroll
      for (int e = 0; e < kE; e += 2) split(mul2(add2(pair(d[e], d[e + 1]), mm), cc), d[e], d[e + 1]);
    }
  }
  // f(step, this lane's vector of it) for the warp's steps; of far rows some
  // vectors are loaded side by side
  template <typename F>
  __device__ __forceinline__ void steps(F f) const {
    if constexpr (is_far(K)) {
      for (int32_t st = st0; st < st1; st += kAhead) {
        uint4 w[kAhead];
        if (st + kAhead <= st1 && x.index(st * 32, 0) >= 0 && x.index((st + kAhead) * 32, 0) <= x.vocab) {
          const uint4 *p = reinterpret_cast<const uint4 *>(x.p + x.index(st * 32 + (int32_t)(threadIdx.x & 31), 0));
#pragma unroll
          for (int k = 0; k < kAhead; k++) w[k] = __ldg(p + 32 * k);
        } else {
          constexpr uint32_t ninf = Elem<T>::kNegInf;
#pragma unroll
          for (int k = 0; k < kAhead; k++) w[k] = st + k < st1 ? x.vec(st + k) : make_uint4(ninf, ninf, ninf, ninf);
        }
#pragma unroll
        for (int k = 0; k < kAhead; k++) f(st + k, w[k]);
      }
    } else {
#pragma unroll 1
      for (int32_t st = st0; st < st1; st++) f(st, x.vec(st));
    }
  }
  // a logit that entries from `from` octaves on reach, with room for roundings
  __device__ __forceinline__ float reached_from(float from) const {
    const float v = m + __fdiv_rn(from, c) * 1.00001f, t = v - (fabsf(v) + fabsf(m)) * 1e-6f;
    return special || !(t > -INFINITY) ? -INFINITY : t;
  }
  // Takes the entries from `from` octaves on out of the warp's segment, if they
  // are few enough: passes over them are short then, whatever their places.
  __device__ __forceinline__ void collect(float from) {
    const int lane = threadIdx.x & 31;
    const float least = reached_from(from);
    uint2 *to = sh.own[threadIdx.x >> 5];
    int n = 0;
    steps([&](int32_t st, uint4 w) {
      if (n > kOwn<K> || !__any_sync(~0u, Elem<T>::vec_max(w, -INFINITY) >= least)) return;
      float d[kE];
      octaves(w, d);
#pragma unroll
      for (int e = 0; e < kE; e++) {
        const bool in = d[e] >= from && d[e] > kFloor;
        const uint32_t who = __ballot_sync(~0u, in);
        const int at = n + __popc(who & ((1u << lane) - 1));
        if (in && at < kOwn<K>) to[at] = make_uint2(key_of(d[e]), (uint32_t)x.index(st * 32 + lane, e));
        n += __popc(who);
      }
    });
    __syncwarp();
    own = n <= kOwn<K> ? n : -1;
    own_from = from;
  }
  // f(octaves, index) of the row's entries from `from` octaves (at least
  // kFloor) up to `to` in this thread
  template <typename F>
  __device__ __forceinline__ void row_entries(float from, float to, F f) const {
    const int lane = threadIdx.x & 31;
    if (own >= 0 && from >= own_from) {
      for (int i = lane; i < own; i += 32) {
        const uint2 v = sh.own[threadIdx.x >> 5][i];
        const float d = -__uint_as_float(v.x);
        if (d >= from && d <= to) f(d, (int32_t)v.y);
      }
      return;
    }
    const float least = reached_from(from);
    steps([&](int32_t st, uint4 w) {
      if (!(Elem<T>::vec_max(w, -INFINITY) >= least)) return;
      float d[kE];
      octaves(w, d);
      bool any = false;
#pragma unroll
      for (int e = 0; e < kE; e++) any |= d[e] >= from && d[e] <= to;
      if (any) {
#pragma unroll
        for (int e = 0; e < kE; e++)
          if (d[e] >= from && d[e] <= to && d[e] > kFloor) f(d[e], x.index(st * 32 + lane, e));
      }
    });
  }
  // The sum of g(octaves, index) over them, where g is 0 for NaN and -inf
  // (without branches: for rows of which many entries count).
  template <typename G>
  __device__ __forceinline__ uint64_t row_sum(float from, G g) const {
    const int lane = threadIdx.x & 31;
    uint64_t sum = 0;
    if (own >= 0 && from >= own_from) {
      for (int i = lane; i < own; i += 32) {
        const uint2 v = sh.own[threadIdx.x >> 5][i];
        sum += g(-__uint_as_float(v.x), (int32_t)v.y);
      }
      return warp_sum(sum);
    }
    const float least = reached_from(from);
    steps([&](int32_t st, uint4 w) {
      if (!(Elem<T>::vec_max(w, -INFINITY) >= least)) return;
      float d[kE];
      octaves(w, d);
#pragma unroll
      for (int e = 0; e < kE; e += 2)
        sum += (uint64_t)g(d[e], x.index(st * 32 + lane, e)) + g(d[e + 1], x.index(st * 32 + lane, e + 1));
    });
    return warp_sum(sum);
  }
  // ... or of the list
  template <typename F>
  __device__ __forceinline__ void list_entries(F f) const {
    for (int32_t i = threadIdx.x; i < listed; i += kThreads) {
      const uint2 v = sh.all[i];
      f(-__uint_as_float(v.x), (int32_t)v.y);
    }
  }

  // ---- searches

  __device__ __forceinline__ void put(uint4 *bins, uint32_t bin, float d) const {
    const uint32_t w = weight(d);
    atomicAdd(&bins[bin].x, 1u);
    atomicAdd(&bins[bin].y, w & 0x7ffu);   // (below 2^21 entries the parts' sums fit 32 bits)
    atomicAdd(&bins[bin].z, w >> 11 & 0x7ffu);
    atomicAdd(&bins[bin].w, w >> 22);
  }
  // Entries that a search goes on in: keys [lo, hi), or, where that is one
  // key, indices [ilo, ihi) of it.  A first split (scale > 0) is even in
  // octaves: by a power of two, from an eighth of an octave, so that
  // differences and products are exact and each bin is a range of keys.
  struct Range {
    uint32_t lo, hi;
    int32_t ilo, ihi;
    float from, scale;
    __device__ __forceinline__ void eighths(int e0, int e1, int32_t vocab) {
      from = e0 * 0.125f;
      lo = __float_as_uint(from), hi = __float_as_uint(e1 * 0.125f);
      ilo = 0, ihi = vocab;
      scale = 8.0f;
      for (int n = e1 - e0; n <= kBins / 2; n *= 2) scale *= 2.0f;
    }
    __device__ __forceinline__ bool ties() const { return hi - lo == 1; }
    __device__ __forceinline__ bool holds(uint32_t key, int32_t i) const {
      return key >= lo && key < hi && (!ties() || (i >= ilo && i < ihi));
    }
    __device__ __forceinline__ int shift() const {
      const uint32_t width = ties() ? (uint32_t)(ihi - ilo) : hi - lo;
      return max(0, 32 - __clz(width - 1) - 8);
    }
    __device__ __forceinline__ void take_bin(int bin) {
      if (scale > 0.0f) {
        const float f = from;
        lo = __float_as_uint(f + bin / scale), hi = __float_as_uint(f + (bin + 1) / scale);
        scale = 0.0f;
      } else if (const int s = shift(); ties()) {
        ilo += bin << s;
        ihi = min(ihi, ilo + (1 << s));
      } else {
        lo += (uint32_t)bin << s;
        hi = min(hi, lo + (1u << s));
      }
    }
  };

  // (What find, sample and count return means nothing where the CTA gave up in them.)

  // Splits the entries of `r` and finds the first bin at which their count (or
  // mass) reaches `need`.  Over the row, entries from `from` octaves on are
  // looked at, and the mass of those before `r` comes before all bins.
  __device__ Found find(bool by_mass, uint64_t need, const Range &r, float from) {
    clear_bins();
    uint64_t front = 0;
    const int shift = r.scale > 0.0f ? 0 : r.shift();
    auto take = [&](float d, int32_t i) {
      const uint32_t key = key_of(d);
      if (r.holds(key, i))
        put(sh.bins, r.scale > 0.0f ? (uint32_t)((-d - r.from) * r.scale) : (r.ties() ? (uint32_t)(i - r.ilo) : key - r.lo) >> shift, d);
    };
    if (listed < 0) {
      const float lo = __uint_as_float(r.lo);
      if (r.scale > 0.0f) post(r.lo > 0 ? row_sum(from, [&](float d, int32_t) { return -d < lo ? weight(d) : 0; }) : 0);
      row_entries(from, -lo, take);
      const uint64_t *box = total_bins(r.scale > 0.0f);
      front = r.scale > 0.0f ? sum_of(box) : 0;
    } else {
      list_entries(take);
      team();
      if (threadIdx.x < kBins) {
        const uint4 v = sh.bins[threadIdx.x];
        const uint64_t w = mass_of(v);
        sh.total[threadIdx.x] = make_uint4(v.x, (uint32_t)w, (uint32_t)(w >> 32), 0);
      }
      team();
      front = 0;
    }
    // Every warp for itself: lane l has bins 8 l to 8 l + 7; then, of the lane
    // whose bins reach it, each of the first eight lanes a bin.
    constexpr int kPer = kBins / 32;
    const int lane = threadIdx.x & 31;
    uint32_t n = 0;
    uint64_t w = 0;
#pragma unroll
    for (int i = 0; i < kPer; i++) {
      const uint4 v = sh.total[lane * kPer + i];
      n += v.x, w += v.y + ((uint64_t)v.z << 32);
    }
    const uint64_t upto = by_mass ? front + warp_scan(w, lane) : warp_scan(n, lane);
    const uint32_t reached = __ballot_sync(~0u, need <= upto);
    Found f = {-1, 0, 0, 0, 0};
    if (reached && !(by_mass && front >= need)) {
      const int o = __ffs(reached) - 1;
      const uint32_t nb = __reduce_add_sync(~0u, lane < o ? n : 0);
      const uint64_t wb = front + warp_sum(lane < o ? w : 0);
      const uint4 v = sh.total[o * kPer + lane % kPer];
      uint32_t n8 = v.x;
      uint64_t w8 = v.y + ((uint64_t)v.z << 32);
#pragma unroll
      for (int d = 1; d < kPer; d <<= 1) {
        const uint32_t nu = __shfl_up_sync(~0u, n8, d);
        const uint64_t wu = __shfl_up_sync(~0u, w8, d);
        if (lane % kPer >= d) n8 += nu, w8 += wu;
      }
      const int at = __ffs(__ballot_sync(~0u, by_mass ? need <= wb + w8 : need <= (uint64_t)nb + n8)) - 1;
      f.bin = o * kPer + at;
      const uint32_t n_at = __shfl_sync(~0u, v.x, at);
      const uint64_t w_at = __shfl_sync(~0u, v.y + ((uint64_t)v.z << 32), at);
      f.count = n_at, f.mass = w_at;
      f.count_before = nb + __shfl_sync(~0u, n8, at) - n_at;
      f.mass_before = wb + __shfl_sync(~0u, w8, at) - w_at;
    }
    team();   // the sums may be written again
    return f;
  }

  // Of at most 32 listed entries in `r`, `n` of them, the one at which the
  // count (or mass) reaches `need`: each lane has one, placed by counting.
  // Its mass and that before it are added to *mass.
  __device__ Place last_few(bool by_mass, uint64_t need, uint32_t n, const Range &r, uint64_t *mass) {
    if (threadIdx.x == 0) sh.small_listed = 0;
    team();
    list_entries([&](float d, int32_t i) {
      const uint32_t key = key_of(d);
      if (r.holds(key, i)) {
        const uint32_t at = atomicAdd(&sh.small_listed, 1u);
        if (at < 32) sh.small[at] = make_uint4(key, (uint32_t)i, weight(d), 0);
      }
    });
    team();
    const uint32_t lane = threadIdx.x & 31;
    const bool have = lane < n;
    const uint4 v = have ? sh.small[lane] : make_uint4(~0u, ~0u, 0, 0);
    uint32_t count = 0;
    uint64_t sum = 0;
#pragma unroll 4
    for (uint32_t j = 0; j < n; j++) {
      const uint4 o = sh.small[j];
      if (o.x < v.x || (o.x == v.x && o.y < v.y)) count++, sum += o.z;
    }
    const bool last = have && (by_mass ? sum < need && need <= sum + v.z : count + 1 == need);
    const int o = max(0, __ffs(__ballot_sync(~0u, last)) - 1);
    *mass += __shfl_sync(~0u, sum + v.z, o);
    const Place p = {__shfl_sync(~0u, v.x, o), (int32_t)__shfl_sync(~0u, v.y, o) + 1};
    team();
    return p;
  }

  // Lists the row's entries in `r`, every CTA all of them.  More than kList of
  // them: `listed` stays -1.
  __device__ void list(const Range &r) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) sh.listed = 0;
    team();
    row_entries(fmaxf(kFloor, -__uint_as_float(r.hi)), -__uint_as_float(r.lo), [&](float d, int32_t i) {
      const uint32_t key = key_of(d);
      if (r.holds(key, i)) {
        const uint32_t at = atomicAdd(&sh.listed, 1u);
        if (at < (uint32_t)kList) sh.list[at] = make_uint2(key, (uint32_t)i);
      }
    });
    team();
    const uint32_t mine = sh.listed;
    if (is_far(K) || size == 1) {
      if (mine <= (uint32_t)kList) {
        for (uint32_t i = threadIdx.x; i < mine; i += kThreads) sh.all[i] = sh.list[i];
        listed = (int32_t)mine;
      }
      team();
      return;
    }
    post(warp == 0 ? mine : 0);
    const uint64_t *box = hear();
    const uint32_t theirs = lane < (int)size ? (uint32_t)box[lane * W] : 0;
    const uint32_t ends = warp_scan(theirs, lane), total = __shfl_sync(~0u, ends, 31);
    agree();
    if (total > (uint32_t)kList || !ok) return;
    // each entry goes to every CTA, whose barrier counts them all
    const uint32_t at = __shfl_sync(~0u, ends - theirs, rank);
    for (uint32_t i = threadIdx.x; i < mine * size; i += kThreads) send(&sh.all[at + i / size], &sh.entries, i % size, sh.list[i / size]);
    if (threadIdx.x == 0) bar_expect(&sh.entries, total * 8);
    wait(&sh.entries, shared_lists++ & 1);
    agree();
    listed = (int32_t)total;
  }

  // The mass of all, and by a sample (the first entry of each vector) the
  // eighths of octaves [e0, e1) that the cut of top-p is in: where the tail's
  // mass, give or take four standard deviations and a twentieth, can be what
  // is left after the cut.  That they hold the cut shows when they are summed.
  __device__ uint64_t sample(float top_p, int &e0, int &e1) {
    const int lane = threadIdx.x & 31;
    constexpr int kPer = kBins / 32;
    clear_bins();
    uint64_t mine = 0;
    steps([&](int32_t, uint4 v) {
      float d[kE];
      octaves(v, d);
      uint64_t of_vec = 0;
#pragma unroll
      for (int e = 0; e < kE; e += 2) of_vec += (uint64_t)weight(d[e]) + weight(d[e + 1]);
      mine += of_vec;
      if (d[0] > kFloor) atomicAdd(&sh.bins[(int)(-d[0] * 8.0f)].x, 1u);
    });
    post(warp_sum(mine));
    const uint64_t *box = total_bins(true);
    const uint64_t all = max((uint64_t)1, sum_of(box)), cut = max((uint64_t)1, share(part_of(top_p), all));
    auto middle = [&](int i) { return ex2(30.9375f - (lane * kPer + i) * 0.125f) * kE; };
    float w[kPer], tail = 0.0f, tail2 = 0.0f;   // the tail's mass from an eighth on, and its variance
#pragma unroll
    for (int i = 0; i < kPer; i++) {
      w[i] = (float)sh.total[lane * kPer + i].x * middle(i);
      tail += w[i], tail2 += w[i] * middle(i);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float u = __shfl_down_sync(~0u, tail, o), u2 = __shfl_down_sync(~0u, tail2, o);
      if (lane + o < 32) tail += u, tail2 += u2;
    }
    tail = __shfl_down_sync(~0u, tail, 1), tail2 = __shfl_down_sync(~0u, tail2, 1);   // after the lane's bins
    if (lane == 31) tail = tail2 = 0.0f;
    const float left = (float)(all - cut);
    int b0 = 0, b1 = kBins;
#pragma unroll
    for (int i = kPer - 1; i >= 0; i--) {
      tail += w[i], tail2 += w[i] * middle(i);
      float root;
      asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(root) : "f"(tail2));
      const float off = 0.05f * tail + 4.0f * root;
      if (tail - off > left) b0 = max(b0, lane * kPer + i);
      if (tail + off <= left) b1 = lane * kPer + i;
    }
    e0 = (int)__reduce_max_sync(~0u, (uint32_t)b0);
    e1 = max((int)__reduce_min_sync(~0u, (uint32_t)b1), e0 + 1);
    return cut;
  }

  // Counts by eighths, exactly, of the entries from `least` octaves on; the
  // eighth in which the k-th is (0 where there are fewer, e1 is 0 then), or
  // those that the cut of top-p can be in: bounds of the mass before each from
  // the counts, from the front and, narrower in the tail, from the back.
  __device__ uint64_t count(int32_t top_k, float least, float top_p, int &e0, int &e1) {
    const int lane = threadIdx.x & 31;
    constexpr int kPer = kBins / 32;
    clear_bins();
    uint64_t mine = 0;
    row_entries(least, 0.0f, [&](float d, int32_t) {
      atomicAdd(&sh.bins[(int)(-d * 8.0f)].x, 1u);
      mine += weight(d);
    });
    post(warp_sum(mine));
    const uint64_t *box = total_bins(true);
    const uint64_t all = max((uint64_t)1, sum_of(box)), cut = max((uint64_t)1, share(part_of(top_p), all));
    uint32_t counts[kPer], n = 0;
#pragma unroll
    for (int i = 0; i < kPer; i++) n += counts[i] = sh.total[lane * kPer + i].x;
    const uint32_t upto = warp_scan(n, lane);
    if (top_k > 0) {
      const uint32_t reached = __ballot_sync(~0u, upto >= (uint32_t)top_k);
      e0 = e1 = 0;
      if (reached) {
        const int o = __ffs(reached) - 1;
        uint32_t before = __shfl_sync(~0u, upto - n, o);
        e0 = o * kPer;
        while (ok && before + sh.total[e0].x < (uint32_t)top_k) before += sh.total[e0++].x;
        e1 = e0 + 1;
        return (uint32_t)top_k - before;
      }
      return 0;
    }
    uint64_t lo[kPer], hi[kPer], least_before = 0, most_before = 0;
#pragma unroll
    for (int i = 0; i < kPer; i++) {
      const float top = ex2(31.0f - (lane * kPer + i) * 0.125f);   // 2^(-1/8) = 0.9170040...
      lo[i] = counts[i] * (uint64_t)fmaxf(top * (0.9170040f * 0.99999f) - 2.0f, 0.0f);
      hi[i] = counts[i] * ((uint64_t)(top * 1.00001f) + 2);
      least_before += lo[i], most_before += hi[i];
    }
    const uint64_t least_mass = least_before, most_mass = most_before;
    least_before = warp_scan(least_before, lane), most_before = warp_scan(most_before, lane);
    const uint64_t least_all = __shfl_sync(~0u, least_before, 31), most_all = __shfl_sync(~0u, most_before, 31);
    least_before -= least_mass, most_before -= most_mass;
    int b0 = 0, b1 = kBins;
#pragma unroll
    for (int i = 0; i < kPer; i++) {
      const uint64_t at_most = min(most_before, all - min(all, least_all - least_before));
      const uint64_t at_least = max(least_before, all - min(all, most_all - most_before));
      if (at_most < cut) b0 = lane * kPer + i;
      if (at_least >= cut) b1 = min(b1, lane * kPer + i);
      least_before += lo[i], most_before += hi[i];
    }
    e0 = (int)__reduce_max_sync(~0u, (uint32_t)b0);
    e1 = max((int)__reduce_min_sync(~0u, (uint32_t)b1), e0 + 1);
    return cut;
  }

  // ---- the kept prefix

  // Where the prefix that top-k and top-p keep ends.  `least` is a lower bound
  // of the k-th largest entry's octaves.  Up to two searches, first for the
  // k-th entry, then for the cut of top-p: the shortest prefix of the order
  // that has k entries, or the cut's mass.
  __device__ Place kept_prefix(int32_t top_k, bool by_p, float top_p, float least) {
    bool by_k = top_k > 0 && top_k < x.vocab;
    enum { kAll, kSample, kCount, kGo } how = by_k && least > kFloor ? kAll : by_k ? kCount : kSample;
    listed = -1;
    Range r;
    int e0 = 0, e1 = kBins;
    uint64_t need = top_k, mass = 0, bin_mass = 0;
    uint32_t bin_count = ~0u;
    float from = kFloor;
    bool sampled = false, all_listed = false;
    while (ok) {
      if (how != kGo) {
        // a search begins
        if (how == kAll) {   // not many more than k entries as a rule: all of them at once
          e0 = 0, e1 = min(kBins, (int)(-least * 8.0f) + 1);
        } else {
          if (how == kSample) {
            need = sample(top_p, e0, e1);
            if (!ok) break;
          } else {
            need = count(by_k ? top_k : 0, least, top_p, e0, e1);
            if (!ok) break;
            if (by_k && e1 == 0) {   // all that weighs anything is among the first k
              if (!by_p) break;
              by_k = false;
              how = kSample;
              continue;
            }
          }
          from = fmaxf(-e1 * 0.125f, kFloor);   // what is counted is what list() lists: all above kFloor in the last eighth
          sampled = how == kSample;
          if (!by_k) collect(from);
        }
        r.eighths(e0, e1, x.vocab);
        mass = 0, bin_count = ~0u;
      }
      if (listed < 0 && (how == kAll || bin_count <= (uint32_t)kList)) {   // few enough
        list(r);
        if (!ok) break;
        all_listed = how == kAll && listed >= 0;
        if (how == kAll && listed < 0) {
          how = kCount;
          continue;
        }
      }
      how = kGo;
      Place end;
      if (bin_count <= 32 && listed >= 0 && r.scale == 0.0f) {
        end = last_few(by_k ? false : true, need, bin_count, r, &mass);
      } else if (r.scale == 0.0f && (bin_count == 1 || need == (by_k ? (uint64_t)bin_count : bin_mass))) {
        mass += bin_mass;
        end = r.ties() ? Place{r.lo, r.ihi} : Place{r.hi, 0};
      } else {
        const Found f = find(!by_k, need, r, from);
        if (!ok) break;
        if (f.bin < 0) {
          if (!sampled) return Place{r.hi, 0};   // (cannot be: what is not reached is less than all)
          how = kCount;                          // the sample misled
          continue;
        }
        need -= by_k ? (uint64_t)f.count_before : f.mass_before;
        mass += f.mass_before;
        bin_count = f.count, bin_mass = f.mass;
        r.take_bin(f.bin);
        continue;
      }
      if (!by_k || !by_p) return end;
      // the second search, among those up to here
      by_k = false;
      need = max((uint64_t)1, share(part_of(top_p), mass));
      const int last = min(kBins, (int)(__uint_as_float(end.key) * 8.0f) + 1);
      if (!all_listed) listed = -1;
      r.eighths(0, last, x.vocab);
      from = fmaxf(-last * 0.125f, kFloor);
      mass = 0, bin_count = ~0u;
    }
    return Place{0x7fffffffu, 0};
  }
};

template <typename T, int W, Kind K>
__global__ __launch_bounds__(W * 32, W == 8 || K == kFarSearch || (K == kFarPlain && W == 16) ? 2 : 1) void sample_kernel(const SampleArgs a) {
  constexpr int kB = kBuffers<K> > 0 ? kBuffers<K> : 1;
  extern __shared__ uint4 buffers[];   // kB buffers of a.steps steps, and the rest
  auto &sh = *reinterpret_cast<Picks<W, K> *>(buffers + kBuffers<K> * a.steps * 32);
  constexpr int kE = Elem<T>::kPerVec, kLog2W = W == 32 ? 5 : W == 16 ? 4 : 3;
  const uint32_t size = cluster_size(), rank = cluster_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t first = blockIdx.x / size, step = gridDim.x / size;
  const uint32_t turns = ((uint32_t)a.rows - first + step - 1) / step;   // (at most one cluster a row)
  const int log2_size = __ffs(size) - 1;
  if (!is_far(K) && threadIdx.x == 0) {
    for (int b = 0; b < kB; b++) {
      bar_init(&sh.full[b], 2);
      bar_init(&sh.empty[b], W);
    }
    for (int b = 0; b < 4; b++) {
      bar_init(&sh.told[b], 1);
      bar_expect(&sh.told[b], size * W * 8);
    }
    bar_init(&sh.parts, 1), bar_expect(&sh.parts, kBins * 8);
    bar_init(&sh.totals, 1), bar_expect(&sh.totals, kBins * 16);
    bar_init(&sh.entries, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  cluster_sync();   // every CTA's barriers are ready

  auto row_of = [&](uint32_t it) { return (int64_t)(first + it * step); };
  auto stream = [&](uint32_t it) {
    Stream<T> x;
    x.set(static_cast<const T *>(a.logits) + row_of(it) * a.stride, a.vocab, rank, log2_size, buffers + it % kB * a.steps * 32);
    return x;
  };
  // The first warp brings rows in, the copy first, later in the same turn what
  // sticks out of it.  (A warp for that alone would leave the others 96
  // registers each, and four times the spills.)
  auto row_at = [&](uint32_t it) { return static_cast<const T *>(a.logits) + row_of(it) * a.stride; };
  {
    Picker<T, W, K> s(sh);
    s.rank = rank, s.size = size, s.limit = a.waits.limit;
    constexpr int kPer = (kMost<K> * W + 31) / 32;
    const uint32_t half = size * W / 2;
    const int log2_segments = log2_size + kLog2W;
    auto place = [&](uint32_t it) {
      if constexpr (is_far(K)) s.x.set(row_at(it), a.vocab);
      else s.x = stream(it);
      s.st0 = s.x.step_of(rank * W + warp, log2_segments) - s.x.begin / 32;
      s.st1 = s.x.step_of(rank * W + warp + 1, log2_segments) - s.x.begin / 32;
    };
    auto temperature_of = [&](int64_t row) { return a.s.temperatures ? a.s.temperatures[row] : a.s.temperature; };
    auto top_k_of = [&](int64_t row) { return a.s.top_ks ? a.s.top_ks[row] : a.s.top_k; };

    // A row's first part: its largest number (NaN is passed over).  Beside it,
    // for a greedy row, its first index; for top-k, the j-th largest of the
    // threads' maxima: j entries each in half of the cluster's warps are k.
    auto look = [&](uint32_t it) {
      place(it);
      const bool greedy = !(temperature_of(row_of(it)) > 0.0f);
      const int32_t top_k = top_k_of(row_of(it));
      if (!is_far(K)) {
        s.wait(&sh.full[it % kB], it / kB & 1);
        s.came = s.came && !a.waits.fails(it, rank * W + warp);
      }
      float m = -INFINITY;
      s.steps([&](int32_t, uint4 v) { m = Elem<T>::vec_max(v, m); });
      const float of_thread = m;
      m = warp_max_all(m);
      uint32_t beside = ordered(-INFINITY);
      if (greedy) {
        beside = 0xffffffffu;
        s.steps([&](int32_t st, uint4 w) {
          float v[kE];
          Elem<T>::unpack(w, v);
#pragma unroll
          for (int e = 0; e < kE; e++)
            if (v[e] == m) beside = min(beside, (uint32_t)s.x.index(st * 32 + lane, e));
        });
        beside = __reduce_min_sync(~0u, beside);
      } else if (searches(K) && top_k > 0 && top_k < a.vocab) {
        const uint32_t j = ((uint32_t)top_k + half - 1) / half;
        if (j <= 32) {
          uint32_t mine = ordered(of_thread);
          beside = ordered(m);
          for (uint32_t i = 1; i < j; i++) {   // without the largest so far, one lane of its
            if (lane == __ffs(__ballot_sync(~0u, mine == beside)) - 1) mine = 0;
            beside = __reduce_max_sync(~0u, mine);
          }
        }
      }
      s.post(((uint64_t)beside << 32) | __float_as_uint(m));
    };

    if (!is_far(K) && warp == 0) {
      for (uint32_t i = 0; i < kB && i < turns; i++) {
        const Stream<T> x = stream(i);
        x.bring_inner(row_at(i), &sh.full[i]);
        x.bring_edges(x.edge(row_at(i)), &sh.full[i]);
      }
      if (lane == 0) sh.begun = sh.whole = min((uint32_t)kB, turns);
    }
    look(0);
    uint32_t it = 0;
    for (; it < turns; it++) {
      // a row goes where the last one was
      const uint32_t next = it + kB - 1;
      float edge = 0.0f;
      bool bring = !is_far(K) && warp == 0 && it > 0 && next < turns;
      if (bring) {
        s.wait(&sh.empty[(it - 1) % kB], (it - 1) / kB & 1);
        bring = s.came;   // (if not, the CTA's next agreement ends it)
      }
      if (bring) {
        const Stream<T> x = stream(next);
        x.bring_inner(row_at(next), &sh.full[next % kB]);
        if (lane == 0) sh.begun = next + 1;
        edge = x.edge(row_at(next));
      }
      // the second part: what is kept of the row, and its mass by warps
      const int64_t row = row_of(it);
      if (it > 0) place(it);
      const float temperature = temperature_of(row);
      const int32_t top_k = top_k_of(row);
      const float top_p = a.s.top_ps ? a.s.top_ps[row] : a.s.top_p;
      const float min_p = a.s.min_ps ? a.s.min_ps[row] : a.s.min_p;
      const bool greedy = !(temperature > 0.0f), by_k = searches(K) && top_k > 0 && top_k < a.vocab, by_p = searches(K) && top_p < 1.0f;
      s.own = -1;
      const uint64_t *box = s.hear();
      uint32_t besides[kPer];
      float tops[kPer], m = -INFINITY;
#pragma unroll
      for (int i = 0; i < kPer; i++) {
        const bool have = i * 32 + lane < (int)(size * W);
        const uint64_t v = have ? box[i * 32 + lane] : 0;
        tops[i] = have ? __uint_as_float((uint32_t)v) : -INFINITY;
        besides[i] = have ? (uint32_t)(v >> 32) : 0;
        m = fmaxf(m, tops[i]);
      }
      m = warp_max_all(m);
      if (by_k || by_p) s.agree();
      if (!s.ok) break;

      Place end = {0x7fffffffu, 0};
      const uint32_t floor_w = min_p > 0.0f ? __float2uint_rn(fminf(min_p, 1.0f) * 2147483648.0f) : 0;
      auto kept = [&](float d, int32_t i) -> uint32_t {
        const uint32_t q = key_of(d), w = weight(d);   // (0 for NaN and -inf)
        return w >= floor_w && (q < end.key || (q == end.key && i < end.index)) ? w : 0;
      };
      const bool draw = m > -INFINITY && !greedy;
      if (m == -INFINITY) {   // nothing left to choose from
        if (s.came && rank == 0 && threadIdx.x == 0) a.tokens[row] = -1, a.logps[row] = -INFINITY;
      } else if (greedy) {
        uint32_t best = 0xffffffffu;
#pragma unroll
        for (int i = 0; i < kPer; i++)
          if (tops[i] == m) best = min(best, besides[i]);
        best = __reduce_min_sync(~0u, best);
        if (s.came && rank == 0 && threadIdx.x == 0) a.tokens[row] = best, a.logps[row] = 0.0f;
      } else {
        s.m = m;
        s.c = __fdiv_rn(1.44269504f, temperature);
        s.special = !(m < INFINITY && s.c < INFINITY);
        if constexpr (searches(K)) if (by_k || by_p) {
          float least = kFloor;
          if (by_k) {
            // a number that one warp of each two reaches: half of them
            uint32_t at;
            if (kPer == 1 || size * W <= 32) at = max(besides[0], __shfl_xor_sync(~0u, besides[0], half));
            else if (kPer == 2 || size * W <= 64) at = max(besides[0], besides[kPer > 1]);
            else at = min(max(besides[0], besides[kPer / 2]), max(besides[kPer > 1], besides[kPer - 1]));
            if (lane >= (int)half) at = ~0u;
            const float v = from_ordered(__reduce_min_sync(~0u, at));
            if (v > -INFINITY) least = fmaxf(kFloor, v == m ? 0.0f : (v - m) * s.c);   // (fmaxf passes NaN over)
          }
          end = s.kept_prefix(top_k, by_p, top_p, least);
          if (!s.ok) break;
        }
        uint64_t mine;
        if (!by_k && !by_p && floor_w == 0) {
          mine = 0;
          s.steps([&](int32_t, uint4 v) {
            float d[kE];
            s.octaves(v, d);
            uint64_t of_vec = 0;
#pragma unroll
            for (int e = 0; e < kE; e += 2) of_vec += (uint64_t)weight(d[e]) + weight(d[e + 1]);   // 0 from kFloor on, and for NaN
            mine += of_vec;
          });
          mine = warp_sum(mine);
        } else {
          mine = s.row_sum(fmaxf(kFloor, -__uint_as_float(end.key)), kept);
        }
        s.post(mine);
      }

      if (bring) {
        stream(next).bring_edges(edge, &sh.full[next % kB]);
        if (lane == 0) sh.whole = next + 1;
      }
      // the next row's first part, while the words of this one travel
      if (it + 1 < turns) look(it + 1);

      // the third part: the entry at which the running sum passes the target
      if (draw) {
        place(it);
        const float u = a.u[row];
        box = s.hear();
        uint64_t upto[kPer], z = 0;
        int owner = 0;
        uint64_t before = 0;
#pragma unroll
        for (int i = 0; i < kPer; i++) {
          upto[i] = z + warp_scan(i * 32 + lane < (int)(size * W) ? box[i * 32 + lane] : 0, lane);
          z = __shfl_sync(~0u, upto[i], 31);
        }
        const uint64_t target = share(u > 0.0f ? (u < 1.0f ? part_of(u) : 0xffffffffull) : 0, z);
#pragma unroll
        for (int i = kPer - 1; i >= 0; i--) {
          const uint32_t above = __ballot_sync(~0u, target < upto[i]);
          if (above) {
            owner = i * 32 + __ffs(above) - 1;
            const uint64_t v = __shfl_sync(~0u, upto[i], __ffs(above) - 1);
            before = v - box[owner];
          }
        }
        s.agree();
        if (!s.ok) break;
        if (owner / W == (int)rank) {
          // all of this CTA's warps take steps of that segment
          const int32_t first_step = s.x.step_of(owner, log2_segments) - s.x.begin / 32,
                        steps = s.x.step_of(owner + 1, log2_segments) - s.x.begin / 32 - first_step;
          auto weights = [&](int32_t st, float *d, uint32_t *w) {
            s.octaves(s.x.vec(first_step + st), d);
            uint64_t sum = 0;
#pragma unroll
            for (int e = 0; e < kE; e++) {
              w[e] = d[e] > kFloor ? kept(d[e], s.x.index((first_step + st) * 32 + lane, e)) : 0;
              sum += w[e];
            }
            return sum;
          };
          float d[kE];
          uint32_t w[kE];
          for (int32_t st = warp; st < steps; st += W) {
            const uint64_t sum = warp_sum(weights(st, d, w));
            if (lane == 0) sh.step_mass[st] = sum;
          }
          s.team();
          int32_t st = 0;
          for (int32_t at = 0;; at += 32) {   // (a segment has hardly more than 32 steps)
            const uint64_t of_step = at + lane < steps ? sh.step_mass[at + lane] : 0, upto_step = before + warp_scan(of_step, lane);
            const uint32_t past = __ballot_sync(~0u, target < upto_step);
            if (past || at + 32 >= steps) {
              const int l = max(0, __ffs(past) - 1);
              before = __shfl_sync(~0u, upto_step - of_step, l);
              st = at + l;
              break;
            }
            before = __shfl_sync(~0u, upto_step, 31);
          }
          if (st % W == warp) {
            const uint64_t of_vec = weights(st, d, w);
            uint64_t sum = before + warp_scan(of_vec, lane) - of_vec;
#pragma unroll
            for (int e = 0; e < kE; e++) {
              if (target >= sum && target < sum + w[e]) {
                a.tokens[row] = s.x.index((first_step + st) * 32 + lane, e);
                a.logps[row] = (d[e] - log2f((float)z * 4.6566128730773926e-10f)) * 0.69314718f;
              }
              sum += w[e];
            }
          }
        }
      } else {
        s.agree();
        if (!s.ok) break;
      }
      __syncwarp();
      if (!is_far(K) && lane == 0) bar_arrive(&sh.empty[it % kB]);
    }
    if (!s.ok) {
      // A wait gave up.  Which CTA has a row's token is not known here, so each
      // marks the rows that it is not done with; where another was done with one,
      // its token or logp may stand beside a mark.
      if (threadIdx.x == 0)
        for (uint32_t i = it; i < turns; i++) a.tokens[row_of(i)] = -1, a.logps[row_of(i)] = NAN;
      // copies in flight land before the CTA goes
      if (warp == 0) {
        __syncwarp();
        const uint32_t begun = sh.begun;
        if (sh.whole < begun) stream(begun - 1).bring_edges(-INFINITY, &sh.full[(begun - 1) % kB]);
        for (uint32_t i = begun > kB ? begun - kB : 0; i < begun; i++) bar_wait(&sh.full[i % kB], i / kB & 1);
      }
    }
    __syncwarp();
    cluster_sync();
    if (!s.ok) stay();
  }
}

constexpr int kDevices = 16;   // whose occupancy is kept (for a function, a number of CTAs and a buffer's size)

template <int W, Kind K>
constexpr int kMostSteps = is_far(K) ? 1 : (int)(((226 << 10) - sizeof(Picks<W, K>)) / (kBuffers<K> * 32 * 16));

static_assert(kMostSteps<8, kSearch> * 32 * 8 < 1 << 16 && kMostSteps<16, kSearch> * 32 * 8 < 1 << 16,
              "the entries of a CTA's slice are counted in 16 bits, their mass of 2^31 each in 48");

template <typename T, int W, Kind K>
int run_sample(SampleArgs a, int size, int log2, cudaStream_t stream) {
  static std::atomic<int> fits[kDevices][4][kMostSteps<W, K> + 1];   // clusters at once, by size and steps (0: not known)
  auto kernel = sample_kernel<T, W, K>;
  constexpr int kThreads = W * 32;
  const size_t shared = (size_t)a.steps * kBuffers<K> * 32 * 16 + sizeof(Picks<W, K>);
  int device = 0, most = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return note_cuda(e);
  if (device < kDevices) most = fits[device][log2][a.steps].load(std::memory_order_relaxed);
  if (most == 0) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSteps<W, K> * kBuffers<K> * 32 * 16 +
                             (int)sizeof(Picks<W, K>));
    if (e == cudaSuccess) e = launch_rows(kernel, a, 1, size, kThreads, shared, stream, &most);
    if (e != cudaSuccess) return note_cuda(e);
    if (most < 1) return SEQSUM_ECUDA;
    if (device < kDevices) fits[device][log2][a.steps].store(most, std::memory_order_relaxed);
  }
  e = launch_rows(kernel, a, a.rows < most ? a.rows : most, size, kThreads, shared, stream);
  return e == cudaSuccess ? SEQSUM_OK : note_cuda(e);
}

// CTAs a row: one, reading far, from half the SMs' number of rows on; else
// enough for two of them to share an SM (66 steps a CTA), more where the rows
// are few.  The tokens do not depend on it: all sums are of integers.
template <typename T>
int choose_sample(SampleArgs a, cudaStream_t stream) {
  constexpr int kE = Elem<T>::kPerVec;
  const int64_t vecs = ((int64_t)a.vocab + kE - 1) / kE + 1;   // whatever the alignment
  const int64_t steps = (vecs + 31) / 32;
  const int sms = multiprocessors();
  bool search = a.s.top_ks || a.s.top_ps || a.s.top_k > 0 || a.s.top_p < 1.0f;
  if (steps > 66 && steps <= kFarSteps && a.rows * 2 >= sms) {
    a.steps = 0;
    if (search) return run_sample<T, 16, kFarSearch>(a, 1, 0, stream);
    // One row an SM where two of each would not stay in L2 (96 of its 129 MB):
    // 512 x 131072 fp32 80 us, two an SM 96; 256 x 131072 bf16 26 and 24.
    return vecs * 16 * 2 * sms > 96 << 20 ? run_sample<T, 32, kFarPlain>(a, 1, 0, stream)
                                          : run_sample<T, 16, kFarPlain>(a, 1, 0, stream);
  }
  int size = 1, log2 = 0;
  while (size < kMaxCluster && (steps > (int64_t)size * 66 || (a.rows * size * 2 <= sms && steps > (int64_t)size * 8)))
    size *= 2, log2++;
  a.steps = (int32_t)((steps + size - 1) / size);
  // (three buffers where there is room for them)
  search |= a.steps > kMostSteps<16, kPlain>;
  if (a.steps > kMostSteps<16, kSearch>) {
    const cudaError_t e = launch_rows(sample_reread_kernel<T, 512>, a, a.rows, kMaxCluster, 512, 0, stream);
    return e == cudaSuccess ? SEQSUM_OK : note_cuda(e);
  }
  // (one CTA an SM from 66 steps on: then twice the warps)
  if (search) return a.steps > 66 ? run_sample<T, 16, kSearch>(a, size, log2, stream) : run_sample<T, 8, kSearch>(a, size, log2, stream);
  return a.steps > 66 ? run_sample<T, 16, kPlain>(a, size, log2, stream) : run_sample<T, 8, kPlain>(a, size, log2, stream);
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
  sq::SampleArgs a = {logits, rows, row_stride, (int32_t)vocab, u, *sampling, tokens, logps, 0, sq::row::waits()};
  if (dtype == SEQSUM_FP32) return sq::choose_sample<float>(a, stream);
  if (dtype == SEQSUM_FP16) return sq::choose_sample<__half>(a, stream);
  return sq::choose_sample<__nv_bfloat16>(a, stream);
}
