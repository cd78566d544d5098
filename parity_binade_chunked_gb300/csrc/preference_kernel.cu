// The loss over pairs of sequences from their tokens' log-probabilities, and
// its gradient (seqsum_preference_loss, _backward).
//
//   a sequence's score = sum of w (logp - ref), or that over the sum of w
//   D = the chosen one's score - the rejected one's, z = beta D - margin
//   sigmoid: (1 - e) softplus(-z) + e softplus(z);  hinge: max(0, 1 - z);
//   ipo: (D - 1 / (2 beta))^2;  the loss is their mean
//
// A sequence is cut into chunks of 1024 tokens, counted from its first: its parts,
// or 32 parts of several chunks where there are more.  A part has 128 sums, of every
// 128th token, joined by one tree, the parts by another, whatever the number of
// warps and CTAs that work on it.
#include "policy_terms.cuh"

#include "row_slice.cuh"

namespace sq {
namespace loss {
namespace {

constexpr int kSums = 128;                        // of a part
constexpr int kBatch = 8;                         // tokens a thread under way
constexpr int64_t kChunk = 1024;
constexpr int kParts = 32;                        // at most: a warp's lanes

// A number in two floats, the first the nearest to it.
struct Pair {
  float hi, lo;
};

struct PairsArgs {
  const float *logps, *ref_logps, *weights;
  int64_t n;
  const int64_t *offsets;
  int64_t pairs;
  Pair beta, margin, half_by_beta;   // the last 1 / (2 beta)
  float smoothing, kept, share;      // kept: 1 - smoothing, rounded by itself; share: 1 / pairs
  int32_t kind;
  bool average;
  float *scores, *slopes, *losses;
  float *dlogps;
  const float *dloss;
  float *loss;
};

__device__ __forceinline__ void add_product(Sum &s, float w, float x) {
  const float p = w * x;
  s.add(p);
  s.lo += __fmaf_rn(w, x, -p);
}

__device__ __forceinline__ void add_product(TwoSums &s, Two w, Two x, Two minus_w) {
  const Two p = mul(w, x);
  s.add(p);
  s.lo = sub(s.lo, fma(minus_w, x, p));
}

__device__ __forceinline__ Pair nearest(const Sum &s) {
  const float hi = s.hi + s.lo;
  if (!(fabsf(s.hi) < INFINITY)) return {s.hi, 0.0f};
  return {hi, s.lo - (hi - s.hi)};
}
__device__ __forceinline__ Pair minus(const Pair &a, const Pair &b) {
  Sum s;
  s.hi = a.hi, s.lo = a.lo;
  s.add(-b.hi);
  s.lo -= b.lo;
  return nearest(s);
}
__device__ __forceinline__ Pair times(const Pair &a, const Pair &b) {
  Sum s;
  s.hi = a.hi * b.hi;
  s.lo = __fmaf_rn(a.hi, b.hi, -s.hi) + (a.hi * b.lo + a.lo * b.hi);
  return nearest(s);
}
// a / b, 0 where b is 0: the quotient of the nearest floats, and that of what it leaves
__device__ __forceinline__ Pair over(const Pair &a, const Pair &b) {
  if (b.hi == 0.0f) return {0.0f, 0.0f};
  Sum s;
  s.hi = __fdiv_rn(a.hi, b.hi);
  s.lo = __fdiv_rn(__fmaf_rn(-s.hi, b.hi, a.hi) + (a.lo - s.hi * b.lo), b.hi);
  return nearest(s);
}

// A pair's loss and its derivative by D, the difference of the scores.  (In pairs
// of floats: a chain of fp64 operations takes longer than all else that a pair
// waits for.)
__device__ __forceinline__ float pair_loss(const PairsArgs &a, const Pair &between, float &slope) {
  if (a.kind == SEQSUM_IPO) {
    const float h = minus(between, a.half_by_beta).hi;
    slope = 2.0f * h;
    return h * h;
  }
  const Pair z = minus(times(a.beta, between), a.margin);
  if (a.kind == SEQSUM_HINGE) {
    const bool inside = z.hi < 1.0f || (z.hi == 1.0f && z.lo < 0.0f), beyond = !inside && z.hi >= 1.0f;
    slope = inside ? -a.beta.hi : beyond ? 0.0f : z.hi;
    return inside ? (1.0f - z.hi) - z.lo : beyond ? 0.0f : z.hi;
  }
  // (the derivative from both sigmoids: smoothing - sigma(-z) would lose the smaller part)
  const float e = expf(-fabsf(z.hi)), soft = log1pf(e), near = __fdiv_rn(1.0f, 1.0f + e), far = __fdiv_rn(e, 1.0f + e);
  slope = a.beta.hi * (a.smoothing * (z.hi >= 0.0f ? near : far) - a.kept * (z.hi >= 0.0f ? far : near));
  float l = a.kept * ((z.hi < 0.0f ? -z.hi : 0.0f) + soft);
  if (a.smoothing != 0.0f) l += a.smoothing * ((z.hi > 0.0f ? z.hi : 0.0f) + soft);
  return l;
}

// Sequence [from, to); none where the pair's offsets are bad.
struct Sequence {
  int64_t from, to, chunks;
  __device__ __forceinline__ void set(int64_t f, int64_t t) {
    from = f, to = t;
    chunks = (t - f + kChunk - 1) / kChunk;
  }
  __device__ __forceinline__ int parts() const { return chunks < kParts ? (int)chunks : kParts; }
  __device__ __forceinline__ int64_t begin(int k) const { return from + (chunks <= kParts ? k : chunks * k / kParts) * kChunk; }
  __device__ __forceinline__ int64_t end(int k) const { return min(begin(k + 1), to); }
};
__device__ __forceinline__ bool load_pair(const PairsArgs &a, int64_t p, Sequence &chosen, Sequence &rejected) {
  const int64_t begin = a.offsets[2 * p], middle = a.offsets[2 * p + 1], last = a.offsets[2 * p + 2];
  const bool good = begin >= 0 && begin <= middle && middle <= last && last <= a.n;
  chosen.set(begin, good ? middle : begin);
  rejected.set(good ? middle : begin, good ? last : begin);
  return good;
}

// The sums of tokens [begin, end) by L threads, `me` of them: sums me, me + L, ... of kSums.
template <int L>
__device__ __forceinline__ void sum_tokens(const PairsArgs &a, int64_t begin, int64_t end, int me, Sum *s, Sum *t) {
  constexpr int kMine = kSums / L;
  static_assert(kBatch % kMine == 0, "a batch is a number of tokens for each sum");
  const int64_t from = begin + me;
  const float *pw = a.weights + from, *px = a.logps + from, *py = a.ref_logps + from;
  const bool weights = a.weights, ref = a.ref_logps;
  constexpr int kTwo = kMine > 1 ? kMine / 2 : 1;
  TwoSums s2[kTwo], t2[kTwo];
  for (int64_t left = end - from; left > 0; left -= kBatch * L, pw += kBatch * L, px += kBatch * L, py += kBatch * L) {
    float w[kBatch], x[kBatch], y[kBatch];
    if (left > (kBatch - 1) * L) {
#pragma unroll
      for (int j = 0; j < kBatch; j++) {
        w[j] = weights ? pw[L * j] : 1.0f;
        x[j] = px[L * j];
        y[j] = ref ? py[L * j] : 0.0f;
      }
    } else {
      const int n = (int)left;
#pragma unroll
      for (int j = 0; j < kBatch; j++) {
        w[j] = L * j < n ? (weights ? pw[L * j] : 1.0f) : 0.0f;
        x[j] = L * j < n ? px[L * j] : 0.0f;
        y[j] = ref && L * j < n ? py[L * j] : 0.0f;
      }
    }
    if constexpr (kMine == 1) {
#pragma unroll
      for (int j = 0; j < kBatch; j++) {
        if (w[j] != 0.0f) {
          add_product(s[0], w[j], x[j]);
          if (ref) add_product(s[0], -w[j], y[j]);
          if (a.average) t[0].add(w[j]);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < kBatch; j += 2) {
        const bool one = w[j] != 0.0f, next = w[j + 1] != 0.0f;
        const Two ww = two(w[j], w[j + 1]), minus = two(-w[j], -w[j + 1]);
        add_product(s2[j / 2 % kTwo], ww, two(one ? x[j] : 0.0f, next ? x[j + 1] : 0.0f), minus);
        if (ref) add_product(s2[j / 2 % kTwo], minus, two(one ? y[j] : 0.0f, next ? y[j + 1] : 0.0f), ww);
        if (a.average) t2[j / 2 % kTwo].add(ww);
      }
    }
  }
  if constexpr (kMine > 1) {
#pragma unroll
    for (int k = 0; k < kTwo; k++) s2[k].get(s[2 * k], s[2 * k + 1]), t2[k].get(t[2 * k], t[2 * k + 1]);
  }
}
template <int L>
__device__ __forceinline__ void write_tokens(const PairsArgs &a, int64_t begin, int64_t end, int me, float slope) {
  const int64_t from = begin + me;
  const float *pw = a.weights + from;
  float *to = a.dlogps + from;
  const bool weights = a.weights;
  for (int64_t left = end - from; left > 0; left -= kBatch * L, pw += kBatch * L, to += kBatch * L) {
    const int n = (int)min(left, (int64_t)(kBatch * L));
    float w[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; j++) w[j] = L * j < n && weights ? pw[L * j] : 1.0f;
#pragma unroll
    for (int j = 0; j < kBatch; j++)
      if (L * j < n) to[L * j] = w[j] != 0.0f ? w[j] * slope : 0.0f;
  }
}
// Tokens of no sequence: before the first pair's and after the last pair's, by `step` threads.
__device__ __forceinline__ void write_rest(const PairsArgs &a, bool first, bool last, int64_t mine, int64_t step) {
  if (first) {
    const int64_t to = min(a.offsets[0], a.n);
    for (int64_t i = mine; i < to; i += step) a.dlogps[i] = 0.0f;
  }
  if (last) {
    const int64_t from = max(a.offsets[2 * a.pairs], (int64_t)0);
    for (int64_t i = from + mine; i < a.n; i += step) a.dlogps[i] = 0.0f;
  }
}

// A part's 128 sums and its weights', and their tree, by a warp.
struct Part {
  uint64_t sum[kSums], total[kSums];
  __device__ __forceinline__ void put(const PairsArgs &a, int me, const Sum &s, const Sum &t) {
    sum[me] = row::pair(s.hi, s.lo);
    if (a.average) total[me] = row::pair(t.hi, t.lo);
  }
  __device__ __forceinline__ void join(const PairsArgs &a, Sum &s, Sum &t) const {
    const int lane = threadIdx.x & 31;
    row::split(sum[lane], s.hi, s.lo);
    if (a.average) row::split(total[lane], t.hi, t.lo);
#pragma unroll
    for (int j = 32; j < kSums; j += 32) {
      Sum u;
      row::split(sum[lane + j], u.hi, u.lo);
      s.add(u);
      if (a.average) {
        row::split(total[lane + j], u.hi, u.lo);
        t.add(u);
      }
    }
    s = warp_add(s);
    if (a.average) t = warp_add(t);
  }
};

// What a sequence's sums give.
struct Score {
  Pair value;
  float scale;   // of the slope by a token's
};
// By a warp, lane k with part k's sums.
__device__ __forceinline__ Score score_of(const PairsArgs &a, Sum sum, Sum total, bool good) {
  sum = warp_add(sum);
  Score r = {nearest(sum), a.share};
  if (a.average) {
    total = warp_add(total);
    const Pair weight = nearest(total);
    r.value = over(r.value, weight);
    r.scale = weight.hi != 0.0f ? __fdiv_rn(a.share, weight.hi) : 0.0f;
  }
  if (!good) r.value.hi = NAN;
  return r;
}

__device__ __forceinline__ float mean_of(const Sum &s, int64_t n) {
  return over(nearest(s), {(float)n, (float)(n - (int64_t)(float)n)}).hi;
}
// Whether all offsets are in order and in [0, n], by all threads of a CTA (the part of each).
__device__ __forceinline__ bool good_offsets(const PairsArgs &a, int threads) {
  bool good = true;
  for (int64_t i = threadIdx.x; i <= 2 * a.pairs; i += threads)
    good &= a.offsets[i] <= (i < 2 * a.pairs ? a.offsets[i + 1] : a.n) && (i > 0 || a.offsets[0] >= 0);
  return good;
}

// A cluster a pair, W warps of each CTA for each of the two sequences, four of
// them for a part at a time.  The sums, where they are asked for, and the
// gradient, whose slopes are the sums' or given.  kFew: a CTA a pair, and one
// cluster has them all: it also does what mean_kernel does for more.
template <bool kValue, bool kGrad, int W, bool kFew>
__global__ __launch_bounds__(2 * W * 32) void pairs_kernel(const PairsArgs a) {
  constexpr int kGroups = W / 4;
  __shared__ float losses[row::kMaxCluster];
  __shared__ Part shared[2][kGroups][kValue ? 2 : 1];     // two parts in turn
  __shared__ uint64_t box[2][2][kParts];                  // of each sequence: the parts' sums and their weights'
  __shared__ Score score[2];
  const uint32_t size = kFew ? 1 : row::cluster_size(), rank = kFew ? 0 : row::cluster_rank();
  if (kValue) row::cluster_begun();
  // (the kernel that comes after waits for the end of this one)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t p = blockIdx.x / size;
  const bool there = !kFew || p < a.pairs, all_good = !kFew || __syncthreads_and(good_offsets(a, 2 * W * 32));
  const int half = threadIdx.x / (W * 32), group = threadIdx.x / 128 % kGroups, me = threadIdx.x % 128, lane = threadIdx.x & 31;
  Sequence chosen = {0, 0, 0}, rejected = chosen;
  const bool good = !there || load_pair(a, p, chosen, rejected);
  const Sequence q = half ? rejected : chosen;
  const int first = (int)rank * kGroups + group, step = (int)size * kGroups, parts = q.parts();
  float slope = 0.0f;
  if constexpr (kValue) {
    row::cluster_wait_begun();
    int turn = 0;
    for (int k = first; k < parts; k += step) {
      Sum s, t;
      sum_tokens<kSums>(a, q.begin(k), q.end(k), me, &s, &t);
      Part &part = shared[half][group][turn];
      part.put(a, me, s, t);
      __syncwarp();
      asm volatile("bar.sync %0, 128;" ::"r"(1 + half * kGroups + group) : "memory");
      turn ^= 1;
      if (me < 32) {
        part.join(a, s, t);
        if (kFew) {
          if (lane == 0) box[half][0][k] = row::pair(s.hi, s.lo), box[half][1][k] = row::pair(t.hi, t.lo);
        } else if (lane < (int)size) {
          row::st_remote(row::remote(&box[half][0][k], lane), row::pair(s.hi, s.lo));
          if (a.average) row::st_remote(row::remote(&box[half][1][k], lane), row::pair(t.hi, t.lo));
        }
      }
    }
    __syncwarp();
    if (size > 1) row::cluster_sync();   // no CTA reads or writes another's memory after this
    else __syncthreads();
    if (group == 0 && me < 32) {
      Sum sum, total;
      if (lane < parts) {
        row::split(box[half][0][lane], sum.hi, sum.lo);
        if (a.average) row::split(box[half][1][lane], total.hi, total.lo);
      }
      const Score r = score_of(a, sum, total, good);
      if (lane == 0) score[half] = r;
    }
    __syncthreads();
    const float loss = pair_loss(a, minus(score[0].value, score[1].value), slope);
    slope = (half ? -slope : slope) * score[half].scale;
    if (there && rank == 0 && group == 0 && me == 0) {
      a.scores[2 * p + half] = score[half].value.hi, a.slopes[2 * p + half] = slope;
      if (half == 0) a.losses[p] = loss;
    }
    if (kFew) {
      if (threadIdx.x == 0) {
        const uint32_t to = row::remote(&losses[p], 0);
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(loss) : "memory");
      }
      __syncwarp();
      row::cluster_sync();   // no CTA writes another's memory after this
      if (p == 0 && threadIdx.x == 0) {
        Sum s;
        for (int i = 0; i < (int)a.pairs; i++) s.add(losses[i]);
        *a.loss = all_good ? mean_of(s, a.pairs) : NAN;
      }
    }
  }
  if constexpr (kGrad) {
    if (kFew && !all_good) {
      for (int64_t i = p * 64 * W + threadIdx.x; i < a.n; i += (int64_t)gridDim.x * 64 * W) a.dlogps[i] = NAN;
      return;
    }
    if (!there) return;
    if (!kValue) slope = a.slopes[2 * p + half] * *a.dloss;
    for (int k = first; k < parts; k += step) write_tokens<kSums>(a, q.begin(k), q.end(k), me, slope);
    write_rest(a, p == 0, p == a.pairs - 1, rank * 64 * W + threadIdx.x, (int64_t)size * 64 * W);
  }
}

// Many pairs: kPairs a CTA of kWarps warps, and the parts of a cluster's sequences
// go to all of its warps in turn, so that a long one keeps none of them waiting.
// Bound by the cluster that has the most tokens: 4096 pairs of sequences of very
// different lengths, 8.3 M tokens with weights, a reference and the gradient, 42 us,
// of equal lengths 33 (20 at the copy rate).
template <bool kValue, bool kGrad, int kPairs, int kCluster, int kWarps>
__global__ __launch_bounds__(kWarps * 32, 28 / kWarps) void many_pairs_kernel(const PairsArgs a) {
  constexpr int kHere = 2 * kPairs, kMost = kCluster * kHere;   // sequences of a CTA, of a cluster
  static_assert(kMost <= 32, "a lane each");
  __shared__ uint64_t box[kHere][2][kParts];             // the CTA's sequences' parts
  __shared__ Sequence sequences[kMost];
  __shared__ bool good[kMost / 2];
  __shared__ __align__(8) float slopes[kMost];
  const uint32_t rank = row::cluster_rank();
  if (kValue) row::cluster_begun();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t first = (int64_t)(blockIdx.x / kCluster) * kCluster * kPairs;
  if (threadIdx.x < kMost / 2) {
    const int64_t i = first + threadIdx.x;
    Sequence chosen = {0, 0, 0}, rejected = chosen;
    good[threadIdx.x] = i >= a.pairs || load_pair(a, i, chosen, rejected);
    sequences[2 * threadIdx.x] = chosen, sequences[2 * threadIdx.x + 1] = rejected;
    if (!kValue && i < a.pairs) {
      const float dloss = *a.dloss;
      slopes[2 * threadIdx.x] = a.slopes[2 * i] * dloss, slopes[2 * threadIdx.x + 1] = a.slopes[2 * i + 1] * dloss;
    }
  }
  __syncthreads();
  const int parts = lane < kMost ? sequences[lane].parts() : 0, up_to = (int)row::warp_scan((uint32_t)parts, lane),
            all_parts = __shfl_sync(~0u, up_to, 31);
  // f(sequence, part) for this warp's parts
  auto each_part = [&](auto f) {
    for (int i = (int)rank * kWarps + warp; i < all_parts; i += kCluster * kWarps) {
      const int w = __popc(__ballot_sync(~0u, up_to <= i));
      f(w, i - __shfl_sync(~0u, up_to - parts, w));
    }
  };
  if constexpr (kValue) {
    __syncwarp();
    row::cluster_wait_begun();
    each_part([&](int w, int k) {
      constexpr int kMine = kSums / 32;
      const Sequence q = sequences[w];
      Sum s[kMine], t[kMine];
      sum_tokens<32>(a, q.begin(k), q.end(k), lane, s, t);
#pragma unroll
      for (int j = 1; j < kMine; j++) s[0].add(s[j]), t[0].add(t[j]);
      s[0] = warp_add(s[0]);
      if (a.average) t[0] = warp_add(t[0]);
      if (lane == 0) {
        row::st_remote(row::remote(&box[w % kHere][0][k], w / kHere), row::pair(s[0].hi, s[0].lo));
        row::st_remote(row::remote(&box[w % kHere][1][k], w / kHere), row::pair(t[0].hi, t[0].lo));
      }
    });
    __syncwarp();
    row::cluster_sync();
    if (warp < kPairs) {
      const int of = (int)rank * kPairs + warp;   // this warp's pair
      const int64_t p = first + of;
      Score r[2];
#pragma unroll
      for (int h = 0; h < 2; h++) {
        Sum sum, total;
        if (lane < sequences[2 * of + h].parts())
          row::split(box[2 * warp + h][0][lane], sum.hi, sum.lo), row::split(box[2 * warp + h][1][lane], total.hi, total.lo);
        r[h] = score_of(a, sum, total, good[of]);
      }
      float slope;
      const float loss = pair_loss(a, minus(r[0].value, r[1].value), slope);
      const float chosen = slope * r[0].scale, rejected = -slope * r[1].scale;
      if (lane == 0 && p < a.pairs) {
        a.scores[2 * p] = r[0].value.hi, a.scores[2 * p + 1] = r[1].value.hi;
        a.slopes[2 * p] = chosen, a.slopes[2 * p + 1] = rejected;
        a.losses[p] = loss;
      }
      if (kGrad && lane < kCluster)
        row::st_remote(row::remote(reinterpret_cast<uint64_t *>(slopes) + of, lane), row::pair(chosen, rejected));
    }
    __syncwarp();
    if (kGrad) row::cluster_sync();   // no CTA writes another's memory after this
  }
  if constexpr (kGrad) {
    each_part([&](int w, int k) { write_tokens<32>(a, sequences[w].begin(k), sequences[w].end(k), lane, slopes[w]); });
    write_rest(a, blockIdx.x == 0, blockIdx.x == gridDim.x - 1, threadIdx.x, 32 * kWarps);
  }
}

// The mean of the pairs' losses.  Offsets out of order or range leave places of
// the gradient that no pair has written: then all of it becomes NaN, as the loss is.
constexpr int kThreads = 1024;
template <bool kValue, bool kGrad>
__global__ __launch_bounds__(kThreads) void mean_kernel(const PairsArgs a) {
  __shared__ uint64_t box[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  bool good = good_offsets(a, kThreads);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Sum s;
  if (kValue)
    for (int64_t i = threadIdx.x; i < a.pairs; i += kThreads) s.add(a.losses[i]);
  s = warp_add(s);
  if (lane == 0) box[warp] = row::pair(s.hi, s.lo);
  good = __syncthreads_and(good);
  if (kValue && warp == 0) {
    Sum t;
    row::split(box[lane], t.hi, t.lo);
    t = warp_add(t);
    if (lane == 0) *a.loss = good ? mean_of(t, a.pairs) : NAN;   // (0 / 0 is 0 here)
  }
  if (kGrad && (!good || a.pairs == 0))
    for (int64_t i = threadIdx.x; i < a.n; i += kThreads) a.dlogps[i] = good ? 0.0f : NAN;
}

template <bool kValue, bool kGrad, int kPairs, int kCluster, int kWarps>
cudaError_t launch_many(const PairsArgs &a, cudaStream_t stream) {
  constexpr int kOf = kPairs * kCluster;
  return launch_after(many_pairs_kernel<kValue, kGrad, kPairs, kCluster, kWarps>, a, (a.pairs + kOf - 1) / kOf * kCluster,
                      32 * kWarps, kCluster, false, stream);
}
template <bool kValue, bool kGrad>
int run_pairs(const PairsArgs &a, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  const int64_t chunks = a.pairs > 0 ? a.n / kChunk / a.pairs : 0;
  // A few pairs of one or two parts on the average: one cluster.  (One pair of 301 tokens: 4.3 us, 5.8 in two launches.)
  if (a.pairs > 0 && a.pairs <= row::kMaxCluster && chunks < 4) {
    int size = 1;
    while (size < a.pairs) size *= 2;
    e = launch_after(pairs_kernel<kValue, kGrad, 4, true>, a, size, 256, size, false, stream);
    return e == cudaSuccess ? SEQSUM_OK : note_cuda(e);
  }
  if (a.pairs > 0) {
    // From 32 pairs on, with a part or more a pair on the average: many_pairs_kernel.  (Gradient, a CTA a pair of pairs_kernel
    // and that kernel: sequences of 700 tokens on the average, 100 pairs 10.5 and 9.2 us, 608 13.9 and 11.5; of 4000, 100 pairs
    // 22 and 12, 300 30 and 17, 608 52 and 26; 300 pairs of 2 x 64 6.3 and 7.5; 50 of 2 x 20000 28 and 36.)  It takes
    //  - as many pairs a CTA as let all run at once (1000 pairs of 4000, one and four a CTA: 44 and 79), but one where they are
    //    long, which find their weights in L2 only if few are under way (4000 pairs of 4000: 127 and 150);
    //  - more warps a CTA for fewer pairs of several parts (4, 8 and 12, 150 pairs of 4000: 17.6, 16.4, 14.2; 300: 18.4, 17.2,
    //    19.9);
    //  - clusters of 8 CTAs with one pair each, of 4 with more (608 pairs of 4000, 8 and 4: 25 and 30; 2048 of 2 x 2048: 40 and
    //    33).
    // Else a CTA a pair, and as many CTAs a pair as it has every four parts, on the average, while there are fewer than would
    // fill the GPU, with four times the warps where each has several parts (2 pairs of 250000: 15 us, 21 with the fewer).
    const int64_t sms = multiprocessors();
    if (a.pairs > 4 * sms || (chunks > 0 && a.pairs >= 32 && (chunks < 16 || 2 * a.pairs > sms))) {
      e = chunks >= 4 && 2 * a.pairs <= 3 * sms  ? launch_many<kValue, kGrad, 1, 8, 12>(a, stream)
          : chunks >= 4 && a.pairs <= 3 * sms    ? launch_many<kValue, kGrad, 1, 8, 8>(a, stream)
          : chunks >= 6 || a.pairs <= 7 * sms    ? launch_many<kValue, kGrad, 1, 8, 4>(a, stream)
          : a.pairs <= 14 * sms                  ? launch_many<kValue, kGrad, 2, 4, 4>(a, stream)
                                                 : launch_many<kValue, kGrad, 4, 4, 4>(a, stream);
    } else {
      int size = 1;
      while (size < row::kMaxCluster && 4 * size <= chunks && a.pairs * size < 2 * sms) size *= 2;
      e = size == row::kMaxCluster && chunks >= 4 * size
              ? launch_after(pairs_kernel<kValue, kGrad, 16, false>, a, a.pairs * size, 1024, size, false, stream)
              : launch_after(pairs_kernel<kValue, kGrad, 4, false>, a, a.pairs * size, 256, size, false, stream);
    }
  }
  if (e == cudaSuccess) e = launch_after(mean_kernel<kValue, kGrad>, a, 1, kThreads, 1, a.pairs > 0, stream);
  return e == cudaSuccess ? SEQSUM_OK : note_cuda(e);
}

Pair pair_of(double x) {
  const float hi = (float)x;
  return {hi, (float)(x - (double)hi)};
}

template <typename T>
bool misplaced(const T *p) { return reinterpret_cast<uintptr_t>(p) % sizeof(T) != 0; }

bool bad_pairs(int64_t n, const int64_t *offsets, int64_t pairs) {
  return n < 0 || n > SEQSUM_MAX_TOKENS || pairs < 0 || pairs > SEQSUM_MAX_ROWS || !offsets || misplaced(offsets);
}

}  // namespace
}  // namespace loss
}  // namespace sq

extern "C" {

int seqsum_preference_loss(const float *logps, const float *ref_logps, const float *weights, int64_t n, const int64_t *offsets,
                           int64_t pairs, const seqsum_preference *s, float *dlogps, float *loss, float *scores, float *slopes,
                           float *losses, cudaStream_t stream) {
  using namespace sq::loss;
  if (bad_pairs(n, offsets, pairs) || !s || !loss || (n > 0 && !logps)) return SEQSUM_EINVAL;
  if (pairs > 0 && (!scores || !slopes || !losses)) return SEQSUM_EINVAL;
  if (s->kind != SEQSUM_SIGMOID && s->kind != SEQSUM_HINGE && s->kind != SEQSUM_IPO) return SEQSUM_EINVAL;
  if (!(s->beta >= 1e-30 && s->beta <= 1e30) || !isfinite((float)s->margin)) return SEQSUM_EINVAL;
  if (!(s->smoothing >= 0.0 && s->smoothing <= 1.0) || (s->smoothing != 0.0 && s->kind != SEQSUM_SIGMOID)) return SEQSUM_EINVAL;
  if (s->margin != 0.0 && s->kind == SEQSUM_IPO) return SEQSUM_EINVAL;
  for (const float *p : {logps, ref_logps, weights, (const float *)dlogps, (const float *)loss, (const float *)scores,
                         (const float *)slopes, (const float *)losses})
    if (misplaced(p)) return SEQSUM_EINVAL;
  const int64_t bytes = n * (int64_t)sizeof(float), each = pairs * (int64_t)sizeof(float);
  if (!apart({place(dlogps, bytes), place(loss, sizeof(float)), place(scores, 2 * each), place(slopes, 2 * each), place(losses, each)},
             {place(logps == dlogps ? nullptr : logps, bytes), place(ref_logps, bytes), place(weights, bytes),
              place(offsets, (2 * pairs + 1) * (int64_t)sizeof(int64_t))}))
    return SEQSUM_EINVAL;
  const PairsArgs a = {logps, ref_logps, weights, n, offsets, pairs, pair_of(s->beta), pair_of(s->margin),
                       pair_of(0.5 / s->beta), (float)s->smoothing, (float)(1.0 - s->smoothing),
                       pairs > 0 ? (float)(1.0 / (double)pairs) : 0.0f, s->kind,
                       s->average != 0, scores, slopes, losses, dlogps, nullptr, loss};
  return dlogps ? run_pairs<true, true>(a, stream) : run_pairs<true, false>(a, stream);
}

int seqsum_preference_backward(const float *weights, int64_t n, const int64_t *offsets, int64_t pairs, const float *slopes,
                               const float *dloss, float *dlogps, cudaStream_t stream) {
  using namespace sq::loss;
  if (bad_pairs(n, offsets, pairs) || (n > 0 && (!dloss || !dlogps)) || (pairs > 0 && !slopes)) return SEQSUM_EINVAL;
  if (misplaced(weights) || misplaced(slopes) || misplaced(dloss) || misplaced(dlogps)) return SEQSUM_EINVAL;
  if (!apart({place(dlogps, n * (int64_t)sizeof(float))},
             {place(weights, n * (int64_t)sizeof(float)), place(offsets, (2 * pairs + 1) * (int64_t)sizeof(int64_t)),
              place(slopes, 2 * pairs * (int64_t)sizeof(float)), place(dloss, sizeof(float))}))
    return SEQSUM_EINVAL;
  PairsArgs a = {};
  a.weights = weights, a.n = n, a.offsets = offsets, a.pairs = pairs, a.slopes = const_cast<float *>(slopes);
  a.dloss = dloss, a.dlogps = dlogps;
  return n > 0 ? run_pairs<false, true>(a, stream) : SEQSUM_OK;
}

}  // extern "C"
