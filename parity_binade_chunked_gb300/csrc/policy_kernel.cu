// The clipped policy loss with a KL term over tokens, from their
// log-probabilities, and its gradient (seqsum_policy_loss, _backward).
//
//   r = exp(logp - old),  s = A min(r, 1 + high)                   (A >= 0)
//                         s = A min(max(r, 1 - low), max_ratio)    (A < 0)
//   k = exp(ref - logp) - (ref - logp) - 1
//   loss = sum of w (-s + kl_coef k - entropy_coef H)
//
// The tokens are cut into chunks of four a thread, the chunks into groups; their
// sizes go by the number of tokens alone.  A thread adds its tokens in order, the
// threads of a warp, the warps and the groups are joined by trees: a sum's order
// does not depend on the GPU or on what else runs (a cluster that has fewer CTAs
// than there are groups takes them in turns).
#include "policy_terms.cuh"

#include <atomic>

#include "row_slice.cuh"

namespace sq {
namespace loss {
namespace {

constexpr int kThreads = 256, kMostThreads = 512;   // of a CTA; of one of a cluster for more tokens
constexpr int kMostGroups = 16;                    // of a cluster, a CTA each where the GPU has room for such clusters
constexpr int kCtas = 3;                               // of an SM
constexpr int kGroups = 152 * kCtas;              // at most: all at once on this GPU
constexpr int kSums = 6;                          // policy, kl, entropy, past, old kl, weight
static_assert(sizeof(float2) * kSums * kGroups <= SEQSUM_POLICY_SCRATCH, "the groups' sums have room");

struct TokensArgs {
  Policy policy;
  const float *logps, *entropies;
  const int64_t *tokens;
  int64_t vocab, n, chunks;
  int32_t groups;
  bool vectors;                     // all arrays are 16-byte aligned
  float *dlogps;
  const float *dloss;               // null: 1
  float *loss, *stats;
  float2 *scratch;                  // [kSums][kGroups]
};

// Four numbers from the i-th on, 0 past the end.
__device__ __forceinline__ float4 load4(const float *p, int64_t i, int64_t n, bool vectors) {
  if (vectors && i + 4 <= n) return *reinterpret_cast<const float4 *>(p + i);
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (i < n) v.x = p[i];
  if (i + 1 < n) v.y = p[i + 1];
  if (i + 2 < n) v.z = p[i + 2];
  if (i + 3 < n) v.w = p[i + 3];
  return v;
}
__device__ __forceinline__ float at(const float4 &v, int e) { return e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w; }

// What stands beside four tokens.
struct Beside {
  float4 w, old, advantage, ref;
};
__device__ __forceinline__ bool any(const float4 &w) { return w.x != 0.0f || w.y != 0.0f || w.z != 0.0f || w.w != 0.0f; }
__device__ __forceinline__ float4 load_weights(const TokensArgs &a, int64_t i) {
  float4 w = load4(a.policy.weights, i, a.n, a.vectors);
  if (a.tokens) {
    auto keep = [&](float &x, int e) {
      if (i + e < a.n && (a.tokens[i + e] < 0 || a.tokens[i + e] >= a.vocab)) x = 0.0f;
    };
    keep(w.x, 0), keep(w.y, 1), keep(w.z, 2), keep(w.w, 3);
  }
  return w;
}
// (what is beside unused tokens is not read; NaN is not 0)
__device__ __forceinline__ void load_rest(const TokensArgs &a, int64_t i, Beside &b) {
  if (!any(b.w)) return;
  b.old = load4(a.policy.old_logps, i, a.n, a.vectors);
  b.advantage = load4(a.policy.advantages, i, a.n, a.vectors);
  if (a.policy.ref_logps) b.ref = load4(a.policy.ref_logps, i, a.n, a.vectors);
}

// Four tokens, the i-th and on.  The first term, whose sum is small beside its
// parts, is added with what its roundings leave; the others, of one sign, are added
// in plain fp32 (which costs no more than the roundings that each has already).
template <bool kValue, bool kGrad>
__device__ __forceinline__ void four_tokens(const TokensArgs &a, int64_t i, const Beside &b, const float4 &lp, const float4 &h,
                                            float dloss, TwoSums &first, Sum *sums) {
  float d[4] = {};
  if (any(b.w)) {
    const Two zero = splat<Two>(0.0f);
    Two part[kSums] = {zero, zero, zero, zero, zero, zero};
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const Two w = two(at(b.w, e), at(b.w, e + 1));
      const Both used = test(w, [](float v) { return v != 0.0f; });
      auto of = [&](const float4 &v) { return pick(used, two(at(v, e), at(v, e + 1)), zero); };
      const Terms<Two> t = policy_terms(a.policy, of(lp), of(b.old), of(b.advantage), of(b.ref));
      if (kGrad) {
        Two g = mul(w, t.slope);
        if (!kValue) g = pick(used, mul(g, splat<Two>(dloss)), zero);   // (of an infinite one too)
        row::split(g.v, d[e], d[e + 1]);
      }
      if (kValue) {
        const Two x = mul(w, t.policy);
        first.add(x);
        first.lo = add(first.lo, add(fma(w, t.policy, sub(zero, x)), mul(w, t.policy_rest)));
        part[1] = add(part[1], mul(w, t.kl)), part[2] = add(part[2], mul(w, of(h)));
        part[3] = add(part[3], mul(w, t.past)), part[4] = add(part[4], mul(w, t.old_kl)), part[5] = add(part[5], w);
      }
    }
    if (kValue) {
#pragma unroll
      for (int k = 1; k < kSums; k++) {
        float x, y;
        row::split(part[k].v, x, y);
        sums[k].add(x + y);
      }
    }
  }
  if (kGrad) {
    if (a.vectors && i + 4 <= a.n) {
      *reinterpret_cast<float4 *>(a.dlogps + i) = make_float4(d[0], d[1], d[2], d[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; e++)
        if (i + e < a.n) a.dlogps[i + e] = d[e];
    }
  }
}

// What the sums give, lane 0 of warp k with the k-th of them; `table` has room for
// all.  (In floats: a chain of fp64 operations by one thread is the longest wait of
// a small call.)
__device__ __forceinline__ void write_loss(const TokensArgs &a, const Sum &s, uint64_t *table) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp < kSums && lane == 0) {
    table[warp] = row::pair(s.hi, s.lo);
    a.stats[warp] = s.nearest();
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    Sum loss;
    row::split(table[0], loss.hi, loss.lo);
    auto add = [&](float f, uint64_t of) {
      Sum x;
      row::split(of, x.hi, x.lo);
      const float p = f * x.hi;
      loss.add(p);
      loss.lo += __fmaf_rn(f, x.hi, -p) + f * x.lo;
    };
    if (a.policy.kl_coef != 0.0f) add(a.policy.kl_coef, table[1]);
    if (a.policy.entropy_coef != 0.0f) add(-a.policy.entropy_coef, table[2]);
    *a.loss = loss.nearest();
  }
}

// Many tokens are bound by latency: a chunk's numbers are asked for while the chunk
// before it is worked out, and the SMs are without a CTA for a fifth of the time (a
// capture of 4 M tokens, half unused: 27% of DRAM, 49% of the issue slots, warps wait
// for loads and, at the end, for the CTA's other warps).  4 M tokens with a reference
// and gradient 26 us (101 MB; 15 at the copy rate), 1 M 11, half of 4 M unused 20.
// (Two tokens an instruction; each by itself 29, 12.6 and 20.  Four CTAs an SM, which
// spill: 30, 13.4 and 20; two: 27, 11 and 20, but 10% more from a cold L2.)
// A group of chunks a CTA.  kCluster: the groups are one cluster's CTAs, whose
// first one ends the call; else finish_kernel does.
template <bool kValue, bool kGrad, bool kCluster, int kThr>
__global__ __launch_bounds__(kThr, kCluster ? 1 : kCtas) void tokens_kernel(const TokensArgs a) {
  constexpr int kWarps = kThr / 32;
  constexpr int64_t kChunk = kThr * 4;
  __shared__ uint64_t box[kSums][(kCluster ? kMostGroups : 1) * kWarps];
  __shared__ uint64_t total[kSums];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t size = kCluster ? row::cluster_size() : 1, rank = kCluster ? row::cluster_rank() : 0;
  if (kCluster) row::cluster_begun();
  // (finish_kernel may come onto an SM, and waits for the end of this one)
  if (kValue && !kCluster) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  auto place = [&](int64_t chunk) { return chunk * kChunk + threadIdx.x * 4; };
  uint32_t group = blockIdx.x;
  do {   // (one, but for a cluster of fewer CTAs than groups)
    const int64_t from = a.chunks * group / a.groups, to = a.chunks * (group + 1) / a.groups;
    Beside b = {};
    if (from < to) {
      b.w = load_weights(a, place(from));
      load_rest(a, place(from), b);
    }
    // (the kernel before writes nothing of what has been read so far)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float dloss = kGrad && a.dloss ? *a.dloss : 1.0f;
    TwoSums first;
    Sum sums[kSums];
    for (int64_t c = from; c < to; c++) {
      float4 lp = {}, h = {}, next = {};
      if (any(b.w)) {
        lp = load4(a.logps, place(c), a.n, a.vectors);
        if (kValue && a.entropies) h = load4(a.entropies, place(c), a.n, a.vectors);
      }
      if (c + 1 < to) next = load_weights(a, place(c + 1));   // here before the chunk that asks for them
      four_tokens<kValue, kGrad>(a, place(c), b, lp, h, dloss, first, sums);
      b.w = next;
      if (c + 1 < to) load_rest(a, place(c + 1), b);
    }
    if constexpr (kValue) {
      Sum other;
      first.get(sums[0], other);
      sums[0].add(other);
      __syncwarp();
      if (kCluster && group == blockIdx.x) row::cluster_wait_begun();
#pragma unroll
      for (int k = 0; k < kSums; k++) {
        const Sum s = warp_add(sums[k]);
        if (lane == 0) {
          if (kCluster) row::st_remote(row::remote(&box[k][group * kWarps + warp], 0), row::pair(s.hi, s.lo));
          else box[k][warp] = row::pair(s.hi, s.lo);
        }
      }
    }
    group += gridDim.x;
  } while (kCluster && group < (uint32_t)a.groups);
  if constexpr (kValue) {
    __syncwarp();
    if (kCluster && size > 1) row::cluster_sync();
    else __syncthreads();
    if (rank != 0) return;
    Sum s;
    if (warp < kSums) {
      const int n = (kCluster ? a.groups : 1) * kWarps;
#pragma unroll
      for (int k = 0; k < (kCluster ? kMostGroups : 1) * kWarps; k += 32) {
        Sum t;
        if (lane + k < n) row::split(box[warp][lane + k], t.hi, t.lo);
        s.add(t);
      }
      s = warp_add(s);
      if (!kCluster && lane == 0) a.scratch[warp * kGroups + blockIdx.x] = make_float2(s.hi, s.lo);
    }
    if (kCluster) write_loss(a, s, total);
  }
}

// The groups' sums, a warp each.
__global__ __launch_bounds__(kSums * 32) void finish_kernel(const TokensArgs a) {
  __shared__ uint64_t total[kSums];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Sum s;
  for (int i = lane; i < a.groups; i += 32 * 8) {
    float2 v[8];
#pragma unroll
    for (int k = 0; k < 8; k++) v[k] = i + 32 * k < a.groups ? a.scratch[warp * kGroups + i + 32 * k] : make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < 8; k++) {
      Sum t;
      t.hi = v[k].x, t.lo = v[k].y;
      s.add(t);
    }
  }
  write_loss(a, warp_add(s), total);
}

// The largest cluster of a kernel that the current device takes: 16 CTAs, or the portable eight (or fewer for a test).
template <void (*kernel)(const TokensArgs), int threads>
int widest() {
  constexpr int kDevices = 16;
  static std::atomic<int> known[kDevices];
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess || device >= kDevices) return min(row::kMaxCluster, row::most_ctas());
  int size = known[device].load(std::memory_order_relaxed);
  if (size == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kMostGroups);
    cfg.blockDim = dim3(threads);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kMostGroups;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    size = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                   cudaOccupancyMaxActiveClusters(&n, (const void *)kernel, &cfg) == cudaSuccess && n > 0
               ? kMostGroups
               : row::kMaxCluster;
    known[device].store(size, std::memory_order_relaxed);
  }
  return min(size, row::most_ctas());
}

bool aligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <bool kValue, bool kGrad>
int run_tokens(TokensArgs &a, bool after, cudaStream_t stream) {
  const Policy &p = a.policy;
  a.vectors = aligned(a.logps) && aligned(p.old_logps) && aligned(p.advantages) && aligned(p.weights) && aligned(p.ref_logps) &&
              aligned(a.entropies) && aligned(a.dlogps);
  const int threads = kValue && a.n > kClusterTokens / 4 && a.n <= kClusterTokens ? kMostThreads : kThreads;
  a.chunks = (a.n + threads * 4 - 1) / (threads * 4);
  cudaError_t e;
  // One cluster while that takes little longer than a second kernel's launch (1000 tokens 3.9 us, 16384 4.7, 65536 7; by
  // many CTAs and finish_kernel 65537 tokens 5.2 and 130000 5.8, but 3.5 us more of the host's time).
  if (kValue && a.n <= kClusterTokens) {
    const int most = threads == kThreads ? widest<tokens_kernel<kValue, kGrad, true, kThreads>, kThreads>()
                                         : widest<tokens_kernel<kValue, kGrad, true, kMostThreads>, kMostThreads>();
    a.groups = 1;
    while (a.groups < kMostGroups && a.groups < a.chunks) a.groups *= 2;
    int size = 1;
    while (2 * size <= most && size < a.groups) size *= 2;
    e = threads == kThreads ? launch_after(tokens_kernel<kValue, kGrad, true, kThreads>, a, size, kThreads, size, after, stream)
                            : launch_after(tokens_kernel<kValue, kGrad, true, kMostThreads>, a, size, kMostThreads, size, after, stream);
  } else {
    if (kValue && !a.scratch) return SEQSUM_EINVAL;
    const int64_t most = kValue ? kGroups : (int64_t)1 << 20;
    a.groups = (int32_t)(a.chunks < most ? a.chunks : most);
    if (a.groups == 0) return SEQSUM_OK;
    e = launch_after(tokens_kernel<kValue, kGrad, false, kThreads>, a, a.groups, kThreads, 1, after, stream);
    if (kValue && e == cudaSuccess) e = launch_after(finish_kernel, a, 1, kSums * 32, 1, true, stream);
  }
  return e == cudaSuccess ? SEQSUM_OK : note_cuda(e);
}

// what the nearest float leaves of x
float rest_of(double x) { return isfinite((float)x) ? (float)(x - (double)(float)x) : 0.0f; }
Bound bound_of(double ratio) { return {(float)log(ratio), rest_of(log(ratio))}; }

bool misplaced(const float *p) { return reinterpret_cast<uintptr_t>(p) % sizeof(float) != 0; }

}  // namespace

bool take_policy(const seqsum_policy *s, int64_t n, bool rows, Policy *to) {
  if (!s || n < 0 || n > SEQSUM_MAX_TOKENS) return false;
  if (!(s->clip_low >= 0.0 && s->clip_low <= 1.0) || !(s->clip_high >= 0.0) || !(s->max_ratio >= 1.0)) return false;
  if (!isfinite((float)s->kl_coef) || (rows && !isfinite((float)s->entropy_coef))) return false;
  if (rows && !(s->temperature >= 1e-30 && s->temperature <= 1e30)) return false;
  if (n > 0 && (!s->old_logps || !s->advantages || !s->weights)) return false;
  if (misplaced(s->old_logps) || misplaced(s->advantages) || misplaced(s->weights) || misplaced(s->ref_logps)) return false;
  // (a bound beyond fp32 is none)
  auto within = [](double x) { return isfinite((float)x) ? x : (double)INFINITY; };
  const double up = within(1.0 + s->clip_high), down = 1.0 - s->clip_low, top = within(s->max_ratio);
  *to = {s->old_logps, s->advantages, s->weights, s->ref_logps, (float)up, (float)down, (float)top, rest_of(up),
         rest_of(down), rest_of(top), bound_of(up), bound_of(down), bound_of(top),
         (float)s->kl_coef, rows ? (float)s->entropy_coef : 0.0f, rows ? (float)(1.0 / s->temperature) : 1.0f};
  return true;
}

int sum_policy(const Policy &policy, const float *logps, const float *entropies, const int64_t *tokens, int64_t vocab,
               int64_t n, float *loss, float *stats, void *scratch, bool after, cudaStream_t stream) {
  TokensArgs a = {policy, logps, entropies, tokens, vocab, n, 0, 0, false, nullptr, nullptr, loss, stats,
                  static_cast<float2 *>(scratch)};
  return run_tokens<true, false>(a, after, stream);
}

}  // namespace loss
}  // namespace sq

extern "C" {

int seqsum_policy_loss(const float *logps, int64_t n, const seqsum_policy *policy, float *dlogps, float *loss, float *stats,
                       void *scratch, cudaStream_t stream) {
  sq::loss::TokensArgs a = {};
  if (!sq::loss::take_policy(policy, n, false, &a.policy) || !loss || !stats || (n > 0 && !logps)) return SEQSUM_EINVAL;
  if (sq::loss::misplaced(logps) || sq::loss::misplaced(dlogps) || sq::loss::misplaced(loss) || sq::loss::misplaced(stats) ||
      reinterpret_cast<uintptr_t>(scratch) % sizeof(float2))
    return SEQSUM_EINVAL;
  const sq::loss::Policy &p = a.policy;
  const int64_t bytes = n * (int64_t)sizeof(float);
  using sq::loss::place;
  if (!sq::loss::apart({place(dlogps, bytes), place(loss, sizeof(float)), place(stats, 6 * sizeof(float)),
                        place(scratch, n > sq::loss::kClusterTokens ? SEQSUM_POLICY_SCRATCH : 0)},
                       {place(logps == dlogps ? nullptr : logps, bytes), place(p.old_logps, bytes), place(p.advantages, bytes),
                        place(p.weights, bytes), place(p.ref_logps, bytes)}))
    return SEQSUM_EINVAL;
  a.logps = logps, a.n = n, a.dlogps = dlogps, a.loss = loss, a.stats = stats, a.scratch = static_cast<float2 *>(scratch);
  return dlogps ? sq::loss::run_tokens<true, true>(a, false, stream) : sq::loss::run_tokens<true, false>(a, false, stream);
}

int seqsum_policy_loss_backward(const float *logps, int64_t n, const seqsum_policy *policy, const float *dloss,
                                float *dlogps, cudaStream_t stream) {
  sq::loss::TokensArgs a = {};
  if (!sq::loss::take_policy(policy, n, false, &a.policy) || (n > 0 && (!logps || !dlogps || !dloss))) return SEQSUM_EINVAL;
  if (sq::loss::misplaced(logps) || sq::loss::misplaced(dlogps) || sq::loss::misplaced(dloss)) return SEQSUM_EINVAL;
  const sq::loss::Policy &p = a.policy;
  const int64_t bytes = n * (int64_t)sizeof(float);
  using sq::loss::place;
  if (!sq::loss::apart({place(dlogps, bytes)}, {place(logps == dlogps ? nullptr : logps, bytes), place(dloss, sizeof(float)),
                                                place(p.old_logps, bytes), place(p.advantages, bytes), place(p.weights, bytes),
                                                place(p.ref_logps, bytes)}))
    return SEQSUM_EINVAL;
  a.logps = logps, a.n = n, a.dlogps = dlogps, a.dloss = dloss;
  return sq::loss::run_tokens<false, true>(a, false, stream);
}

}  // extern "C"
