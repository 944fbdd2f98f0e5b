// Log probabilities of given tokens, entropy and the top alternatives of rows of
// logits, in one pass over them.
//
// With M the row's largest logit (one of them, where several are equal) and the sums
// over all others
//   R = sum e^(x - M),  W = sum (x - M) e^(x - M):
//   lse = M + ln(1 + R),  logprob = (x[token] - M) - ln(1 + R),
//   entropy = ln(1 + R) - W / (1 + R).
// Leaving the largest term, 1, out of R and W keeps the digits of a likely token's
// log probability, -ln(1 + R) with R far below 1.  Entropy is a sum of two terms of
// one sign.  R and W are fp32; a running maximum a warp rescales them.
//
// Alternatives: a thread keeps, for each of its runs of 16-byte words, the best word
// by (largest logit, lower place).  The n best words of all runs name the n runs
// that hold the n best logits (each of those n words holds a logit that beats all
// of another run's), and only these runs are read again.
//
// Bound: HBM where there are many rows; a few rows are split over a cluster of CTAs
// and are bound by latency.
#include <cuda_bf16.h>

#include "csa2_device.cuh"
#include "csa2_internal.h"

namespace csa2 {
namespace {

constexpr int kLpThreads = 256, kLpWarps = kLpThreads / 32;
constexpr int kBatch = 4;     // 16-byte words a thread loads at a time
constexpr int kMaxRuns = 8;   // runs of a thread
constexpr int kMaxList = 1024;  // candidates that are sorted from a list; more are merged one by one
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kFar = -200.f;  // e^x is 0 in fp32 from -104 on

struct LogprobParams {
  const void* logits;
  long long ld;
  int V;
  const int* token;
  float* logprob;
  float* entropy;
  float* lse;
  int* top_id;
  float* top_logprob;
  long long ld_top;
  int n;
  uint32_t* err;
};

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// e^x for x <= 0 (relative error about 2^-22 and |x| 2^-24)
__device__ __forceinline__ float exp_neg(float x) { return exp2_fast(x * kLog2e); }

// Sums over some logits: the largest of them, m (-inf: none), and R, W over the others.
struct Sums {
  float m, r, w;
};
__device__ __forceinline__ Sums merge(Sums a, Sums b) {
  if (b.m > a.m) {
    const Sums t = a;
    a = b;
    b = t;
  }
  if (b.m == -INFINITY) return a;
  const float d = fmaxf(b.m - a.m, kFar), f = exp_neg(d), s = 1.f + b.r;
  a.r += s * f;
  a.w += (b.w + s * d) * f;
  return a;
}

// Order of (value, lower place first) as a 64-bit key; 0: nothing.
__device__ __forceinline__ unsigned long long top_key(float x, uint32_t place) {
  return (static_cast<unsigned long long>(ord_key(x + 0.f)) << 32) | (0xFFFFFFFFu - place);  // -0 is 0
}
__device__ __forceinline__ float key_value(unsigned long long k) { return ord_to_float(static_cast<uint32_t>(k >> 32)); }
__device__ __forceinline__ uint32_t key_place(unsigned long long k) { return 0xFFFFFFFFu - static_cast<uint32_t>(k); }

// One step of a bitonic network over the warp's lanes: the pair (lane, lane ^ d).
__device__ __forceinline__ unsigned long long bitonic_step(unsigned long long k, int d, bool larger) {
  const unsigned long long o = __shfl_xor_sync(0xffffffffu, k, d);
  return (k > o) == larger ? k : o;
}
// Sorts the lanes' keys ascending.
__device__ __forceinline__ unsigned long long sort_up(unsigned long long k) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int s = 2; s <= 32; s <<= 1)
#pragma unroll
    for (int d = s >> 1; d > 0; d >>= 1) k = bitonic_step(k, d, ((lane & s) == 0) == ((lane & d) != 0));
  return k;
}
// The 32 best of a list (descending over the lanes) and of keys that ascend over
// the lanes, descending.
__device__ __forceinline__ unsigned long long merge_best(unsigned long long list, unsigned long long up) {
  const int lane = threadIdx.x & 31;
  unsigned long long k = list > up ? list : up;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) k = bitonic_step(k, d, (lane & d) == 0);
  return k;
}
// Adds the lanes' keys to the warp's list, unless none of them is among its n best.
__device__ __forceinline__ void add_keys(unsigned long long& list, unsigned long long k, int n) {
  const unsigned long long least = __shfl_sync(0xffffffffu, list, n - 1);
  if (__any_sync(0xffffffffu, k > least)) list = merge_best(list, sort_up(k));
}
// The best of the warps' lists, in warp 0.  s: [kLpWarps][32].
__device__ __forceinline__ unsigned long long join_lists(unsigned long long list, unsigned long long (*s)[32]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int h = kLpWarps / 2; h > 0; h >>= 1) {
    if (warp >= h && warp < 2 * h) s[warp][lane] = list;
    __syncthreads();
    if (warp < h) list = merge_best(list, s[warp + h][31 - lane]);
  }
  return list;
}

__device__ __forceinline__ unsigned long long ld_cluster_u64(uint32_t addr) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr));
  return v;
}

// A row's logits as 16-byte aligned words; the first and the last may be part of the row.
template <bool F32>
struct Row {
  static constexpr int kSize = F32 ? 4 : 2, kEl = 16 / kSize;
  const uint8_t* words;  // the word that holds the row's first logit
  int lead, V, n;        // logits of the first word before the row; the row's logits and words
  __device__ __forceinline__ Row(const void* logits, long long at, int v) {
    const uint8_t* p = static_cast<const uint8_t*>(logits) + at * kSize;
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u;
    words = p - off;
    lead = off / kSize;
    V = v;
    n = static_cast<int>((static_cast<long long>(v) + lead + kEl - 1) / kEl);
  }
  // Logits of word i (-inf where there is none).
  __device__ __forceinline__ void load(int i, float (&x)[kEl]) const {
    if (i < n && (i > 0 || lead == 0) && static_cast<long long>(i + 1) * kEl - lead <= V) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(words) + i);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (F32) {
          x[j] = __uint_as_float(w[j]);
        } else {
          x[2 * j] = __uint_as_float(w[j] << 16);
          x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < kEl; ++j) {
        const long long e = static_cast<long long>(i) * kEl + j - lead;
        x[j] = -INFINITY;
        if (i < n && e >= 0 && e < V) x[j] = at(static_cast<int>(e));
      }
    }
  }
  __device__ __forceinline__ float at(int e) const {
    const uint8_t* p = words + (static_cast<long long>(lead) + e) * kSize;
    return F32 ? __ldg(reinterpret_cast<const float*>(p))
               : __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(p))) << 16);
  }
};

// A cluster of gridDim.x / rows CTAs takes a row, each a run of its words.
template <bool F32, bool TOP>
__global__ void __launch_bounds__(kLpThreads) logprobs_kernel(const __grid_constant__ LogprobParams p, int splits) {
  constexpr int kEl = Row<F32>::kEl;
  __shared__ Sums s_sums[kLpWarps];
  __shared__ Sums s_part;
  __shared__ unsigned long long s_keys[TOP ? kLpThreads * kMaxRuns : 1];
  __shared__ unsigned long long s_cand[TOP ? kMaxList : 1];
  __shared__ unsigned long long s_lists[TOP ? kLpWarps : 1][32];
  __shared__ unsigned long long s_best[32];
  __shared__ int s_count;
  pdl_wait();
  pdl_trigger();
  const long long t = blockIdx.x / splits;
  const int rank = blockIdx.x % splits;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Row<F32> row(p.logits, t * p.ld, p.V);
  const int share = (row.n + splits - 1) / splits;
  const int first = min(row.n, rank * share), words = min(row.n, first + share) - first;
  const int batches = (words + kLpThreads * kBatch - 1) / (kLpThreads * kBatch);  // of this CTA's threads
  const int run_batches = max(1, (batches + kMaxRuns - 1) / kMaxRuns);
  int token = -1;
  float given = -INFINITY;
  if (rank == 0 && tid == 0 && p.token) {
    token = __ldg(p.token + t);
    if (token >= p.V || token < -1) {
      set_error(p.err, kErrBounds);
      token = -1;
    }
    if (token >= 0) given = row.at(token);
  }

  // ---- one pass
  float m = -INFINITY;  // the warp's largest logit so far
  float r = 0.f, w = 0.f;
  float run_max = -INFINITY;
  uint32_t run_word = 0;
  int run = 0, left = run_batches;
  for (int b = 0; b < batches; ++b) {
    float x[kBatch][kEl];
    float best = -INFINITY;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = (b * kBatch + u) * kLpThreads + tid;
      if (i < words) {
        row.load(first + i, x[u]);
      } else {
#pragma unroll
        for (int j = 0; j < kEl; ++j) x[u][j] = -INFINITY;
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      float g = x[u][0];
#pragma unroll
      for (int j = 1; j < kEl; ++j) g = fmaxf(g, x[u][j]);  // drops a NaN
      if (g == INFINITY) {
        g = -INFINITY;
#pragma unroll
        for (int j = 0; j < kEl; ++j) {
          if (x[u][j] == INFINITY) x[u][j] = -INFINITY;
          g = fmaxf(g, x[u][j]);
        }
      }
      if (TOP && g > run_max) {
        run_max = g;
        run_word = first + (b * kBatch + u) * kLpThreads + tid;
      }
      best = fmaxf(best, g);
    }
    if (__any_sync(0xffffffffu, best > m)) {
      float top = best;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      // the old maximum joins the sums (lane 0), one of the new leaves them
      const float d = fmaxf(m - top, kFar), f = exp_neg(d);
      if (lane == 0 && m > -INFINITY) r += 1.f;
      w = (w + r * d) * f;
      r *= f;
      m = top;
      if (lane == __ffs(__ballot_sync(0xffffffffu, best == top)) - 1) {
        bool out = false;
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
#pragma unroll
          for (int j = 0; j < kEl; ++j)
            if (!out && x[u][j] == top) {
              x[u][j] = -INFINITY;
              out = true;
            }
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
#pragma unroll
      for (int j = 0; j < kEl; ++j) {
        const float d = fmaxf(x[u][j] - m, kFar);  // masked logits and NaN: e^d is 0
        const float e = exp_neg(d);
        r += e;
        w = fmaf(e, d, w);
      }
    if (TOP && (--left == 0 || b + 1 == batches)) {
      s_keys[run++ * kLpThreads + tid] = run_max > -INFINITY ? top_key(run_max, run_word) : 0ull;
      run_max = -INFINITY;
      left = run_batches;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    r += __shfl_xor_sync(0xffffffffu, r, o);
    w += __shfl_xor_sync(0xffffffffu, w, o);
  }
  if (lane == 0) s_sums[warp] = Sums{m, r, w};
  if (tid == 0) s_count = 0;
  __syncthreads();
  Sums all = s_sums[0];
#pragma unroll
  for (int i = 1; i < kLpWarps; ++i) all = merge(all, s_sums[i]);

  // ---- this CTA's best logits, descending over warp 0's lanes
  unsigned long long list = 0;
  if (TOP) {
    for (int i = warp * 32; i < run * kLpThreads; i += kLpThreads) add_keys(list, s_keys[i + lane], p.n);
    list = join_lists(list, s_lists);
    if (warp == 0) s_best[lane] = lane < p.n ? list : 0ull;
    __syncthreads();
    const unsigned long long least = s_best[p.n - 1];
    const int run_words = run_batches * kBatch;
    // logits of the best runs that are no worse than the n-th best word
    auto candidates = [&](auto&& take) {
      for (int i = warp * 32; i < p.n * run_words; i += kLpThreads) {
        const int at = i + lane;
        float x[kEl];
        uint32_t word = 0;
        bool in = false;
        if (at < p.n * run_words && s_best[at / run_words]) {
          const uint32_t local = key_place(s_best[at / run_words]) - first;  // of the run's best word
          const int j = static_cast<int>(local / kLpThreads) / run_words * run_words + at % run_words;
          const int k = j * kLpThreads + static_cast<int>(local % kLpThreads);
          in = k < words;
          word = first + k;
        }
        if (in) {
          row.load(static_cast<int>(word), x);
        } else {
#pragma unroll
          for (int j = 0; j < kEl; ++j) x[j] = -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < kEl; ++j) {
          const bool is = selectable(x[j]) && top_key(x[j], word) >= least;
          take(is ? top_key(x[j], word * kEl + j - row.lead) : 0ull);
        }
      }
    };
    candidates([&](unsigned long long k) {
      if (k) {
        const int at = atomicAdd(&s_count, 1);
        if (at < kMaxList) s_cand[at] = k;  // any order: the keys differ and are sorted
      }
    });
    __syncthreads();
    const int count = s_count;
    list = 0;
    if (count <= kMaxList) {
      for (int i = warp * 32; i < count; i += kLpThreads) add_keys(list, i + lane < count ? s_cand[i + lane] : 0ull, p.n);
    } else {
      candidates([&](unsigned long long k) { add_keys(list, k, p.n); });
    }
    list = join_lists(list, s_lists);
  }

  // ---- the cluster's CTAs
  if (splits > 1) {
    if (tid == 0) s_part = all;
    if (TOP && warp == 0) s_best[lane] = list;
    cluster_sync();
    if (rank == 0) {
      for (int i = 1; i < splits; ++i) {
        const uint32_t at = map_rank(smem_u32(&s_part), static_cast<uint32_t>(i));
        all = merge(all, Sums{ld_cluster_f32(at), ld_cluster_f32(at + 4), ld_cluster_f32(at + 8)});
      }
      if (TOP) {
        list = 0;
        for (int i = warp; i < splits; i += kLpWarps) {
          const unsigned long long k = ld_cluster_u64(map_rank(smem_u32(&s_best[31 - lane]), static_cast<uint32_t>(i)));
          list = merge_best(list, k);
        }
        list = join_lists(list, s_lists);
      }
    }
  }
  if (rank == 0) {
    const float log_total = all.m > -INFINITY ? log1pf(all.r) : 0.f;
    if (tid == 0) {
      if (p.lse) p.lse[t] = all.m + log_total;
      if (p.entropy) p.entropy[t] = all.m > -INFINITY ? log_total - all.w / (1.f + all.r) : 0.f;
      if (p.logprob) p.logprob[t] = token < 0 ? 0.f : (selectable(given) ? (given - all.m) - log_total : -INFINITY);
    }
    if (TOP && warp == 0 && lane < p.n) {
      if (p.top_id) p.top_id[t * p.ld_top + lane] = list ? static_cast<int>(key_place(list)) : -1;
      if (p.top_logprob) p.top_logprob[t * p.ld_top + lane] = list ? (key_value(list) - all.m) - log_total : -INFINITY;
    }
  }
  if (splits > 1) cluster_sync();  // no CTA leaves while its part may still be read
}

template <bool F32, bool TOP>
cudaError_t launch(const LogprobParams& p, int T, const DeviceCtx& ctx, cudaStream_t st) {
  // Rows that leave SMs idle are split, down to 4,096 logits a CTA.
  int splits = 1;
  while (splits < 8 && static_cast<long long>(T) * splits * 2 <= 4LL * ctx.num_sms && p.V / (splits * 2) >= 4096) splits *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(T) * splits);
  cfg.blockDim = dim3(kLpThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<F32, TOP>, p, splits);
}

}  // namespace

cudaError_t launch_logprobs(const csa2_logprobs_args& a, const DeviceCtx& ctx, cudaStream_t st) {
  const LogprobParams p{a.logits, a.ld_logits, a.V, a.token, a.logprob, a.entropy, a.lse, a.top_id, a.top_logprob,
                        a.ld_top, a.n_top, ctx.err};
  if (a.logits_f32) return a.n_top ? launch<true, true>(p, a.T, ctx, st) : launch<true, false>(p, a.T, ctx, st);
  return a.n_top ? launch<false, true>(p, a.T, ctx, st) : launch<false, false>(p, a.T, ctx, st);
}

}  // namespace csa2
