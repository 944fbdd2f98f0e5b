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
// Alternatives: a thread keeps the largest logit of each of its runs of 16-byte words.
// No logit below the n-th largest of the threads' largest ones, tau, is among the n best,
// as n threads hold one that is not below it; so only the runs with a logit of at least
// tau are read again, and of those logits, few more than n, the n best by (value, lower
// token) are sorted out.  Where many runs tie with tau, all of the row is read again.
//
// Bound: HBM where there are many rows (2,048 x 131,072 bf16 with the best token: 86 us,
// 6.2 TB/s of a copy's 6.8; issue slots 82 % full), latency where there are few, which a
// cluster of CTAs a row splits (8 x 131,072 fp32: 3.6 us, 7.7 with 20 alternatives).
#include <cuda_bf16.h>

#include <atomic>

#include "csa2_device.cuh"
#include "csa2_internal.h"

namespace csa2 {
namespace {

constexpr int kLpWarps = 8, kLpThreads = kLpWarps * 32;
// 16-byte words of a thread at a time, and how many such batches its ring holds
template <bool F32>
constexpr int kBatch = F32 ? 4 : 2;
template <bool F32, bool DEEP>
constexpr int kStages = F32 && !DEEP ? 2 : 4;
template <bool F32, bool DEEP>
constexpr int kRingBytes = kStages<F32, DEEP> * kBatch<F32> * kLpThreads * 16;
// Runs of a thread, at most, and their batches, at least; fewer if there are fewer, but 8
// words, which are read again by more warps than 2 would be (8 rows of 131,072 fp32 logits
// with 20 alternatives: 8.3 us with runs of 16 words, 7.8 with 8; of 20,000 bf16: 6.6 us with
// 2, 6.3 with 8).
constexpr int kMaxRuns = 4, kRunBatches = 4, kRunWords = 8;
// Logits are summed as if none were below this: e^(x - M) of one further down is 0 next
// to any M above it, and x - M stays finite.  A row whose M is not above it is summed
// as it is.
constexpr float kLowest = -1.2676506e30f;  // -2^100, exact in bf16
// Of a row: candidates that are sorted from a list (more are merged as they are read),
// and runs that are read again (with more, all are).
template <int NW>
constexpr int kMaxList = NW == 1 ? 256 : 1024;
constexpr int kMaxTied = 128;
constexpr int kMaxSplits = 16;  // CTAs of a row
constexpr float kLargestFloat = 3.402823466e38f;
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

// The N first lanes' sums merged, in every lane.
template <int N>
__device__ __forceinline__ Sums merge_lanes(Sums a) {
#pragma unroll
  for (int o = 1; o < N; o <<= 1)
    a = merge(a, Sums{__shfl_down_sync(0xffffffffu, a.m, o), __shfl_down_sync(0xffffffffu, a.r, o),
                      __shfl_down_sync(0xffffffffu, a.w, o)});
  return Sums{__shfl_sync(0xffffffffu, a.m, 0), __shfl_sync(0xffffffffu, a.r, 0), __shfl_sync(0xffffffffu, a.w, 0)};
}

// The place of a lane's item, if it has one, at the end of a row's list of *count.  The
// items of a row's only warp come many at a time and take their places together; of a
// CTA's warps few lanes have one at a time.
template <int NW>
__device__ __forceinline__ int append(int* count, bool is) {
  if (NW > 1) return is ? atomicAdd(count, 1) : 0;
  const uint32_t mask = __ballot_sync(0xffffffffu, is);
  const int lane = threadIdx.x & 31, before = *count;
  __syncwarp();
  if (lane == 0) *count = before + __popc(mask);
  __syncwarp();
  return before + __popc(mask & ((1u << lane) - 1));
}
// Order of a value, and of (value, lower place first) as a 64-bit key; 0: nothing.
__device__ __forceinline__ uint32_t value_key(float x) { return ord_key(x + 0.f); }  // -0 is 0
__device__ __forceinline__ uint32_t run_key(float x) { return x > -INFINITY ? value_key(x) : 0u; }
__device__ __forceinline__ unsigned long long top_key(float x, uint32_t place) {
  return (static_cast<unsigned long long>(value_key(x)) << 32) | (0xFFFFFFFFu - place);
}
__device__ __forceinline__ float key_value(unsigned long long k) { return ord_to_float(static_cast<uint32_t>(k >> 32)); }
__device__ __forceinline__ uint32_t key_place(unsigned long long k) { return 0xFFFFFFFFu - static_cast<uint32_t>(k); }

// One step of a bitonic network over the warp's lanes: the pair (lane, lane ^ d).
// K: the 64-bit keys, or the upper halves alone.
template <class K>
__device__ __forceinline__ K bitonic_step(K k, int d, bool larger) {
  const K o = __shfl_xor_sync(0xffffffffu, k, d);
  return (k > o) == larger ? k : o;
}
// Sorts the lanes' keys ascending.
template <class K>
__device__ __forceinline__ K sort_up(K k) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int s = 2; s <= 32; s <<= 1)
#pragma unroll
    for (int d = s >> 1; d > 0; d >>= 1) k = bitonic_step(k, d, ((lane & s) == 0) == ((lane & d) != 0));
  return k;
}
// The 32 best of a list (descending over the lanes) and of keys that ascend over
// the lanes, descending.
template <class K>
__device__ __forceinline__ K merge_best(K list, K up) {
  const int lane = threadIdx.x & 31;
  K k = list > up ? list : up;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) k = bitonic_step(k, d, (lane & d) == 0);
  return k;
}
// Adds the lanes' keys to the warp's list, unless none of them is among its n best.
// n == 1: every lane keeps its best.
template <class K>
__device__ __forceinline__ void add_keys(K& list, K k, int n) {
  if (n == 1) {
    list = list > k ? list : k;
    return;
  }
  const K least = __shfl_sync(0xffffffffu, list, n - 1);
  if (!__any_sync(0xffffffffu, k > least)) return;
  const K up = sort_up(k);
  // a list without keys takes them as they are
  list = __any_sync(0xffffffffu, list != 0) ? merge_best(list, up) : __shfl_sync(0xffffffffu, up, 31 - (threadIdx.x & 31));
}
template <class K>
__device__ __forceinline__ K warp_best(K k) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) k = bitonic_step(k, d, true);
  return k;
}
// Barrier of a row's NW warps: one of the CTA's, or all.
template <int NW>
__device__ __forceinline__ void sync_row() {
  if (NW == 1) __syncwarp();
  else __syncthreads();
}
// The best of the NW warps' lists, in the row's first warp (n == 1: of all lanes' keys, in
// every lane).  s: [NW][32].
template <int NW, class K>
__device__ __forceinline__ K join_lists(K list, K (*s)[32], int n) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (n == 1) list = warp_best(list);
  if (NW == 1) return list;
  if (n == 1) {
    if (lane == 0) s[0][warp] = list;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NW; ++i) list = list > s[0][i] ? list : s[0][i];
    __syncthreads();
    return list;
  }
#pragma unroll
  for (int h = NW / 2; h > 0; h >>= 1) {
    if (warp >= h && warp < 2 * h) s[warp][lane] = list;
    __syncthreads();
    if (warp < h) list = merge_best(list, s[warp + h][31 - lane]);
  }
  return list;
}

__device__ __forceinline__ void st_cluster_u64(uint32_t addr, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

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
  // The words that are all the row's: from whole0() up to whole1().
  __device__ __forceinline__ int whole0() const { return lead ? 1 : 0; }
  __device__ __forceinline__ int whole1() const { return static_cast<int>((static_cast<long long>(V) + lead) / kEl); }
  // Word i; -inf where there is no logit.
  __device__ __forceinline__ uint4 load(int i) const {
    if (i >= whole0() && i < whole1()) return __ldg(reinterpret_cast<const uint4*>(words) + i);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const long long e = static_cast<long long>(i) * kEl + (F32 ? j : 2 * j) - lead;
      if (F32) {
        w[j] = bits(i, e);
      } else {
        w[j] = bits(i, e) | (bits(i, e + 1) << 16);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ uint32_t bits(int i, long long e) const {
    if (i >= n || e < 0 || e >= V) return F32 ? 0xFF800000u : 0xFF80u;
    const uint8_t* p = words + (static_cast<long long>(lead) + e) * kSize;
    return F32 ? __ldg(reinterpret_cast<const uint32_t*>(p)) : __ldg(reinterpret_cast<const unsigned short*>(p));
  }
  __device__ __forceinline__ float at(int e) const {
    const uint8_t* p = words + (static_cast<long long>(lead) + e) * kSize;
    return F32 ? __ldg(reinterpret_cast<const float*>(p))
               : __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(p))) << 16);
  }
};

// A 16-byte copy global -> shared that the thread waits for by group.
__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {  // drops a NaN
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// A 16-byte word's logits.
template <bool F32>
struct Word {
  static constexpr int kEl = F32 ? 4 : 8;
  // The largest of N words; NaN only where all logits are.
  template <int N>
  static __device__ __forceinline__ float largest(const uint4 (&v)[N]) {
    if (F32) {
      float m = -INFINITY;
#pragma unroll
      for (int u = 0; u < N; ++u)
        m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(v[u].x), __uint_as_float(v[u].y)),
                           fmaxf(__uint_as_float(v[u].z), __uint_as_float(v[u].w))));
      return m;
    }
    uint32_t m = 0xFF80FF80u;
#pragma unroll
    for (int u = 0; u < N; ++u) m = max_bf16x2(m, max_bf16x2(max_bf16x2(v[u].x, v[u].y), max_bf16x2(v[u].z, v[u].w)));
    return fmaxf(bf16_lo(m), bf16_hi(m));
  }
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[kEl]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (F32) {
        x[j] = __uint_as_float(w[j]);
      } else {
        x[2 * j] = bf16_lo(w[j]);
        x[2 * j + 1] = bf16_hi(w[j]);
      }
    }
  }
  // Makes one logit equal to top -inf, if the word has one.
  static __device__ __forceinline__ bool remove(uint4& v, float top) {
    const uint4 one[1] = {v};
    if (largest(one) != top) return false;
    if (!remove(v.x, top) && !remove(v.y, top) && !remove(v.z, top)) remove(v.w, top);
    return true;
  }
  static __device__ __forceinline__ bool remove(uint32_t& w, float top) {
    if (F32) {
      if (__uint_as_float(w) != top) return false;
      w = 0xFF800000u;
      return true;
    }
    if (bf16_lo(w) == top) {
      w = (w & 0xFFFF0000u) | 0xFF80u;
      return true;
    }
    if (bf16_hi(w) != top) return false;
    w = (w & 0xFFFFu) | 0xFF800000u;
    return true;
  }
  // +inf made -inf
  static __device__ __forceinline__ void drop_inf(uint32_t& w) {
    if (F32) {
      if (w == 0x7F800000u) w = 0xFF800000u;
    } else {
      if ((w & 0xFFFFu) == 0x7F80u) w |= 0x8000u;
      if ((w >> 16) == 0x7F80u) w |= 0x80000000u;
    }
  }
  // Adds the terms of two logits of the word, both raised to kLowest (which a NaN
  // becomes as well).
  static __device__ __forceinline__ void add(float a, float b, uint64_t minus_m, uint64_t& r, uint64_t& w) {
    const uint64_t d = add_f32x2(pack_f32x2(a, b), minus_m);
    const float2 e2 = unpack_f32x2(mul_f32x2(d, pack_f32x2(kLog2e, kLog2e)));
    const uint64_t e = pack_f32x2(exp2_fast(e2.x), exp2_fast(e2.y));
    r = add_f32x2(r, e);
    w = fma_f32x2(e, d, w);
  }
  static __device__ __forceinline__ void add_word(const uint4& v, uint64_t minus_m, uint64_t& r, uint64_t& w) {
    const uint32_t q[4] = {v.x, v.y, v.z, v.w};
    if (F32) {
#pragma unroll
      for (int j = 0; j < 4; j += 2)
        add(fmaxf(__uint_as_float(q[j]), kLowest), fmaxf(__uint_as_float(q[j + 1]), kLowest), minus_m, r, w);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t c = max_bf16x2(q[j], 0xF180F180u);  // kLowest twice
        add(bf16_lo(c), bf16_hi(c), minus_m, r, w);
      }
    }
  }
};

// A row is NW warps' work: one warp's, or a CTA's, or that of a cluster of `splits` CTAs,
// each with a run of its words.  A thread copies its words ahead into places of its own
// in shared memory, so the pass has no barrier.
template <bool F32, bool TOP, int NW, bool DEEP, bool SPLIT>
__global__ void __launch_bounds__(kLpThreads) logprobs_kernel(const __grid_constant__ LogprobParams p, int T, int splits) {
  constexpr int kEl = Row<F32>::kEl, B = kBatch<F32>, S = kStages<F32, DEEP>, kThreads = NW * 32, kRows = kLpWarps / NW;
  constexpr uint32_t kNone = F32 ? 0xFF800000u : 0xFF80FF80u;
  constexpr int kRing = S * B * kThreads, kList = kMaxList<NW>;
  static_assert((NW * 32 + kList) * 8 <= kRing * 16, "the lists fit the row's ring");
  __shared__ Sums s_sums[kLpWarps];
  __shared__ Sums s_parts[SPLIT ? kMaxSplits : 1];  // of the cluster's CTAs, in its first
  __shared__ float s_all_runs[kRows][TOP ? kThreads * kMaxRuns : 1];  // the runs' largest logits
  __shared__ int s_all_tied[kRows][TOP ? kMaxTied : 1];
  __shared__ unsigned long long s_bests[SPLIT && TOP ? kMaxSplits : 1][32];
  __shared__ float s_taus[kRows];
  __shared__ int s_counts[kRows], s_tied_counts[kRows];
  extern __shared__ uint4 s_all[];  // [kRows][S][B][kThreads]; behind the pass, lists and candidates
  if (SPLIT) cluster_arrive();  // waited for before the first CTA's shared memory is written
  pdl_wait();
  pdl_trigger();
  const int mine = NW == 1 ? threadIdx.x >> 5 : 0;  // of the CTA's rows
  const long long t = NW == 1 ? static_cast<long long>(blockIdx.x) * kRows + mine : SPLIT ? blockIdx.x / splits : blockIdx.x;
  if (NW == 1 && t >= T) return;
  const int rank = SPLIT ? blockIdx.x % splits : 0;
  const int tid = threadIdx.x % kThreads, warp = tid >> 5, lane = tid & 31;
  uint4* s_ring = s_all + mine * kRing;
  unsigned long long(*s_lists)[32] = reinterpret_cast<unsigned long long(*)[32]>(s_ring);
  unsigned long long* s_cand = reinterpret_cast<unsigned long long*>(s_ring) + NW * 32;
  float* s_runs = s_all_runs[mine];
  int* s_tied = s_all_tied[mine];
  int &s_count = s_counts[mine], &s_tied_count = s_tied_counts[mine];
  float& s_tau = s_taus[mine];
  const Row<F32> row(p.logits, t * p.ld, p.V);
  const int share = SPLIT ? (row.n + splits - 1) / splits : row.n;
  const int first = min(row.n, rank * share), words = min(row.n, first + share) - first;
  const int batches = (words + kThreads * B - 1) / (kThreads * B);
  const int run_batches =
      max(NW == 1 ? 1 : min(kRunBatches, max(batches, kRunWords / B)), (batches + kMaxRuns - 1) / kMaxRuns);
  const int whole0 = row.whole0(), whole1 = min(row.whole1(), first + words);
  uint4* place = s_ring + tid;
  auto fetch = [&](int b) {
    if (b < batches) {
      const int w0 = first + b * kThreads * B, st = b % S;
      if (w0 >= whole0 && w0 + kThreads * B <= whole1) {
        const uint8_t* src = row.words + (static_cast<long long>(w0) + tid) * 16;
#pragma unroll
        for (int u = 0; u < B; ++u) copy16(place + (st * B + u) * kThreads, src + u * kThreads * 16);
      } else {  // the row's ends, and what is behind them
#pragma unroll 1
        for (int u = 0; u < B; ++u) {
          const int i = w0 + u * kThreads + tid;
          if (i >= whole0 && i < whole1) copy16(place + (st * B + u) * kThreads, row.words + static_cast<long long>(i) * 16);
          else place[(st * B + u) * kThreads] = i < first + words ? row.load(i) : make_uint4(kNone, kNone, kNone, kNone);
        }
      }
    }
    copy_commit();
  };
#pragma unroll
  for (int b = 0; b < S - 1; ++b) fetch(b);
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
  float run_max = -INFINITY, thread_max = -INFINITY;
  int run = 0, left = run_batches;
  for (int b = 0; b < batches; ++b) {
    copy_wait<S - 2>();
    uint4 x[B];
#pragma unroll
    for (int u = 0; u < B; ++u) x[u] = place[(b % S * B + u) * kThreads];
    fetch(b + S - 1);
    float best = Word<F32>::largest(x);
    if (best == INFINITY) {
#pragma unroll
      for (int u = 0; u < B; ++u) {
        Word<F32>::drop_inf(x[u].x);
        Word<F32>::drop_inf(x[u].y);
        Word<F32>::drop_inf(x[u].z);
        Word<F32>::drop_inf(x[u].w);
      }
      best = Word<F32>::largest(x);
    }
    run_max = fmaxf(run_max, best);
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
        for (int u = 0; u < B; ++u)
          if (!out) out = Word<F32>::remove(x[u], top);
      }
    }
    if (m > kLowest) {
      const uint64_t minus_m = pack_f32x2(-m, -m);
      uint64_t r2 = pack_f32x2(r, 0.f), w2 = pack_f32x2(w, 0.f);
#pragma unroll
      for (int u = 0; u < B; ++u) Word<F32>::add_word(x[u], minus_m, r2, w2);
      const float2 rs = unpack_f32x2(r2), ws = unpack_f32x2(w2);
      r = rs.x + rs.y;
      w = ws.x + ws.y;
    } else {
#pragma unroll
      for (int u = 0; u < B; ++u) {
        float y[kEl];
        Word<F32>::unpack(x[u], y);
#pragma unroll
        for (int j = 0; j < kEl; ++j) {
          const float d = fmaxf(y[j] - m, kFar);  // masked logits and NaN: e^d is 0
          const float e = exp_neg(d);
          r += e;
          w = fmaf(e, d, w);
        }
      }
    }
    if (TOP && (--left == 0 || b + 1 == batches)) {
      s_runs[run++ * kThreads + tid] = run_max;
      thread_max = fmaxf(thread_max, run_max);
      run_max = -INFINITY;
      left = run_batches;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    r += __shfl_xor_sync(0xffffffffu, r, o);
    w += __shfl_xor_sync(0xffffffffu, w, o);
  }
  Sums all = {m, r, w};
  if (NW > 1 && lane == 0) s_sums[warp] = all;
  if (tid == 0) s_count = s_tied_count = 0;
  sync_row<NW>();
  if (NW > 1 && warp == 0) all = merge_lanes<NW>(lane < NW ? s_sums[lane] : Sums{-INFINITY, 0.f, 0.f});

  // ---- the best of these logits, descending over the first warp's lanes
  unsigned long long list = 0;
  if (TOP) {
    const int run_words = run_batches * B;
    uint32_t largest = 0;
    if (NW == 1) {  // 32 threads are few for n of them: their runs
      for (int i = 0; i < run; ++i) add_keys(largest, run_key(s_runs[i * kThreads + tid]), p.n);
    } else {
      add_keys(largest, run_key(thread_max), p.n);
    }
    largest = join_lists<NW>(largest, reinterpret_cast<uint32_t(*)[32]>(s_lists), p.n);
    if (warp == 0) {
      largest = __shfl_sync(0xffffffffu, largest, p.n - 1);
      // fewer threads than n have a logit: all runs that have one
      if (lane == 0) s_tau = largest ? ord_to_float(largest) : -kLargestFloat;
    }
    sync_row<NW>();
    const float tau = s_tau;
    for (int i = 0; i < run; ++i) {
      const bool is = s_runs[i * kThreads + tid] >= tau;
      const int at = append<NW>(&s_tied_count, is);
      if (is && at < kMaxTied) s_tied[at] = i * kThreads + tid;
    }
    sync_row<NW>();
    const int tied = s_tied_count;
    const bool all_runs = tied > kMaxTied;
    const int again = all_runs ? batches * B * kThreads : tied * run_words;
    // the logits of these runs that are at least tau (0: none), a word a lane
    auto candidates = [&](auto&& take) {
      for (int i = warp * 32; i < again; i += kThreads) {
        int k = i + lane;  // the word, from this CTA's first
        bool in = k < again;
        if (in && !all_runs) {
          const int at = s_tied[k / run_words];
          k = (at / kThreads * run_words + k % run_words) * kThreads + at % kThreads;
        }
        in = in && k < words;
        const int word = first + (in ? k : 0);
        float y[kEl];
        Word<F32>::unpack(row.load(in ? word : row.n), y);
#pragma unroll
        for (int j = 0; j < kEl; ++j) {
          const bool is = y[j] >= tau && y[j] <= kLargestFloat;
          take(is, y[j], static_cast<uint32_t>(word) * kEl + j - row.lead);
        }
      }
    };
    if (!all_runs)
      candidates([&](bool is, float y, uint32_t id) {
        const int at = append<NW>(&s_count, is);
        if (is && at < kList) s_cand[at] = top_key(y, id);  // any order: the keys differ and are sorted
      });
    sync_row<NW>();
    const int count = all_runs ? kList + 1 : s_count;
    if (count <= 64) {  // one warp sorts them in less time than the warps' lists are joined
      if (warp == 0)
        for (int i = 0; i < count; i += 32) add_keys(list, i + lane < count ? s_cand[i + lane] : 0ull, p.n);
      if (p.n == 1) list = warp_best(list);
    } else {
      if (count <= kList) {
        for (int i = warp * 32; i < count; i += kThreads) add_keys(list, i + lane < count ? s_cand[i + lane] : 0ull, p.n);
      } else {
        candidates([&](bool is, float y, uint32_t id) { add_keys(list, is ? top_key(y, id) : 0ull, p.n); });
      }
      list = join_lists<NW>(list, s_lists, p.n);
    }
  }

  // ---- the cluster's CTAs
  if constexpr (SPLIT) {
    static_assert(kMaxSplits <= 2 * NW, "a warp joins two CTAs' lists");
    __syncwarp();
    cluster_wait();  // the first CTA has started
    if (warp == 0) {
      if (lane == 0) {
        const uint32_t to = map_rank(smem_u32(&s_parts[rank]), 0u);
        st_cluster_f32(to, all.m);
        st_cluster_f32(to + 4, all.r);
        st_cluster_f32(to + 8, all.w);
      }
      if (TOP) st_cluster_u64(map_rank(smem_u32(&s_bests[rank][lane]), 0u), list);
      __syncwarp();
    }
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;  // nothing of its shared memory is read from outside
    if (warp == 0) all = merge_lanes<kMaxSplits>(lane < splits ? s_parts[lane] : Sums{-INFINITY, 0.f, 0.f});
    if (TOP) {
      list = warp < splits ? s_bests[warp][lane] : 0;
      if (warp + NW < splits) list = merge_best(list, s_bests[warp + NW][31 - lane]);
      list = join_lists<NW>(list, s_lists, p.n);
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
}

template <bool F32, bool TOP, int NW, bool DEEP, bool SPLIT>
cudaError_t launch(const LogprobParams& p, int T, int splits, const DeviceCtx& ctx, cudaStream_t st) {
  constexpr int kSmem = kRingBytes<F32, DEEP>;
  constexpr auto kern = logprobs_kernel<F32, TOP, NW, DEEP, SPLIT>;
  cudaError_t e = prefer_max_smem_once<kern>(ctx.device, kSmem);
  if (e != cudaSuccess) return e;
  static std::atomic<bool> above8[64];  // clusters of more CTAs have to be allowed, once a device
  if (splits > 8 && !above8[ctx.device].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    above8[ctx.device].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(NW == 1 ? (T + kLpWarps - 1) / kLpWarps : T * splits);
  cfg.blockDim = dim3(kLpThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = SPLIT ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p, T, splits);
}

template <bool F32, bool TOP>
cudaError_t launch_type(const LogprobParams& p, int T, const DeviceCtx& ctx, cudaStream_t st) {
  // A warp a row where the rows are short and many: 2,048 rows of 1,000 fp32 logits with
  // 5 alternatives take 6.9 us, 18.5 with a CTA each; 2,048 of 10,000: 21.8 and 27.4; 333
  // of 2,000: 8.5 and 6.1; 700 of 10,000: 13.5 and 11.3; 2,048 of 20,000: 43 and 37.
  if (p.V <= 512 || (p.V <= 10000 && T >= 5 * ctx.num_sms)) return launch<F32, TOP, 1, false, false>(p, T, 1, ctx, st);
  // A cluster a row where the rows leave SMs idle, down to 2,048 logits a CTA (64 rows of
  // 131,072 fp32 logits with 20 alternatives: 12.7 us split by 4, 16.9 whole; 128 rows: 18.7
  // by 2, 16.9 whole; 8 rows of 20,000 bf16: 6.6 by 8, 7.1 by 4); 16 CTAs while each has an
  // SM to itself (8 rows of 131,072: 8.1 and 8.2 by 8; 2 of 1,000,000: 13.0 and 17.0; 16
  // rows of 131,072: 8.4 and 8.1).
  int splits = 1;
  if (2 * T <= ctx.num_sms)
    while (splits < 8 && T * splits <= ctx.num_sms && p.V / (splits * 2) >= 2048) splits *= 2;
  if (splits == 8 && T * kMaxSplits <= ctx.num_sms && p.V / kMaxSplits >= 2048) splits = kMaxSplits;
  if (splits > 1) return launch<F32, TOP, kLpWarps, false, true>(p, T, splits, ctx, st);
  // With an SM or half of one to itself a whole row's CTA needs more bytes on their way
  // (rows of 131,072 fp32 logits, 128 of them: 16.9 us, 26 with two stages), but the larger
  // ring leaves fewer CTAs an SM (512: 58 and 46).  Between them the SMs' uneven shares of rows
  // decide, with 5 alternatives: 250 rows 29.4 and 30.5, 304 35.9 and 32.5, 333 37.6 and 34.5,
  // 400 41.1 and 46.8, 512 56.7 and 54.2.
  if constexpr (F32)
    if (T <= 2 * ctx.num_sms) return launch<F32, TOP, kLpWarps, true, false>(p, T, 1, ctx, st);
  return launch<F32, TOP, kLpWarps, false, false>(p, T, 1, ctx, st);
}

}  // namespace

cudaError_t launch_logprobs(const csa2_logprobs_args& a, const DeviceCtx& ctx, cudaStream_t st) {
  const LogprobParams p{a.logits, a.ld_logits, a.V, a.token, a.logprob, a.entropy, a.lse, a.top_id, a.top_logprob,
                        a.ld_top, a.n_top, ctx.err};
  if (a.logits_f32) return a.n_top ? launch_type<true, true>(p, a.T, ctx, st) : launch_type<true, false>(p, a.T, ctx, st);
  return a.n_top ? launch_type<false, true>(p, a.T, ctx, st) : launch_type<false, false>(p, a.T, ctx, st);
}

}  // namespace csa2
