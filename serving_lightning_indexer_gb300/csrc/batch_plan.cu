// The batch's rows, pages and slots from its sequences' lengths, in one launch.
//
// Per sequence: rows, new entries and new pages; an exclusive prefix sum of the
// three places every row, entry and page.  Each CTA makes the sums that it needs
// for itself (two loads a sequence, B <= 8192, in shared memory), which costs less
// than a second launch or a wait between CTAs, and then fills its share of the
// outputs: 32 rows at a time, or a thread an entry or a page.  Bound: launch and load
// latency (8 sequences: 2.8 us; 256 with 8,260 rows: 5.5 us for 4.5 MB).
#include <limits.h>

#include "csa2_device.cuh"
#include "csa2_internal.h"

namespace csa2 {
namespace {

constexpr int kPlanThreads = 256;

struct PlanParams {
  csa2_batch_plan_args a;
  int row_ctas;  // CTAs that fill the rows; the others fill the pages and entries
  int vec;       // swa_slot in 16-byte pieces
  uint32_t* err;
};

// Sum of two counts, at most INT_MAX (as every place that is used is).
__device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) { return min(a + b, static_cast<uint32_t>(INT_MAX)); }
__device__ __forceinline__ int pages_of(int entries) { return (entries >> 6) + ((entries & 63) != 0); }
__device__ __forceinline__ int clip(long long v) { return static_cast<int>(min(v, static_cast<long long>(INT_MAX))); }

// Largest b in [0, n) with start[b] <= i: the sequence that place i belongs to
// (sequences without a place have start[b] == start[b + 1]).
__device__ __forceinline__ int owner_of(const int* start, int n, int i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= i) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Rows of this CTA, 32 at a time: a lane of the first warp finds a row's sequence and
// place and writes its words, then the warps write four rows' windows each.
constexpr int kPlanRows = 32;
struct RowPlace {
  int pos, base, at, kept;  // position, first ring slot (-1: no ring), own place in it, first position that is kept
};

__device__ __forceinline__ void fill_rows(const PlanParams& p, const int* ctx, const int* row0, const int* ring) {
  const csa2_batch_plan_args& a = p.a;
  const int B = a.B, rows = row0[B], W = a.n_swa, R = a.swa_ring;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = a.pad ? a.max_rows : min(rows, a.max_rows);
  __shared__ RowPlace place[2][kPlanRows];  // two sets: the next rows are placed while these are written
  int set = 0;
  for (long long t0 = static_cast<long long>(blockIdx.x) * kPlanRows; t0 < n;
       t0 += static_cast<long long>(p.row_ctas) * kPlanRows, set ^= 1) {
    const int count = static_cast<int>(min(static_cast<long long>(kPlanRows), n - t0));
    if (warp == 0 && lane < count) {
      const int t = static_cast<int>(t0) + lane;
      int seq = -1;
      RowPlace r{-1, -1, 0, 0};
      if (t < rows) {
        seq = owner_of(row0, B, t);
        r.pos = ctx[seq] + t - row0[seq];
        if (a.swa_new || a.swa_slot) {
          r.kept = max(ctx[seq] + row0[seq + 1] - row0[seq] - R, 0);
          const long long slot0 = static_cast<long long>(ring[seq]) * R;
          r.base = ring[seq] >= 0 && slot0 + R - 1 <= INT_MAX ? static_cast<int>(slot0) : -1;
          const int need = a.swa_slot ? max(ctx[seq] - W + 1, 0) : ctx[seq];
          if (r.base < 0 || r.kept > need) set_error(p.err, kErrBounds);
          r.at = r.pos % R;
        }
      }
      place[set][lane] = r;
      if (a.row_seq) a.row_seq[t] = seq;
      if (a.row_pos) a.row_pos[t] = r.pos;
      if (a.swa_new) a.swa_new[t] = r.base >= 0 && r.pos >= r.kept ? r.base + r.at : -1;
    }
    if (!a.swa_slot) continue;
    __syncthreads();
    for (int i = warp; i < count; i += kPlanThreads / 32) {
      const RowPlace r = place[set][i];
      auto slot = [&](int j) {
        const int back = W - 1 - j;  // tokens before the row's
        return r.base >= 0 && r.pos - back >= r.kept ? r.base + (r.at >= back ? r.at - back : r.at - back + R) : -1;
      };
      int* out = a.swa_slot + (t0 + i) * a.ld_swa;
      if (p.vec) {
        const int j = lane * 4;
        if (j < W) *reinterpret_cast<int4*>(out + j) = make_int4(slot(j), slot(j + 1), slot(j + 2), slot(j + 3));
      } else {
        for (int j = lane; j < W; j += 32) out[j] = slot(j);
      }
    }
  }
}

__global__ void __launch_bounds__(kPlanThreads) batch_plan_kernel(const __grid_constant__ PlanParams p) {
  extern __shared__ int sm[];
  const csa2_batch_plan_args& a = p.a;
  const int B = a.B, m = a.ratio_m, sh = m - 1;  // lengths / m: m is 1 or 2
  int* ctx = sm;               // [B]
  int* row0 = ctx + B;         // [B + 1]; first new_len, then its prefix sum
  int* ent0 = row0 + B + 1;    // [B + 1]
  int* pag0 = ent0 + B + 1;    // [B + 1]
  int* ring = pag0 + B + 1;    // [B]; ring_id
  __shared__ uint32_t warp_sum[3][kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool first = blockIdx.x == 0, is_rows = static_cast<int>(blockIdx.x) < p.row_ctas;
  pdl_wait();
  pdl_trigger();
  const long long head = a.free_head ? static_cast<long long>(__ldg(a.free_head)) : 0;  // on its way under the sums
  for (int b = tid; b < B; b += kPlanThreads) {
    int c = __ldg(a.ctx_len + b), n = __ldg(a.new_len + b);
    const bool bad = c < 0 || n < 0 || c > INT_MAX - max(n, 0);
    if (bad) {
      c = max(c, 0);
      n = 0;
      if (first) set_error(p.err, kErrBounds);
    }
    ctx[b] = c;
    row0[b] = n;
    ring[b] = a.ring_id ? __ldg(a.ring_id + b) : b;
  }
  __syncthreads();
  // prefix sums: a thread's run of sequences, then across threads; the CTAs of the
  // rows, which are most, sum the rows only
  const int sums = is_rows && !first ? 1 : 3;
  const int per = (B + kPlanThreads - 1) / kPlanThreads;
  const int lo = min(tid * per, B), hi = min(lo + per, B);
  uint32_t s[3] = {0, 0, 0}, incl[3], run[3];
  for (int b = lo; b < hi; ++b) {
    const int n = row0[b], e0 = ctx[b] >> sh, e1 = (ctx[b] + n) >> sh;
    s[0] = add(s[0], n);
    s[1] = add(s[1], e1 - e0);
    s[2] = add(s[2], pages_of(e1) - pages_of(e0));
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (k >= sums) break;
    incl[k] = s[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, incl[k], o);
      if (lane >= o) incl[k] = add(incl[k], v);
    }
    if (lane == 31) warp_sum[k][warp] = incl[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (k >= sums) break;
    run[k] = __shfl_up_sync(0xffffffffu, incl[k], 1);
    if (lane == 0) run[k] = 0;
    for (int w = 0; w < warp; ++w) run[k] = add(run[k], warp_sum[k][w]);
    // the last thread's sum is the total
    if (tid == kPlanThreads - 1) (k == 0 ? row0 : k == 1 ? ent0 : pag0)[B] = static_cast<int>(add(run[k], s[k]));
  }
  for (int b = lo; b < hi; ++b) {
    const int n = row0[b], e0 = ctx[b] >> sh, e1 = (ctx[b] + n) >> sh;
    row0[b] = static_cast<int>(run[0]);
    run[0] = add(run[0], n);
    if (sums == 1) continue;
    ent0[b] = static_cast<int>(run[1]);
    pag0[b] = static_cast<int>(run[2]);
    run[1] = add(run[1], e1 - e0);
    run[2] = add(run[2], pages_of(e1) - pages_of(e0));
    if (first) {
      if (a.row_start) a.row_start[b] = row0[b];
      if (a.entry_start) a.entry_start[b] = ent0[b];
      if (a.n_visible) a.n_visible[b] = e1;
      if (a.page_table && pages_of(e1) > a.pt_stride) set_error(p.err, kErrBounds);
    }
  }
  __syncthreads();
  if (is_rows && !first) {
    fill_rows(p, ctx, row0, ring);
    return;
  }
  const int rows = row0[B], entries = ent0[B], pages = pag0[B];
  const bool has_rows = a.row_seq || a.row_pos || a.swa_new || a.swa_slot;
  const bool has_entries = a.entry_slot || a.entry_pos || a.entry_row;
  // the free list's page for the i-th new page of the batch, -1 if there is none
  auto new_page = [&](long long i) {
    const long long at = head + i;
    return at >= 0 && at < a.n_free ? __ldg(a.free_pages + at) : -1;
  };
  if (first && tid == 0) {
    if (a.row_start) a.row_start[B] = rows;
    if (a.entry_start) a.entry_start[B] = entries;
    if (a.free_head_out) a.free_head_out[0] = clip(head + (a.free_pages ? pages : 0));
    // sums stop at INT_MAX, which may then be short of the rows (the other counts are smaller)
    if (rows == INT_MAX || (has_rows && rows > a.max_rows) || (has_entries && entries > a.max_entries))
      set_error(p.err, kErrBounds);
  }
  if (is_rows) {
    fill_rows(p, ctx, row0, ring);
    return;
  }
  const int gtid = (blockIdx.x - p.row_ctas) * kPlanThreads + tid, gthreads = (gridDim.x - p.row_ctas) * kPlanThreads;

  // ---- new pages
  if (a.free_pages) {
    for (long long i = gthreads - 1 - gtid; i < pages; i += gthreads) {  // from the end: not the entries' first threads
      const int b = owner_of(pag0, B, static_cast<int>(i));
      const int e0 = ctx[b] >> sh;
      const int lp = pages_of(e0) + static_cast<int>(i) - pag0[b];
      const int page = new_page(i);
      if (page < 0) set_error(p.err, kErrBounds);
      if (lp < a.pt_stride) a.page_table[static_cast<long long>(b) * a.pt_stride + lp] = page < 0 ? -1 : page;
    }
  }
  // ---- new entries
  if (has_entries) {
    const int n = a.pad ? a.max_entries : min(entries, a.max_entries);
    for (long long i = gtid; i < n; i += gthreads) {
      int slot = -1, pos = 0, row = -1;
      if (i < entries) {
        const int b = owner_of(ent0, B, static_cast<int>(i));
        const int e0 = ctx[b] >> sh, e = e0 + static_cast<int>(i) - ent0[b];
        const int old_pages = pages_of(e0), lp = e / 64;
        pos = e * m;
        row = clip(static_cast<long long>(row0[b]) + (pos + m - 1 - ctx[b]));
        if (a.entry_slot) {
          int page = -1;
          if (lp < a.pt_stride)
            page = a.free_pages && lp >= old_pages ? new_page(static_cast<long long>(pag0[b]) + lp - old_pages)
                                                   : a.page_table[static_cast<long long>(b) * a.pt_stride + lp];
          if (page >= 0 && page <= (INT_MAX - 63) / 64) slot = page * 64 + e % 64;
          else set_error(p.err, kErrBounds);
        }
      }
      if (a.entry_slot) a.entry_slot[i] = slot;
      if (a.entry_pos) a.entry_pos[i] = pos;
      if (a.entry_row) a.entry_row[i] = row;
    }
  }
}

}  // namespace

cudaError_t launch_batch_plan(const csa2_batch_plan_args& a, const DeviceCtx& ctx, cudaStream_t st) {
  const bool rows = a.row_seq || a.row_pos || a.swa_new || a.swa_slot;
  const bool rest = a.free_pages || a.entry_slot || a.entry_pos || a.entry_row;
  PlanParams p{a, 0, 0, ctx.err};
  p.vec = a.swa_slot && reinterpret_cast<uintptr_t>(a.swa_slot) % 16 == 0 && a.ld_swa % 4 == 0 && a.n_swa % 4 == 0;
  const size_t smem = (static_cast<size_t>(a.B) * 5 + 3) * sizeof(int);
  cudaError_t e = prefer_max_smem_once<batch_plan_kernel>(ctx.device, (kPlanMaxSeqs * 5 + 3) * sizeof(int));
  if (e != cudaSuccess) return e;
  // 32 rows a CTA, and CTAs of their own for the pages and entries (an entry's page
  // is a load that would hold up the rows behind it); the sums are made in every
  // CTA, so no more of them than four an SM for the rows and one for the rest.
  auto ctas = [](long long items, long long each, long long most) {
    const long long n = (items + each - 1) / each;
    return static_cast<int>(n > most ? most : n);
  };
  p.row_ctas = rows ? ctas(a.max_rows, kPlanRows, 4LL * ctx.num_sms) : 0;
  const long long places = a.max_entries > a.B ? a.max_entries : a.B;
  int grid = p.row_ctas + (rest ? ctas(places, kPlanThreads, ctx.num_sms) : 0);
  if (grid < 1) grid = 1;
  return launch_pdl(batch_plan_kernel, dim3(grid), dim3(kPlanThreads), smem, st, p);
}

}  // namespace csa2
