// The batch's rows, pages and slots from its sequences' lengths, in one launch.
//
// Per sequence: rows, new entries and new pages; an exclusive prefix sum of the
// three places every row, entry and page.  Each CTA makes the sums for itself
// (two loads a sequence, B <= 8192, in shared memory), which costs less than a
// second launch or a wait between CTAs, and then fills its share of the
// outputs: a warp a row, a thread an entry or a page.  Bound: launch latency for
// a decode batch, the stores of swa_slot (4 * n_swa bytes a row) for prompts.
#include <limits.h>

#include "csa2_device.cuh"
#include "csa2_internal.h"

namespace csa2 {
namespace {

constexpr int kPlanThreads = 256;

struct PlanParams {
  csa2_batch_plan_args a;
  uint32_t* err;
};

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

__global__ void __launch_bounds__(kPlanThreads) batch_plan_kernel(const __grid_constant__ PlanParams p) {
  extern __shared__ int sm[];
  const csa2_batch_plan_args& a = p.a;
  const int B = a.B, m = a.ratio_m;
  int* ctx = sm;               // [B]
  int* row0 = ctx + B;         // [B + 1]; first new_len, then its prefix sum
  int* ent0 = row0 + B + 1;    // [B + 1]
  int* pag0 = ent0 + B + 1;    // [B + 1]
  __shared__ long long warp_sum[3][kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool first = blockIdx.x == 0;
  pdl_wait();
  pdl_trigger();
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
  }
  __syncthreads();
  // prefix sums: a thread's run of sequences, then across threads
  const int per = (B + kPlanThreads - 1) / kPlanThreads;
  const int lo = min(tid * per, B), hi = min(lo + per, B);
  long long s[3] = {0, 0, 0};
  for (int b = lo; b < hi; ++b) {
    const int n = row0[b], e0 = ctx[b] / m, e1 = (ctx[b] + n) / m;
    s[0] += n;
    s[1] += e1 - e0;
    s[2] += (e1 / 64 + (e1 % 64 != 0)) - (e0 / 64 + (e0 % 64 != 0));
  }
  long long incl[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    incl[k] = s[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl[k], o);
      if (lane >= o) incl[k] += v;
    }
    if (lane == 31) warp_sum[k][warp] = incl[k];
  }
  __syncthreads();
  long long run[3], total[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    run[k] = incl[k] - s[k];
    total[k] = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w < warp) run[k] += warp_sum[k][w];
      total[k] += warp_sum[k][w];
    }
  }
  auto clip = [](long long v) { return static_cast<int>(min(v, static_cast<long long>(INT_MAX))); };
  for (int b = lo; b < hi; ++b) {
    const int n = row0[b], e0 = ctx[b] / m, e1 = (ctx[b] + n) / m;
    row0[b] = clip(run[0]);
    ent0[b] = clip(run[1]);
    pag0[b] = clip(run[2]);
    run[0] += n;
    run[1] += e1 - e0;
    const int p1 = e1 / 64 + (e1 % 64 != 0);
    run[2] += p1 - (e0 / 64 + (e0 % 64 != 0));
    if (first) {
      if (a.row_start) a.row_start[b] = row0[b];
      if (a.entry_start) a.entry_start[b] = ent0[b];
      if (a.n_visible) a.n_visible[b] = e1;
      if (a.page_table && p1 > a.pt_stride) set_error(p.err, kErrBounds);
    }
  }
  if (tid == 0) {
    row0[B] = clip(total[0]);
    ent0[B] = clip(total[1]);
    pag0[B] = clip(total[2]);
  }
  __syncthreads();
  const int rows = row0[B], entries = ent0[B], pages = pag0[B];
  const bool has_rows = a.row_seq || a.row_pos || a.swa_new || a.swa_slot;
  const bool has_entries = a.entry_slot || a.entry_pos || a.entry_row;
  const long long head = a.free_head ? static_cast<long long>(__ldg(a.free_head)) : 0;
  // the free list's page for the i-th new page of the batch, -1 if there is none
  auto new_page = [&](long long i) {
    const long long at = head + i;
    return at >= 0 && at < a.n_free ? __ldg(a.free_pages + at) : -1;
  };
  if (first && tid == 0) {
    if (a.row_start) a.row_start[B] = rows;
    if (a.entry_start) a.entry_start[B] = entries;
    if (a.free_head_out) a.free_head_out[0] = clip(head + (a.free_pages ? pages : 0));
    if ((has_rows && rows > a.max_rows) || (has_entries && entries > a.max_entries)) set_error(p.err, kErrBounds);
  }
  const int gtid = blockIdx.x * kPlanThreads + tid, gthreads = gridDim.x * kPlanThreads;

  // ---- new pages
  if (a.free_pages) {
    for (long long i = gtid; i < pages; i += gthreads) {
      const int b = owner_of(pag0, B, static_cast<int>(i));
      const int e0 = ctx[b] / m;
      const int lp = e0 / 64 + (e0 % 64 != 0) + static_cast<int>(i) - pag0[b];
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
        const int e0 = ctx[b] / m, e = e0 + static_cast<int>(i) - ent0[b];
        const int old_pages = e0 / 64 + (e0 % 64 != 0), lp = e / 64;
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
  // ---- rows: a warp each
  if (has_rows) {
    const int n = a.pad ? a.max_rows : min(rows, a.max_rows);
    const int W = a.n_swa, R = a.swa_ring;
    for (long long t = blockIdx.x * (kPlanThreads / 32) + warp; t < n; t += gridDim.x * (kPlanThreads / 32)) {
      int b = -1, pos = -1;
      long long base = -1;  // first slot of the ring; -1: no ring
      int kept = 0;         // first position whose slot this step leaves in place
      if (t < rows) {
        b = owner_of(row0, B, static_cast<int>(t));
        pos = ctx[b] + static_cast<int>(t) - row0[b];
        if (a.swa_new || a.swa_slot) {
          const int last = ctx[b] + row0[b + 1] - row0[b];  // the sequence's length after the step
          const int id = a.ring_id ? __ldg(a.ring_id + b) : b;
          const long long at = static_cast<long long>(id) * R;
          base = id >= 0 && at + R - 1 <= INT_MAX ? at : -1;
          kept = max(last - R, 0);
          const int need = a.swa_slot ? max(ctx[b] - W + 1, 0) : ctx[b];
          if (lane == 0 && (base < 0 || kept > need)) set_error(p.err, kErrBounds);
        }
      }
      if (lane == 0) {
        if (a.row_seq) a.row_seq[t] = b;
        if (a.row_pos) a.row_pos[t] = pos;
      }
      if (a.swa_new || a.swa_slot) {
        const int at = base >= 0 ? pos % R : 0;  // the row's own place in the ring
        if (lane == 0 && a.swa_new) a.swa_new[t] = base >= 0 && pos >= kept ? static_cast<int>(base) + at : -1;
        if (a.swa_slot) {
          for (int j = lane; j < W; j += 32) {
            const int back = W - 1 - j;
            const int q = pos - back;
            int slot = -1;
            if (base >= 0 && q >= kept) slot = static_cast<int>(base) + (at >= back ? at - back : at - back + R);
            a.swa_slot[t * a.ld_swa + j] = slot;
          }
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_batch_plan(const csa2_batch_plan_args& a, const DeviceCtx& ctx, cudaStream_t st) {
  PlanParams p{a, ctx.err};
  const size_t smem = (static_cast<size_t>(a.B) * 4 + 3) * sizeof(int);
  cudaError_t e = prefer_max_smem_once<batch_plan_kernel>(ctx.device, (kPlanMaxSeqs * 4 + 3) * sizeof(int));
  if (e != cudaSuccess) return e;
  // four rows a warp; the sums are made in every CTA, so no more CTAs than four an SM
  long long grid = (static_cast<long long>(a.max_rows) + 31) / 32;
  const long long by_entries = (static_cast<long long>(a.max_entries) + kPlanThreads - 1) / kPlanThreads;
  grid = grid > by_entries ? grid : by_entries;
  grid = grid < 1 ? 1 : (grid > 4LL * ctx.num_sms ? 4LL * ctx.num_sms : grid);
  return launch_pdl(batch_plan_kernel, dim3(static_cast<unsigned>(grid)), dim3(kPlanThreads), smem, st, p);
}

}  // namespace csa2
