// plan.cu — the step plan of a batch over a paged cache, from its request
// lengths: block table entries for the new pages, and for every new token its
// position, its sequence and its row of the page pool.
//
//   cu[b]   = sum_{i < b} new[i]                       (packed token offsets)
//   have[b] = ceil(cached[b] / page),  need[b] = ceil((cached[b] + new[b]) / page)
//   table[b, have[b] + j] = free[first[b] + j],  j < need[b] - have[b],
//   first[b] = sum_{i < b} (need[i] - have[i])
//   token t of sequence b (cu[b] <= t < cu[b+1]): position p = cached[b] + t - cu[b],
//   slot = table[b, p / page] * page + p % page
//
// One launch. The work is a prefix sum over the requests, then 16 bytes a token:
// a few microseconds of latency, not bandwidth (65536 tokens write 1 MB; 64 single-token requests
// take 8.3 us, 999 mixed ones 10.4). A second
// launch for the token rows would cost more than the scan, so every block scans
// all requests by itself (kChunk at a time, from L2) and fills its own token
// range. No block reads what another one writes: the page of a new token is read
// from the free list, and the token in the first row of a new page writes that
// page's table entry.
#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace gmla {

namespace {

constexpr int kPlanThreads = 256;
constexpr int kPlanItems = 16;                            // requests a thread scans per chunk, at most
constexpr int kChunk = kPlanThreads * kPlanItems;         // requests per chunk
constexpr int kPlanTok = 4;                               // token rows a thread fills at a time (16-byte stores)

struct Pair {
  long long tok, page;
};

// Exclusive prefix sums of (tok, page) over the block; *total gets the sums.
__device__ __forceinline__ Pair block_scan2(Pair v, Pair* s_warp, Pair* s_total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  Pair inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, inc.tok, o), b = __shfl_up_sync(0xffffffffu, inc.page, o);
    if (lane >= o) {
      inc.tok += a;
      inc.page += b;
    }
  }
  if (lane == 31) s_warp[w] = inc;
  __syncthreads();
  Pair r{inc.tok - v.tok, inc.page - v.page};
  Pair t{0, 0};
#pragma unroll
  for (int i = 0; i < kPlanThreads / 32; ++i) {
    const Pair x = s_warp[i];
    if (i < w) {
      r.tok += x.tok;
      r.page += x.page;
    }
    t.tok += x.tok;
    t.page += x.page;
  }
  *s_total = t;
  __syncthreads();
  return r;
}

// a / page and its ceiling (no overflow near 2^31); page sizes are mostly powers of two
__device__ __forceinline__ int page_of(const PlanArgs& a, int x) { return a.page_shift >= 0 ? x >> a.page_shift : x / a.page; }
__device__ __forceinline__ int pages_for(const PlanArgs& a, int x) {
  const int q = page_of(a, x);
  return q + (x != q * a.page);
}

}  // namespace

__global__ void __launch_bounds__(kPlanThreads) plan_batch_kernel(PlanArgs a) {
  __shared__ int s_cu[kChunk + 1];       // packed token offset of each request of the chunk
  __shared__ int s_first[kChunk];        // its first free page
  __shared__ Pair s_warp[kPlanThreads / 32], s_total;
  __shared__ int s_bad;
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  const long long limit = static_cast<long long>(a.max_pages) * a.page;
  if (tid == 0) s_bad = 0;
  __syncthreads();

  const int n_chunk = (a.B + kChunk - 1) / kChunk;
  // tokens and pages of request b; a length that cannot be is a fault of the whole plan
  auto request = [&](int b, bool& bad) {
    const int c = a.cached[b], n = a.fresh[b];
    if (c < 0 || n < 0 || static_cast<long long>(c) + n > limit) {
      bad = true;
      return Pair{0, 0};
    }
    return Pair{n, pages_for(a, c + n) - pages_for(a, c)};
  };
  Pair total{0, 0};
  if (n_chunk > 1) {   // the sums of the whole batch come first: nothing is written for a batch that does not fit
    bool bad = false;
    Pair v{0, 0};
    for (int b = tid; b < a.B; b += kPlanThreads) {
      const Pair r = request(b, bad);
      v.tok += r.tok;
      v.page += r.page;
    }
    if (bad) s_bad = 1;
    block_scan2(v, s_warp, &s_total);
    total = s_total;
    __syncthreads();
  }
  Pair carry{0, 0};
  for (int chunk = 0; chunk < n_chunk || chunk == 0; ++chunk) {
    const int base = chunk * kChunk;
    const int n = max(0, min(kChunk, a.B - base));
    const int items = (n + kPlanThreads - 1) / kPlanThreads;
    {
      bool bad = false;
      Pair sum{0, 0}, only{0, 0};
      for (int i = 0; i < items; ++i) {
        const int k = tid * items + i;
        if (k < n) {
          const Pair r = request(base + k, bad);
          only = r;
          sum.tok += r.tok;
          sum.page += r.page;
        }
      }
      if (bad) s_bad = 1;
      Pair at = block_scan2(sum, s_warp, &s_total);
      at.tok += carry.tok;
      at.page += carry.page;
      if (n_chunk <= 1) total = s_total;
      for (int i = 0; i < items; ++i) {
        const int k = tid * items + i;
        if (k < n) {
          s_cu[k] = static_cast<int>(at.tok);
          s_first[k] = static_cast<int>(at.page);
          const Pair r = items == 1 ? only : request(base + k, bad);
          at.tok += r.tok;
          at.page += r.page;
        }
      }
      carry.tok += s_total.tok;
      carry.page += s_total.page;
      if (tid == 0) s_cu[n] = static_cast<int>(carry.tok);
    }
    __syncthreads();
    const bool ok = !s_bad && total.tok <= a.T && total.page <= a.n_free;
    if (!ok && blockIdx.x == 0 && tid == 0) report_status(a.status, kStatusRange);
    if (blockIdx.x == 0) {
      for (int k = tid; k < n; k += kPlanThreads) {
        a.seq_lens[base + k] = ok ? a.cached[base + k] + a.fresh[base + k] : 0;
        a.cu[base + k] = ok ? s_cu[k] : 0;
      }
      if (tid == 0 && chunk == max(n_chunk, 1) - 1) {
        a.cu[a.B] = ok ? static_cast<int>(total.tok) : 0;
        a.pages_used[0] = ok ? static_cast<int>(total.page) : 0;
      }
    }
    // token rows [lo, hi) belong to this chunk; the last chunk also marks the rows behind the last sequence
    const bool last = chunk >= n_chunk - 1;
    const int lo = ok ? (n > 0 ? s_cu[0] : 0) : 0;
    const int live = ok ? (n > 0 ? s_cu[n] : 0) : 0;
    const int hi = last ? a.T : live;
    const int q0 = lo / kPlanTok, q1 = (hi + kPlanTok - 1) / kPlanTok;
    for (int q = q0 + blockIdx.x * kPlanThreads + tid; q < q1; q += gridDim.x * kPlanThreads) {
      int pos[kPlanTok], seq[kPlanTok];
      long long slot[kPlanTok];
      int k = -1, b = 0, cached = 0, have = 0;
#pragma unroll
      for (int i = 0; i < kPlanTok; ++i) {
        const int t = q * kPlanTok + i;
        pos[i] = seq[i] = -1;
        slot[i] = -1;
        if (t < lo || t >= live) continue;
        if (k < 0 || t >= s_cu[k + 1]) {   // the last request whose offset is not above t (it has tokens)
          int x = max(k, 0), y = n;
          while (y - x > 1) {
            const int m = (x + y) >> 1;
            if (s_cu[m] <= t)
              x = m;
            else
              y = m;
          }
          k = x;
          b = base + k;
          cached = a.cached[b];
          have = pages_for(a, cached);
        }
        const int p = cached + (t - s_cu[k]);
        const int pi = page_of(a, p), off = p - pi * a.page;
        int* entry = a.table + static_cast<int64_t>(b) * a.max_pages + pi;
        int page;
        if (pi >= have) {
          page = a.free_pages[s_first[k] + (pi - have)];
          if (off == 0) *entry = page;
        } else {
          page = *entry;
        }
        if (page < 0) report_status(a.status, kStatusRange);
        pos[i] = p;
        seq[i] = b;
        slot[i] = page < 0 ? -1 : static_cast<long long>(page) * a.page + off;
      }
      const int t = q * kPlanTok;
      if (t >= lo && t + kPlanTok <= hi) {
        reinterpret_cast<int4*>(a.positions)[q] = make_int4(pos[0], pos[1], pos[2], pos[3]);
        reinterpret_cast<int4*>(a.seq_ids)[q] = make_int4(seq[0], seq[1], seq[2], seq[3]);
        reinterpret_cast<longlong2*>(a.slots)[2 * q] = make_longlong2(slot[0], slot[1]);
        reinterpret_cast<longlong2*>(a.slots)[2 * q + 1] = make_longlong2(slot[2], slot[3]);
      } else {
#pragma unroll
        for (int i = 0; i < kPlanTok; ++i)
          if (t + i >= lo && t + i < hi) {
            a.positions[t + i] = pos[i];
            a.seq_ids[t + i] = seq[i];
            a.slots[t + i] = slot[i];
          }
      }
    }
    __syncthreads();   // the next chunk overwrites the offsets
  }
}

cudaError_t launch_plan_batch(PlanArgs a, int num_sms, cudaStream_t st) {
  a.page_shift = -1;
  if ((a.page & (a.page - 1)) == 0)
    for (a.page_shift = 0; (1 << a.page_shift) < a.page;) ++a.page_shift;
  const int per_block = kPlanThreads * kPlanTok;
  int grid = (a.T + per_block - 1) / per_block;
  grid = grid < 1 ? 1 : (grid > 4 * num_sms ? 4 * num_sms : grid);
  prof_begin(st, "plan_batch");
  cudaError_t e = launch_pdl(plan_batch_kernel, dim3(grid), dim3(kPlanThreads), 0, st, 1, a);
  prof_end(st);
  return e;
}

}  // namespace gmla
