// One serving step's bookkeeping on the GPU: block tables, slot mappings,
// positions and query offsets from the requests' lengths (kvq_plan_step).
//
// Request s holds old_s tokens in ceil(old_s / bs) pages and brings new_s more.
// With cu_s = sum_{i<s} new_i and fresh_s = ceil((old_s + new_s) / bs) -
// ceil(old_s / bs), page j >= ceil(old_s / bs) of request s takes free block
// number sum_{i<s} fresh_i + j - ceil(old_s / bs), and new token t of the
// packed batch belongs to the request with cu_s <= t < cu_{s+1}, at position
// old_s + t - cu_s.
//
// Every quantity is a prefix sum over the requests plus a search, so one launch
// does it all: each CTA scans all requests itself (kThreads at a time, two
// sums a warp shuffle tree wide) instead of waiting for another CTA's scan, and
// writes its own run of tokens and its share of the fresh pages.  A token whose
// page is fresh reads the block from the free list, not from the table, so no
// CTA reads what another writes.  Latency-bound: the scan's two barriers and
// three dependent loads (lengths, table or free list) set the time of a decode
// step (64 requests of one token: 4.5 us on the GPU); a large step adds 12 bytes
// written per token (256 requests with 521,000 tokens: 9.5 us).
#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {

KVQ_ERROR_ACCESSOR(take_error_bits_plan)

namespace {

constexpr int kThreads = 512;  // requests scanned at a time
constexpr int kRun = 4;        // consecutive tokens per thread (one 16-byte store of positions)
constexpr int kWarps = kThreads / 32;

struct Chunk {            // one scanned chunk of requests, in shared memory
  int cu[kThreads + 1];   // first token of each request (cu[kThreads]: behind the last)
  int page[kThreads + 1]; // first fresh page of each request, counted over all requests
  int old[kThreads];
};

// The entry of v[0..kThreads] (non-decreasing) that holds x: the largest i with
// v[i] <= x, given v[0] <= x < v[kThreads].
__device__ __forceinline__ int holder(const int* v, int x) {
  int lo = 0;
#pragma unroll
  for (int step = kThreads / 2; step >= 1; step >>= 1)
    if (v[lo + step] <= x) lo += step;
  return lo;
}

__global__ void __launch_bounds__(kThreads) plan_step_kernel(const PlanArgs a) {
  __shared__ Chunk ch;
  __shared__ long long sums[2][kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bs = 1 << a.block_shift;
  const long long cap = static_cast<long long>(a.max_blocks_per_seq) << a.block_shift;
  // the usable part of the free list
  const int f0 = a.free_range[0], f1 = a.free_range[1];
  const int first = min(max(f0, 0), a.free_capacity);
  const int avail = max(min(f1, a.free_capacity), first) - first;  // no difference that could wrap: f1 is any int
  unsigned err = (f0 != first || f1 > a.free_capacity || f1 < f0) ? 128u : 0u;  // KVQ_DEVERR_FREE_BLOCKS

  const long long t0 = (static_cast<long long>(blockIdx.x) * kThreads + tid) * kRun;  // this thread's tokens
  const long long run0 = static_cast<long long>(blockIdx.x) * kThreads * kRun;  // this CTA's
  int pos[kRun];
  long long slot[kRun];
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    pos[i] = 0;
    slot[i] = -1;
  }

  // block id of fresh page number f (counted over all requests), or -1
  auto fresh_block = [&](int f) {
    if (f >= avail) {
      err |= 128u;
      return -1;
    }
    const int b = a.free_blocks[first + f];
    if (b >= 0 && b < a.num_blocks) return b;
    err |= 2u;  // KVQ_DEVERR_BLOCK_RANGE
    return -1;
  };

  long long tokens = 0, pages = 0;  // of the chunks before
  for (int base = 0; base < a.num_seqs; base += kThreads) {
    const int s = base + tid;
    int old = 0, add = 0, have = 0, fresh = 0;
    if (s < a.num_seqs) {
      const int o = a.context_lens[s], n = a.new_lens[s];
      old = static_cast<int>(min(static_cast<long long>(max(o, 0)), cap));
      add = static_cast<int>(min(static_cast<long long>(max(n, 0)), cap - old));
      if (old != o || add != n) err |= 4u;  // KVQ_DEVERR_CONTEXT_RANGE
      have = (old + bs - 1) >> a.block_shift;  // cap <= 2^30 (checked on the host): no overflow
      fresh = ((old + add + bs - 1) >> a.block_shift) - have;
    }
    // inclusive sums over the chunk
    long long ti = add, pi = fresh;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, ti, o), y = __shfl_up_sync(0xffffffffu, pi, o);
      if (lane >= o) {
        ti += x;
        pi += y;
      }
    }
    if (lane == 31) {
      sums[0][warp] = ti;
      sums[1][warp] = pi;
    }
    __syncthreads();
    long long tb = tokens, pb = pages, tt = tokens, pp = pages;
    for (int w = 0; w < kWarps; ++w) {
      const long long x = sums[0][w], y = sums[1][w];
      if (w < warp) {
        tb += x;
        pb += y;
      }
      tt += x;
      pp += y;
    }
    // counts past 2^31 - 1 saturate: the batch is refused below (too many tokens)
    auto clip = [](long long x) { return static_cast<int>(min(x, 0x7fffffffll)); };
    const int cu = clip(tb + ti - add), pg = clip(pb + pi - fresh);
    ch.cu[tid] = cu;
    ch.page[tid] = pg;
    ch.old[tid] = old;
    if (tid == kThreads - 1) {
      ch.cu[kThreads] = clip(tt);
      ch.page[kThreads] = clip(pp);
    }
    __syncthreads();
    if (s < a.num_seqs && (base / kThreads) % gridDim.x == blockIdx.x) {
      a.context_lens_out[s] = old + add;
      a.cu_new[s] = cu;
    }
    // this CTA's share of the chunk's fresh pages
    for (long long f = pages + static_cast<long long>(blockIdx.x) * kThreads + tid; f < ch.page[kThreads];
         f += static_cast<long long>(gridDim.x) * kThreads) {
      const int i = holder(ch.page, static_cast<int>(f));
      const int j = ((ch.old[i] + bs - 1) >> a.block_shift) + static_cast<int>(f) - ch.page[i];
      a.block_table[static_cast<size_t>(base + i) * a.max_blocks_per_seq + j] = fresh_block(static_cast<int>(f));
    }
    // this thread's tokens that fall in the chunk
    const long long lo = max(t0, static_cast<long long>(ch.cu[0]));
    const long long hi = min(min(t0 + kRun, a.max_tokens), static_cast<long long>(ch.cu[kThreads]));
    if (lo < hi) {
      int i = holder(ch.cu, static_cast<int>(lo));
      int at_page = -1, at_seq = -1, blk = -1;
#pragma unroll
      for (int u = 0; u < kRun; ++u) {
        const long long t = t0 + u;
        if (t < lo || t >= hi) continue;
        while (ch.cu[i + 1] <= t) ++i;  // t < cu[kThreads]: ends
        const int p = ch.old[i] + static_cast<int>(t) - ch.cu[i];
        const int page = p >> a.block_shift, held = (ch.old[i] + bs - 1) >> a.block_shift;
        if (page != at_page || i != at_seq) {
          at_page = page;
          at_seq = i;
          if (page >= held) {
            blk = fresh_block(ch.page[i] + page - held);
          } else {
            blk = a.block_table[static_cast<size_t>(base + i) * a.max_blocks_per_seq + page];
            if (blk < 0 || blk >= a.num_blocks) {
              err |= 2u;
              blk = -1;
            }
          }
        }
        pos[u] = p;
        slot[u] = blk < 0 ? -1 : (static_cast<long long>(blk) << a.block_shift) + (p & (bs - 1));
      }
    }
    tokens = tt;
    pages = pp;
    __syncthreads();  // the chunk is read before the next one overwrites it
  }

  if (run0 < a.max_tokens) {
    if (t0 + kRun <= a.max_tokens) {  // buffers are 16-byte aligned
      *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      *reinterpret_cast<longlong2*>(a.slot_mapping + t0) = make_longlong2(slot[0], slot[1]);
      *reinterpret_cast<longlong2*>(a.slot_mapping + t0 + 2) = make_longlong2(slot[2], slot[3]);
    } else {
#pragma unroll
      for (int u = 0; u < kRun; ++u)
        if (t0 + u < a.max_tokens) {
          a.positions[t0 + u] = pos[u];
          a.slot_mapping[t0 + u] = slot[u];
        }
    }
  }
  if (blockIdx.x == 0 && tid == 0) {
    if (tokens > a.max_tokens) err |= 256u;  // KVQ_DEVERR_TOKENS
    if (pages > avail) err |= 128u;
    a.cu_new[a.num_seqs] = static_cast<int>(min(tokens, 0x7fffffffll));
    a.free_range_out[0] = first + static_cast<int>(min(pages, static_cast<long long>(avail)));
    a.free_range_out[1] = first + avail;
  }
  if (err) raise_error(err);
}

}  // namespace

cudaError_t launch_plan(const PlanArgs& a, cudaStream_t st) {
  const long long per = kThreads * kRun;
  long long grid = (a.max_tokens + per - 1) / per;
  if (grid < 1) grid = 1;
  plan_step_kernel<<<static_cast<unsigned>(grid), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq
