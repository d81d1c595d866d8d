// lla_page_plan.cu — block tables and slot maps built on the GPU from request lengths
// (lla_page_plan): what the paged encode, the 4-bit store and the paged decode calls of a
// step take, made without the host seeing a length ("Enabling dynamic computation in
// Looped LMs", App. A.1: a logical-to-physical page table per sequence).
//
// One launch.  Every block scans all B requests by itself (a few KB from L2, a few
// microseconds), so no block waits for another, and then writes its own stretch of the
// token maps and its own requests' table rows; a slot never depends on a table entry
// that this call writes, because pages taken now are read from the free list.
#include <algorithm>
#include <atomic>

#include "lla_kernels.h"

using namespace lla;

namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanMaxB = 8192;        // requests of a plan (shared memory: 16 bytes each)
constexpr int kTokPerThread = 8;

struct PlanArgs {
  int B, page_size, max_pages, n_free, n_tok;
  int64_t num_pages;
  const int32_t* ctx;
  const int32_t* fresh;
  const int32_t* free_pages;
  const int32_t* free_head;
  int32_t* table;
  int32_t* seq_lens;
  int32_t* tok_start;
  int32_t* granted;
  int32_t* seq_idx;
  int32_t* pos;
  int64_t* slots;
  int32_t* counts;
  uint32_t* status;
};

// Inclusive block scan of one pair of 64-bit sums.
__device__ __forceinline__ void block_scan(int64_t& a, int64_t& b, int64_t (*tot)[2]) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t ua = __shfl_up_sync(0xffffffffu, a, o), ub = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) { a += ua; b += ub; }
  }
  if (lane == 31) { tot[w][0] = a; tot[w][1] = b; }
  __syncthreads();
  int64_t pa = 0, pb = 0;
  for (int i = 0; i < w; ++i) { pa += tot[i][0]; pb += tot[i][1]; }
  a += pa;
  b += pb;
  __syncthreads();
}

__device__ __forceinline__ int64_t pages_of(int64_t tokens, int P) { return (tokens + P - 1) / P; }

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const __grid_constant__ PlanArgs a) {
  // per request: first token (requested), cached length, first page taken, 1 if granted
  extern __shared__ int32_t sh[];
  int32_t* start = sh;
  int32_t* len0 = sh + a.B;
  int32_t* page0 = sh + 2 * a.B;
  int32_t* ok = sh + 3 * a.B;
  __shared__ int64_t tot[kPlanThreads / 32][2];
  const int tid = threadIdx.x;
  const bool first = blockIdx.x == 0;
  int64_t head = a.free_head ? static_cast<int64_t>(__ldg(a.free_head)) : 0;
  if (head < 0 || head > a.n_free) {
    if (first && tid == 0) record_status(a.status, LLA_ERR_DEVICE_ARG);
    head = a.n_free;   // nothing to take
  }
  const int64_t avail = a.n_free - head;
  const int64_t cap = static_cast<int64_t>(a.max_pages) * a.page_size;
  // a thread's requests: a contiguous stretch, so that one block scan serves them all
  const int per = (a.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  int64_t toks = 0;
  for (int b = b0; b < b1; ++b) {
    const int c = __ldg(a.ctx + b), n = __ldg(a.fresh + b);
    if ((c < 0 || n < 0) && first) record_status(a.status, LLA_ERR_DEVICE_ARG);
    toks += max(n, 0);
  }
  int64_t tok_end = toks, zero = 0;
  block_scan(tok_end, zero, tot);
  // pages: a request that cannot hold its tokens (table too short, maps too short) takes none
  int64_t need_sum = 0;
  int64_t t = tok_end - toks;
  for (int b = b0; b < b1; ++b) {
    const int64_t c = max(__ldg(a.ctx + b), 0), n = max(__ldg(a.fresh + b), 0);
    t += n;
    if (c + n <= cap && t <= a.n_tok) need_sum += pages_of(c + n, a.page_size) - pages_of(c, a.page_size);
  }
  int64_t page_end = need_sum;
  zero = 0;
  block_scan(page_end, zero, tot);
  int64_t taken = 0, live = 0;
  t = tok_end - toks;
  int64_t pg = page_end - need_sum;
  for (int b = b0; b < b1; ++b) {
    const int64_t c = max(__ldg(a.ctx + b), 0), n = max(__ldg(a.fresh + b), 0);
    const bool fits = c + n <= cap && t + n <= a.n_tok;
    const int64_t need = fits ? pages_of(c + n, a.page_size) - pages_of(c, a.page_size) : 0;
    // the free list serves requests in order: the first that it cannot fill ends it for
    // every later one that needs a page
    const bool g = fits && (need == 0 || pg + need <= avail);
    start[b] = static_cast<int32_t>(min(t, static_cast<int64_t>(INT32_MAX)));
    len0[b] = static_cast<int32_t>(c);
    page0[b] = static_cast<int32_t>(min(head + pg, static_cast<int64_t>(INT32_MAX)));
    ok[b] = g ? 1 : 0;
    if (first) {
      a.seq_lens[b] = static_cast<int32_t>(g ? c + n : c);
      a.tok_start[b] = start[b];
      a.granted[b] = g ? 1 : 0;
    }
    if (g) { taken += need; live += n; }
    t += n;
    pg += need;
  }
  if (first) {
    if (tid == kPlanThreads - 1) a.tok_start[a.B] = static_cast<int32_t>(min(tok_end, static_cast<int64_t>(INT32_MAX)));
    block_scan(taken, live, tot);
    if (tid == kPlanThreads - 1) {
      a.counts[0] = static_cast<int32_t>(head + taken);
      a.counts[1] = static_cast<int32_t>(live);
    }
  }
  __syncthreads();

  // ---- table rows: one warp per request, its new pages in order off the free list
  const int warps = kPlanThreads / 32, lane = tid & 31;
  for (int b = blockIdx.x * warps + (tid >> 5); b < a.B; b += gridDim.x * warps) {
    if (!ok[b]) continue;
    const int64_t c = len0[b], n = max(__ldg(a.fresh + b), 0);
    const int held = static_cast<int>(pages_of(c, a.page_size)), need = static_cast<int>(pages_of(c + n, a.page_size)) - held;
    for (int i = lane; i < need; i += 32) {
      const int p = __ldg(a.free_pages + page0[b] + i);
      if (p < 0 || p >= a.num_pages) record_status(a.status, LLA_ERR_DEVICE_ARG);
      a.table[static_cast<int64_t>(b) * a.max_pages + held + i] = p;
    }
  }

  // ---- token maps: entry i belongs to the last request that starts at or before it
  const int64_t total = min(tok_end, static_cast<int64_t>(INT32_MAX));   // of the last thread only: broadcast
  __shared__ int64_t all;
  if (tid == kPlanThreads - 1) all = total;
  __syncthreads();
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kPlanThreads * kTokPerThread;
#pragma unroll 1
  for (int k = 0; k < kTokPerThread; ++k) {
    const int64_t i = i0 + k * kPlanThreads + tid;
    if (i >= a.n_tok) break;
    int sb = -1, sp = -1;
    int64_t slot = -1;
    if (i < all) {
      int lo = 0, hi = a.B;   // the last b with start[b] <= i
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= i) lo = mid;
        else hi = mid;
      }
      if (ok[lo]) {
        const int p = len0[lo] + static_cast<int>(i - start[lo]);
        const int lp = p / a.page_size;
        const int held = static_cast<int>(pages_of(len0[lo], a.page_size));
        const int page = lp < held ? __ldg(a.table + static_cast<int64_t>(lo) * a.max_pages + lp)
                                   : __ldg(a.free_pages + page0[lo] + lp - held);
        sb = lo;
        sp = p;
        if (page < 0 || page >= a.num_pages) record_status(a.status, LLA_ERR_DEVICE_ARG);
        else slot = static_cast<int64_t>(page) * a.page_size + (p - lp * a.page_size);
      }
    }
    a.seq_idx[i] = sb;
    a.pos[i] = sp;
    a.slots[i] = slot;
  }
}

}  // namespace

extern "C" lla_status lla_page_plan(int B, int page_size, int max_pages, int64_t num_pages, const int32_t* ctx_lens,
                                    const int32_t* new_lens, const int32_t* free_pages, int n_free,
                                    const int32_t* free_head, int32_t* block_table, int32_t* seq_lens,
                                    int32_t* tok_start, int32_t* granted, int n_tok, int32_t* seq_idx, int32_t* pos,
                                    int64_t* slots, int32_t* counts, void* workspace, size_t ws_bytes, void* stream) {
  if (B < 0 || page_size < 1 || max_pages < 1 || num_pages < 1 || n_free < 0 || n_tok < 0) return LLA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(max_pages) * page_size > (int64_t(1) << 30) || num_pages >= (int64_t(1) << 31) ||
      static_cast<int64_t>(B) * max_pages >= (int64_t(1) << 31) || B > kPlanMaxB)
    return LLA_ERR_UNSUPPORTED;
  if (ws_bytes < 256 || !workspace || !counts || !tok_start) return LLA_ERR_INVALID_ARG;
  if (B > 0 && (!ctx_lens || !new_lens || !block_table || !seq_lens || !granted)) return LLA_ERR_INVALID_ARG;
  if (n_tok > 0 && (!seq_idx || !pos || !slots)) return LLA_ERR_INVALID_ARG;
  if (n_free > 0 && !free_pages) return LLA_ERR_INVALID_ARG;
  const void* words[] = {ctx_lens, new_lens, free_pages, free_head, block_table, seq_lens, tok_start, granted, seq_idx,
                         pos, counts, workspace};
  for (const void* p : words)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return LLA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(slots) & 7u) return LLA_ERR_INVALID_ARG;
  // every block reads the lengths and the list while others write: no output may be an input
  struct Range { const void* p; int64_t bytes; };
  const int64_t b4 = static_cast<int64_t>(B) * 4, t4 = static_cast<int64_t>(n_tok) * 4;
  const Range in[] = {{ctx_lens, b4}, {new_lens, b4}, {free_pages, static_cast<int64_t>(n_free) * 4}, {free_head, 4}};
  const Range out[] = {{block_table, b4 * max_pages}, {seq_lens, b4}, {tok_start, b4 + 4}, {granted, b4}, {seq_idx, t4},
                       {pos, t4}, {slots, 2 * t4}, {counts, 8}};
  for (const Range& o : out)
    for (const Range& i : in) {
      const uintptr_t x = reinterpret_cast<uintptr_t>(i.p), y = reinterpret_cast<uintptr_t>(o.p);
      if (x && y && x < y + o.bytes && y < x + i.bytes) return LLA_ERR_INVALID_ARG;
    }
  PlanArgs a{B, page_size, max_pages, n_free, n_tok, num_pages, ctx_lens, new_lens, free_pages, free_head, block_table,
             seq_lens, tok_start, granted, seq_idx, pos, slots, counts, static_cast<uint32_t*>(workspace)};
  const size_t smem = static_cast<size_t>(B) * 16;
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPlanMaxB * 16) != cudaSuccess)
    return LLA_ERR_CUDA;
  const int64_t tok_blocks = (static_cast<int64_t>(n_tok) + kPlanThreads * kTokPerThread - 1) / (kPlanThreads * kTokPerThread);
  const unsigned blocks = static_cast<unsigned>(std::max<int64_t>(1, tok_blocks));
  page_plan_kernel<<<blocks, kPlanThreads, smem, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? LLA_OK : LLA_ERR_CUDA;
}
