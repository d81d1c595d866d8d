// lla_page_plan.cu — block tables and slot maps built on the GPU from request lengths
// (lla_page_plan): what the paged encode, the 4-bit store and the paged decode calls of a
// step take, made without the host seeing a length ("Enabling dynamic computation in
// Looped LMs", App. A.1: a logical-to-physical page table per sequence).
//
// One launch.  Every block scans all B requests by itself (a few KB from L2, held in shared
// memory), so no block waits for another, and then writes its own stretch of the token maps and of
// the new table entries, each found by a binary search of the scan; a slot never depends on a
// table entry that this call writes, because pages taken now are read from the free list.
// Latency-bound: the lengths are read once, the rest runs out of shared memory.
#include <algorithm>

#include "lla_kernels.h"

using namespace lla;

namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanMaxB = 8192;        // requests of a plan (shared memory: 16 bytes each)

struct PlanArgs {
  int B, max_pages, n_free, n_tok;
  FastDiv page;                      // page size
  int64_t num_pages;
  int per_thread;                    // token entries of a thread
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

// (lengths are below 2^31: 64-bit divisions took a tenth of the kernel's time)
__device__ __forceinline__ int pages_of(int tokens, const FastDiv& P) {
  const uint32_t whole = P.div(static_cast<uint32_t>(tokens));
  return static_cast<int>(whole + (whole * P.d != static_cast<uint32_t>(tokens)));
}

// The last of n ascending starts that is at or before i (starts[0] <= i).
__device__ __forceinline__ int owner(const int32_t* starts, int n, int64_t i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int32_t clamp32(int64_t x) { return static_cast<int32_t>(min(x, static_cast<int64_t>(INT32_MAX))); }

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const __grid_constant__ PlanArgs a) {
  // per request: first token (requested), cached length, first page taken (counted from the list's
  // head), tokens brought; -1 - tokens where it is not granted
  extern __shared__ int32_t sh[];
  int32_t* start = sh;
  int32_t* len0 = sh + a.B;
  int32_t* page0 = sh + 2 * a.B;
  int32_t* fresh = sh + 3 * a.B;
  __shared__ int64_t tot[kPlanThreads / 32][2];
  __shared__ int64_t total[2];           // tokens requested, pages taken
  const int tid = threadIdx.x, P = static_cast<int>(a.page.d);
  const bool first = blockIdx.x == 0;
  int64_t head = a.free_head ? static_cast<int64_t>(__ldg(a.free_head)) : 0;
  if (head < 0 || head > a.n_free) {
    if (first && tid == 0) record_status(a.status, LLA_ERR_DEVICE_ARG);
    head = a.n_free;   // nothing to take
  }
  const int64_t avail = a.n_free - head;
  const int64_t cap = static_cast<int64_t>(a.max_pages) * P;
  for (int b = tid; b < a.B; b += kPlanThreads) {
    const int c = __ldg(a.ctx + b), n = __ldg(a.fresh + b);
    if ((c < 0 || n < 0) && first) record_status(a.status, LLA_ERR_DEVICE_ARG);
    len0[b] = max(c, 0);
    fresh[b] = max(n, 0);
  }
  __syncthreads();
  // a thread's requests: a contiguous stretch, so that one block scan serves them all
  const int per = (a.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  int64_t toks = 0, zero = 0;
  for (int b = b0; b < b1; ++b) toks += fresh[b];
  int64_t tok_end = toks;
  block_scan(tok_end, zero, tot);
  // pages: a request that cannot hold its tokens (table too short, maps too short) takes none
  auto fits = [&](int64_t c, int64_t n, int64_t before) { return c + n <= cap && before + n <= a.n_tok; };
  auto need_of = [&](int64_t c, int64_t n) {   // (fits: below 2^30)
    return pages_of(static_cast<int>(c + n), a.page) - pages_of(static_cast<int>(c), a.page);
  };
  int64_t need_sum = 0, t = tok_end - toks;
  for (int b = b0; b < b1; ++b) {
    const int64_t c = len0[b], n = fresh[b];
    if (fits(c, n, t)) need_sum += need_of(c, n);
    t += n;
  }
  int64_t page_end = need_sum;
  zero = 0;
  block_scan(page_end, zero, tot);
  int64_t taken = 0, live = 0, pg = page_end - need_sum;
  t = tok_end - toks;
  for (int b = b0; b < b1; ++b) {
    const int64_t c = len0[b], n = fresh[b];
    const bool f = fits(c, n, t);
    const int64_t need = f ? need_of(c, n) : 0;
    // the free list serves requests in order: the first that it cannot fill ends it for
    // every later one that needs a page
    const bool g = f && (need == 0 || pg + need <= avail);
    start[b] = clamp32(t);
    page0[b] = clamp32(pg);
    if (!g) fresh[b] = -1 - static_cast<int32_t>(n);
    if (first) {
      a.seq_lens[b] = static_cast<int32_t>(g ? c + n : c);
      a.tok_start[b] = start[b];
      a.granted[b] = g ? 1 : 0;
    }
    if (g) { taken += need; live += n; }
    t += n;
    pg += need;
  }
  block_scan(taken, live, tot);
  if (tid == kPlanThreads - 1) {
    total[0] = tok_end;
    total[1] = taken;
    if (first) {
      a.tok_start[a.B] = clamp32(tok_end);
      a.counts[0] = static_cast<int32_t>(head + taken);
      a.counts[1] = static_cast<int32_t>(live);
    }
  }
  __syncthreads();

  // ---- new table entries: page k of those taken belongs to the last request that starts at or before it
  // (the granted requests that take pages come before every other that needs one)
  for (int64_t k = static_cast<int64_t>(blockIdx.x) * kPlanThreads + tid; k < total[1]; k += static_cast<int64_t>(gridDim.x) * kPlanThreads) {
    const int b = owner(page0, a.B, k), p = __ldg(a.free_pages + head + k);
    if (p < 0 || p >= a.num_pages) record_status(a.status, LLA_ERR_DEVICE_ARG);
    a.table[static_cast<int64_t>(b) * a.max_pages + pages_of(len0[b], a.page) + (k - page0[b])] = p;
  }

  // ---- token maps
  int64_t i = static_cast<int64_t>(blockIdx.x) * kPlanThreads * a.per_thread + tid;
#pragma unroll 1
  for (int k = 0; k < a.per_thread && i < a.n_tok; ++k, i += kPlanThreads) {
    int sb = -1, sp = -1;
    int64_t slot = -1;
    if (i < total[0]) {
      const int b = owner(start, a.B, i);
      if (fresh[b] >= 0) {
        const int p = len0[b] + static_cast<int>(i - start[b]), lp = static_cast<int>(a.page.div(static_cast<uint32_t>(p)));
        const int held = pages_of(len0[b], a.page);
        const int page = lp < held ? __ldg(a.table + static_cast<int64_t>(b) * a.max_pages + lp)
                                   : __ldg(a.free_pages + head + page0[b] + lp - held);
        sb = b;
        sp = p;
        if (page < 0 || page >= a.num_pages) record_status(a.status, LLA_ERR_DEVICE_ARG);
        else slot = static_cast<int64_t>(page) * P + (p - lp * P);
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
  const int sms = device_sm_count();
  if (sms <= 0) return LLA_ERR_CUDA;
  // two blocks per SM at most: each repeats the scan
  const int64_t stretch = static_cast<int64_t>(kPlanThreads) * 2 * sms;
  PlanArgs a{B, max_pages, n_free, n_tok, FastDiv(page_size), num_pages, static_cast<int>((n_tok + stretch - 1) / stretch), ctx_lens,
             new_lens, free_pages, free_head, block_table, seq_lens, tok_start, granted, seq_idx, pos, slots, counts,
             static_cast<uint32_t*>(workspace)};
  a.per_thread = std::max(a.per_thread, 1);
  const size_t smem = static_cast<size_t>(B) * 16;
  // (the most any call takes, at every call: what needs no opt-in is 48 KB less the kernel's static part)
  if (cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPlanMaxB * 16) != cudaSuccess)
    return LLA_ERR_CUDA;
  const int64_t per_block = static_cast<int64_t>(kPlanThreads) * a.per_thread;
  const unsigned blocks = static_cast<unsigned>(std::max<int64_t>(1, (n_tok + per_block - 1) / per_block));
  page_plan_kernel<<<blocks, kPlanThreads, smem, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? LLA_OK : LLA_ERR_CUDA;
}
