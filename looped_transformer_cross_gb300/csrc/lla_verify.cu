// lla_verify.cu — what follows the model in a step that verifies drafted tokens: the logits of
// every node under its request's rules (lla_logits_adjust) and the walk down the tree along the
// chosen tokens (lla_tree_accept).
//
// Logits: one pass.  A block takes a slice of the vocabulary of one sequence and up to `group` of
// its nodes: the slice's counts (output part of the history) and prompt marks are made once in
// shared memory, each node adds the tokens on its own path and takes them away again, and only
// stretches of 64 tokens in which anything is counted or biased look at them.  Best token and
// log-sum-exp come out of the same pass, a partial result per (node, slice) that a second launch
// merges in a fixed order.  Memory-bound: each logit is read and written once.
#include <algorithm>

#include "lla_kernels.h"

using namespace lla;

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxNodes = LLA_TREE_MAX_NODES;
constexpr int kSlice = 4096;            // tokens of a slice
constexpr int kLogitThreads = 256;
constexpr int kStretch = 64;            // tokens a warp takes at a time
constexpr int kSteps = kSlice / (kLogitThreads / 32 * kStretch);
constexpr uint32_t kPrompt = 0x80000000u;   // mark of a token of the prompt part; the rest is the count
constexpr int kMaxVocab = 1 << 22;

struct Partial {
  float m, s;      // largest value; sum of exp(x - ref(m))
  int32_t best;    // its lowest index, -1: none
  int32_t pad;
};

struct LogitArgs {
  int B, n_tok, max_nodes, vocab, slices, group;
  const int32_t* tok_start;
  const int32_t* parent;
  const int32_t* token;
  const void* logits;
  void* out;
  int64_t row_stride, out_stride;
  lla_logit_rules r;
  int mask_words;                    // 32-bit words of a mask
  Partial* partials;                 // [n_tok][slices]
  int32_t* best;
  float* lse;
  uint32_t* status;
};

// Nodes of sequence b, or 0 (see lla_tree).
__device__ __forceinline__ int nodes_of(const int32_t* tok_start, int b, int n_tok, int max_nodes, int& first, uint32_t* status) {
  const int s0 = __ldg(tok_start + b), s1 = __ldg(tok_start + b + 1);
  first = s0;
  if (s0 < 0 || s1 < s0 || s1 > n_tok || s1 - s0 > max_nodes) {
    record_status(status, LLA_ERR_DEVICE_ARG);
    return 0;
  }
  return s1 - s0;
}

// The value that a partial sum's exponentials are relative to: its maximum, or 0 where that is
// infinite (so that infinities give sums of 0 and infinity, not NaN).
__device__ __forceinline__ float ref_of(float m) { return fabsf(m) == INFINITY ? 0.f : m; }

// A sum relative to `from`, relative to `to`.
__device__ __forceinline__ float rebase(float s, float from, float to) {
  return s == 0.f ? 0.f : s * exp2f((from - to) * kLog2e);
}

// Maximum, its lowest index and the sum over a warp.
__device__ __forceinline__ void warp_merge(float& m, float& s, int& best) {
  const float mw = warp_max(m);
  s = warp_sum(rebase(s, ref_of(m), ref_of(mw)));
  const uint32_t i = m == mw && best >= 0 ? static_cast<uint32_t>(best) : 0x7FFFFFFFu;
  const uint32_t lo = __reduce_min_sync(0xffffffffu, i);
  best = lo == 0x7FFFFFFFu ? -1 : static_cast<int>(lo);
  m = mw;
}

// Two neighbouring tokens' logits (or, unpaired, tokens 32 apart).
template <typename T, bool kPair>
__device__ __forceinline__ float2 load2(const T* p, int lane, int left) {
  float2 v = make_float2(-INFINITY, -INFINITY);
  if constexpr (kPair) {
    // (a row of an odd vocabulary ends within a pair)
    const int i = 2 * lane;
    if constexpr (sizeof(T) == 2) {
      if (i + 1 < left) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(p + i);
        v = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
      } else if (i < left) {
        v.x = __bfloat162float(p[i]);
      }
    } else {
      if (i + 1 < left) v = *reinterpret_cast<const float2*>(p + i);
      else if (i < left) v.x = p[i];
    }
  } else {
    if constexpr (sizeof(T) == 2) {
      if (lane < left) v.x = __bfloat162float(p[lane]);
      if (lane + 32 < left) v.y = __bfloat162float(p[lane + 32]);
    } else {
      if (lane < left) v.x = p[lane];
      if (lane + 32 < left) v.y = p[lane + 32];
    }
  }
  return v;
}

template <typename T, bool kPair>
__device__ __forceinline__ void store2(T* p, int lane, int left, float2 v) {
  const int i0 = kPair ? 2 * lane : lane, i1 = kPair ? 2 * lane + 1 : lane + 32;
  if constexpr (sizeof(T) == 2) {
    if (kPair && i1 < left) {
      *reinterpret_cast<__nv_bfloat162*>(p + i0) = __floats2bfloat162_rn(v.x, v.y);
    } else {
      if (i0 < left) p[i0] = __float2bfloat16_rn(v.x);
      if (i1 < left) p[i1] = __float2bfloat16_rn(v.y);
    }
  } else {
    if (kPair && i1 < left) {
      *reinterpret_cast<float2*>(p + i0) = v;
    } else {
      if (i0 < left) p[i0] = v.x;
      if (i1 < left) p[i1] = v.y;
    }
  }
}

template <typename T, bool kPair>
__global__ void __launch_bounds__(kLogitThreads) logits_kernel(const __grid_constant__ LogitArgs a) {
  __shared__ uint32_t cnt[kSlice];
  __shared__ float bias[kSlice];
  __shared__ uint32_t touched[kSlice / kStretch];
  __shared__ int32_t tok[kMaxNodes];
  __shared__ int32_t jump[2][kMaxNodes];
  __shared__ uint32_t path[2][kMaxNodes][kMaxNodes / 32];
  __shared__ Partial red[2][kLogitThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / a.slices, slice = blockIdx.x - b * a.slices;
  int first;
  const int n = nodes_of(a.tok_start, b, a.n_tok, a.max_nodes, first, a.status);
  const int row0 = blockIdx.y * a.group;
  if (row0 >= n) return;
  const bool flag = slice == 0 && blockIdx.y == 0;      // the block that reports what it skips
  const int lo = slice * kSlice, width = min(kSlice, a.vocab - lo);

  for (int i = tid; i < kSlice; i += kLogitThreads) { cnt[i] = 0; bias[i] = 0.f; }
  if (tid < kSlice / kStretch) touched[tid] = 0;
  for (int i = tid; i < n; i += kLogitThreads) {
    const int t = __ldg(a.token + first + i);
    int p = __ldg(a.parent + first + i);
    if (p < -1 || p >= i) {
      if (flag) record_status(a.status, LLA_ERR_DEVICE_ARG);
      p = -1;
    }
    if (flag && (t < 0 || t >= a.vocab)) record_status(a.status, LLA_ERR_DEVICE_ARG);
    tok[i] = t;
    jump[0][i] = p;
#pragma unroll
    for (int w = 0; w < kMaxNodes / 32; ++w) path[0][i][w] = i >> 5 == w ? 1u << (i & 31) : 0u;
  }
  __syncthreads();
  // ---- the nodes on each node's path, by pointer doubling
  int cur = 0;
  for (int reach = 1; reach < n; reach *= 2, cur ^= 1) {
    if (tid < n) {
      const int j = jump[cur][tid];
#pragma unroll
      for (int w = 0; w < kMaxNodes / 32; ++w) path[cur ^ 1][tid][w] = path[cur][tid][w] | (j >= 0 ? path[cur][j][w] : 0u);
      jump[cur ^ 1][tid] = j >= 0 ? jump[cur][j] : -1;
    }
    __syncthreads();
  }
  // ---- counts of the history and biases
  if (a.r.max_history > 0) {
    int hl = __ldg(a.r.hist_len + b);
    int pl = a.r.prompt_len ? __ldg(a.r.prompt_len + b) : 0;
    if (hl < 0 || hl > a.r.max_history || pl < 0 || pl > hl) {
      if (flag) record_status(a.status, LLA_ERR_DEVICE_ARG);
      hl = min(max(hl, 0), a.r.max_history);
      pl = min(max(pl, 0), hl);
    }
    const int32_t* hist = a.r.history + static_cast<int64_t>(b) * a.r.max_history;
    for (int i = tid; i < hl; i += kLogitThreads) {
      const int t = __ldg(hist + i);
      if (t >= lo && t < lo + width) {
        if (i < pl) atomicOr(&cnt[t - lo], kPrompt);
        else atomicAdd(&cnt[t - lo], 1u);
        touched[(t - lo) / kStretch] = 1;
      } else if (flag && (t < 0 || t >= a.vocab)) {
        record_status(a.status, LLA_ERR_DEVICE_ARG);
      }
    }
  }
  if (a.r.max_bias > 0) {
    const int32_t* bt = a.r.bias_token + static_cast<int64_t>(b) * a.r.max_bias;
    const float* bv = a.r.bias + static_cast<int64_t>(b) * a.r.max_bias;
    for (int i = tid; i < a.r.max_bias; i += kLogitThreads) {
      const int t = __ldg(bt + i);
      if (t >= lo && t < lo + width) {
        // the first entry of a token adds up all of them, in list order
        bool again = false;
        for (int j = 0; j < i; ++j) again |= __ldg(bt + j) == t;
        if (!again) {
          float sum = __ldg(bv + i);
          for (int j = i + 1; j < a.r.max_bias; ++j)
            if (__ldg(bt + j) == t) sum += __ldg(bv + j);
          bias[t - lo] = sum;
          touched[(t - lo) / kStretch] = 1;
        }
      } else if (flag && t >= a.vocab) {
        record_status(a.status, LLA_ERR_DEVICE_ARG);
      }
    }
  }
  const float rep = a.r.repetition ? __ldg(a.r.repetition + b) : 1.f;
  const float pres = a.r.presence ? __ldg(a.r.presence + b) : 0.f;
  const float freq = a.r.frequency ? __ldg(a.r.frequency + b) : 0.f;

  const int row1 = min(n, row0 + a.group);
  for (int row = row0; row < row1; ++row) {
    // ---- this node's path joins the counts
    auto on_path = [&]() {
      return tid < n && (path[cur][row][tid >> 5] >> (tid & 31) & 1u) && tok[tid] >= lo && tok[tid] < lo + width;
    };
    // (the counts of the history, or the undoing of the node before, may still be under way in
    // other warps: additions commute, and the barrier below comes before any is read)
    if (on_path()) {
      atomicAdd(&cnt[tok[tid] - lo], 1u);
      touched[(tok[tid] - lo) / kStretch] = 1;
    }
    __syncthreads();
    const int64_t at = first + row;
    const T* src = static_cast<const T*>(a.logits) + at * a.row_stride + lo;
    T* dst = a.out ? static_cast<T*>(a.out) + at * a.out_stride + lo : nullptr;
    float2 x[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int g = (k * (kLogitThreads / 32) + warp) * kStretch;
      x[k] = load2<T, kPair>(src + g, lane, width - g);
    }
    const uint32_t* mask = nullptr;
    if (a.r.n_masks > 0) {
      const int mr = __ldg(a.r.allowed_row + at);
      if (mr >= a.r.n_masks) {
        if (slice == 0 && tid == 0) record_status(a.status, LLA_ERR_DEVICE_ARG);
      } else if (mr >= 0) {
        mask = a.r.allowed + static_cast<int64_t>(mr) * a.mask_words + lo / 32;
      }
    }
    float m = -INFINITY;
    int best = -1;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int g = (k * (kLogitThreads / 32) + warp) * kStretch;
      const int i0 = g + (kPair ? 2 * lane : lane), i1 = g + (kPair ? 2 * lane + 1 : lane + 32);
      if (touched[g / kStretch]) {
        float* v = &x[k].x;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = e == 0 ? i0 : i1;
          const uint32_t c = cnt[i];
          // each step rounded by itself, as the formulas are written
          if (c != 0) {
            const uint32_t times = c & ~kPrompt;
            v[e] = v[e] > 0.f ? __fdiv_rn(v[e], rep) : __fmul_rn(v[e], rep);
            v[e] = __fsub_rn(v[e], __fmul_rn(freq, static_cast<float>(times)));
            if (times) v[e] = __fsub_rn(v[e], pres);
          }
          if (a.r.max_bias > 0) v[e] = __fadd_rn(v[e], bias[i]);
        }
      }
      if (mask && g < width) {
        const uint32_t w0 = __ldg(mask + g / 32), w1 = g + 32 < width ? __ldg(mask + g / 32 + 1) : 0u;
        const uint32_t bits = kPair ? (lane < 16 ? w0 : w1) >> ((2 * lane) & 31) : (w0 >> lane & 1u) | (w1 >> lane & 1u) << 1;
        if (!(bits & 1u)) x[k].x = -INFINITY;
        if (!(bits & 2u)) x[k].y = -INFINITY;
      }
      if (dst) store2<T, kPair>(dst + g, lane, width - g, x[k]);
      // (tokens past the end of the vocabulary take no part, whatever was added to them)
      if (i0 >= width) x[k].x = -INFINITY;
      if (i1 >= width) x[k].y = -INFINITY;
      if (x[k].x > m) { m = x[k].x; best = lo + i0; }
      if (x[k].y > m) { m = x[k].y; best = lo + i1; }
    }
    const float ref = ref_of(m);
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) s += exp2f((x[k].x - ref) * kLog2e) + exp2f((x[k].y - ref) * kLog2e);
    warp_merge(m, s, best);
    if (lane == 0) red[row & 1][warp] = Partial{m, s, best, 0};
    __syncthreads();
    if (warp == 0) {
      const Partial p = lane < kLogitThreads / 32 ? red[row & 1][lane] : Partial{-INFINITY, 0.f, -1, 0};
      m = p.m;
      s = p.s;
      best = p.best;
      warp_merge(m, s, best);
      if (lane == 0) a.partials[at * a.slices + slice] = Partial{m, s, best, 0};
    }
    if (on_path()) atomicSub(&cnt[tok[tid] - lo], 1u);
  }
}

// A warp merges one node's partial results, slices in order.
__global__ void __launch_bounds__(kLogitThreads) logits_merge_kernel(const __grid_constant__ LogitArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int first;
  const int n = nodes_of(a.tok_start, blockIdx.x, a.n_tok, a.max_nodes, first, a.status);
  const int row = blockIdx.y * (kLogitThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= n) return;
  const int64_t at = first + row;
  float m = -INFINITY, s = 0.f;
  int best = -1;
  for (int i = lane; i < a.slices; i += 32) {
    const Partial p = a.partials[at * a.slices + i];
    const float mn = fmaxf(m, p.m);
    s = rebase(s, ref_of(m), ref_of(mn)) + rebase(p.s, ref_of(p.m), ref_of(mn));
    if (p.m > m) best = p.best;       // (slices ascend: an equal value further on is not the lowest)
    m = mn;
  }
  warp_merge(m, s, best);
  if (lane == 0) {
    if (a.best) a.best[at] = best;
    if (a.lse) a.lse[at] = ref_of(m) + logf(s);
  }
}

// ------------------------------------------------------------------ acceptance

constexpr int kAcceptWarps = 4;

struct AcceptArgs {
  int B, n_tok, max_nodes;
  const int32_t* tok_start;
  const int32_t* parent;
  const int32_t* token;
  const int32_t* chosen;
  const int32_t* ctx_lens;
  int32_t* count;
  int32_t* next_token;
  int32_t* seq_lens;
  int32_t* path;
  int32_t* seq_idx;
  int32_t* pos;
  uint32_t* status;
};

// A warp takes one sequence, four nodes a lane.  Every node whose token is the one chosen after
// its parent offers itself to the parent, which keeps the lowest; lane 0 follows these links from
// node 0.  Latency-bound: three loads a node, then shared memory.
__global__ void __launch_bounds__(32 * kAcceptWarps) tree_accept_kernel(const __grid_constant__ AcceptArgs a) {
  __shared__ int32_t link[kAcceptWarps][kMaxNodes], said[kAcceptWarps][kMaxNodes], rank[kAcceptWarps][kMaxNodes];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x * kAcceptWarps + w;
  if (b >= a.B) return;
  int first;
  const int n = nodes_of(a.tok_start, b, a.n_tok, a.max_nodes, first, a.status);
  int ctx = __ldg(a.ctx_lens + b);
  if (ctx < 0) {
    if (lane == 0) record_status(a.status, LLA_ERR_DEVICE_ARG);
    ctx = 0;
  }
  constexpr int kPer = kMaxNodes / 32;
  int par[kPer], tok[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = k * 32 + lane;
    par[k] = -1;
    tok[k] = 0;
    if (i < n) {
      par[k] = __ldg(a.parent + first + i);
      tok[k] = __ldg(a.token + first + i);
      said[w][i] = __ldg(a.chosen + first + i);
      link[w][i] = kMaxNodes;
      rank[w][i] = -1;
      if (par[k] < -1 || par[k] >= i) {
        record_status(a.status, LLA_ERR_DEVICE_ARG);
        par[k] = -1;
      }
    }
  }
  __syncwarp();
#pragma unroll
  for (int k = 0; k < kPer; ++k)
    if (par[k] >= 0 && tok[k] == said[w][par[k]]) atomicMin(&link[w][par[k]], k * 32 + lane);
  __syncwarp();
  int count = 0, last = 0;
  if (lane == 0 && n > 0) {
    for (int i = 0; i < kMaxNodes; i = link[w][i]) {
      rank[w][i] = count++;
      last = i;
    }
    a.next_token[b] = said[w][last];
  }
  if (lane == 0 && n == 0) a.next_token[b] = -1;
  __syncwarp();
  count = __shfl_sync(0xffffffffu, count, 0);
  if (lane == 0) {
    a.count[b] = count;
    a.seq_lens[b] = ctx + count;
  }
  int behind = count;          // place of the next node that does not stay
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = k * 32 + lane;
    const int r = i < n ? rank[w][i] : 0;
    const uint32_t left = __ballot_sync(0xffffffffu, i < n && r < 0);
    if (i < n) {
      if (i >= count) a.path[first + i] = -1;
      if (r >= 0) a.path[first + r] = first + i;
      a.seq_idx[first + i] = b;
      a.pos[first + i] = ctx + (r >= 0 ? r : behind + __popc(left & ((1u << lane) - 1u)));
    }
    behind += __popc(left);
  }
}

bool at4(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool opt4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
int slices_of(int vocab) { return (vocab + kSlice - 1) / kSlice; }

struct Range { const void* p; int64_t bytes; };
bool overlap(const Range& x, const Range& y) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
  return x.p && y.p && a < b + y.bytes && b < a + x.bytes;
}

}  // namespace

extern "C" {

size_t lla_logits_workspace_size(int n_tok, int vocab) {
  if (n_tok < 0 || vocab < 1 || vocab > kMaxVocab) return 0;
  return 256 + static_cast<size_t>(n_tok) * slices_of(vocab) * sizeof(Partial);
}

lla_status lla_logits_adjust(const lla_tree* tree, const int32_t* token, int dtype, const void* logits,
                             int64_t row_stride, int vocab, const lla_logit_rules* rules, void* out,
                             int64_t out_stride, int32_t* best, float* lse, void* workspace, size_t ws_bytes,
                             void* stream) {
  if (!tree || !rules || tree->B < 0 || tree->n_tok < 0 || tree->max_nodes < 1 || vocab < 1 || rules->max_history < 0 ||
      rules->max_bias < 0 || rules->n_masks < 0 || (dtype != LLA_BF16 && dtype != LLA_F32))
    return LLA_ERR_INVALID_ARG;
  const int slices = slices_of(std::min(vocab, kMaxVocab));
  if (tree->max_nodes > kMaxNodes || vocab > kMaxVocab || static_cast<int64_t>(tree->B) * slices >= (int64_t(1) << 31))
    return LLA_ERR_UNSUPPORTED;
  if (!out && !best && !lse) return LLA_ERR_INVALID_ARG;
  if (tree->B == 0 || tree->n_tok == 0) return LLA_OK;
  const uintptr_t es = dtype == LLA_BF16 ? 2 : 4;
  const int64_t most = int64_t(1) << 40;
  if (!logits || reinterpret_cast<uintptr_t>(logits) % es || reinterpret_cast<uintptr_t>(out) % es || row_stride < vocab ||
      row_stride > most || (out && (out_stride < vocab || out_stride > most)))
    return LLA_ERR_INVALID_ARG;
  if (!at4(tree->tok_start) || !at4(tree->parent) || !at4(token) || !opt4(best) || !opt4(lse)) return LLA_ERR_INVALID_ARG;
  const lla_logit_rules& r = *rules;
  if (r.max_history > 0 && (!at4(r.history) || !at4(r.hist_len) || !opt4(r.prompt_len))) return LLA_ERR_INVALID_ARG;
  if (!opt4(r.repetition) || !opt4(r.presence) || !opt4(r.frequency)) return LLA_ERR_INVALID_ARG;
  if (r.max_bias > 0 && (!at4(r.bias_token) || !at4(r.bias))) return LLA_ERR_INVALID_ARG;
  if (r.n_masks > 0 && (!at4(r.allowed) || !at4(r.allowed_row))) return LLA_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15u) || ws_bytes < lla_logits_workspace_size(tree->n_tok, vocab))
    return LLA_ERR_INVALID_ARG;
  if (out && !(out == logits && out_stride == row_stride) &&
      overlap({logits, static_cast<int64_t>(((tree->n_tok - 1) * row_stride + vocab) * es)},
              {out, static_cast<int64_t>(((tree->n_tok - 1) * out_stride + vocab) * es)}))
    return LLA_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return LLA_ERR_CUDA;
  LogitArgs a{};
  a.B = tree->B;
  a.n_tok = tree->n_tok;
  a.max_nodes = tree->max_nodes;
  a.vocab = vocab;
  a.slices = slices;
  // nodes a block: as many as leave eight blocks an SM, so that a slice's counts are made once for them
  a.group = static_cast<int>(std::min<int64_t>(tree->max_nodes, std::max<int64_t>(1, static_cast<int64_t>(tree->n_tok) * slices / (8 * sms))));
  a.tok_start = tree->tok_start;
  a.parent = tree->parent;
  a.token = token;
  a.logits = logits;
  a.out = out;
  a.row_stride = row_stride;
  a.out_stride = out_stride;
  a.r = r;
  a.mask_words = (vocab + 31) / 32;
  a.status = static_cast<uint32_t*>(workspace);
  a.partials = reinterpret_cast<Partial*>(static_cast<uint8_t*>(workspace) + 256);
  a.best = best;
  a.lse = lse;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(tree->B) * slices, (tree->max_nodes + a.group - 1) / a.group);
  // a thread takes two neighbouring tokens at once where every row starts on a pair
  const uintptr_t pair = 2 * es;
  const bool paired = reinterpret_cast<uintptr_t>(logits) % pair == 0 && row_stride % 2 == 0 &&
                      (!out || (reinterpret_cast<uintptr_t>(out) % pair == 0 && out_stride % 2 == 0));
  if (dtype == LLA_BF16) {
    if (paired) logits_kernel<__nv_bfloat16, true><<<grid, kLogitThreads, 0, s>>>(a);
    else logits_kernel<__nv_bfloat16, false><<<grid, kLogitThreads, 0, s>>>(a);
  } else {
    if (paired) logits_kernel<float, true><<<grid, kLogitThreads, 0, s>>>(a);
    else logits_kernel<float, false><<<grid, kLogitThreads, 0, s>>>(a);
  }
  if (cudaGetLastError() != cudaSuccess) return LLA_ERR_CUDA;
  if (!best && !lse) return LLA_OK;
  const dim3 merge(tree->B, (tree->max_nodes + kLogitThreads / 32 - 1) / (kLogitThreads / 32));
  return launch_pdl(logits_merge_kernel, merge, dim3(kLogitThreads), 0, s, a) == cudaSuccess ? LLA_OK : LLA_ERR_CUDA;
}

lla_status lla_tree_accept(const lla_tree* tree, const int32_t* token, const int32_t* chosen,
                           const int32_t* ctx_lens, int32_t* count, int32_t* next_token, int32_t* seq_lens,
                           int32_t* path, int32_t* seq_idx, int32_t* pos, void* workspace, size_t ws_bytes,
                           void* stream) {
  if (!tree || tree->B < 0 || tree->n_tok < 0 || tree->max_nodes < 1) return LLA_ERR_INVALID_ARG;
  if (tree->max_nodes > kMaxNodes) return LLA_ERR_UNSUPPORTED;
  if (tree->B == 0) return LLA_OK;
  if (!at4(tree->tok_start) || !at4(ctx_lens) || !at4(count) || !at4(next_token) || !at4(seq_lens) || !at4(workspace) ||
      ws_bytes < 256)
    return LLA_ERR_INVALID_ARG;
  const void* per_token[] = {tree->parent, token, chosen, path, seq_idx, pos};
  for (const void* p : per_token)
    if (tree->n_tok > 0 ? !at4(p) : !opt4(p)) return LLA_ERR_INVALID_ARG;
  // warps read while others write: no output may be an input
  const int64_t b4 = static_cast<int64_t>(tree->B) * 4, t4 = static_cast<int64_t>(tree->n_tok) * 4;
  const Range in[] = {{tree->tok_start, b4 + 4}, {tree->parent, t4}, {token, t4}, {chosen, t4}, {ctx_lens, b4}};
  const Range outs[] = {{count, b4}, {next_token, b4}, {seq_lens, b4}, {path, t4}, {seq_idx, t4}, {pos, t4}};
  for (const Range& o : outs)
    for (const Range& i : in)
      if (overlap(o, i)) return LLA_ERR_INVALID_ARG;
  AcceptArgs a{tree->B, tree->n_tok, tree->max_nodes, tree->tok_start, tree->parent, token, chosen, ctx_lens, count,
               next_token, seq_lens, path, seq_idx, pos, static_cast<uint32_t*>(workspace)};
  tree_accept_kernel<<<(tree->B + kAcceptWarps - 1) / kAcceptWarps, 32 * kAcceptWarps, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? LLA_OK : LLA_ERR_CUDA;
}

}  // extern "C"
