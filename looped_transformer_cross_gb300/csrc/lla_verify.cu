// lla_verify.cu — what follows the model in a step that verifies drafted tokens: the logits of
// every node under its request's rules (lla_logits_adjust) and the walk down the tree along the
// chosen tokens (lla_tree_accept).
//
// Logits: one pass.  A block takes a slice of the vocabulary of one sequence and some of its nodes; each of
// its warps owns a window of the slice, for all of these nodes, and never waits for another while it
// goes through them.  What the history and the biases touch is counted once per block in shared memory,
// and listed per window; a node's pass streams the window's logits and takes the listed ones through the whole
// formula.  The tokens on a node's path join the window's counts and list for that node and leave them
// again.  Best token and log-sum-exp come out of the same pass, a partial result per (node, slice) that a
// second launch merges in a fixed order.
// Each logit is read and written once; bound by instruction issue (66 % of the slots): 400 nodes x 131072 in bf16 93 us
// (2.3 TB/s), 300 x 49999 in fp32, rows without 16-byte alignment, 61 us (2.0 TB/s).
#include <algorithm>

#include "lla_kernels.h"

using namespace lla;

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxNodes = LLA_TREE_MAX_NODES;
constexpr int kSlice = 4096;            // tokens of a slice
constexpr int kLogitThreads = 256;
constexpr int kLogitWarps = kLogitThreads / 32;
constexpr int kWindow = kSlice / kLogitWarps;          // tokens of a warp
constexpr int kPerLane = kWindow / 32;
constexpr int kGroup = 16;              // most nodes of a block
constexpr int kHeldBiases = 256;        // biases of a slice that shared memory has room for
constexpr int kMaxVocab = 1 << 22;

struct Partial {
  float m, s;      // largest value; sum of exp(x - ref(m))
  int32_t best;    // its lowest index, -1: none
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

__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}

// 2^x (sums of logits' exponentials: an error of 2^-22 a term).
__device__ __forceinline__ float exp2_of(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A sum relative to `from`, relative to `to`.
__device__ __forceinline__ float rebase(float s, float from, float to) {
  return s == 0.f ? 0.f : s * exp2_of((from - to) * kLog2e);
}

// Maximum, its lowest index and the sum over a warp.
__device__ __forceinline__ void warp_merge(float& m, float& s, int& best) {
  const float mw = warp_max_redux(m);
  s = warp_sum(rebase(s, ref_of(m), ref_of(mw)));
  const uint32_t i = m == mw && best >= 0 ? static_cast<uint32_t>(best) : 0x7FFFFFFFu;
  const uint32_t lo = __reduce_min_sync(0xffffffffu, i);
  best = lo == 0x7FFFFFFFu ? -1 : static_cast<int>(lo);
  m = mw;
}

// Which of a window's tokens a lane takes: 16 of them, in rising order.  Rows that start on 16 bytes
// (kVec): stretches of 16 bytes; others: every 32nd token.
template <typename T, bool kVec>
struct Lanes {
  static constexpr int kRun = kVec ? 16 / static_cast<int>(sizeof(T)) : 1;   // neighbouring tokens
  __device__ static int token(int lane, int e) { return (e / kRun) * 32 * kRun + lane * kRun + e % kRun; }
  // Where a lane's logit e, or a token's, lies in shared memory: lane by lane, so that neither side's
  // accesses meet in a bank more often than they have to.
  __device__ static int place(int lane, int e) { return 32 * e + lane; }
  __device__ static int place_of(int t) {
    const int run = t / kRun, e = (run / 32) * kRun + t % kRun;
    return 32 * e + run % 32;
  }
  // Bits of the lane's tokens out of a bitmap of the window (`words` of its words exist).
  __device__ static uint32_t bits(const uint32_t* map, int lane, int words) {
    uint32_t r = 0;
    if constexpr (kVec) {
#pragma unroll
      for (int v = 0; v < kPerLane / kRun; ++v) {
        const int bit = v * 32 * kRun + lane * kRun, w = bit >> 5;
        if (w < words) r |= ((map[w] >> (bit & 31)) & ((1u << kRun) - 1u)) << (v * kRun);
      }
    } else {
#pragma unroll 4
      for (int e = 0; e < kPerLane; ++e)
        if (e < words) r |= ((map[e] >> lane) & 1u) << e;
    }
    return r;
  }
  // The lane's logits as they lie in memory (a node's are requested while the one before it is worked on).
  struct Raw {
    uint4 v[kVec ? kPerLane / kRun : 1];
    T one[kVec ? 1 : kPerLane];
  };
  __device__ static T nothing() { return static_cast<T>(-INFINITY); }
  __device__ static void fetch(const T* p, int lane, int left, Raw& r) {
    if constexpr (kVec) {
#pragma unroll
      for (int v = 0; v < kPerLane / kRun; ++v) {
        const int i = v * 32 * kRun + lane * kRun;
        if (i + kRun <= left) {
          r.v[v] = *reinterpret_cast<const uint4*>(p + i);
        } else {                                    // -inf past the end
          T t[kRun];
#pragma unroll
          for (int k = 0; k < kRun; ++k) t[k] = i + k < left ? p[i + k] : nothing();
          r.v[v] = *reinterpret_cast<const uint4*>(t);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < kPerLane; ++e) r.one[e] = 32 * e + lane < left ? p[32 * e + lane] : nothing();
    }
  }
  __device__ static void unpack(const Raw& r, float (&x)[kPerLane]) {
    if constexpr (kVec) {
#pragma unroll
      for (int v = 0; v < kPerLane / kRun; ++v) {
        const uint32_t u[4] = {r.v[v].x, r.v[v].y, r.v[v].z, r.v[v].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (sizeof(T) == 2) {
            x[v * kRun + 2 * k] = __uint_as_float(u[k] << 16);
            x[v * kRun + 2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
          } else {
            x[v * kRun + k] = __uint_as_float(u[k]);
          }
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < kPerLane; ++e) x[e] = static_cast<float>(r.one[e]);
    }
  }
  __device__ static void store(T* p, int lane, int left, const float (&x)[kPerLane]) {
    if constexpr (kVec) {
#pragma unroll
      for (int v = 0; v < kPerLane / kRun; ++v) {
        const int i = v * 32 * kRun + lane * kRun;
        if (i + kRun <= left) {
          uint4 w;
          if constexpr (sizeof(T) == 2) {
            uint32_t u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __nv_bfloat162 h = __floats2bfloat162_rn(x[v * kRun + 2 * k], x[v * kRun + 2 * k + 1]);
              u[k] = *reinterpret_cast<const uint32_t*>(&h);
            }
            w = make_uint4(u[0], u[1], u[2], u[3]);
          } else {
            w = make_uint4(__float_as_uint(x[v * kRun]), __float_as_uint(x[v * kRun + 1]), __float_as_uint(x[v * kRun + 2]),
                           __float_as_uint(x[v * kRun + 3]));
          }
          *reinterpret_cast<uint4*>(p + i) = w;
        } else {
#pragma unroll
          for (int k = 0; k < kRun; ++k)
            if (i + k < left) p[i + k] = static_cast<T>(x[v * kRun + k]);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < kPerLane; ++e)
        if (32 * e + lane < left) p[32 * e + lane] = static_cast<T>(x[e]);
    }
  }
};

// Occurrences of a slice's tokens, with two marks (in the prompt part, has a bias) above them: 16 bits a token
// where no history is longer than 14 bits can count, else 32.
template <int kBits>
struct Counts {
  static constexpr uint32_t kPrompt = 1u << (kBits - 1), kBiased = 1u << (kBits - 2), kTimes = kBiased - 1;
  static constexpr int kPer = 32 / kBits;           // tokens of a word
  uint32_t word[kSlice / kPer];
  __device__ uint32_t get(int i) const { return kPer == 1 ? word[i] : (word[i >> 1] >> (16 * (i & 1))) & 0xFFFFu; }
  __device__ uint32_t mark(int i, uint32_t m) {     // the count before
    return kPer == 1 ? atomicOr(&word[i], m) : (atomicOr(&word[i >> 1], m << (16 * (i & 1))) >> (16 * (i & 1))) & 0xFFFFu;
  }
  __device__ uint32_t add(int i) {
    return kPer == 1 ? atomicAdd(&word[i], 1u) : (atomicAdd(&word[i >> 1], 1u << (16 * (i & 1))) >> (16 * (i & 1))) & 0xFFFFu;
  }
  __device__ void take(int i) {
    if (kPer == 1) atomicSub(&word[i], 1u);
    else atomicSub(&word[i >> 1], 1u << (16 * (i & 1)));
  }
};
constexpr int kMaxTimes16 = (1 << 14) - 1;

template <int kBits>
struct LogitShared {
  Counts<kBits> cnt;
  uint32_t touched[kSlice / 32];                    // tokens with a count or a mark, as bits
  int32_t tok[kMaxNodes];
  uint32_t path[kMaxNodes][kMaxNodes / 32];         // the nodes on each node's path, as bits
  Partial part[kGroup][kLogitWarps];
  uint16_t list[kSlice];                            // per window: its touched tokens
  union {
    float stage[kLogitWarps][kWindow];              // a window's logits while they are worked on
    struct {                                        // before that, steps of the paths' doubling
      int32_t jump[2][kMaxNodes];
      uint32_t path[2][kMaxNodes][kMaxNodes / 32];
    } walk;
  };
  int biases;                                       // of the slice
  int16_t bias_at[kHeldBiases];                     // their tokens
  int32_t bias_entry[kHeldBiases];                  // and entries of the list
};

template <typename T, bool kVec, int kBits>
__global__ void __launch_bounds__(kLogitThreads, 4) logits_kernel(const __grid_constant__ LogitArgs a) {
  __shared__ LogitShared<kBits> sh;
  using C = Counts<kBits>;
  C& cnt = sh.cnt;
  uint32_t* touched = sh.touched;
  int32_t* tok = sh.tok;
  auto& jump = sh.walk.jump;
  auto& path = sh.walk.path;
  auto& part = sh.part;
  using L = Lanes<T, kVec>;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / a.slices, slice = blockIdx.x - b * a.slices;
  // (the chain of loads below is what a block with one node takes: everything is requested as early as it can be)
  const int lo = slice * kSlice, width = min(kSlice, a.vocab - lo);
  const int w0 = warp * kWindow, left = width - w0, row0 = blockIdx.y * a.group;
  int hl = 0, pl = 0;
  constexpr int kEarly = 8;
  int hist_early[kEarly], bias_early = -1;
  const int32_t* hist = a.r.history + static_cast<int64_t>(b) * a.r.max_history;
  const int32_t* bt = a.r.bias_token + static_cast<int64_t>(b) * a.r.max_bias;
  const float* bv = a.r.bias + static_cast<int64_t>(b) * a.r.max_bias;
  if (a.r.max_history > 0) {
    hl = __ldg(a.r.hist_len + b);
    pl = a.r.prompt_len ? __ldg(a.r.prompt_len + b) : 0;
  }
#pragma unroll
  for (int k = 0; k < kEarly; ++k) {
    const int i = tid + k * kLogitThreads;
    hist_early[k] = i < a.r.max_history ? __ldg(hist + i) : -1;
  }
  if (tid < a.r.max_bias) bias_early = __ldg(bt + tid);
  const float rep = a.r.repetition ? __ldg(a.r.repetition + b) : 1.f;
  const float pres = a.r.presence ? __ldg(a.r.presence + b) : 0.f;
  const float freq = a.r.frequency ? __ldg(a.r.frequency + b) : 0.f;
  int first;
  const int n = nodes_of(a.tok_start, b, a.n_tok, a.max_nodes, first, a.status);
  if (row0 >= n) return;
  const bool flag = slice == 0 && blockIdx.y == 0;      // the block that reports what it skips
  const T* src = static_cast<const T*>(a.logits) + (static_cast<int64_t>(first) + row0) * a.row_stride + lo + w0;
  typename L::Raw raw;
  if (left > 0) L::fetch(src, lane, left, raw);

  for (int i = tid; i < kSlice / C::kPer / 4; i += kLogitThreads) reinterpret_cast<uint4*>(cnt.word)[i] = make_uint4(0, 0, 0, 0);
  if (tid < kSlice / 32) touched[tid] = 0;
  if (tid == 0) sh.biases = 0;
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
  if (tid < n) {
#pragma unroll
    for (int w = 0; w < kMaxNodes / 32; ++w) sh.path[tid][w] = path[cur][tid][w];
  }
  // ---- counts of the history and biases
  if (hl < 0 || hl > a.r.max_history || pl < 0 || pl > hl) {
    if (flag) record_status(a.status, LLA_ERR_DEVICE_ARG);
    hl = min(max(hl, 0), a.r.max_history);
    pl = min(max(pl, 0), hl);
  }
  auto count = [&](int i, int t) {
    if (t >= lo && t < lo + width) {
      const int at = t - lo;
      if ((i < pl ? cnt.mark(at, C::kPrompt) : cnt.add(at)) == 0) atomicOr(&touched[at >> 5], 1u << (at & 31));
    } else if (flag && (t < 0 || t >= a.vocab)) {
      record_status(a.status, LLA_ERR_DEVICE_ARG);
    }
  };
#pragma unroll
  for (int k = 0; k < kEarly; ++k)
    if (tid + k * kLogitThreads < hl) count(tid + k * kLogitThreads, hist_early[k]);
#pragma unroll 4
  for (int i = tid + kEarly * kLogitThreads; i < hl; i += kLogitThreads) count(i, __ldg(hist + i));
  if (a.r.max_bias > 0) {
    for (int i = tid; i < a.r.max_bias; i += kLogitThreads) {
      const int t = i < kLogitThreads ? bias_early : __ldg(bt + i);
      if (t >= lo && t < lo + width) {
        const int at = t - lo;
        if (cnt.mark(at, C::kBiased) == 0) atomicOr(&touched[at >> 5], 1u << (at & 31));
        const int k = atomicAdd(&sh.biases, 1);
        if (k < kHeldBiases) {
          sh.bias_at[k] = static_cast<int16_t>(at);
          sh.bias_entry[k] = i;
        }
      } else if (flag && t >= a.vocab) {
        record_status(a.status, LLA_ERR_DEVICE_ARG);
      }
    }
  }
  __syncthreads();
  // The bias of a token: the sum of its entries in list order (found by their index, as the order in
  // which they came into shared memory is open).
  auto bias_of = [&](int at) {
    float sum = 0.f;
    if (sh.biases <= kHeldBiases) {
      for (int last = -1;;) {
        int next = INT32_MAX;
        for (int k = 0; k < sh.biases; ++k)
          if (sh.bias_at[k] == at && sh.bias_entry[k] > last) next = min(next, sh.bias_entry[k]);
        if (next == INT32_MAX) break;
        sum = last < 0 ? __ldg(bv + next) : __fadd_rn(sum, __ldg(bv + next));
        last = next;
      }
    } else {
      bool any = false;
      for (int k = 0; k < a.r.max_bias; ++k)
        if (__ldg(bt + k) == lo + at) {
          sum = any ? __fadd_rn(sum, __ldg(bv + k)) : __ldg(bv + k);
          any = true;
        }
    }
    return sum;
  };

  // ---- from here on a warp is on its own with its window
  uint32_t* map = touched + w0 / 32;
  // its touched tokens: sixteen neighbouring bits a lane, places by a scan
  uint16_t* list = sh.list + w0;
  int listed = 0;
  {
    uint32_t bits = (map[lane >> 1] >> (16 * (lane & 1))) & 0xFFFFu;
    int end = __popc(bits);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += v;
    }
    listed = __shfl_sync(0xffffffffu, end, 31);
    for (int k = end - __popc(bits); bits; bits &= bits - 1) list[k++] = static_cast<uint16_t>(16 * lane + __ffs(bits) - 1);
    __syncwarp();
  }
  uint32_t here[kMaxNodes / 32];                    // nodes whose token lies in the window
#pragma unroll
  for (int k = 0; k < kMaxNodes / 32; ++k) {
    const int t = 32 * k + lane < n ? tok[32 * k + lane] - lo - w0 : -1;
    here[k] = __ballot_sync(0xffffffffu, t >= 0 && t < min(left, kWindow));
  }
  const int row1 = min(n, row0 + a.group), words = left > 0 ? min(kPerLane, (left + 31) / 32) : 0;

  for (int row = row0; row < row1 && left > 0; ++row, src += a.row_stride) {
    const int64_t at = first + row;
    T* dst = a.out ? static_cast<T*>(a.out) + at * a.out_stride + lo + w0 : nullptr;
    float x[kPerLane];
    L::unpack(raw, x);
    if (row + 1 < row1) L::fetch(src + a.row_stride, lane, left, raw);
    const uint32_t* mask = nullptr;
    if (a.r.n_masks > 0) {
      const int mr = __ldg(a.r.allowed_row + at);
      if (mr >= a.r.n_masks) {
        if (slice == 0 && tid == 0) record_status(a.status, LLA_ERR_DEVICE_ARG);
      } else if (mr >= 0) {
        mask = a.r.allowed + static_cast<int64_t>(mr) * a.mask_words + (lo + w0) / 32;
      }
    }
    // ---- this node's path joins the counts and the list
    uint32_t on = 0;                                // of the lane's four nodes: in the window
    int more = 0;
#pragma unroll
    for (int k = 0; k < kMaxNodes / 32; ++k) {
      const uint32_t nodes = here[k] & sh.path[row][k];
      if (nodes == 0) continue;
      const bool in = nodes >> lane & 1u;
      const int t = in ? tok[32 * k + lane] - lo - w0 : 0;
      const bool fresh = in && cnt.add(w0 + t) == 0;
      const uint32_t f = __ballot_sync(0xffffffffu, fresh);
      if (in) on |= 1u << k;
      if (fresh) list[listed + more + __popc(f & ((1u << lane) - 1u))] = static_cast<uint16_t>(t);
      more += __popc(f);
      __syncwarp();
    }
    // ---- tokens that the history, the biases or the path touch: each step rounded by itself, as the formulas
    // are written.  The window goes through shared memory, where a lane takes every 32nd of the list.
    const int work = listed + more;
    if (work > 0) {
      float* stage = sh.stage[warp];
#pragma unroll
      for (int e = 0; e < kPerLane; ++e) stage[L::place(lane, e)] = x[e];
      __syncwarp();
#pragma unroll 1
      for (int j = lane; j < work; j += 32) {
        const int t = list[j], at_t = L::place_of(t);
        const uint32_t c = cnt.get(w0 + t), times = c & C::kTimes;
        float v = stage[at_t];
        if (c & ~C::kBiased) v = v > 0.f ? __fdiv_rn(v, rep) : __fmul_rn(v, rep);
        if (times) v = __fsub_rn(__fsub_rn(v, __fmul_rn(freq, static_cast<float>(times))), pres);
        if (c & C::kBiased) v = __fadd_rn(v, bias_of(w0 + t));
        stage[at_t] = v;
      }
      __syncwarp();
#pragma unroll
      for (int e = 0; e < kPerLane; ++e) x[e] = stage[L::place(lane, e)];
      // the path leaves the counts again
#pragma unroll
      for (int k = 0; k < kMaxNodes / 32; ++k)
        if (on >> k & 1u) cnt.take(tok[32 * k + lane] - lo);
      __syncwarp();
    }
    if (mask) {
      const uint32_t allowed = L::bits(mask, lane, words);
#pragma unroll
      for (int e = 0; e < kPerLane; ++e)
        if (!(allowed >> e & 1u)) x[e] = -INFINITY;
    }
    // (in place, a window that nothing changes stays as it is)
    if (dst && (mask || work > 0 || static_cast<const void*>(dst) != src)) L::store(dst, lane, left, x);
    float m = x[0];
#pragma unroll
    for (int e = 1; e < kPerLane; ++e) m = fmaxf(m, x[e]);
    if (m != m) m = -INFINITY;                      // nothing but NaN
    // (the difference first: it is exact where it matters, at any size of the logits)
    const float ref = ref_of(m);
    float s;
    {
      const uint64_t scale = pair2(kLog2e, kLog2e), off = pair2(-ref, -ref);
      uint64_t sum = 0;
#pragma unroll
      for (int e = 0; e < kPerLane; e += 2) {
        uint64_t d = pair2(x[e], x[e + 1]);
        float d0, d1;
        asm("add.rn.f32x2 %0, %0, %1;" : "+l"(d) : "l"(off));
        asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(d) : "l"(scale));
        asm("mov.b64 {%0, %1}, %2;" : "=f"(d0), "=f"(d1) : "l"(d));
        asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum) : "l"(pair2(exp2_of(d0), exp2_of(d1))));
      }
      float s0, s1;
      asm("mov.b64 {%0, %1}, %2;" : "=f"(s0), "=f"(s1) : "l"(sum));
      s = s0 + s1;
    }
    int best = -1;
    if (m == warp_max_redux(m) && m > -INFINITY) {  // (only a lane that may hold the warp's best looks for it)
      int at_e = 0;
#pragma unroll
      for (int e = kPerLane - 1; e > 0; --e)
        if (x[e] == m) at_e = e;
      if (x[0] == m) at_e = 0;
      best = lo + w0 + L::token(lane, at_e);
    }
    warp_merge(m, s, best);
    if (lane == 0) part[row - row0][warp] = Partial{m, s, best};
  }
  __syncthreads();
  // ---- the windows of each node, in order
  const int windows = (width + kWindow - 1) / kWindow;
  for (int r = tid; r < row1 - row0; r += kLogitThreads) {
    Partial p = part[r][0];
    for (int w = 1; w < windows; ++w) {
      const Partial y = part[r][w];
      const float m2 = fmaxf(p.m, y.m), r2 = ref_of(m2);
      p.s = rebase(p.s, ref_of(p.m), r2) + rebase(y.s, ref_of(y.m), r2);
      if (y.m > p.m) p.best = y.best;
      p.m = m2;
    }
    a.partials[(first + row0 + r) * static_cast<int64_t>(a.slices) + slice] = p;
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
  const int64_t n = tree->n_tok, B4 = product({tree->B, 4});
  const bool in_place = out == logits && out_stride == row_stride;
  const Span outs[] = {{out, row_bytes(n, out_stride, vocab, es)}, {best, n * 4}, {lse, n * 4},
                       {workspace, static_cast<int64_t>(lla_logits_workspace_size(tree->n_tok, vocab))}};
  const Span ins[] = {{in_place ? nullptr : logits, row_bytes(n, row_stride, vocab, es)}, {token, n * 4}, {tree->tok_start, B4 + 4}, {tree->parent, n * 4},
                      {r.max_history > 0 ? r.history : nullptr, product({tree->B, r.max_history, 4})},
                      {r.max_history > 0 ? r.hist_len : nullptr, B4}, {r.max_history > 0 ? r.prompt_len : nullptr, B4},
                      {r.repetition, B4}, {r.presence, B4}, {r.frequency, B4},
                      {r.max_bias > 0 ? r.bias_token : nullptr, product({tree->B, r.max_bias, 4})},
                      {r.max_bias > 0 ? r.bias : nullptr, product({tree->B, r.max_bias, 4})},
                      {r.n_masks > 0 ? r.allowed : nullptr, product({r.n_masks, (vocab + 31) / 32, 4})},
                      {r.n_masks > 0 ? r.allowed_row : nullptr, n * 4}};
  if (outputs_meet(outs, ins)) return LLA_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return LLA_ERR_CUDA;
  LogitArgs a{};
  a.B = tree->B;
  a.n_tok = tree->n_tok;
  a.max_nodes = tree->max_nodes;
  a.vocab = vocab;
  a.slices = slices;
  // nodes a block: as many as leave eight blocks an SM, so that a slice's counts are made once for them
  a.group = static_cast<int>(std::min<int64_t>(std::min(tree->max_nodes, kGroup), std::max<int64_t>(1, static_cast<int64_t>(tree->n_tok) * slices / (8 * sms))));
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
  // a lane takes 16 bytes of neighbouring tokens at once where every row starts on 16 bytes
  const int64_t run = 16 / static_cast<int64_t>(es);
  const bool vec = reinterpret_cast<uintptr_t>(logits) % 16 == 0 && row_stride % run == 0 &&
                   (!out || (reinterpret_cast<uintptr_t>(out) % 16 == 0 && out_stride % run == 0));
  if (r.max_history + kMaxNodes <= kMaxTimes16) {
    auto kern = dtype == LLA_BF16 ? (vec ? logits_kernel<__nv_bfloat16, true, 16> : logits_kernel<__nv_bfloat16, false, 16>)
                                  : (vec ? logits_kernel<float, true, 16> : logits_kernel<float, false, 16>);
    kern<<<grid, kLogitThreads, 0, s>>>(a);
  } else {
    auto kern = dtype == LLA_BF16 ? (vec ? logits_kernel<__nv_bfloat16, true, 32> : logits_kernel<__nv_bfloat16, false, 32>)
                                  : (vec ? logits_kernel<float, true, 32> : logits_kernel<float, false, 32>);
    kern<<<grid, kLogitThreads, 0, s>>>(a);
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
  const Span in[] = {{tree->tok_start, b4 + 4}, {tree->parent, t4}, {token, t4}, {chosen, t4}, {ctx_lens, b4}};
  const Span outs[] = {{count, b4}, {next_token, b4}, {seq_lens, b4}, {path, t4}, {seq_idx, t4}, {pos, t4}, {workspace, 256}};
  if (outputs_meet(outs, in)) return LLA_ERR_INVALID_ARG;
  AcceptArgs a{tree->B, tree->n_tok, tree->max_nodes, tree->tok_start, tree->parent, token, chosen, ctx_lens, count,
               next_token, seq_lens, path, seq_idx, pos, static_cast<uint32_t*>(workspace)};
  tree_accept_kernel<<<(tree->B + kAcceptWarps - 1) / kAcceptWarps, 32 * kAcceptWarps, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? LLA_OK : LLA_ERR_CUDA;
}

}  // extern "C"
