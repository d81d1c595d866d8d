// lla_tree.cu — attention of drafted tokens over a latent cache (lla_tree_attn): entry points,
// the plain kernel (fp32 arithmetic, either storage type) and the finish kernel.
//
// A node's softmax runs over the cached tokens, whose keys are reconstructed from their
// latents, and over the nodes on its path, whose keys are exact.  The first part is split along
// the cache; each split leaves, per node, its running maximum m, sum l and latent sum
// acc = sum_j 2^(s_j - m) c_v,j, because sum_j p_j (W c_j + mu) = W (sum_j p_j c_j) + mu sum_j p_j:
// V is never reconstructed per token.  The finish kernel merges the splits, adds the path's
// part and applies W_up,v once per node.
#include <algorithm>
#include <cmath>

#include "lla_tree.h"

namespace lla {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kInvSqrtD = 0.08838834764831845f;   // 1/sqrt(128)
constexpr int kPlainThreads = 256;
constexpr int kKeyStride = kHeadDim + 4;            // floats between rows of keys and queries in shared memory
constexpr int kFinishThreads = 128;
constexpr int kFinishRows = 8;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float x, float* p) { *p = x; }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16* p) { *p = __float2bfloat16_rn(x); }

// Four consecutive elements (aligned to four) as floats.
__device__ __forceinline__ float4 ld4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 ld4(const __nv_bfloat16* p) {
  const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xFFFF0000u));
}

// First and second member of frequency pair f.
__device__ __forceinline__ int pair0(int style, int f) { return style == 0 ? f : 2 * f; }
__device__ __forceinline__ int pair1(int style, int f) { return style == 0 ? f + 64 : 2 * f + 1; }

__device__ __forceinline__ int64_t node_pos(const TreeArgs& a, int entry, bool flag) {
  const int p = __ldg(a.pos + entry);
  if (p >= 0 && p < a.rope_len) return p;
  if (flag) record_status(a.status, LLA_ERR_DEVICE_ARG);
  return p < 0 ? 0 : a.rope_len - 1;
}

// W_up,k of the loop in fp32 as [H][r_k][128], dimensions in the paired layout, and W_up,v as [H][r_v][128]: the
// other kernels' threads read neighbouring dimensions of one column (from L1; in shared memory the first left
// room for one block an SM).  Block = 32 columns of a head.
template <typename T>
__global__ void __launch_bounds__(kPlainThreads) tree_turn_kernel(const __grid_constant__ TreeArgs a) {
  __shared__ float t[32][kHeadDim + 1];
  const int k_tiles = (a.r_k + 31) / 32;
  const bool key = blockIdx.y < k_tiles;
  const int r = key ? a.r_k : a.r_v, h = blockIdx.x, c0 = (key ? blockIdx.y : blockIdx.y - k_tiles) * 32, cols = min(32, r - c0);
  const T* W = static_cast<const T*>(key ? a.w_up_k : a.w_up_v) + static_cast<int64_t>(h) * kHeadDim * r + c0;
  const int c = threadIdx.x & 31, e0 = threadIdx.x >> 5;
  if (c < cols) {
    float x[kHeadDim * 32 / kPlainThreads];           // every load under way before the first is used
#pragma unroll
    for (int k = 0; k < kHeadDim * 32 / kPlainThreads; ++k) {
      const int e = e0 + k * (kPlainThreads / 32);
      x[k] = to_f(W[static_cast<int64_t>(!key ? e : e < 64 ? pair0(a.rope_style, e) : pair1(a.rope_style, e - 64)) * r + c]);
    }
#pragma unroll
    for (int k = 0; k < kHeadDim * 32 / kPlainThreads; ++k) t[c][e0 + k * (kPlainThreads / 32)] = x[k];
  }
  __syncthreads();
  float* out = (key ? a.w_turned : a.v_turned) + (static_cast<int64_t>(h) * r + c0) * kHeadDim;
  for (int i = threadIdx.x; i < kHeadDim * cols; i += kPlainThreads) out[i] = t[i >> 7][i & 127];
}

// Block = (unit, split of the cache) x 32 nodes.  32 tokens at a time: their K latents transposed in shared
// memory, keys by a thread per 4 tokens x 4 dimensions, rotated in place, then eight threads a node take
// its scores, its softmax and a share of its latent sum.
// Bound by its multiply-adds (2 * 128 * r_k a token for the keys, repeated for every 32 nodes) and the shared-memory
// reads that feed them: 4 x 2000 tokens of 16 heads at (96, 160) with 16 nodes 288 us, a fifth of the fp32 rate.
template <typename T>
__global__ void __launch_bounds__(kPlainThreads, 2) tree_plain_kernel(const __grid_constant__ TreeArgs a) {
  extern __shared__ float4 sh4[];
  constexpr int kTokStride = kTreePlainTile + 4;
  float* qs = reinterpret_cast<float*>(sh4);                    // [32][kKeyStride]
  float* ks = qs + kTreePlainRows * kKeyStride;                 // [32][kKeyStride]
  float* ct = ks + kTreePlainTile * kKeyStride;                 // [r_k][kTokStride]: latents transposed
  float* vs = ct + a.r_k * kTokStride;                          // [32][r_v]
  float* ps = vs + kTreePlainTile * a.r_v;                      // [32][33]
  const int tid = threadIdx.x;
  const int64_t unit = blockIdx.x / a.splits;
  const int split = static_cast<int>(blockIdx.x - unit * a.splits);
  const int b = static_cast<int>(unit / a.H), h = static_cast<int>(unit - static_cast<int64_t>(b) * a.H);
  const int row0 = blockIdx.y * kTreePlainRows;
  int first;
  const int n = tree_nodes(a, b, first, false);
  const int L = tree_cached(a, b, false);
  const int64_t j0 = split * a.chunk, j1 = min(static_cast<int64_t>(L), j0 + a.chunk);
  if (row0 >= n || j0 >= j1) return;
  const int rows = min(kTreePlainRows, n - row0);

  // ---- queries: rotated, scaled to log2 units; rows past the last node are zeros
  for (int i = tid; i < kTreePlainRows * 64; i += kPlainThreads) {
    const int r = i >> 6, f = i & 63;
    float y0 = 0.f, y1 = 0.f;
    if (r < rows) {
      const int entry = first + row0 + r;
      const T* qv = static_cast<const T*>(a.q) + entry * a.q_stride + h * kHeadDim;
      const int64_t p = node_pos(a, entry, false);
      const float c = __ldg(a.rope_cos + p * 64 + f), s = __ldg(a.rope_sin + p * 64 + f);
      const float x0 = to_f(qv[pair0(a.rope_style, f)]), x1 = to_f(qv[pair1(a.rope_style, f)]);
      const float sc = kLog2e * kInvSqrtD;
      y0 = (x0 * c - x1 * s) * sc;
      y1 = (x0 * s + x1 * c) * sc;
    }
    qs[r * kKeyStride + f] = y0;          // pairs (f, f + 64), like the keys below
    qs[r * kKeyStride + 64 + f] = y1;
  }

  const int row = tid >> 3, part = tid & 7;     // eight threads a node
  // its latent sum: columns 4 part .. of every 32
  float4 acc[kMaxRankPerHead / 32];
#pragma unroll
  for (int i = 0; i < kMaxRankPerHead / 32; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, l = 0.f;
  const float* W = a.w_turned + static_cast<int64_t>(h) * a.r_k * kHeadDim;
  const int tg = tid >> 5, dg = tid & 31;       // keys: tokens 4 tg .., dimensions 4 dg .. (paired layout)
  float mu[4];
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const int e = 4 * dg + d;
    mu[d] = __ldg(a.mu_k + h * a.mu_hstride + (e < 64 ? pair0(a.rope_style, e) : pair1(a.rope_style, e - 64)));
  }
  for (int64_t t0 = j0; t0 < j1; t0 += kTreePlainTile) {
    const int cnt = static_cast<int>(min(static_cast<int64_t>(kTreePlainTile), j1 - t0));
    __syncthreads();
    // ---- latents of the tile, four tokens a warp, their loads together; zeros past its last token
    const int gk = a.r_k >> 2, gv = a.r_v >> 2;
    {
      int64_t at[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int t = 4 * tg + u;
        at[u] = t < cnt ? latent_row(a.block_table, a.page_size, a.max_pages, a.num_pages, a.L_max, a.H, b, h, t0 + t, a.status) : 0;
      }
      for (int c = dg; c < gk + gv; c += 32) {
        float4 x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          x[u] = c < gk ? ld4(static_cast<const T*>(a.cache_k) + at[u] * a.r_k + 4 * c)
                        : ld4(static_cast<const T*>(a.cache_v) + at[u] * a.r_v + 4 * (c - gk));
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (4 * tg + u >= cnt) x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < gk) {
          float* to = ct + 4 * c * kTokStride + 4 * tg;
          *reinterpret_cast<float4*>(to) = make_float4(x[0].x, x[1].x, x[2].x, x[3].x);
          *reinterpret_cast<float4*>(to + kTokStride) = make_float4(x[0].y, x[1].y, x[2].y, x[3].y);
          *reinterpret_cast<float4*>(to + 2 * kTokStride) = make_float4(x[0].z, x[1].z, x[2].z, x[3].z);
          *reinterpret_cast<float4*>(to + 3 * kTokStride) = make_float4(x[0].w, x[1].w, x[2].w, x[3].w);
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u) *reinterpret_cast<float4*>(vs + (4 * tg + u) * a.r_v + 4 * (c - gk)) = x[u];
        }
      }
    }
    // ---- keys before rotation
    float k[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int d = 0; d < 4; ++d) k[t][d] = mu[d];
    __syncthreads();
#pragma unroll 8
    for (int r = 0; r < a.r_k; ++r) {
      const float4 w = __ldg(reinterpret_cast<const float4*>(W + r * kHeadDim + 4 * dg));
      const float4 c = *reinterpret_cast<const float4*>(ct + r * kTokStride + 4 * tg);
      const float wv[4] = {w.x, w.y, w.z, w.w}, cv[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int d = 0; d < 4; ++d) k[t][d] = fmaf(cv[t], wv[d], k[t][d]);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
      *reinterpret_cast<float4*>(ks + (4 * tg + t) * kKeyStride + 4 * dg) = make_float4(k[t][0], k[t][1], k[t][2], k[t][3]);
    __syncthreads();
    // ---- rotation by each token's row of the table: frequency tid mod 64 of every fourth token
    {
      const int f = tid & 63, t1 = tid >> 6;
      float c[8], sn[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int64_t at = (t0 + min(t1 + 4 * u, cnt - 1)) * 64 + f;
        c[u] = __ldg(a.rope_cos + at);
        sn[u] = __ldg(a.rope_sin + at);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        float* kk = ks + (t1 + 4 * u) * kKeyStride + f;
        const float x0 = kk[0], x1 = kk[64];
        kk[0] = x0 * c[u] - x1 * sn[u];
        kk[64] = x0 * sn[u] + x1 * c[u];
      }
    }
    __syncthreads();
    // ---- scores of the thread's four tokens (part, part + 8, ..), softmax over the node's eight threads
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    for (int d = 0; d < kHeadDim; d += 4) {
      const float4 q = *reinterpret_cast<const float4*>(qs + row * kKeyStride + d);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 kk = *reinterpret_cast<const float4*>(ks + (part + 8 * i) * kKeyStride + d);
        s[i] = fmaf(q.x, kk.x, fmaf(q.y, kk.y, fmaf(q.z, kk.z, fmaf(q.w, kk.w, s[i]))));
      }
    }
    float mt = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (part + 8 * i >= cnt) s[i] = -INFINITY;
      mt = fmaxf(mt, s[i]);
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
    const float m_new = fmaxf(m, mt);
    const float alpha = m == -INFINITY ? 0.f : exp2f(m - m_new);
    m = m_new;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p = part + 8 * i < cnt ? exp2f(s[i] - m) : 0.f;
      ps[row * 33 + part + 8 * i] = p;
      sum += p;
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = l * alpha + sum;
    __syncwarp();
    // ---- latent sum
#pragma unroll
    for (int i = 0; i < kMaxRankPerHead / 32; ++i) {
      if (32 * i < a.r_v) { acc[i].x *= alpha; acc[i].y *= alpha; acc[i].z *= alpha; acc[i].w *= alpha; }
    }
#pragma unroll 2
    for (int t = 0; t < kTreePlainTile; ++t) {
      const float p = ps[row * 33 + t];
#pragma unroll
      for (int i = 0; i < kMaxRankPerHead / 32; ++i) {
        if (32 * i + 4 * part < a.r_v) {
          const float4 v = *reinterpret_cast<const float4*>(vs + t * a.r_v + 32 * i + 4 * part);
          acc[i].x = fmaf(p, v.x, acc[i].x); acc[i].y = fmaf(p, v.y, acc[i].y);
          acc[i].z = fmaf(p, v.z, acc[i].z); acc[i].w = fmaf(p, v.w, acc[i].w);
        }
      }
    }
  }
  if (row < rows) {
    float* rec = a.records + ((unit * a.splits + split) * a.rec_rows + row0 + row) * (a.r_v + kTreeHead);
    if (part == 0) { rec[0] = m; rec[1] = l; rec[2] = rec[3] = rec[4] = 0.f; }
#pragma unroll
    for (int i = 0; i < kMaxRankPerHead / 32; ++i)
      if (32 * i + 4 * part < a.r_v) *reinterpret_cast<float4*>(rec + kTreeHead + 32 * i + 4 * part) = acc[i];
  }
}

// Block = (unit, up to eight nodes).  A warp takes a key at a time, rotates it and has its products with all
// nodes; sixteen threads a node make its softmax over its path and the records; thread e then forms
// out_e = (W_e . A + mu_e P + sum_a p_a v_a,e) / l of all nodes, so that a key, a value and a weight are read
// once for eight.  Bound by the latency of its steps.  16 sequences of 12 heads with 35 nodes each over 76 tokens
// 48 us, 128 nodes of 16 heads over 1000 tokens 59, 4 x 16 nodes of 16 heads over 2000 38 (one node at a time, rows of
// W_up,v read as they lie by the threads: 177, 130, 31).
template <typename T>
__global__ void __launch_bounds__(kFinishThreads, 5) tree_finish_kernel(const __grid_constant__ TreeArgs a) {
  __shared__ int32_t par[kTreeMaxNodes];
  __shared__ uint32_t path[kFinishRows][4], used[4];
  __shared__ __align__(16) float sc[kTreeMaxNodes][kFinishRows];       // scores, then weights
  __shared__ __align__(16) float A[kMaxRankPerHead][kFinishRows];
  __shared__ float q[kFinishRows][kHeadDim];
  __shared__ float factor[16][kFinishRows];
  __shared__ float4 stat[kFinishRows];                // {reference, cached sum, sum, -}
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t unit = blockIdx.x;
  const int b = static_cast<int>(unit / a.H), h = static_cast<int>(unit - static_cast<int64_t>(b) * a.H);
  const bool flag = h == 0 && blockIdx.y == 0;
  int first;
  const int n = tree_nodes(a, b, first, flag);
  const int L = tree_cached(a, b, flag);
  constexpr int kMost = kFinishRows * kMaxRankPerHead / 4 / kFinishThreads;     // quads of latent sums a thread holds
  const int row0 = blockIdx.y * a.finish_rows;
  if (row0 >= n) return;
  const int rows = min(a.finish_rows, n - row0), nk = row0 + rows;
  const int nsplit = static_cast<int>((L + a.chunk - 1) / a.chunk), stride = a.r_v + kTreeHead;
  for (int i = tid; i < n; i += kFinishThreads) {
    int p = __ldg(a.parent + first + i);
    if (p < -1 || p >= i) {
      if (flag) record_status(a.status, LLA_ERR_DEVICE_ARG);
      p = -1;
    }
    par[i] = p;
    if (flag) node_pos(a, first + i, true);
  }
  for (int i = tid; i < kFinishRows * 64; i += kFinishThreads) {
    const int r = i >> 6, f = i & 63;
    float y0 = 0.f, y1 = 0.f;
    if (r < rows) {
      const int entry = first + row0 + r;
      const T* qv = static_cast<const T*>(a.q) + entry * a.q_stride + h * kHeadDim;
      const int64_t p = node_pos(a, entry, false);
      const float c = __ldg(a.rope_cos + p * 64 + f), s = __ldg(a.rope_sin + p * 64 + f);
      const float x0 = to_f(qv[pair0(a.rope_style, f)]), x1 = to_f(qv[pair1(a.rope_style, f)]);
      y0 = (x0 * c - x1 * s) * (kLog2e * kInvSqrtD);
      y1 = (x0 * s + x1 * c) * (kLog2e * kInvSqrtD);
    }
    q[r][f] = y0;
    q[r][64 + f] = y1;
  }
  if (tid < 4) used[tid] = 0;
  __syncthreads();
  // ---- the nodes on each node's path, as bits
  if (tid < kFinishRows) {
    uint32_t on[4] = {0, 0, 0, 0};
    if (tid < rows) {
      for (int i = row0 + tid; i >= 0; i = par[i]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) on[k] |= (i >> 5) == k ? 1u << (i & 31) : 0u;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      path[tid][k] = on[k];
      if (on[k]) atomicOr(&used[k], on[k]);
    }
  }
  __syncthreads();
  // ---- scores: four keys of a warp at a time, their loads under way together
  constexpr int kWarps = kFinishThreads / 32, kAtOnce = 4;
  for (int j0 = warp; j0 < nk; j0 += kWarps * kAtOnce) {
    float y0[kAtOnce][2], y1[kAtOnce][2];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int j = min(j0 + i * kWarps, nk - 1);
      const T* kv = static_cast<const T*>(a.k) + (first + j) * a.k_stride + h * kHeadDim;
      const int64_t p = node_pos(a, first + j, false);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int f = lane + 32 * k;
        const float c = __ldg(a.rope_cos + p * 64 + f), s = __ldg(a.rope_sin + p * 64 + f);
        const float x0 = to_f(kv[pair0(a.rope_style, f)]), x1 = to_f(kv[pair1(a.rope_style, f)]);
        y0[i][k] = x0 * c - x1 * s;
        y1[i][k] = x0 * s + x1 * c;
      }
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int j = j0 + i * kWarps;
      if (j >= nk || !(used[j >> 5] >> (j & 31) & 1)) continue;
      float d[kFinishRows];
#pragma unroll
      for (int r = 0; r < kFinishRows; ++r) d[r] = q[r][lane] * y0[i][0];
#pragma unroll
      for (int r = 0; r < kFinishRows; ++r)
        d[r] = fmaf(q[r][lane + 32], y0[i][1], fmaf(q[r][lane + 64], y1[i][0], fmaf(q[r][lane + 96], y1[i][1], d[r])));
      // the eight sums over the lanes: half of them go on in half of the lanes, three times
      float x[4], y[2];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float give = __shfl_xor_sync(0xffffffffu, lane & 16 ? d[r] : d[r + 4], 16);
        x[r] = (lane & 16 ? d[r + 4] : d[r]) + give;
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float give = __shfl_xor_sync(0xffffffffu, lane & 8 ? x[r] : x[r + 2], 8);
        y[r] = (lane & 8 ? x[r + 2] : x[r]) + give;
      }
      const float give = __shfl_xor_sync(0xffffffffu, lane & 4 ? y[0] : y[1], 4);
      float z = (lane & 4 ? y[1] : y[0]) + give;
      z += __shfl_xor_sync(0xffffffffu, z, 2);
      z += __shfl_xor_sync(0xffffffffu, z, 1);
      if ((lane & 3) == 0) sc[j][(lane >> 4) * 4 + (lane >> 3 & 1) * 2 + (lane >> 2 & 1)] = z;
    }
  }
  __syncthreads();
  // ---- softmax over the path and the records: sixteen threads a node
  {
    const int r = tid >> 4, x = tid & 15;
    const float* rec0 = a.records + (unit * a.splits * a.rec_rows + row0 + r) * stride;
    const int64_t next = static_cast<int64_t>(a.rec_rows) * stride;
    const int held_by = r < rows ? nsplit : 0;
    float m = -INFINITY;
    for (int j = x; j < nk; j += 16)
      if (path[r][j >> 5] >> (j & 31) & 1) m = fmaxf(m, sc[j][r]);
    for (int i = x; i < held_by; i += 16) m = fmaxf(m, rec0[i * next]);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.f, held = 0.f;
    for (int j = x; j < nk; j += 16) {
      const float p = path[r][j >> 5] >> (j & 31) & 1 ? exp2f(sc[j][r] - m) : 0.f;
      sc[j][r] = p;
      l += p;
    }
    for (int i = x; i < held_by; i += 16) {
      const float* rec = rec0 + i * next;
      held = fmaf(exp2f(rec[0] - m), (rec[1] + rec[2]) + (rec[3] + rec[4]), held);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
      l += __shfl_xor_sync(0xffffffffu, l, o);
      held += __shfl_xor_sync(0xffffffffu, held, o);
    }
    if (x == 0) stat[r] = make_float4(m, held, l + held, 0.f);
  }
  __syncthreads();
  // ---- the records' latent sums, sixteen records' factors at a time
  if (nsplit > 0) {
    const float* rec0 = a.records + (unit * a.splits * a.rec_rows + row0) * stride;
    const int64_t next = static_cast<int64_t>(a.rec_rows) * stride;
    const int quads = a.r_v / 4;
    float4 sum[kMost];
#pragma unroll
    for (int e = 0; e < kMost; ++e) sum[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < nsplit; s0 += 16) {
      const int r = tid & 7, k = tid >> 3, parts = min(16, nsplit - s0);
      __syncthreads();
      factor[k][r] = r < rows && k < parts ? exp2f(rec0[(s0 + k) * next + r * stride] - stat[r].x) : 0.f;
      __syncthreads();
#pragma unroll
      for (int e = 0; e < kMost; ++e) {
        const int i = tid + e * kFinishThreads, row = i / quads;
        if (row >= rows) break;
        const float* at = rec0 + s0 * next + row * stride + kTreeHead + 4 * (i - row * quads);
#pragma unroll 8
        for (int x = 0; x < parts; ++x, at += next) {
          const float4 y = ld4(at);
          const float f = factor[x][row];
          sum[e].x = fmaf(f, y.x, sum[e].x); sum[e].y = fmaf(f, y.y, sum[e].y);
          sum[e].z = fmaf(f, y.z, sum[e].z); sum[e].w = fmaf(f, y.w, sum[e].w);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < kMost; ++e) {
      const int i = tid + e * kFinishThreads, row = i / quads, c = 4 * (i - row * quads);
      if (row >= kFinishRows) break;
      A[c][row] = sum[e].x; A[c + 1][row] = sum[e].y; A[c + 2][row] = sum[e].z; A[c + 3][row] = sum[e].w;
    }
  }
  __syncthreads();
  // ---- dimension tid of every node
  float o[kFinishRows];
  auto add = [&](const float (&by)[kFinishRows], float w) {
    const float4 lo = *reinterpret_cast<const float4*>(by), hi = *reinterpret_cast<const float4*>(by + 4);
    o[0] = fmaf(lo.x, w, o[0]); o[1] = fmaf(lo.y, w, o[1]); o[2] = fmaf(lo.z, w, o[2]); o[3] = fmaf(lo.w, w, o[3]);
    o[4] = fmaf(hi.x, w, o[4]); o[5] = fmaf(hi.y, w, o[5]); o[6] = fmaf(hi.z, w, o[6]); o[7] = fmaf(hi.w, w, o[7]);
  };
  const float mu = nsplit > 0 ? __ldg(a.mu_v + h * a.mu_hstride + tid) : 0.f;
#pragma unroll
  for (int r = 0; r < kFinishRows; ++r) o[r] = stat[r].y * mu;
  for (int j0 = 0; j0 < nk; j0 += 8) {                // (eight values under way together)
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f(static_cast<const T*>(a.v)[(first + min(j0 + i, nk - 1)) * a.v_stride + h * kHeadDim + tid]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int j = j0 + i;
      if (j >= nk || !(used[j >> 5] >> (j & 31) & 1)) continue;
      if (isfinite(v[i])) {
        add(sc[j], v[i]);
      } else {                                        // (0 times it is not 0 where the node is not on the path)
#pragma unroll 1
        for (int r = 0; r < rows; ++r)
          if (path[r][j >> 5] >> (j & 31) & 1) {
            const float x = sc[j][r] * v[i];
#pragma unroll
            for (int k = 0; k < kFinishRows; ++k) o[k] += k == r ? x : 0.f;
          }
      }
    }
  }
  if (nsplit > 0) {
    const float* w = a.v_turned + static_cast<int64_t>(h) * a.r_v * kHeadDim + tid;
#pragma unroll 16
    for (int c = 0; c < a.r_v; ++c) add(A[c], __ldg(w + c * kHeadDim));
  }
#pragma unroll
  for (int r = 0; r < kFinishRows; ++r) {
    if (r >= rows) break;
    const int64_t at = (static_cast<int64_t>(first) + row0 + r) * a.H + h;
    const float4 st = stat[r];
    from_f(o[r] / st.z, static_cast<T*>(a.out) + at * kHeadDim + tid);
    if (tid == 0 && a.lse) a.lse[at] = (st.x + log2f(st.z)) * kLn2;
  }
}

size_t plain_smem(int r_k, int r_v) {
  return sizeof(float) * ((kTreePlainRows + kTreePlainTile) * kKeyStride + (kTreePlainTile + 4) * r_k + kTreePlainTile * r_v +
                          kTreePlainRows * 33);
}

}  // namespace

cudaError_t launch_tree_plain(const TreeArgs& a, bool bf16, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(a.B) * a.H * a.splits),
                  (a.max_nodes + kTreePlainRows - 1) / kTreePlainRows);
  auto kern = bf16 ? tree_plain_kernel<__nv_bfloat16> : tree_plain_kernel<float>;
  // (the most any shape takes, at every call)
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(plain_smem(kMaxRankPerHead, kMaxRankPerHead)));
  if (e != cudaSuccess) return e;
  auto turn = bf16 ? tree_turn_kernel<__nv_bfloat16> : tree_turn_kernel<float>;
  turn<<<dim3(a.H, (a.r_k + 31) / 32 + (a.r_v + 31) / 32), kPlainThreads, 0, s>>>(a);
  kern<<<grid, kPlainThreads, plain_smem(a.r_k, a.r_v), s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_tree_finish(const TreeArgs& a, bool bf16, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(a.B) * a.H), (a.max_nodes + a.finish_rows - 1) / a.finish_rows);
  if (bf16) tree_finish_kernel<__nv_bfloat16><<<grid, kFinishThreads, 0, s>>>(a);
  else tree_finish_kernel<float><<<grid, kFinishThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace lla

using namespace lla;

namespace {

bool at16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool at4(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The cache of a call: dense, or a page pool with a block table.
struct View {
  const void* k;
  const void* v;
  int B;
  int64_t L_max;
  const int32_t* bt;
  int page_size, max_pages;
  int64_t num_pages;
};

// Shapes of the tensor-core kernel: those whose operands fit for any number of nodes.
bool tensor_path(const lla_dims* d) {
  TreePlan p;
  return d->dtype == LLA_BF16 && make_tree_plan(d->r_k, d->r_v, tree_group(d->r_v), &p);
}

// Workspace: status word; tensor-core kernel: the plan, the mu and the query operands; the records.
struct TreeWs {
  int64_t chunk;
  int splits, grid;
  size_t turned, v_turned, tile_start, cta_start, head_top, unit_top, bias, qimg, qback, khat, kback, paths, records, total;
};

TreeWs tree_ws(const lla_dims* d, int B, int max_nodes, int64_t L_max, int sms, bool tensor) {
  TreeWs w{};
  const int64_t units = std::max<int64_t>(1, static_cast<int64_t>(B) * d->H);
  const int group = tree_group(d->r_v), groups = (max_nodes + group - 1) / group;
  const size_t rec = static_cast<size_t>(tensor ? std::min(max_nodes, group) : max_nodes) * (d->r_v + kTreeHead) * 4;
  auto al = [](size_t x) { return (x + 255) / 256 * 256; };
  if (tensor) {
    const int64_t most = units * groups * std::max<int64_t>(1, (L_max + kTile - 1) / kTile);
    w.grid = static_cast<int>(std::min<int64_t>(std::min(sms, kMaxGrid), most));
    w.tile_start = 256;
    w.cta_start = al(w.tile_start + (static_cast<size_t>(B) + 1) * 4);
    w.head_top = w.cta_start + static_cast<size_t>(w.grid) * 16;
    w.unit_top = w.head_top + static_cast<size_t>(d->H) * 8;
    w.bias = al(w.unit_top + static_cast<size_t>(units) * 4);
    w.qimg = w.bias + static_cast<size_t>(d->H) * 4096;
    w.qback = w.qimg + static_cast<size_t>(units * groups) * tree_rows(max_nodes, d->r_v) * 512;
    w.khat = al(w.qback + static_cast<size_t>(units * groups) * tree_rows(max_nodes, d->r_v) * 4);
    w.kback = w.khat + static_cast<size_t>(units) * max_nodes * 512;
    w.paths = al(w.kback + static_cast<size_t>(units) * max_nodes * 4);
    w.records = al(w.paths + static_cast<size_t>(std::max(B, 1)) * max_nodes * 16);
    w.total = w.records + static_cast<size_t>(units * groups + w.grid) * rec;
    return w;
  }
  // plain kernel: about four blocks an SM, splits of whole tiles
  const int64_t tiles = std::max<int64_t>(1, (L_max + kTreePlainTile - 1) / kTreePlainTile);
  const int64_t want = std::min(tiles, std::max<int64_t>(1, 4 * sms / units));
  const int64_t per = (tiles + want - 1) / want;
  w.chunk = per * kTreePlainTile;
  w.splits = static_cast<int>((tiles + per - 1) / per);
  w.turned = 256;
  w.v_turned = 256 + static_cast<size_t>(d->H) * d->r_k * kHeadDim * 4;
  w.records = w.v_turned + static_cast<size_t>(d->H) * d->r_v * kHeadDim * 4;
  // (units x splits is at most max(units, 4 sms), a bound that does not fall as the batch grows)
  w.total = w.records + static_cast<size_t>(std::min(units * tiles, std::max<int64_t>(units, 4 * sms))) * rec;
  return w;
}

// bf16 tensor of up to four dimensions as a map; strides in bytes of dimensions 1.., swizzle of the box's rows.
bool map_4d(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* strides, const uint32_t* box) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t d[4], st[3];
  cuuint32_t b[4], one[4] = {1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
    if (i > 0) st[i - 1] = strides[i - 1];
  }
  const CUtensorMapSwizzle sw = box[0] == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : box[0] == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B;
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), d, st, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool tree_maps(const TreeArgs& a, TreeMaps* m) {
  *m = TreeMaps{};
  // rows of one (sequence or page, head): L_max or page_size of them
  const uint64_t rows = static_cast<uint64_t>(a.block_table ? a.page_size : a.L_max);
  const uint64_t outer = static_cast<uint64_t>(a.block_table ? a.num_pages : a.B) * a.H;
  const uint32_t box_rows = a.block_table ? a.piece : kTile;
  const uint64_t rk = a.r_k, rv = a.r_v;
  const bool copies = !a.block_table || a.piece >= 8;       // else row by row, without a map
  auto latents = [&](CUtensorMap* map, const void* base, uint64_t r, uint32_t width) {
    const uint64_t d[3] = {r, rows, outer}, st[2] = {2 * r, 2 * r * rows};
    const uint32_t box[3] = {width, box_rows, 1};
    return map_4d(map, base, 3, d, st, box);
  };
  for (int c = 0; c < a.plan.kplan.n; ++c) {
    const uint32_t width = a.plan.kplan.width[c];
    const int i = chunk_map_index(width);
    if (copies && !latents(&m->k[i], a.cache_k, rk, width)) return false;
    // row pair_index of member 0 or 1: f and f + 64, or 2 f and 2 f + 1
    const uint64_t step = a.rope_style == 0 ? 1 : 2, member = a.rope_style == 0 ? 64 : 1;
    const uint64_t d[4] = {rk, 64, 2, static_cast<uint64_t>(a.H)}, st[3] = {2 * rk * step, 2 * rk * member, 2 * rk * kHeadDim};
    const uint32_t box[4] = {width, 64, 2, 1};
    if (!map_4d(&m->w[i], a.w_up_k, 4, d, st, box)) return false;
  }
  if (!copies) return true;
  if (rv % 32 == 0) {
    const uint64_t d[4] = {32, rows, rv / 32, outer}, st[3] = {2 * rv, 64, 2 * rv * rows};
    const uint32_t box[4] = {32, box_rows, static_cast<uint32_t>(rv / 32), 1};
    if (!map_4d(&m->v4, a.cache_v, 4, d, st, box)) return false;
  }
  return latents(&m->v, a.cache_v, rv, 32);
}

lla_status tree_attn(const lla_dims* dims, int loop_t, const lla_tree* tree, const void* q, int64_t q_stride, const void* k,
                     int64_t k_stride, const void* v, int64_t v_stride, const View& cache, const int32_t* seq_lens,
                     const void* w_up_k, const void* w_up_v, const float* mu_k, const float* mu_v, const float* rope_cos,
                     const float* rope_sin, int64_t rope_len, void* out, float* lse, void* workspace, size_t ws_bytes,
                     void* stream) {
  if (!tree || loop_t < 0 || loop_t >= dims->T || tree->B < 0 || tree->n_tok < 0 || tree->max_nodes < 1 ||
      cache.B != tree->B || cache.L_max < 1)
    return LLA_ERR_INVALID_ARG;
  // (tiles: of every block of nodes, which the tensor-core kernels count in 32 bits)
  const int64_t blocks = tensor_path(dims) ? (tree->max_nodes + tree_group(dims->r_v) - 1) / tree_group(dims->r_v) : 1;
  if (tree->max_nodes > kTreeMaxNodes || cache.L_max > (int64_t(1) << 30) ||
      static_cast<int64_t>(tree->B) * dims->H > (int64_t(1) << 24) ||
      static_cast<int64_t>(tree->n_tok) * dims->H >= (int64_t(1) << 31) ||
      static_cast<int64_t>(tree->B) * dims->H * blocks * ((cache.L_max + kTile - 1) / kTile) >= (int64_t(1) << 30))
    return LLA_ERR_UNSUPPORTED;
  if (tree->B == 0 || tree->n_tok == 0) return LLA_OK;
  if (rope_len < cache.L_max || rope_len < kTile) return LLA_ERR_INVALID_ARG;
  const int64_t es = dims->dtype == LLA_BF16 ? 2 : 4, width = static_cast<int64_t>(dims->H) * kHeadDim;
  const int64_t strides[] = {q_stride, k_stride, v_stride};
  for (int64_t x : strides)
    if (x < width || x * es % 16 || x > (int64_t(1) << 40)) return LLA_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k, v, cache.k, cache.v, w_up_k, w_up_v, mu_k, mu_v, rope_cos, rope_sin, out, workspace};
  for (const void* p : ptrs)
    if (!at16(p)) return LLA_ERR_INVALID_ARG;
  const void* words[] = {tree->tok_start, tree->parent, tree->pos, seq_lens};
  for (const void* p : words)
    if (!at4(p)) return LLA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(lse) & 3u) || ws_bytes < 256) return LLA_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  TreeArgs a{};
  const bool tensor = tensor_path(dims) && make_tree_plan(dims->r_k, dims->r_v, tree_rows(tree->max_nodes, dims->r_v), &a.plan);
  const TreeWs w = tree_ws(dims, tree->B, tree->max_nodes, cache.L_max, std::max(1, sms), tensor);
  if (ws_bytes < w.total) return LLA_ERR_INVALID_ARG;
  // (blocks read what belongs to other nodes while they write)
  const int64_t n = tree->n_tok, H = dims->H, TH = static_cast<int64_t>(dims->T) * H;
  const int64_t rows = cache.bt ? product({cache.num_pages, H, cache.page_size}) : product({cache.B, H, cache.L_max});
  const Span outs[] = {{out, product({n, width, es})}, {lse, product({n, H, 4})}, {workspace, static_cast<int64_t>(w.total)}};
  const Span ins[] = {{q, row_bytes(n, q_stride, width, es)}, {k, row_bytes(n, k_stride, width, es)}, {v, row_bytes(n, v_stride, width, es)},
                      {cache.k, product({rows, dims->r_k, es})}, {cache.v, product({rows, dims->r_v, es})},
                      {w_up_k, product({TH, kHeadDim, dims->r_k, es})}, {w_up_v, product({TH, kHeadDim, dims->r_v, es})},
                      {mu_k, product({TH, kHeadDim, 4})}, {mu_v, product({TH, kHeadDim, 4})},
                      {rope_cos, product({rope_len, kHeadDim / 2, 4})}, {rope_sin, product({rope_len, kHeadDim / 2, 4})},
                      {seq_lens, product({tree->B, 4})}, {tree->tok_start, product({tree->B, 4}) + 4}, {tree->parent, n * 4}, {tree->pos, n * 4},
                      {cache.bt, product({cache.B, cache.max_pages, 4})}};
  if (outputs_meet(outs, ins)) return LLA_ERR_INVALID_ARG;
  if (sms <= 0) return LLA_ERR_CUDA;
  a.B = tree->B;
  a.H = dims->H;
  a.r_k = dims->r_k;
  a.r_v = dims->r_v;
  a.rope_style = dims->rope_style;
  a.n_tok = tree->n_tok;
  a.max_nodes = tree->max_nodes;
  a.L_max = cache.L_max;
  a.rope_len = rope_len;
  a.mu_hstride = static_cast<int64_t>(dims->T) * kHeadDim;
  a.tok_start = tree->tok_start;
  a.parent = tree->parent;
  a.pos = tree->pos;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.seq_lens = seq_lens;
  a.cache_k = cache.k;
  a.cache_v = cache.v;
  a.block_table = cache.bt;
  a.page_size = cache.page_size;
  a.max_pages = cache.max_pages;
  a.num_pages = cache.num_pages;
  a.piece = std::min(kTile, cache.page_size & -cache.page_size);
  a.w_up_k = static_cast<const uint8_t*>(w_up_k) + static_cast<size_t>(loop_t) * width * dims->r_k * es;
  a.w_up_v = static_cast<const uint8_t*>(w_up_v) + static_cast<size_t>(loop_t) * width * dims->r_v * es;
  a.mu_k = mu_k + static_cast<size_t>(loop_t) * kHeadDim;
  a.mu_v = mu_v + static_cast<size_t>(loop_t) * kHeadDim;
  a.rope_cos = rope_cos;
  a.rope_sin = rope_sin;
  a.out = out;
  a.lse = lse;
  a.status = static_cast<uint32_t*>(workspace);
  a.records = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + w.records);
  a.rec_rows = a.max_nodes;
  a.splits = w.splits;
  // nodes of a finish block: few enough that there are four blocks an SM, at most eight (which share W_up,v in L1)
  a.finish_rows = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(8, static_cast<int64_t>(tree->n_tok) * dims->H / (4 * sms))));
  a.chunk = w.chunk;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf16 = dims->dtype == LLA_BF16;
  if (tensor) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.group = tree_group(a.r_v);
    a.groups = (a.max_nodes + a.group - 1) / a.group;
    a.rows = tree_rows(a.max_nodes, a.r_v);
    a.v_whole = a.r_v % 32 == 0;
    a.rec_rows = std::min(a.max_nodes, a.group);
    a.grid = w.grid;
    a.tile_start = reinterpret_cast<int32_t*>(ws + w.tile_start);
    a.cta_start = reinterpret_cast<int4*>(ws + w.cta_start);
    a.head_top = reinterpret_cast<float2*>(ws + w.head_top);
    a.unit_top = reinterpret_cast<float*>(ws + w.unit_top);
    a.bias = ws + w.bias;
    a.qimg = ws + w.qimg;
    a.qback = reinterpret_cast<float*>(ws + w.qback);
    a.khat = ws + w.khat;
    a.kback = reinterpret_cast<float*>(ws + w.kback);
    a.paths = reinterpret_cast<uint4*>(ws + w.paths);
    TreeMaps maps;
    if (!tree_maps(a, &maps)) return LLA_ERR_CUDA;
    return launch_tree_tensor(a, maps, s) == cudaSuccess ? LLA_OK : LLA_ERR_CUDA;
  }
  a.w_turned = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + w.turned);
  a.v_turned = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + w.v_turned);
  if (launch_tree_plain(a, bf16, s) != cudaSuccess || launch_tree_finish(a, bf16, s) != cudaSuccess) return LLA_ERR_CUDA;
  return LLA_OK;
}

}  // namespace

extern "C" {

const char* lla_tree_kernel(const lla_dims* dims, int page_size) {
  if (checked_dims(dims) != LLA_OK || dims->variant != LLA_PER_HEAD || page_size < 0) return nullptr;
  return tensor_path(dims) ? "tensor" : "plain";
}

size_t lla_tree_workspace_size(const lla_dims* dims, int B, int max_nodes, int64_t L_max) {
  if (checked_dims(dims) != LLA_OK || dims->variant != LLA_PER_HEAD || B < 0 || max_nodes < 1 ||
      max_nodes > kTreeMaxNodes || L_max < 0)
    return 0;
  return tree_ws(dims, B, max_nodes, L_max, std::max(1, device_sm_count()), tensor_path(dims)).total;
}

lla_status lla_tree_attn(const lla_dims* dims, int loop_t, const lla_tree* tree, const void* q, int64_t q_stride,
                         const void* k, int64_t k_stride, const void* v, int64_t v_stride, lla_cache cache,
                         const int32_t* seq_lens, const void* w_up_k, const void* w_up_v, const float* mu_k,
                         const float* mu_v, const float* rope_cos, const float* rope_sin, int64_t rope_len,
                         void* out, float* lse, void* workspace, size_t ws_bytes, void* stream) {
  const lla_status st = checked_dims(dims);
  if (st != LLA_OK) return st;
  if (dims->variant != LLA_PER_HEAD) return LLA_ERR_UNSUPPORTED;
  return tree_attn(dims, loop_t, tree, q, q_stride, k, k_stride, v, v_stride,
                   View{cache.k, cache.v, cache.B, cache.L_max, nullptr, 0, 0, 0}, seq_lens, w_up_k, w_up_v, mu_k, mu_v,
                   rope_cos, rope_sin, rope_len, out, lse, workspace, ws_bytes, stream);
}

lla_status lla_tree_attn_paged(const lla_dims* dims, int loop_t, const lla_tree* tree, const void* q,
                               int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                               lla_paged_cache cache, const int32_t* seq_lens, const void* w_up_k,
                               const void* w_up_v, const float* mu_k, const float* mu_v, const float* rope_cos,
                               const float* rope_sin, int64_t rope_len, void* out, float* lse, void* workspace,
                               size_t ws_bytes, void* stream) {
  const lla_status st = checked_dims(dims);
  if (st != LLA_OK) return st;
  if (dims->variant != LLA_PER_HEAD) return LLA_ERR_UNSUPPORTED;
  if (cache.B < 0 || cache.max_pages < 1 || cache.page_size < 1 || cache.num_pages < 1) return LLA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(cache.max_pages) * cache.page_size > (int64_t(1) << 30) || cache.num_pages >= (int64_t(1) << 31) ||
      cache.num_pages * static_cast<int64_t>(dims->H) >= (int64_t(1) << 31) ||
      static_cast<int64_t>(cache.B) * cache.max_pages >= (int64_t(1) << 31))
    return LLA_ERR_UNSUPPORTED;
  if (cache.B > 0 && !at4(cache.block_table)) return LLA_ERR_INVALID_ARG;
  return tree_attn(dims, loop_t, tree, q, q_stride, k, k_stride, v, v_stride,
                   View{cache.k, cache.v, cache.B, static_cast<int64_t>(cache.max_pages) * cache.page_size, cache.block_table,
                        cache.page_size, cache.max_pages, cache.num_pages},
                   seq_lens, w_up_k, w_up_v, mu_k, mu_v, rope_cos, rope_sin, rope_len, out, lse, workspace, ws_bytes,
                   stream);
}

}  // extern "C"
