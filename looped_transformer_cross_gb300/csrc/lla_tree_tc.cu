// lla_tree_tc.cu — lla_tree_attn over bf16 latents on the tensor cores: the cached tokens'
// part of every node's softmax, one record (m, l, latent sum) per (unit, CTA, node).
//
// A unit is (sequence, head, block of up to 64 nodes); the flat list of the units' 128-token tiles is
// cut into equal contiguous ranges, one persistent CTA per SM.  Per tile, three matrix products,
// tokens in the rows of the first two:
//   U = C_k W^T + mu          128 tokens x 128 dimensions, latents by TMA
//   S = K^ Q^^T               128 tokens x nodes: K^ is U rotated by the warps below, over U in TMEM; Q^
//                             (rotated, scaled to log2 units) from tree_prepare_kernel
//   D += C_v^T P              r_v x nodes, both operands MN-major from shared memory
// K^, Q^ and P are each the sum of two 16-bit parts: one rounding to bf16 of each made the log-sum-exp 1e-3
// off and an output 1.5 times as far off as its own rounding.  K^ and Q^ are f16 + f16 (22 bits; products
// high x high, high x low, low x high), scaled by powers of two first: a row of Q^ to 1..2, a unit's keys by
// what brings a bound of them (row sums of |W| times a latent's largest value, and |mu|) to 16..32 at the upper
// quartile of 16 of its tokens.  A component is then off by 2^-22 of itself, or of 2^-8 of that bound where it is
// smaller, at any sizes of latents and weights; keys 2^11 times beyond the bound make the sums NaN, and the join then
// takes the cached tokens again in fp32.  P is
// bf16 + bf16 (16 bits at any size).
// A key is reconstructed and rotated once for all nodes of its block, V never is, and the
// products and exponentials of S and D are made for 16, 32 or 64 nodes, not for a full 128 rows.
// Weights are 2^(s - ref) with one reference per node and unit: the largest score of the unit's first
// tile.  Scores further on only have to stay below ref + 32 (bf16 keeps its digits at any size, and
// fp32 sums have the range); the softmax warps vote on that for every tile, and a tile that breaks it
// moves the references and rescales D.
//
// Roles: warp 0 copies K and V tiles, warp 1 issues U (and copies W and RoPE rows), warp 2 issues S
// (and copies Q^), warp 3 issues D; warps 4..11 rotate (two per TMEM lane quadrant, 32 frequencies
// each, one token per lane), warps 12..15 do the softmax, one token per lane.  cos/sin of a token's
// angle are the angle sum of the tile's base row (shared memory, without a factor that the table's rows may
// have) and the lane's own row (registers, or TMEM
// for up to 16 nodes: 5 % of the call at 32 x 4096; those kernels do not spill, those for 32 nodes 104 bytes a
// thread, those for 64 48).  The roles' loops are kept short on purpose: with bodies
// unrolled all the way, instruction fetch took more time than anything else.
//
// Measured (the whole call, 16 heads; bytes of the latents over the time): 32 x 4096 tokens at (96, 160) with up to
// 16 nodes 187 us, 5.4 TB/s of the 6.8 that a copy reaches; 8 x 16384 in 64-token pages with up to 64 nodes 265 us,
// 3.9 TB/s, where the softmax warps and 2,900 cycles of products a tile bound it; 128 x 4096 at (16, 32) with up to 8
// nodes 455 us, 1.4 TB/s: a tile's fixed part, 2,600 cycles, most of them the rotation's.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include <cuda_fp16.h>

#include "lla_tree.h"

namespace lla {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kInvSqrtD = 0.08838834764831845f;   // 1/sqrt(128)
constexpr float kHeadroom = 32.f;                   // a score this far above its reference (log2 units) moves it
// The tensor core cuts its sums off at 24 bits: up to 2^-23 of a sum is lost with every 16 tokens, always downwards
// (65536 tokens in one sum: log-sum-exp 1e-4 off, outputs 5e-4).  So a unit's latent sums go to its record, and
// start anew, every 64 tiles (512 steps, 2^-14 at most), and the sums of weights of 64 nodes to shared memory every 8
// (8 x 16384 with 64 nodes: 8 us of 259).
constexpr int kSumTiles = 64, kWeightTiles = 8;
constexpr int kPrepThreads = 256, kPrepWarps = kPrepThreads / 32;
constexpr int kRotWarps = 8;
constexpr int kSoftWarp0 = 4 + kRotWarps;
constexpr int kTreeThreads = 32 * (kSoftWarp0 + 4);
constexpr int kSCol = 256;                          // TMEM columns: U, then K^ in its place 0..255 (two), S (two), D

struct alignas(16) TreeMisc {
  uint64_t kfull[kMaxStages], kempty[kMaxStages], vfull[kMaxStages], vempty[kMaxStages];
  uint64_t wfull, wfree, qfull, qfree;              // the unit's W and bias; its queries
  uint64_t ufull[2];                                // U computed and the tile's base RoPE row written
  uint64_t rfull[2];                                // K^ written over U, the base row read
  uint64_t sfull[2], sfree[2];                      // S computed (and K^ read); S read
  uint64_t pfull[2], vdone[2];                      // P written; D += C_v^T P done
  uint64_t vote;                                    // the four softmax warps
  uint64_t done[3];
  uint32_t tmem_base;
  int abort;
  int over[2];                                      // tile + 1 in which a score passed its headroom
};
static_assert(sizeof(TreeMisc) <= 768, "misc region");

struct Walk {
  int b, h, g, t, ng, nb, L;        // block g of ng of the sequence's nodes; tile t of nb
};

// Tiles of sequence b: none without nodes.
__device__ __forceinline__ void walk_load(Walk& w, const TreeArgs& a) {
  int first;
  const int n = tree_nodes(a, w.b, first, false);
  w.L = tree_cached(a, w.b, false);
  w.ng = (n + a.group - 1) / a.group;
  w.nb = n > 0 ? (w.L + kTile - 1) / kTile : 0;
}

__device__ __forceinline__ void walk_next(Walk& w, const TreeArgs& a) {
  if (++w.t < w.nb) return;
  w.t = 0;
  if (++w.g < w.ng) return;
  w.g = 0;
  if (++w.h < a.H) return;
  w.h = 0;
  while (true) {
    if (++w.b >= a.B) { w.nb = 0; return; }
    walk_load(w, a);
    if (w.nb > 0) return;
  }
}

struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++slot == n) { slot = 0; phase ^= 1u; }
  }
};

// warp_wait with everything past the first test out of line: one copy of that code instead of one for
// each place that waits (instruction fetch bounds this kernel).
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort, uint32_t* status) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = mbar_wait(bar, parity, abort, status);
  __syncwarp();
  return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
}
__device__ __forceinline__ bool tile_wait(uint32_t bar, uint32_t parity, volatile int* abort, uint32_t* status) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return wait_on(bar, parity, abort, status);
}

// True in one lane of the warp, the same at every call.  Products are issued from a block that only this lane
// enters: one takes 24..110 cycles there (M 128, N 16..128) and 110..145 where the whole warp runs along with
// the instruction predicated, or where the lane is chosen by its number.
__device__ __forceinline__ bool elected() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Two fp32 lanes in one 64-bit register, and packed arithmetic on them.
__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t x, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x)); }
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
// x = hi + lo in f16: hi with x's first 11 bits, lo with the next 11 (both lanes).
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void split2(uint64_t x, uint32_t& hi, uint32_t& lo) {
  float x0, x1;
  unpack2(x, x0, x1);
  hi = pack_f16(x0, x1);
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tfma.rn.f32.f16 %0, l, %5, %3;\n\tfma.rn.f32.f16 %1, h, %5, %4;\n\t}"
      : "=f"(x0), "=f"(x1)
      : "r"(hi), "f"(x0), "f"(x1), "h"(static_cast<unsigned short>(0xBC00)));
  lo = pack_f16(x0, x1);
}
__device__ __forceinline__ void split_f16(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  hi = pack_f16(x0, x1);
  const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  lo = pack_f16(x0 - h.x, x1 - h.y);
}
// x = hi + mid + lo in bf16: 24 bits, all that fp32 has (both lanes).
__device__ __forceinline__ void less_bf16(uint32_t part, float& x0, float& x1) {       // x minus the part
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tfma.rn.f32.bf16 %0, l, %3, %0;\n\tfma.rn.f32.bf16 %1, h, %3, %1;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "r"(part), "h"(static_cast<unsigned short>(0xBF80)));
}
__device__ __forceinline__ void split_bf16(float x0, float x1, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  hi = pack_bf16(x0, x1);
  less_bf16(hi, x0, x1);
  mid = pack_bf16(x0, x1);
  less_bf16(mid, x0, x1);
  lo = pack_bf16(x0, x1);
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Store 8 consecutive 32-bit columns of this thread's lane.
__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// What the cached keys of a (sequence, head) are scaled by, and what undoes it: the power of two that brings the
// bound of its keys (see above) to 16..32, within what products of these powers with others leave finite.
__device__ __forceinline__ float2 key_scale(const TreeArgs& a, int b, int h) {
  const float2 top = __ldcg(&a.head_top[h]);
  const float bound = fmaf(top.x, __ldcg(a.unit_top + b * a.H + h), top.y);
  const int power = min(60, max(-60, 131 - static_cast<int>((__float_as_uint(bound) >> 23) & 255u)));
  return make_float2(__int_as_float((127 + power) << 23), __int_as_float((127 - power) << 23));
}

__device__ __forceinline__ int page_at(const TreeArgs& a, int b, int lp) {
  const int pg = __ldg(a.block_table + static_cast<int64_t>(b) * a.max_pages + lp);
  return min(max(pg, 0), static_cast<int>(a.num_pages) - 1);
}

// A chunk of a latent tile as the copying warp needs it (in shared memory: reading the plan's arrays
// out of the launch parameters for every copy cost more than the copies).
struct Chunk {
  int off, start, row, map;          // byte offset in a tile, first column, bytes of a row, tensor map
};

// Where the latents of a tile lie: the sequence or the tile's page or, with pieces, the lane's piece's page, as the
// maps' outer coordinate, and the first row in it.
struct Place {
  int y, page;                       // (the table's entry as it was read: what depends on it waits for the load)
};
template <int kPage>
__device__ __forceinline__ Place place_of(const TreeArgs& a, const Walk& w, int my_piece) {
  Place p{w.t * kTile, 0};
  if constexpr (kPage == 1 || kPage == 2) {
    if (kPage == 2) p.y += my_piece * a.piece;
    if (kPage == 1 || p.y < w.L) {
      const int lp = p.y / a.page_size;
      p.page = __ldg(a.block_table + static_cast<int64_t>(w.b) * a.max_pages + lp);
      p.y -= lp * a.page_size;
    }
  }
  return p;
}
template <int kPage>
__device__ __forceinline__ int outer_of(const TreeArgs& a, const Walk& w, const Place& p) {
  if constexpr (kPage == 1 || kPage == 2) return min(max(p.page, 0), static_cast<int>(a.num_pages) - 1) * a.H + w.h;
  return w.b * a.H + w.h;
}

// One latent tile into dst, completing on fb (the whole warp calls it).  A lane issues the boxes of one
// piece (those that hold tokens) or of the tile, every `every`-th chunk from its first on.
template <int kPage>
__device__ __forceinline__ void load_tile(const Walk& w, int y, int z, uint32_t dst, uint32_t fb, const Chunk* chunks, int n, int bytes,
                                          const CUtensorMap* maps, int piece, int my_piece, int first, int every) {
  int np = 1;
  if constexpr (kPage == 2) np = (min(kTile, w.L - w.t * kTile) + piece - 1) / piece;
  if ((threadIdx.x & 31) == 0) mbar_arrive_expect_tx(fb, kPage == 2 ? bytes / kTile * piece * np : bytes);
  __syncwarp();
  if (my_piece < np) {
    for (int c = first; c < n; c += every) {
      const Chunk k = chunks[c];
      tma_load_3d(dst + k.off + (kPage == 2 ? my_piece * piece * k.row : 0), maps + k.map, fb, k.start, y, z);
    }
  }
}

// Rows of one latent (width r) of a tile through the block table, into dst: 16 bytes a lane and step, as many
// rows at a time as a warp covers, to where the tile's chunks (n of them) have them; they complete on fb, on
// which every lane arrives.  `rows` holds the pool row of the tile's tokens lane, lane + 32, ..; tokens past the
// sequence's end are left out.
__device__ __forceinline__ void gather_tile(const void* pool, int r, const int64_t (&rows)[4], int valid, uint8_t* dst, uint32_t fb,
                                            const Chunk* chunks, int n) {
  const int lane = threadIdx.x & 31, gran = r >> 3, at_once = 32 / gran;      // (a row is 32 pieces of 16 bytes at most)
  const int sub = lane / gran, g = lane - sub * gran;
  int c = 0;
  while (c + 1 < n && 8 * g >= chunks[c + 1].start) ++c;
  const Chunk k = chunks[c];
  const uint32_t to = smem_u32(dst + k.off) + sub * k.row, col = (8 * g - k.start) * 2;
  const uint32_t mask = k.row == 128 ? 7u : k.row == 64 ? 3u : 1u, shift = k.row == 128 ? 0u : k.row == 64 ? 1u : 2u;
  const uint8_t* from = static_cast<const uint8_t*>(pool) + 16 * g;
  // (steps without a branch between them, so that their shuffles overlap; eight where a step is a few rows: 32 x 4096
  // tokens one a page 864 us, 1148 with a branch, 1395 two at a time; at the small ranks four, 1342 and 1473; both with what else there was then)
  auto steps = [&](auto most) {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int64_t mine = rows[b] * (2 * r);
      const int m = min(32, valid - 32 * b);
#pragma unroll 1
      for (int t0 = 0; t0 < m; t0 += most * at_once) {
#pragma unroll
        for (int i = 0; i < most; ++i) {
          const int t = t0 + i * at_once;
          const uint8_t* src = from + __shfl_sync(0xffffffffu, mine, (t + sub) & 31);
          const uint32_t row = 32 * b + t + sub;      // (its place in the swizzle: 16-byte pieces exchanged by rows)
          if (sub < at_once && t + sub < m)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + (32 * b + t) * k.row + (col ^ (((row >> shift) & mask) << 4))), "l"(src)
                         : "memory");
        }
      }
    }
  };
  if (at_once < 8) steps(std::integral_constant<int, 8>{});
  else steps(std::integral_constant<int, 4>{});
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(fb) : "memory");
}

// ---------------------------------------------------------------- preparation

// Eight frequency pairs of a vector: first and second members, from f0 on.
__device__ __forceinline__ void load_pairs8(const __nv_bfloat16* v, int style, int f0, float (&x0)[8], float (&x1)[8]) {
  if (style == 0) {
    unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(v + f0)), x0);
    unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(v + 64 + f0)), x1);
  } else {
    float lo[8], hi[8];
    unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(v + 2 * f0)), lo);
    unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(v + 2 * f0 + 8)), hi);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x0[k] = lo[2 * k]; x1[k] = lo[2 * k + 1];
      x0[4 + k] = hi[2 * k]; x1[4 + k] = hi[2 * k + 1];
    }
  }
}

// The pairs rotated, times `scale`: first members, then second members.
__device__ __forceinline__ void turn_pairs8(const float (&x0)[8], const float (&x1)[8], const float* c, const float* s, float scale,
                                            float (&z)[16]) {
#pragma unroll
  for (int k = 0; k < 8; k += 4) {
    const float4 c4 = __ldg(reinterpret_cast<const float4*>(c + k)), s4 = __ldg(reinterpret_cast<const float4*>(s + k));
    const float cc[4] = {c4.x, c4.y, c4.z, c4.w}, ss[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      z[k + e] = (x0[k + e] * cc[e] - x1[k + e] * ss[e]) * scale;
      z[8 + k + e] = (x0[k + e] * ss[e] + x1[k + e] * cc[e]) * scale;
    }
  }
}

// First a warp a (sequence, head): the size of its K latents, by which its cached keys are scaled.  Then a block a
// unit: its query operand, RoPE(q, pos) log2(e)/sqrt(d) as two f16 parts, each the
// shared-memory image (two chunks of 64 columns, 128-byte rows, swizzled), and its drafted keys, RoPE(k, pos)
// likewise, row by row; dimensions in the order first members of the pairs, then second members, as U's.
// Then B blocks: the nodes on each node's path as bits, and the checks of a sequence's values.  Then H
// blocks: mu of a head as an operand that ones multiply, in three bf16 parts (24 bits), and the largest row sum of
// |W_up,k| and |mu|.  The last
// block: tiles per sequence, and every CTA's first tile.
__global__ void __launch_bounds__(kPrepThreads, 5) tree_prepare_kernel(const __grid_constant__ TreeArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  const int units = a.B * a.H * a.groups;
  const int sized = (a.B * a.H + kPrepWarps - 1) / kPrepWarps;
  if (blockIdx.x < sized) {
    // a warp a (sequence, head): the largest values of the K latents of 16 tokens from the first to the last, 16 bytes
    // a lane, and their upper quartile, without zeros
    constexpr int kSampled = 16, kAtOnce = 4;
    __shared__ uint32_t most[kPrepWarps][kSampled];
    const int warp = tid >> 5, lane = tid & 31, bh = blockIdx.x * kPrepWarps + warp;
    if (bh >= a.B * a.H) return;
    int first;
    const int b = bh / a.H, h = bh - b * a.H, L = tree_cached(a, b, false), gran = a.r_k >> 3;
    const int pieces = L > 0 && tree_nodes(a, b, first, false) > 0 ? kSampled * gran : 0;    // (none of a sequence without nodes is read)
    if (lane < kSampled) most[warp][lane] = 0;
    __syncwarp();
    for (int i0 = lane; i0 < pieces; i0 += 32 * kAtOnce) {
      uint4 x[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int i = min(i0 + 32 * k, pieces - 1), s = i / gran;
        const int64_t at = latent_row(a.block_table, a.page_size, a.max_pages, a.num_pages, a.L_max, a.H, b, h,
                                      static_cast<int64_t>(L - 1) * s / (kSampled - 1), a.status);
        x[k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.cache_k) + at * a.r_k + 8 * (i - s * gran)));
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        float y[8], m = 0.f;
        unpack_bf16x8(x[k], y);
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(y[e]));
        atomicMax(&most[warp][min(i0 + 32 * k, pieces - 1) / gran], __float_as_uint(m));
      }
    }
    __syncwarp();
    const uint32_t m = lane < kSampled ? most[warp][lane] : 0u;
    int below = 0;
#pragma unroll
    for (int k = 0; k < kSampled; ++k) below += most[warp][k] < m || (most[warp][k] == m && k < lane) ? 1 : 0;
    const int zeros = __popc(__ballot_sync(0xffffffffu, lane < kSampled && m == 0));
    const bool pick = zeros == kSampled ? lane == 0 : below == zeros + 3 * (kSampled - 1 - zeros) / 4;
    if (lane < kSampled && pick) a.unit_top[bh] = __uint_as_float(m);
    return;
  }
  const int block = blockIdx.x - sized;
  if (block < units) {
    const int bh = block / a.groups, g = block - bh * a.groups;
    const int b = bh / a.H, h = bh - b * a.H;
    int first;
    const int n = tree_nodes(a, b, first, false) - g * a.group;
    if (n <= 0) return;
    first += g * a.group;
    uint8_t* img = a.qimg + static_cast<int64_t>(block) * a.rows * 512;
    float* back_q = a.qback + static_cast<int64_t>(block) * a.rows;
    uint8_t* keys = a.khat + (static_cast<int64_t>(bh) * a.max_nodes + g * a.group) * 512;
    float* back_k = a.kback + static_cast<int64_t>(bh) * a.max_nodes + g * a.group;
    for (int i = tid; i < a.rows * 16; i += kPrepThreads) {      // (whole warps: rows is a multiple of 16)
      const bool key = i >= a.rows * 8;
      const int it = key ? i - a.rows * 8 : i, r = it >> 3, f0 = (it & 7) * 8;
      float z[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) z[k] = 0.f;
      if (r < n) {
        const int64_t entry = first + r;
        const __nv_bfloat16* v = key ? static_cast<const __nv_bfloat16*>(a.k) + entry * a.k_stride
                                     : static_cast<const __nv_bfloat16*>(a.q) + entry * a.q_stride;
        float x0[8], x1[8];
        load_pairs8(v + h * kHeadDim, a.rope_style, f0, x0, x1);
        int p = __ldg(a.pos + entry);
        p = p < 0 ? 0 : (p >= a.rope_len ? static_cast<int>(a.rope_len - 1) : p);
        const int64_t at = static_cast<int64_t>(p) * 64 + f0;
        turn_pairs8(x0, x1, a.rope_cos + at, a.rope_sin + at, key ? 1.f : kLog2e * kInvSqrtD, z);
      }
      // the row times the power of two that brings its largest value to 1..2 (eight lanes hold a row)
      float top = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) top = fmaxf(top, fabsf(z[k]));
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const uint32_t e = min(max(__float_as_uint(top) >> 23, 1u), 253u);
      const float scale = __uint_as_float((254u - e) << 23);
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) split_f16(z[2 * k] * scale, z[2 * k + 1] * scale, hi[k], lo[k]);
      const uint4 h0 = make_uint4(hi[0], hi[1], hi[2], hi[3]), h1 = make_uint4(hi[4], hi[5], hi[6], hi[7]);
      const uint4 l0 = make_uint4(lo[0], lo[1], lo[2], lo[3]), l1 = make_uint4(lo[4], lo[5], lo[6], lo[7]);
      if (!key) {
        const uint32_t o = swizzle_offset(r * 128 + f0 * 2, 128);
        *reinterpret_cast<uint4*>(img + o) = h0;
        *reinterpret_cast<uint4*>(img + a.rows * 128 + o) = h1;
        *reinterpret_cast<uint4*>(img + a.rows * 256 + o) = l0;
        *reinterpret_cast<uint4*>(img + a.rows * 384 + o) = l1;
        if (f0 == 0) back_q[r] = __uint_as_float(e << 23);
      } else if (r < n) {
        uint8_t* to = keys + r * 512 + f0 * 2;
        *reinterpret_cast<uint4*>(to) = h0;
        *reinterpret_cast<uint4*>(to + 128) = h1;
        *reinterpret_cast<uint4*>(to + 256) = l0;
        *reinterpret_cast<uint4*>(to + 384) = l1;
        if (f0 == 0) back_k[r] = __uint_as_float(e << 23);
      }
    }
    return;
  }
  if (block < units + a.B) {
    const int b = block - units;
    __shared__ int32_t jump[2][kTreeMaxNodes];
    __shared__ uint4 path[2][kTreeMaxNodes];
    int first;
    const int n = tree_nodes(a, b, first, true), L = tree_cached(a, b, true);
    if (n == 0) return;
    if (a.block_table) {
      const int used = (L + a.page_size - 1) / a.page_size;
      for (int lp = tid; lp < used; lp += kPrepThreads) {
        const int pg = __ldg(a.block_table + static_cast<int64_t>(b) * a.max_pages + lp);
        if (pg < 0 || pg >= a.num_pages) record_status(a.status, LLA_ERR_DEVICE_ARG);
      }
    }
    if (tid < n) {
      int p = __ldg(a.parent + first + tid);
      const int at = __ldg(a.pos + first + tid);
      if (p < -1 || p >= tid || at < 0 || at >= a.rope_len) record_status(a.status, LLA_ERR_DEVICE_ARG);
      if (p < -1 || p >= tid) p = -1;
      jump[0][tid] = p;
      const uint32_t bit = 1u << (tid & 31), w = tid >> 5;
      path[0][tid] = make_uint4(w == 0 ? bit : 0, w == 1 ? bit : 0, w == 2 ? bit : 0, w == 3 ? bit : 0);
    }
    __syncthreads();
    // by pointer doubling
    int cur = 0;
    for (int reach = 1; reach < n; reach *= 2, cur ^= 1) {
      if (tid < n) {
        const int j = jump[cur][tid];
        uint4 m = path[cur][tid];
        if (j >= 0) {
          const uint4 o = path[cur][j];
          m = make_uint4(m.x | o.x, m.y | o.y, m.z | o.z, m.w | o.w);
        }
        path[cur ^ 1][tid] = m;
        jump[cur ^ 1][tid] = j >= 0 ? jump[cur][j] : -1;
      }
      __syncthreads();
    }
    if (tid < n) a.paths[static_cast<int64_t>(b) * a.max_nodes + tid] = path[cur][tid];
    return;
  }
  if (block < units + a.B + a.H) {
    const int h = block - units - a.B;
    __shared__ float2 most[kPrepThreads / 32];
    // the largest sum of a row's |W|, and |mu|, two threads a row
    const int dim = tid >> 1;
    const __nv_bfloat16* W = static_cast<const __nv_bfloat16*>(a.w_up_k) + (static_cast<int64_t>(h) * kHeadDim + dim) * a.r_k;
    float sum = 0.f;
#pragma unroll 4
    for (int c = (tid & 1) * 8; c < a.r_k; c += 16) {
      float x[8];
      unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(W + c)), x);
#pragma unroll
      for (int k = 0; k < 8; ++k) sum += fabsf(x[k]);
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum = warp_max(sum);
    const float mean = warp_max(fabsf(__ldg(a.mu_k + h * a.mu_hstride + dim)));
    if ((tid & 31) == 0) most[tid >> 5] = make_float2(sum, mean);
    if (tid < kHeadDim) {
      const int src = tid < 64 ? (a.rope_style == 0 ? tid : 2 * tid) : (a.rope_style == 0 ? tid : 2 * (tid - 64) + 1);
      const float mu = __ldg(a.mu_k + h * a.mu_hstride + src);
      const float hi = __bfloat162float(__float2bfloat16_rn(mu));
      const float mid = __bfloat162float(__float2bfloat16_rn(mu - hi));
      uint8_t* ab = a.bias + h * 4096;
      *reinterpret_cast<uint4*>(ab + swizzle_offset(tid * 32, 32)) = make_uint4(pack_bf16(hi, mid), pack_bf16(mu - hi - mid, 0.f), 0, 0);
      *reinterpret_cast<uint4*>(ab + swizzle_offset(tid * 32 + 16, 32)) = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    if (tid == 0) {
      float2 top = most[0];
      for (int k = 1; k < kPrepThreads / 32; ++k) top = make_float2(fmaxf(top.x, most[k].x), fmaxf(top.y, most[k].y));
      a.head_top[h] = top;
    }
    return;
  }
  // ---- the plan: prefix of the sequences' tiles, then each CTA's first (sequence, head, tile)
  constexpr int kHeld = 2048;
  __shared__ int tot[kPrepThreads];
  __shared__ int starts[kHeld];
  const int per = (a.B + kPrepThreads - 1) / kPrepThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  auto tiles = [&](int b) {          // of one head
    Walk w;
    w.b = b;
    walk_load(w, a);
    return w.nb * w.ng;
  };
  int sum = 0;
  for (int b = b0; b < b1; ++b) sum += tiles(b);
  tot[tid] = sum;
  __syncthreads();
  for (int o = 1; o < kPrepThreads; o <<= 1) {
    const int v = tid >= o ? tot[tid - o] : 0;
    __syncthreads();
    tot[tid] += v;
    __syncthreads();
  }
  const int64_t total = static_cast<int64_t>(tot[kPrepThreads - 1]) * a.H;
  const int64_t share = max(static_cast<int64_t>(1), (total + a.grid - 1) / a.grid);
  int at = tot[tid] - sum;
  for (int b = b0; b < b1; ++b) {
    a.tile_start[b] = at;
    if (b < kHeld) starts[b] = at;
    at += tiles(b);
  }
  if (tid == 0) a.tile_start[a.B] = tot[kPrepThreads - 1];
  __syncthreads();
  for (int c = tid; c < a.grid; c += kPrepThreads) {
    int4 s = make_int4(0, 0, 0, 0);
    const int64_t f0 = c * share;
    if (f0 < total) {
      // the last sequence that starts at or before this tile (one without tiles starts where the next does)
      int lo = 0, hi = a.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        const int64_t st = mid < kHeld ? starts[mid] : __ldcg(a.tile_start + mid);
        if (st * a.H <= f0) lo = mid;
        else hi = mid;
      }
      const int64_t rem = f0 - static_cast<int64_t>(lo < kHeld ? starts[lo] : __ldcg(a.tile_start + lo)) * a.H;
      // (z: the tile among the head's, over all its blocks of nodes)
      const int nt = tiles(lo);
      s = make_int4(lo, static_cast<int>(rem / nt), static_cast<int>(rem % nt), static_cast<int>(min(share, total - f0)));
    }
    a.cta_start[c] = s;
  }
}

// ---------------------------------------------------------------- the cached tokens

// kPage: 0 dense, 1 pages of a multiple of 128 tokens, 2 tiles in pieces of 8..64 tokens, each within a page, 3
// any page size, row by row.  kRows: nodes that S and D have room for (16, 32 or 64).
template <int kPage, int kRows>
__global__ void __launch_bounds__(kTreeThreads, 1)
tree_tile_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ TreeMaps maps) {
  // Up to 32 nodes (kBoth): D is r_v x nodes in blocks of 128 rows, B = P with the two parts side by side in a
  // token's row, into columns of their own.  64 nodes: D is its transpose, A = P^T with both parts' nodes one below
  // the other, 128 rows (8 products a tile where the other form takes 16 of N = 128 or 32 of N = 64, with
  // 109 and 78 cycles each against 46 + r_v / 2), and there is one buffer of P (shared memory) and of S (TMEM).
  constexpr bool kBoth = kRows <= 32;
  constexpr int kSBuf = kBoth ? 2 : 1, kPBuf = kBoth ? 2 : 1, kDCols = 2 * kRows;
  constexpr int kDCol = kSCol + kSBuf * kRows;        // (64 nodes: r_v columns, up to 176, and 16 of the weights' sums)
  static_assert(kDCol + (kBoth ? 2 * kDCols : 192) <= 512, "TMEM columns");
  constexpr uint32_t kPRow = kBoth ? kRows * 4 : kRows * 2;        // bytes of a token's weights
  constexpr uint32_t kPTile = kTile * kRows * 4, kLow = kBoth ? kRows * 2 : kTile * kPRow;     // (the lower parts' place)
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const TreePlan& P = a.plan;
  const uint32_t sbase = smem_u32(sm);
  TreeMisc* misc = reinterpret_cast<TreeMisc*>(sm + P.misc);
  volatile int* abort = &misc->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto bar = [&](const uint64_t& m) { return smem_u32(&m); };
  auto wait = [&](const uint64_t& m, uint32_t parity) { return tile_wait(smem_u32(&m), parity & 1u, abort, a.status); };

  if (tid == 0) {
    misc->abort = 0;
    misc->over[0] = misc->over[1] = 0;
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(bar(misc->kfull[s]), kPage == 3 ? 32 : 1); mbar_init(bar(misc->kempty[s]), 1);
      mbar_init(bar(misc->vfull[s]), kPage == 3 ? 32 : 1); mbar_init(bar(misc->vempty[s]), 1);
    }
    mbar_init(bar(misc->wfull), 1); mbar_init(bar(misc->wfree), 1);
    mbar_init(bar(misc->qfull), 1); mbar_init(bar(misc->qfree), 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(misc->ufull[s]), 2);
      mbar_init(bar(misc->rfull[s]), kRotWarps);
      mbar_init(bar(misc->sfull[s]), 1); mbar_init(bar(misc->sfree[s]), 4);
      mbar_init(bar(misc->pfull[s]), 4); mbar_init(bar(misc->vdone[s]), 1);
    }
    mbar_init(bar(misc->vote), 4);
    for (int s = 0; s < 3; ++s) mbar_init(bar(misc->done[s]), 1);
    fence_mbar_init();
  }
  if (warp == 0 && lane < 16) {
    const ChunkPlan& c = lane < 8 ? P.kplan : P.vplan;
    const int k = lane & 7;
    reinterpret_cast<Chunk*>(sm + P.chunks)[lane] = Chunk{c.off[k], c.start[k], c.width[k] * 2, lane < 8 ? chunk_map_index(c.width[k]) : 0};
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc(smem_u32(&misc->tmem_base), 512);
  }
  if (warp >= kSoftWarp0) {
    // ones that meet the three parts of mu: eight rows, the same for every eight tokens
    const int r = tid - 32 * kSoftWarp0;
    if (r < 8) {
      *reinterpret_cast<uint4*>(sm + P.ones + swizzle_offset(r * 32, 32)) = make_uint4(0x3F803F80u, 0x00003F80u, 0, 0);
      *reinterpret_cast<uint4*>(sm + P.ones + swizzle_offset(r * 32 + 16, 32)) = make_uint4(0, 0, 0, 0);
    }
    // and ones that sum weights
    if (!kBoth && r < 16) *reinterpret_cast<uint4*>(sm + P.ones + 256 + r * 16) = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = misc->tmem_base;
  const int4 first_tile = __ldcg(a.cta_start + blockIdx.x);
  const int count = first_tile.w;
  Walk w;
  w.b = first_tile.x;
  w.h = first_tile.y;
  w.g = w.t = 0;
  if (count > 0) {
    walk_load(w, a);
    w.g = first_tile.z / w.nb;
    w.t = first_tile.z - w.g * w.nb;
  }
  // this warp's products complete before TMEM is released
  auto products_done = [&](uint64_t& m) {
    umma_commit_warp(bar(m));
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar(m), 0) && global_timer_ns() - t0 < kWaitLimitNs) {}
  };
  // the copy that completes phase `phase` (from 0 on; below 0: none) of a barrier lands before the CTA can exit
  auto landed = [&](uint64_t& m, int phase) {
    const uint64_t t0 = global_timer_ns();
    while (phase >= 0 && !mbar_try_wait(bar(m), phase & 1) && global_timer_ns() - t0 < kWaitLimitNs) {}
  };

  if (warp == 0) {
    // ======================================================== K and V tiles
    // V tile i - 1 after K tile i: it is needed only once tile i - 1 has weights.  Page ids are read one
    // tile ahead.  (A copy costs this warp some hundred cycles: the fewer the better.)
    const int piece = a.piece, pieces = kPage == 2 ? kTile / piece : 1;
    const int my_piece = lane % pieces, first = lane / pieces, every = 32 / pieces;
    const Chunk* kc = reinterpret_cast<const Chunk*>(sm + P.chunks);
    const Chunk* vc = kc + 8;
    const int SK = P.SK, SV = P.SV, nk = P.kplan.n, nv = P.vplan.n, k_bytes = P.kplan.bytes, v_bytes = P.vplan.bytes;
    const uint32_t k_ring = sbase + P.k_ring, v_ring = sbase + P.v_ring;
    const uint32_t k_stage = P.k_stage, v_stage = P.v_stage;
    const bool v_whole = a.v_whole;
    Walk wv = w;
    Ring kr, vr;
    int issued_k = 0, issued_v = 0;
    Place at = {}, at_v = {};
    if (count > 0) at = place_of<kPage>(a, w, my_piece);
    // (row by row: the pool rows of this tile's tokens and of the one before it)
    int64_t rows[4] = {}, rows_v[4] = {};
    auto find_rows = [&]() {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = w.t * kTile + 32 * k + lane, lp = j / a.page_size;
        rows[k] = j < w.L ? (static_cast<int64_t>(page_at(a, w.b, lp)) * a.H + w.h) * a.page_size + (j - lp * a.page_size) : 0;
      }
    };
    for (int i = 0; i <= count && count > 0; ++i) {
      const Walk wt = w;
      Place at_k = at;
      if (i < count) {
        if (!wait(misc->kempty[kr.slot], kr.phase ^ 1u)) break;
        if constexpr (kPage == 3) {
          find_rows();
          gather_tile(a.cache_k, a.r_k, rows, w.L - w.t * kTile < kTile ? w.L - w.t * kTile : kTile, sm + P.k_ring + kr.slot * k_stage,
                      bar(misc->kfull[kr.slot]), kc, nk);
        } else {
          load_tile<kPage>(w, at.y, outer_of<kPage>(a, w, at), k_ring + kr.slot * k_stage, bar(misc->kfull[kr.slot]), kc, nk, k_bytes, maps.k, piece, my_piece,
                           first, every);
        }
        issued_k = i + 1;
        kr.next(SK);
        walk_next(w, a);
        if (i + 1 < count) at = place_of<kPage>(a, w, my_piece);
      }
      if (i > 0) {
        if (!wait(misc->vempty[vr.slot], vr.phase ^ 1u)) break;
        if constexpr (kPage == 3) {
          gather_tile(a.cache_v, a.r_v, rows_v, min(kTile, wv.L - wv.t * kTile), sm + P.v_ring + vr.slot * v_stage,
                      bar(misc->vfull[vr.slot]), vc, nv);
        } else if (v_whole) {                         // all of a tile's, or a piece's, columns in one copy
          const int np = kPage == 2 ? (min(kTile, wv.L - wv.t * kTile) + piece - 1) / piece : 1;
          const uint32_t vb = bar(misc->vfull[vr.slot]), region = kPage == 2 ? piece * nv * 64 : v_bytes;
          if (lane == 0) mbar_arrive_expect_tx(vb, region * np);
          __syncwarp();
          if (lane < np) tma_load_4d(v_ring + vr.slot * v_stage + lane * region, &maps.v4, vb, 0, at_v.y, 0, outer_of<kPage>(a, wv, at_v));
        } else {
          load_tile<kPage>(wv, at_v.y, outer_of<kPage>(a, wv, at_v), v_ring + vr.slot * v_stage, bar(misc->vfull[vr.slot]), vc, nv, v_bytes, &maps.v, piece, my_piece,
                           first, every);
        }
        issued_v = i;
        vr.next(SV);
      }
      wv = wt;
      at_v = at_k;
      if constexpr (kPage == 3) {
#pragma unroll
        for (int k = 0; k < 4; ++k) rows_v[k] = rows[k];
      }
    }
    if (lane == 0) {
      for (int i = max(0, issued_k - P.SK); i < issued_k; ++i) landed(misc->kfull[i % P.SK], i / P.SK);
      for (int i = max(0, issued_v - P.SV); i < issued_v; ++i) landed(misc->vfull[i % P.SV], i / P.SV);
    }
  } else if (warp == 1) {
    // ======================================================== U = C_k W^T + mu
    const uint32_t idesc = umma_idesc_bf16(128, 128, false, false);
    const uint64_t d_ones = umma_desc(sbase + P.ones, 16, 0, kSw32), d_mu = umma_desc(sbase + P.mu, 16, 256, kSw32);
    const int r_k = a.r_k, n64 = r_k / 64, k32 = r_k & 32, k16 = r_k & 16;
    const int o32 = r_k / 64 * 16384, o16 = o32 + (r_k & 32) * 256;
    const uint32_t k_ring = sbase + P.k_ring, wb = sbase + P.w, kst = static_cast<uint32_t>(P.k_stage) >> 4;
    const uint64_t a64 = umma_desc(k_ring, 16, 1024, kSw128), b64 = umma_desc(wb, 16, 1024, kSw128);
    const uint64_t a32 = umma_desc(k_ring + o32, 16, 512, kSw64), b32 = umma_desc(wb + o32, 16, 512, kSw64);
    const uint64_t a16 = umma_desc(k_ring + o16, 16, 256, kSw32), b16 = umma_desc(wb + o16, 16, 256, kSw32);
    const int SK = P.SK;
    Ring kr;
    int unit = -1;
    // the tile's base row of the RoPE table too: a lane takes four cosines or sines, read one tile ahead
    const float* table = lane < 16 ? a.rope_cos + 4 * lane : a.rope_sin + 4 * (lane - 16);
    float4 ahead = make_float4(0.f, 0.f, 0.f, 0.f);
    auto fetch = [&]() { ahead = __ldg(reinterpret_cast<const float4*>(table + static_cast<int64_t>(w.t) * kTile * 64)); };
    // what the base row is multiplied by: the scale of the unit's keys, and what undoes the factor on the table's rows
    // (the cosines of row 0), which the lanes' own rows bring once already
    const float4 on_rows = __ldg(reinterpret_cast<const float4*>(a.rope_cos + 4 * (lane & 15)));
    float4 scale = make_float4(1.f, 1.f, 1.f, 1.f);
    if (count > 0) fetch();
    for (int i = 0; i < count; ++i) {
      if (i == 0 || w.t == 0) {
        if (unit >= 0 && !wait(misc->wfree, unit)) break;
        ++unit;
        if (lane == 0) {
          const uint32_t wf = bar(misc->wfull);
          mbar_arrive_expect_tx(wf, P.kplan.bytes + 4096);
          for (int c = 0; c < P.kplan.n; ++c)
            tma_load_4d(sbase + P.w + P.kplan.off[c], &maps.w[chunk_map_index(P.kplan.width[c])], wf, P.kplan.start[c], 0, 0, w.h);
          bulk_load(sbase + P.mu, a.bias + static_cast<int64_t>(w.h) * 4096, 4096, wf);
        }
        __syncwarp();
        const float keys = key_scale(a, w.b, w.h).x;  // (with the copies under way)
        scale = make_float4(__fdividef(keys, on_rows.x), __fdividef(keys, on_rows.y), __fdividef(keys, on_rows.z), __fdividef(keys, on_rows.w));
        if (!wait(misc->wfull, unit)) break;
      }
      if (!wait(misc->kfull[kr.slot], kr.phase)) break;
      if constexpr (kPage == 3) fence_proxy_async_smem();       // (plain copies, read by the products)
      if (i >= 2 && !wait(misc->sfull[i & 1], (i - 2) >> 1)) break;      // S(i - 2) has read the K^ in U(i)'s place
      reinterpret_cast<float4*>(sm + P.base + (i & 1) * 512)[lane] = make_float4(ahead.x * scale.x, ahead.y * scale.y, ahead.z * scale.z, ahead.w * scale.w);
      tc_fence_after();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(misc->ufull[i & 1]));
      // (chunks of 64 columns, then one of 32, then one of 16)
      const uint32_t d = tmem + (i & 1) * 128, so = kr.slot * kst;
      if (elected()) {
        umma_bf16(d, d_ones, d_mu, idesc, 0);
#pragma unroll 1
        for (int c = 0; c < n64; ++c) {
          const uint64_t ac = a64 + so + c * 1024, bc = b64 + c * 1024;
#pragma unroll
          for (int k = 0; k < 4; ++k) umma_bf16(d, ac + 2 * k, bc + 2 * k, idesc, 1);
        }
        if (k32) {
          umma_bf16(d, a32 + so, b32, idesc, 1);
          umma_bf16(d, a32 + so + 2, b32 + 2, idesc, 1);
        }
        if (k16) umma_bf16(d, a16 + so, b16, idesc, 1);
        umma_commit(bar(misc->ufull[i & 1]));
        umma_commit(bar(misc->kempty[kr.slot]));
        if (w.t == w.nb - 1) umma_commit(bar(misc->wfree));
      }
      __syncwarp();
      kr.next(SK);
      walk_next(w, a);
      if (i + 1 < count) fetch();
    }
    products_done(misc->done[0]);
    landed(misc->wfull, unit);
  } else if (warp == 2) {
    // ======================================================== S = K^ Q^^T
    const uint32_t idesc = umma_idesc_f16(128, kRows);
    const uint64_t d_q = umma_desc(sbase + P.q, 16, 1024, kSw128);
    int unit = -1;
    for (int i = 0; i < count; ++i) {
      const int sb = i % kSBuf;
      if (i == 0 || w.t == 0) {
        if (unit >= 0 && !wait(misc->qfree, unit)) break;
        ++unit;
        if (lane == 0) {
          const uint32_t qf = bar(misc->qfull);
          mbar_arrive_expect_tx(qf, kRows * 512);
          bulk_load(sbase + P.q, a.qimg + (static_cast<int64_t>(w.b * a.H + w.h) * a.groups + w.g) * (kRows * 512), kRows * 512, qf);
        }
        __syncwarp();
        if (!wait(misc->qfull, unit)) break;
      }
      if (!wait(misc->rfull[i & 1], i >> 1)) break;
      if (i >= kSBuf && !wait(misc->sfree[(i - kSBuf) & 1], (i - kSBuf) >> 1)) break;
      // the weights of tile i - 2 have been read: those of S(i) take their place (one wait here instead of one for
      // each softmax warp)
      if (kPBuf == 2 && i >= 2 && !wait(misc->vdone[i & 1], (i - 2) >> 1)) break;
      tc_fence_after();
      if (elected()) {
        const uint32_t d = tmem + kSCol + sb * kRows, high = tmem + (i & 1) * 128;
#pragma unroll 1
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint64_t q_high = d_q + c * (kRows * 128 / 16) + k * 2;
            umma_bf16_ts(d, high + 64 * c + 16 * k, q_high, idesc, c + k > 0);
            umma_bf16_ts(d, high + 64 * c + 16 * k, q_high + kRows * 256 / 16, idesc, 1);
            umma_bf16_ts(d, high + 64 * c + 16 * k + 8, q_high, idesc, 1);
          }
        umma_commit(bar(misc->sfull[i & 1]));
        if (w.t == w.nb - 1) umma_commit(bar(misc->qfree));
      }
      __syncwarp();
      walk_next(w, a);
    }
    products_done(misc->done[1]);
    landed(misc->qfull, unit);
  } else if (warp == 3) {
    // ======================================================== D += C_v^T P
    // (two blocks of 128 rows of r_v; rows past r_v read whatever follows the tile in shared memory and
    // are not looked at)
    const uint32_t idesc = umma_idesc_bf16(128, kBoth ? kDCols : a.r_v, true, true);
    // V: chunks of 32 columns, their 128 token rows of 64 bytes one after the other; with one copy per piece of
    // 8..64 tokens, piece by piece, each [chunk][piece rows]
    const bool by_piece = kPage == 2 && a.v_whole;
    const int nv = P.vplan.n, rows = by_piece ? a.piece : kTile;             // rows of a chunk that lie together
    const uint32_t region = rows * nv * 64;
    const uint64_t d_v = umma_desc(sbase + P.v_ring, rows * 64, rows >= 16 ? 512 : region, kSw64);
    const uint32_t block_step = 4 * rows * 64 / 16;
    const uint32_t idesc_sum = umma_idesc_bf16(128, 16, true, false);
    const uint64_t d_sum = umma_desc(sbase + P.ones + 256, 16, 0, kSw32);
    const int log_rows = 31 - __clz(rows);
    const uint64_t d_p = umma_desc(sbase + P.p, kTile * kPRow, 8 * kPRow, sw_mode_for_row_bytes(kPRow));     // (64 nodes: lower parts a tile on)
    const uint32_t vst = static_cast<uint32_t>(P.v_stage) >> 4;
    const int SV = P.SV, blocks = kBoth ? P.blocks : 1;
    Ring vr;
    for (int j = 0; j < count; ++j, vr.next(SV)) {
      if (!wait(misc->vfull[vr.slot], vr.phase)) break;
      if constexpr (kPage == 3) fence_proxy_async_smem();
      // rows past the sequence's end: whole steps of 16 tokens are left out, the rest of a partial step
      // is zeroed (it may hold anything; its weights are 0 and 0 * x stays 0)
      const int valid = min(kTile, w.L - w.t * kTile);
      const int steps = (valid + 15) / 16;
      if (valid < steps * 16) {
        uint8_t* vs = sm + P.v_ring + vr.slot * P.v_stage;
        const int per = (steps * 16 - valid) * 4;
        for (int x = lane; x < nv * per; x += 32) {
          const int c = x / per, r = valid + (x - c * per) / 4, g = x & 3;
          *reinterpret_cast<uint4*>(vs + (r >> log_rows) * region + c * rows * 64 + swizzle_offset((r & (rows - 1)) * 64 + g * 16, 64)) =
              make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (!wait(misc->pfull[j & 1], j >> 1)) break;
      tc_fence_after();
      const uint64_t a0 = d_v + vr.slot * vst, b0 = d_p + (j % kPBuf) * (kPTile / 16);
      // a unit's first product starts the sums, and every kSumTiles-th or kWeightTiles-th does again
      const uint32_t sum = j > 0 && w.t % kSumTiles != 0, sum_w = j > 0 && w.t % kWeightTiles != 0;
      if (elected()) {
#pragma unroll 1
        for (int blk = 0; blk < blocks; ++blk)
#pragma unroll 2
          for (int k = 0; k < steps; ++k) {
            // (rows is a power of two; a whole tile is one region)
            const uint32_t o = (16 * k >> log_rows) * (region / 16) + (16 * k & (rows - 1)) * 4;
            if (kBoth) umma_bf16(tmem + kDCol + blk * kDCols, a0 + blk * block_step + o, b0 + k * kPRow, idesc, k > 0 || sum);
            else {
              umma_bf16(tmem + kDCol, b0 + k * kPRow, a0 + o, idesc, k > 0 || sum);
              umma_bf16(tmem + kDCol + a.r_v, b0 + k * kPRow, d_sum, idesc_sum, k > 0 || sum_w);
            }
          }
        umma_commit(bar(misc->vdone[j & 1]));
        umma_commit(bar(misc->vempty[vr.slot]));
      }
      __syncwarp();
      walk_next(w, a);
    }
    products_done(misc->done[2]);
  } else if (warp < kSoftWarp0) {
    // ======================================================== rotation: U -> K^
    const int quad = warp & 3, row = 32 * quad + lane, f0 = 32 * ((warp - 4) >> 2);
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quad) << 16);
    // the lane's own row of the table, by twos: in registers, or, where TMEM has room for it (up to 16 nodes), there,
    // and the loop over the frequencies stays rolled
    constexpr bool kTable = kRows == 16;
    constexpr int kTabCol = kDCol + 2 * kDCols;
    uint64_t cl[kTable ? 8 : 16], sl[kTable ? 8 : 16];
    if constexpr (kTable) {
      uint4 x[16];                                    // cosines, then sines
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] = __ldg(reinterpret_cast<const uint4*>((k < 8 ? a.rope_cos : a.rope_sin) + row * 64 + f0 + 4 * (k & 7)));
#pragma unroll
      for (int c = 0; c < 16; c += 4) {
        const uint32_t y[16] = {x[c].x, x[c].y, x[c].z, x[c].w, x[c + 1].x, x[c + 1].y, x[c + 1].z, x[c + 1].w,
                                x[c + 2].x, x[c + 2].y, x[c + 2].z, x[c + 2].w, x[c + 3].x, x[c + 3].y, x[c + 3].z, x[c + 3].w};
        tmem_st_x16(lanes + kTabCol + (c >> 3) * 64 + f0 + (c & 7) * 4, y);
      }
      tmem_wait_st();
    } else {
#pragma unroll
      for (int f = 0; f < 16; f += 2) {
        const float4 c = __ldg(reinterpret_cast<const float4*>(a.rope_cos + row * 64 + f0 + 2 * f));
        const float4 s = __ldg(reinterpret_cast<const float4*>(a.rope_sin + row * 64 + f0 + 2 * f));
        cl[f] = pair2(c.x, c.y); cl[f + 1] = pair2(c.z, c.w);
        sl[f] = pair2(s.x, s.y); sl[f + 1] = pair2(s.z, s.w);
      }
    }
    const uint64_t minus = pair2(-1.f, -1.f);
    const float* rows = reinterpret_cast<const float*>(sm + P.base) + f0;
    for (int i = 0; i < count; ++i) {
      const uint32_t t_u = lanes + (i & 1) * 128 + f0;
      const float* base = rows + (i & 1) * 128;       // cos, then sin
      if (!wait(misc->ufull[i & 1], i >> 1)) break;
      tc_fence_after();
#pragma unroll(kTable ? 1 : 2)
      for (int g = 0; g < 2; ++g) {
        float u0[16], u1[16];
        tmem_ld_x16(t_u + 16 * g, u0);
        tmem_ld_x16(t_u + 64 + 16 * g, u1);
        if constexpr (kTable) {
          float c[16], sn[16];
          tmem_ld_x16(lanes + kTabCol + f0 + 16 * g, c);
          tmem_ld_x16(lanes + kTabCol + 64 + f0 + 16 * g, sn);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            cl[k] = pair2(c[2 * k], c[2 * k + 1]);
            sl[k] = pair2(sn[2 * k], sn[2 * k + 1]);
          }
        } else {
          tmem_wait_ld();
        }
        uint32_t y0[16], y1[16];                      // (higher parts, then lower)
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          const float4 c4 = *reinterpret_cast<const float4*>(base + 16 * g + 2 * k);
          const float4 s4 = *reinterpret_cast<const float4*>(base + 64 + 16 * g + 2 * k);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint64_t cb = e == 0 ? pair2(c4.x, c4.y) : pair2(c4.z, c4.w), sb = e == 0 ? pair2(s4.x, s4.y) : pair2(s4.z, s4.w);
            const int f = (kTable ? 0 : 8 * g) + k + e;
            const uint64_t c = fma2(mul2(sb, sl[f]), minus, mul2(cb, cl[f])), sn = fma2(sb, cl[f], mul2(cb, sl[f]));
            const uint64_t x0 = pair2(u0[2 * (k + e)], u0[2 * (k + e) + 1]), x1 = pair2(u1[2 * (k + e)], u1[2 * (k + e) + 1]);
            split2(fma2(mul2(x1, sn), minus, mul2(x0, c)), y0[k + e], y0[8 + k + e]);
            split2(fma2(x0, sn, mul2(x1, c)), y1[k + e], y1[8 + k + e]);
          }
        }
        tmem_st_x16(t_u + 16 * g, y0);
        tmem_st_x16(t_u + 64 + 16 * g, y1);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(misc->rfull[i & 1]));
    }
  } else {
    // ======================================================== softmax: S -> P, records
    const int quad = warp & 3, row = 32 * quad + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quad) << 16);
    // Of this unit's nodes: what brings a score to log2 units, minus the reference, and what the sums were
    // multiplied by when the references moved.  A lane holds the first two of nodes lane and lane + 32; for
    // all lanes they are in shared memory, where all four warps write the same values after a vote.  The
    // warps' maxima (two sets in turn).
    constexpr int kMine = (kRows + 31) / 32;
    float back[kMine], refs[kMine];
    float* scale = reinterpret_cast<float*>(sm + P.refs);
    float* minus_ref = scale + kRows;
    float* factor = minus_ref + kRows;
    float* maxima = factor + kRows;
    int votes = 0, moves = 0;
    auto vote = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(misc->vote));
      return wait(misc->vote, votes++);
    };
    const uint64_t minus = pair2(-1.f, -1.f);
    // sums of the weights of this lane's tokens, nodes by twos (64 nodes: D has them, and the lane's node in shared
    // memory, where only this lane reads, what has left it)
    uint64_t l[kBoth ? kRows / 2 : 1];
    float* l_node = maxima + 8 * kRows + row;
    // whether the record has latent sums of this unit, and what they are relative to (each warp has its own
    // copy; of 64 nodes there is one, written after all four have read it)
    bool held = false;
    float* held_ref = maxima + 8 * kRows + (kBoth ? quad * kRows : kTile);
    int cur_b = w.b, cur_h = w.h, cur_g = w.g;
    // the largest score of every node in tile S (t_s), over the four warps, becomes its reference if that
    // is higher, or if it is the unit's first
    auto move = [&](uint32_t t_s, bool live, bool fresh) -> bool {
      float* mine = maxima + ((moves & 1) * 4 + quad) * kRows;
#pragma unroll 1
      for (int c = 0; c < kRows; c += 16) {
        float s[16];
        tmem_ld_x16(t_s + c, s);
        tmem_wait_ld();
        float keep = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float m = warp_max_redux(live ? s[k] : -INFINITY);
          if (lane == k) keep = m;
        }
        if (lane < 16) mine[c + lane] = keep;
      }
      if (!vote()) return false;
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        const int c = lane + 32 * j;
        if (c >= kRows) break;
        const float* m = maxima + (moves & 1) * 4 * kRows + c;
        float top = fmaxf(fmaxf(m[0], m[kRows]), fmaxf(m[2 * kRows], m[3 * kRows])) * back[j];
        if (fresh) top = top == -INFINITY ? 0.f : top;
        else top = fmaxf(top, refs[j]);
        factor[c] = exp2f(refs[j] - top);              // (not looked at for a new unit)
        refs[j] = top;
        minus_ref[c] = -top;
        scale[c] = back[j];
      }
      ++moves;
      __syncwarp();
      return true;
    };
    // the unit's sums (the last product was tile `last`) into its record; `whole`: it is finished.  D's lanes are
    // columns of the latent
    auto finish = [&](int last, bool whole) -> bool {
      if (!wait(misc->vdone[last & 1], last >> 1)) return false;
      tc_fence_after();
      int first;
      const int n = min(a.group, tree_nodes(a, cur_b, first, false) - cur_g * a.group);
      const int64_t slot = (static_cast<int64_t>(cur_b) * a.H + cur_h) * a.groups + cur_g + blockIdx.x;
      const int stride = a.r_v + kTreeHead;
      float* rec = a.records + slot * a.rec_rows * stride;
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        if (quad == 0 && lane + 32 * j < n) rec[(lane + 32 * j) * stride] = refs[j];
        const int c = lane + 32 * j;
        if (c < kRows) {
          if (held) factor[c] = exp2f(held_ref[c] - refs[j]);
          if (kBoth && !whole) held_ref[c] = refs[j];
        }
      }
      __syncwarp();
      if constexpr (kBoth) {
        // the lanes' sums through the warp's own rows of the weights, which have been read
        if (whole) {
          float* own = reinterpret_cast<float*>(sm + P.p + (last % kPBuf) * kPTile + quad * (32 * kPRow));
#pragma unroll
          for (int k = 0; k < kRows / 2; ++k) {
            float l0, l1;
            unpack2(l[k], l0, l1);
            own[64 * k + lane] = l0;
            own[64 * k + 32 + lane] = l1;
          }
          __syncwarp();
          if (lane < n) {
            float sum = 0.f;
#pragma unroll 4
            for (int k = 0; k < 32; ++k) sum += own[32 * lane + ((k + lane) & 31)];
            rec[lane * stride + 1 + quad] = sum;
          }
        }
        for (int blk = 0; blk < P.blocks; ++blk) {
          const int r = blk * 128 + row;
#pragma unroll 1
          for (int c = 0; c < n; c += 16) {
            float v[16], low[16];
            tmem_ld_x16(lanes + kDCol + blk * kDCols + c, v);
            tmem_ld_x16(lanes + kDCol + blk * kDCols + kRows + c, low);
            tmem_wait_ld();
            float* to = rec + c * stride + kTreeHead + r;
            if (held) {
              float before[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) before[k] = c + k < n && r < a.r_v ? to[k * stride] : 0.f;
#pragma unroll
              for (int k = 0; k < 16; ++k) low[k] = fmaf(before[k], factor[c + k], low[k]);
            }
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (c + k < n && r < a.r_v) to[k * stride] = v[k] + low[k];
          }
        }
      } else {
        // lanes are nodes: the lower parts' sums reach the upper parts' warps through the weights' memory, which
        // has been read, 16 columns at a time
        float* pass = reinterpret_cast<float*>(sm + P.p) + (row & 63) * 20;
#pragma unroll 1
        for (int c = 0; whole ? c <= a.r_v : c < a.r_v; c += 16) {
          float v[16];
          float4 before[4];
          float* to = rec + row * stride + kTreeHead + c;
          const bool more = held && quad < 2 && row < n && c < a.r_v;
#pragma unroll
          for (int k = 0; k < 4; ++k) before[k] = more ? *reinterpret_cast<const float4*>(to + 4 * k) : make_float4(0.f, 0.f, 0.f, 0.f);
          tmem_ld_x16(lanes + kDCol + c, v);
          tmem_wait_ld();
          if (c == a.r_v) v[0] += *l_node;
          if (quad >= 2) {
#pragma unroll
            for (int k = 0; k < 16; k += 4) *reinterpret_cast<float4*>(pass + (c & 16) * 80 + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
          }
          if (!vote()) return false;                   // (two places in turn: one vote a step keeps them apart)
          if (quad < 2 && row < n) {
#pragma unroll
            for (int k = 0; k < 16; k += 4) {
              const float4 y = *reinterpret_cast<const float4*>(pass + (c & 16) * 80 + k);
              const float f = more ? factor[row & 63] : 0.f;
              const float4 o = before[k / 4];
              const float4 z = make_float4(v[k] + fmaf(o.x, f, y.x), v[k + 1] + fmaf(o.y, f, y.y), v[k + 2] + fmaf(o.z, f, y.z),
                                           v[k + 3] + fmaf(o.w, f, y.w));
              if (c < a.r_v) *reinterpret_cast<float4*>(to + k) = z;
              else rec[row * stride + 1 + k / 4] = k == 0 ? z.x : 0.f;
            }
          }
        }
      }
      if (!kBoth && !whole && quad == 0) {            // (votes lie between)
#pragma unroll
        for (int j = 0; j < kMine; ++j) held_ref[lane + 32 * j] = refs[j];
      }
      tc_fence_before();
      held = !whole;
      return true;
    };
    for (int i = 0; i <= count && count > 0; ++i) {
      const uint32_t t_s = lanes + kSCol + i % kSBuf * kRows;
      const bool fresh = i == 0 || w.t == 0;
      if (fresh && i < count) {
        const float* from = a.qback + (static_cast<int64_t>(w.b * a.H + w.h) * a.groups + w.g) * kRows;
        const float undo = key_scale(a, w.b, w.h).y;
#pragma unroll
        for (int j = 0; j < kMine; ++j) back[j] = (lane + 32 * j < kRows ? __ldcg(from + lane + 32 * j) : 1.f) * undo;
      }
      if (i > 0 && (i == count || w.t % kSumTiles == 0)) {
        if (!finish(i - 1, fresh || i == count)) break;
        cur_b = w.b; cur_h = w.h; cur_g = w.g;
      }
      if (i == count || !wait(misc->sfull[i & 1], i >> 1)) break;
      tc_fence_after();
      const bool live = w.t * kTile + row < w.L, partial = (w.t + 1) * kTile > w.L;
      uint8_t* p = sm + P.p + (i % kPBuf) * kPTile;
      if (fresh) {
        if (!move(t_s, live, true)) break;
#pragma unroll
        for (int k = 0; k < (kBoth ? kRows / 2 : 0); ++k) l[k] = 0;
        if (!kBoth) *l_node = 0.f;
      }
      // Weights, in two bf16 parts as the product takes them.  Where a score is too far above its reference, the
      // references move and the weights are made again.
      bool settled = fresh, ok = true;
      uint32_t x[kRows / 2], y[kRows / 2];
      uint64_t pp[kBoth ? kRows / 2 : 1];
      while (true) {
        float top = -INFINITY;
        // (all of the lane's scores at once: the waits of one chain hide behind the others)
        float s[kRows];
        if constexpr (kRows == 16) tmem_ld_x16(t_s, s);
        else tmem_ld_x32(t_s, *reinterpret_cast<float(*)[32]>(s));
        if constexpr (kRows == 64) tmem_ld_x32(t_s + 32, *reinterpret_cast<float(*)[32]>(s + 32));
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < kRows / 2; k += 2) {
          const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(scale + 2 * k);
          const ulonglong2 m = *reinterpret_cast<const ulonglong2*>(minus_ref + 2 * k);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float d0, d1;
            unpack2(fma2(pair2(s[2 * (k + e)], s[2 * (k + e) + 1]), e == 0 ? f.x : f.y, e == 0 ? m.x : m.y), d0, d1);
            top = fmaxf(top, fmaxf(d0, d1));
            const float p0 = exp2_fast(d0), p1 = exp2_fast(d1);
            const uint32_t h = pack_bf16(p0, p1);
            if (kBoth) pp[k + e] = pair2(p0, p1);
            x[k + e] = h;
            asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tfma.rn.f32.bf16 %0, l, %5, %3;\n\tfma.rn.f32.bf16 %1, h, %5, %4;\n\t}"
                : "=f"(d0), "=f"(d1)
                : "r"(h), "f"(p0), "f"(p1), "h"(static_cast<unsigned short>(0xBF80)));
            y[k + e] = pack_bf16(d0, d1);
          }
        }
        if (settled) break;
        if (__any_sync(0xffffffffu, live && top > kHeadroom) && lane == 0) misc->over[i & 1] = i + 1;
        ok = vote();
        if (!ok || *const_cast<volatile int*>(&misc->over[i & 1]) != i + 1) break;
        settled = true;
        // (D is at rest once the product of tile i - 1 is done)
        ok = move(t_s, live, false) && wait(misc->vdone[(i - 1) & 1], (i - 1) >> 1);
        if (!ok) break;
        tc_fence_after();
        const int columns = kBoth ? P.blocks * kDCols : a.r_v + 16;
#pragma unroll 1
        for (int c = 0; c < columns; c += 8) {
          float v[8];
          tmem_ld_x8(lanes + kDCol + c, v);
          tmem_wait_ld();
          uint32_t z[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) z[k] = __float_as_uint(v[k] * factor[(kBoth ? c + k : row) % kRows]);
          tmem_st_x8(lanes + kDCol + c, z);
        }
        tmem_wait_st();
        if (!kBoth) *l_node *= factor[row % kRows];
#pragma unroll
        for (int k = 0; k < (kBoth ? kRows / 2 : 0); ++k) l[k] = mul2(l[k], *reinterpret_cast<const uint64_t*>(factor + 2 * k));
      }
      if (!ok) break;
      if constexpr (kPBuf == 1) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(misc->sfree[i & 1]));
        if (i > 0 && !wait(misc->vdone[(i - 1) & 1], (i - 1) >> 1)) break;     // the last weights have been read
        if (!fresh && w.t % kWeightTiles == 0) {      // (their sum starts anew with this tile's)
          float v[8];
          tc_fence_after();
          tmem_ld_x8(lanes + kDCol + a.r_v, v);
          tmem_wait_ld();
          *l_node += v[0];
        }
      }
      if (partial) {                                    // a token past the end has none
#pragma unroll
        for (int k = 0; k < kRows / 2; ++k) {
          x[k] = live ? x[k] : 0u;
          y[k] = live ? y[k] : 0u;
          if (kBoth) pp[k] = live ? pp[k] : 0;
        }
      }
#pragma unroll
      for (int k = 0; k < (kBoth ? kRows / 2 : 0); ++k) l[k] = add2(l[k], pp[k]);
#pragma unroll
      for (int k = 0; k < kRows / 2; k += 4) {
        *reinterpret_cast<uint4*>(p + swizzle_offset(row * kPRow + 4 * k, kPRow)) = make_uint4(x[k], x[k + 1], x[k + 2], x[k + 3]);
        *reinterpret_cast<uint4*>(p + swizzle_offset(row * kPRow + 4 * k + kLow, kPRow)) = make_uint4(y[k], y[k + 1], y[k + 2], y[k + 3]);
      }
      tc_fence_before();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(misc->pfull[i & 1]));
        if (kPBuf == 2) mbar_arrive(bar(misc->sfree[i & 1]));
      }
      walk_next(w, a);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- joining the parts

constexpr int kJoinThreads = 128;

// acc (16 x 8, fp32) += A (16 x 16) B (16 x 8), bf16.
__device__ __forceinline__ void mma16816(float (&acc)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(acc[0]), "+f"(acc[1]), "+f"(acc[2]), "+f"(acc[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two steps over 32 values of K: a lane's 16 bytes of a row of A (rows g and g + 8) and of B are K values
// 8 q .. 8 q + 7 (q = lane mod 4); both operands give them to the same places of the two steps, so the
// order of K is another one and the sum the same.
__device__ __forceinline__ void mma_k32(float (&acc)[4], const uint4& lo, const uint4& hi, const uint4& b) {
  mma16816(acc, lo.x, hi.x, lo.y, hi.y, b.x, b.y);
  mma16816(acc, lo.z, hi.z, lo.w, hi.w, b.z, b.w);
}

__device__ __forceinline__ void mma16816_f16(float (&acc)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(acc[0]), "+f"(acc[1]), "+f"(acc[2]), "+f"(acc[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_k32_f16(float (&acc)[4], const uint4& lo, const uint4& hi, const uint4& b) {
  mma16816_f16(acc, lo.x, hi.x, lo.y, hi.y, b.x, b.y);
  mma16816_f16(acc, lo.z, hi.z, lo.w, hi.w, b.z, b.w);
}

// Of two bf16 values, those that are not finite become 0; whether there was one.
__device__ __forceinline__ bool drop_odd(uint32_t& x) {
  const uint32_t hi = (x & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u, lo = (x & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u;
  x &= ~(hi | lo);
  return (hi | lo) != 0;
}

// Shared memory of a join block (bytes): V rows of the keys, scores and then weights, latent sums, per row
// {reference, cached sum, 1 / sum}.
struct JoinPlan {
  int keys, s_pitch, a_pitch;                        // pitches in elements
  int v, s, a, row, bytes;
};
constexpr int kJoinRows = 16;           // nodes of a join block
constexpr int kAgainStep = 8;           // cached tokens that join_again takes at a time
__host__ __device__ inline JoinPlan join_plan(int max_nodes, int r_k, int r_v) {
  constexpr int rows = kJoinRows;
  JoinPlan j{};
  j.keys = (max_nodes + 15) / 16 * 16;
  j.s_pitch = j.keys + 4;
  j.a_pitch = (r_v + 31) / 32 * 32 + 4;
  int off = 0;
  j.v = off;   off += j.keys * (kHeadDim + 8) * 2;
  j.s = off;   off += rows * j.s_pitch * 4;
  j.a = off;   off += rows * j.a_pitch * 4 > kAgainStep * (r_k + r_v) * 2 ? rows * j.a_pitch * 4 : kAgainStep * (r_k + r_v) * 2;
  j.row = off; off += rows * 16;
  j.bytes = off;
  return j;
}

// The cached tokens of a join block's nodes once more, in fp32, eight at a time: for sums that are NaN, which a
// component of a scaled cached key beyond the range of f16 makes them (and NaN and infinities in the cache, whose
// results stay NaN: it stops once every row's is).  Leaves them in rec, the block's rows of the unit's first record, as
// the one record there is, and the keys' values to be read again (their place holds the step's keys).  Keys by warp-level products of the bf16
// latents and weights (exact, fp32 sums), then eight lanes a row.  One block goes through its whole sequence, 0.9 us a token
// (rank 96, bound by the latency of the few dependent parts of a step: 3653 tokens 3.2 ms, 15393 14.0 ms).
__device__ __noinline__ void join_again(const TreeArgs& a, uint8_t* sm, int b, int h, int row0, int nr, float* rec) {
  constexpr int kStep = kAgainStep, kPitch = kHeadDim + 8;       // (16 rows of values are eight of keys)
  const JoinPlan J = join_plan(a.max_nodes, a.r_k, a.r_v);
  float* u = reinterpret_cast<float*>(sm + J.v);
  const int tid = threadIdx.x, lane = tid & 31, r = tid >> 3, x = tid & 7;
  const int L = tree_cached(a, b, false);
  // (what the loops need of the arguments, read once: they lie in memory here, which the loops' stores might change)
  const int H = a.H, r_k = a.r_k, r_v = a.r_v, page_size = a.page_size, max_pages = a.max_pages;
  const int64_t num_pages = a.num_pages, L_max = a.L_max;
  const int32_t* block_table = a.block_table;
  const __nv_bfloat16* cache_k = static_cast<const __nv_bfloat16*>(a.cache_k);
  const __nv_bfloat16* cache_v = static_cast<const __nv_bfloat16*>(a.cache_v);
  const float* rope_cos = a.rope_cos;
  const float* rope_sin = a.rope_sin;
  uint32_t* status = a.status;
  const int64_t unit = (static_cast<int64_t>(b) * a.H + h) * a.groups + row0 / a.group;
  const int ir = row0 % a.group + r;
  float q[16];                                        // components 4 x .. of every 32
  const float back = __ldcg(a.qback + unit * a.rows + ir);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint8_t* chunk = a.qimg + unit * (a.rows * 512) + (c >> 1) * a.rows * 128 + swizzle_offset(ir * 128 + (c & 1) * 64 + x * 8, 128);
    const uint2 hi = __ldcg(reinterpret_cast<const uint2*>(chunk)), lo = __ldcg(reinterpret_cast<const uint2*>(chunk + a.rows * 256));
    const __half2* y = reinterpret_cast<const __half2*>(&hi);
    const __half2* z = reinterpret_cast<const __half2*>(&lo);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float2 v = __half22float2(y[k]), w = __half22float2(z[k]);
      q[4 * c + 2 * k] = (v.x + w.x) * back;
      q[4 * c + 2 * k + 1] = (v.y + w.y) * back;
    }
  }
  // keys: a warp makes 32 components (8 i + .. of its own), the step's tokens in the first eight rows of its products
  constexpr int kWarps = kJoinThreads / 32, kTiles = 16 / kWarps;
  const int g = lane >> 2, k8 = 8 * (lane & 3), e0 = (tid >> 5) * (kHeadDim / kWarps);
  auto source = [&](int e) { return a.rope_style == 0 ? e : e < 64 ? 2 * e : 2 * (e - 64) + 1; };
  const __nv_bfloat16* W = static_cast<const __nv_bfloat16*>(a.w_up_k) + static_cast<int64_t>(h) * kHeadDim * r_k + k8;
  float mu[kTiles][2];
  int w_row[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    w_row[i] = source(e0 + 8 * i + g) * r_k;
#pragma unroll
    for (int k = 0; k < 2; ++k) mu[i][k] = __ldg(a.mu_k + h * a.mu_hstride + source(e0 + 8 * i + (k8 >> 2) + k));
  }
  float m = -INFINITY, held = 0.f, acc[4][8];         // columns 8 x .. of every 64
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[k][e] = 0.f;
  // a step's latents, K then V of a token, 16 bytes a piece: read one step ahead, and where the latent sums go in the
  // end (past the sequence's end: the last token, whose weight is then 0)
  constexpr int kPieces = kStep * 2 * kMaxRankPerHead / 8 / kJoinThreads;
  const int gk = r_k >> 3, gran = gk + (r_v >> 3);
  uint4* held_rows = reinterpret_cast<uint4*>(sm + J.a);
  uint4 ahead[kPieces];
  float turn[kStep];                                  // and cosine and sine of frequency tid mod 64 of every other token
  auto read = [&](int t0) {
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int i = tid + k * kJoinThreads, t = i / gran, c = i - t * gran;
      if (t < kStep) {
        const int64_t at = latent_row(block_table, page_size, max_pages, num_pages, L_max, H, b, h, min(t0 + t, L - 1), status);
        ahead[k] = __ldg(reinterpret_cast<const uint4*>(c < gk ? cache_k + at * r_k + 8 * c
                                                               : cache_v + at * r_v + 8 * (c - gk)));
      }
    }
#pragma unroll
    for (int k = 0; k < kStep; k += 2) {
      const int64_t at = static_cast<int64_t>(min(t0 + k + (tid >> 6), L - 1)) * 64 + (tid & 63);
      turn[k] = __ldg(rope_cos + at);
      turn[k + 1] = __ldg(rope_sin + at);
    }
  };
  if (L > 0) read(0);
  for (int t0 = 0; t0 < L; t0 += kStep) {
    if (__syncthreads_and(r >= nr || held != held)) break;
#pragma unroll
    for (int k = 0; k < kPieces; ++k)
      if (tid + k * kJoinThreads < kStep * gran) held_rows[tid + k * kJoinThreads] = ahead[k];
    __syncthreads();
    float key[kTiles][4];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) { key[i][0] = mu[i][0]; key[i][1] = mu[i][1]; key[i][2] = key[i][3] = 0.f; }
    const uint4 none = make_uint4(0, 0, 0, 0);
#pragma unroll 1
    for (int c = 0; c < r_k; c += 32) {
      const bool in = c + k8 < r_k;
      const uint4 y = in ? held_rows[g * gran + ((c + k8) >> 3)] : none;
      uint4 w[kTiles];
#pragma unroll
      for (int i = 0; i < kTiles; ++i) w[i] = in ? __ldg(reinterpret_cast<const uint4*>(W + w_row[i] + c)) : none;
#pragma unroll
      for (int i = 0; i < kTiles; ++i) mma_k32(key[i], y, none, w[i]);
    }
#pragma unroll
    for (int i = 0; i < kTiles; ++i) *reinterpret_cast<float2*>(u + g * kPitch + e0 + 8 * i + (k8 >> 2)) = make_float2(key[i][0], key[i][1]);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kStep; k += 2) {
      float* y = u + (k + (tid >> 6)) * kPitch + (tid & 63);
      const float x0 = y[0], x1 = y[64];
      y[0] = x0 * turn[k] - x1 * turn[k + 1];
      y[64] = x0 * turn[k + 1] + x1 * turn[k];
    }
    if (t0 + kStep < L) read(t0 + kStep);
    __syncthreads();
    float s[kStep];
#pragma unroll
    for (int t = 0; t < kStep; ++t) {
      s[t] = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float4 y = *reinterpret_cast<const float4*>(u + t * kPitch + 32 * c + 4 * x);
        s[t] = fmaf(q[4 * c], y.x, fmaf(q[4 * c + 1], y.y, fmaf(q[4 * c + 2], y.z, fmaf(q[4 * c + 3], y.w, s[t]))));
      }
    }
    // the eight sums over a row's lanes: half of them go on in half of the lanes, three times; lane x has token x
    float s4[4], s2[2];
#pragma unroll
    for (int t = 0; t < 4; ++t) s4[t] = (x & 4 ? s[t + 4] : s[t]) + __shfl_xor_sync(0xffffffffu, x & 4 ? s[t] : s[t + 4], 4);
#pragma unroll
    for (int t = 0; t < 2; ++t) s2[t] = (x & 2 ? s4[t + 2] : s4[t]) + __shfl_xor_sync(0xffffffffu, x & 2 ? s4[t] : s4[t + 2], 2);
    float mine = (x & 1 ? s2[1] : s2[0]) + __shfl_xor_sync(0xffffffffu, x & 1 ? s2[0] : s2[1], 1);
    if (t0 + x >= L) mine = -INFINITY;
    float top = fmaxf(m, mine);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float ref = top == -INFINITY ? 0.f : top, f = exp2f(m - ref), p = t0 + x < L ? exp2f(mine - ref) : 0.f;
    float sum = p;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    m = top;
    held = fmaf(held, f, sum);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[k][e] *= f;
#pragma unroll 1
    for (int t = 0; t < kStep; ++t) {                 // (rolled: a long body waits for its instructions)
      const float w = __shfl_sync(0xffffffffu, p, (lane & 24) + t);
      const uint4* from = held_rows + t * gran + gk + x;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (64 * k + 8 * x >= r_v) break;
        float v[8];
        unpack_bf16x8(from[8 * k], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[k][e] = fmaf(w, v[e], acc[k][e]);
      }
      __syncwarp();
    }
  }
  if (r < nr) {
    float* to = rec + static_cast<int64_t>(r) * (r_v + kTreeHead);
    if (x == 0) {
      *reinterpret_cast<float4*>(to) = make_float4(m, held, 0.f, 0.f);
      to[4] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = 8 * x + 64 * k;
      if (c >= r_v) break;
      *reinterpret_cast<float4*>(to + kTreeHead + c) = make_float4(acc[k][0], acc[k][1], acc[k][2], acc[k][3]);
      *reinterpret_cast<float4*>(to + kTreeHead + c + 4) = make_float4(acc[k][4], acc[k][5], acc[k][6], acc[k][7]);
    }
  }
}

// Block = 16 nodes of a (sequence, head); its four warps split the keys, then the output's dimensions.
//   S = Q^ K^^T over the nodes' keys, masked to each node's path; reference M over S and the records
//   P = 2^(S - M), A = sum of the records' latent sums times 2^(m - M), both fp32
//   out = (A W_up,v^T + P V + held mu_v) / l
// by warp-level products whose operands come straight from global memory (L2) where they are read
// along K (Q^ and K^ in two f16 parts; P and A as the three bf16 parts that hold an fp32 value, split where a
// product takes them: with two parts, 16 bits, one output in 500 took the other neighbour in its rounding).  Bound by
// the latency of its few steps; blocks are small so that many run at a time: 17 us for 512 blocks, 75 for 2048 with 128 keys (of which the third parts 7) (80 registers and six blocks an
// SM instead of four, with half of the values held at a time: no faster).  The
// scores need nothing of the tile kernel, so they are made before the wait for it (its blocks let this
// grid start only once they have seen the preparation complete, and leave room for it as they end).
__global__ void __launch_bounds__(kJoinThreads, 4) tree_join_kernel(const __grid_constant__ TreeArgs a) {
  extern __shared__ uint4 shared[];
  constexpr int kSplit = kJoinThreads / 32, kRows = kJoinRows, kTiles = 16 / kSplit;      // 8-dimension tiles of a warp
  uint8_t* sm = reinterpret_cast<uint8_t*>(shared);
  const JoinPlan J = join_plan(a.max_nodes, a.r_k, a.r_v);
  __nv_bfloat16* sv = reinterpret_cast<__nv_bfloat16*>(sm + J.v);
  float* ss = reinterpret_cast<float*>(sm + J.s);
  float* sa = reinterpret_cast<float*>(sm + J.a);
  float4* srow = reinterpret_cast<float4*>(sm + J.row);
  const int tid = threadIdx.x, lane = tid & 31, part = tid >> 5, g = lane >> 2, q = lane & 3;
  const int bh = blockIdx.x, b = bh / a.H, h = bh - b * a.H, row0 = blockIdx.y * kRows, grp = row0 / a.group;
  int first;
  const int n = tree_nodes(a, b, first, false);
  if (row0 >= n) {
    // (where no block has nodes too, this grid has to end after the tile kernel: the next call waits for it alone
    // before it writes the plan that the tile kernel reads)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const int nr = min(kRows, n - row0), nk = min(n, row0 + kRows), nk16 = (nk + 15) & ~15;

  // ---- values of the keys; NaN and infinities are left out (0 times them is not 0 for the nodes that do not have
  // the key on their path) and added at the end
  bool odd = false;
  auto read_values = [&]() {
    for (int i = tid; i < nk16 * 16; i += kJoinThreads) {
      const int r = i >> 4, c = (i & 15) * 8;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (r < nk) x = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.v) + (first + r) * a.v_stride + h * kHeadDim + c));
      odd |= drop_odd(x.x) | drop_odd(x.y) | drop_odd(x.z) | drop_odd(x.w);
      *reinterpret_cast<uint4*>(sv + r * (kHeadDim + 8) + c) = x;
    }
  };
  read_values();
  // ---- scores of this warp's 16 nodes against every kSplit-th tile of eight keys
  {
    const int64_t unit = static_cast<int64_t>(bh) * a.groups + grp;
    const uint8_t* img = a.qimg + unit * (a.rows * 512);
    const int ir = row0 - grp * a.group + g;       // row of the image
    uint4 x0[2][4], x1[2][4];                         // rows ir and ir + 8, both parts
#pragma unroll
    for (int c = 0; c < 8; ++c) {                     // K values 32 c + 8 q .. of chunk c / 2
      const uint32_t o = (c & 1) * 64 + q * 16;
      const uint8_t* chunk = img + (c >> 1) * a.rows * 128;
      x0[c >> 2][c & 3] = __ldcg(reinterpret_cast<const uint4*>(chunk + swizzle_offset(ir * 128 + o, 128)));
      x1[c >> 2][c & 3] = __ldcg(reinterpret_cast<const uint4*>(chunk + swizzle_offset((ir + 8) * 128 + o, 128)));
    }
    const float f0 = __ldcg(a.qback + unit * a.rows + ir), f1 = __ldcg(a.qback + unit * a.rows + ir + 8);
    const uint8_t* keys = a.khat + static_cast<int64_t>(bh) * a.max_nodes * 512;
    const float* back = a.kback + static_cast<int64_t>(bh) * a.max_nodes;
    uint4 m0 = make_uint4(0, 0, 0, 0), m1 = m0;
    const int r0 = row0 + g;
    if (r0 < n) m0 = __ldcg(a.paths + static_cast<int64_t>(b) * a.max_nodes + r0);
    if (r0 + 8 < n) m1 = __ldcg(a.paths + static_cast<int64_t>(b) * a.max_nodes + r0 + 8);
    for (int kt = part; kt < nk16 / 8; kt += kSplit) {
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      uint4 y[2][4];
#pragma unroll
      for (int c = 0; c < 8; ++c)
        y[c >> 2][c & 3] = 8 * kt + g < nk ? __ldcg(reinterpret_cast<const uint4*>(keys + (8 * kt + g) * 512 + c * 64 + q * 16)) : make_uint4(0, 0, 0, 0);
      const int col = 8 * kt + 2 * q, wd = col >> 5, bit = col & 31;
      const float k0 = col < nk ? __ldcg(back + col) : 0.f, k1 = col + 1 < nk ? __ldcg(back + col + 1) : 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        mma_k32_f16(acc, x0[0][c], x1[0][c], y[0][c]);
        mma_k32_f16(acc, x0[0][c], x1[0][c], y[1][c]);
        mma_k32_f16(acc, x0[1][c], x1[1][c], y[0][c]);
      }
      const uint32_t b0 = (wd == 0 ? m0.x : wd == 1 ? m0.y : wd == 2 ? m0.z : m0.w) >> bit;
      const uint32_t b1 = (wd == 0 ? m1.x : wd == 1 ? m1.y : wd == 2 ? m1.z : m1.w) >> bit;
      float* s0 = ss + g * J.s_pitch + col;
      float* s1 = s0 + 8 * J.s_pitch;
      s0[0] = b0 & 1 ? acc[0] * f0 * k0 : -INFINITY;
      s0[1] = b0 & 2 ? acc[1] * f0 * k1 : -INFINITY;
      s1[0] = b1 & 1 ? acc[2] * f1 * k0 : -INFINITY;
      s1[1] = b1 & 2 ? acc[3] * f1 * k1 : -INFINITY;
    }
  }
  // ---- the unit's records: consecutive
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int ng = (n + a.group - 1) / a.group, stride = a.r_v + kTreeHead;
  const uint32_t t0 = __ldcg(a.tile_start + b), nb = (__ldcg(a.tile_start + b + 1) - t0) / ng;
  const uint32_t total = static_cast<uint32_t>(__ldcg(a.tile_start + a.B)) * a.H;     // (below 2^30)
  const uint32_t share = max(1u, (total + a.grid - 1) / a.grid);
  const uint32_t f0 = t0 * a.H + (h * ng + grp) * nb, c0 = f0 / share;
  int nrec = nb > 0 ? static_cast<int>((f0 + nb - 1) / share + 1 - c0) : 0;
  const int64_t next = static_cast<int64_t>(a.rec_rows) * stride;
  float* recs = a.records + (static_cast<int64_t>(bh) * a.groups + grp + c0) * next + (row0 - grp * a.group) * stride;
  // ---- their references and sums: eight lanes a row
  float top, held;
  auto read_records = [&]() {
    const int r = tid >> 3, x = tid & 7;
    const float* rec = recs + r * stride;
    top = -INFINITY;
    held = 0.f;
    for (int i = x; i < nrec && r < nr; i += 8) top = fmaxf(top, __ldcg(rec + i * next));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    for (int i = x; i < nrec && r < nr; i += 8) {
      const float4 head = __ldcg(reinterpret_cast<const float4*>(rec + i * next));
      held = fmaf(exp2f(head.x - top), (head.y + head.z) + (head.w + __ldcg(rec + i * next + 4)), held);
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) held += __shfl_xor_sync(0xffffffffu, held, o);
  };
  read_records();
  if (__syncthreads_or(odd || held != held)) {
    odd = __syncthreads_or(odd);
    // (a node whose score of itself is NaN has a result that nothing mends)
    const int r = tid >> 3;
    const float own = r < nr ? ss[r * J.s_pitch + row0 + r] : 0.f;
    if (__syncthreads_or(r < nr && held != held && own == own)) {
      join_again(a, sm, b, h, row0, nr, recs);
      nrec = 1;
      __syncthreads();
      read_values();
      read_records();
    }
  }
  // ---- reference, weights (over the scores) and sums
  {
    const int r = tid >> 3, x = tid & 7;
    const bool row = r < nr;
    float m = top;
    for (int c = x; c < nk && row; c += 8) m = fmaxf(m, ss[r * J.s_pitch + c]);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.f;
    for (int c = x; c < nk16; c += 8) {
      const float w = row && c < nk ? exp2f(ss[r * J.s_pitch + c] - m) : 0.f;
      ss[r * J.s_pitch + c] = w;
      l += w;
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (nrec > 0) held *= exp2f(top - m);
    l += held;
    if (x == 0) {
      srow[r] = make_float4(m, held, row ? 1.f / l : 0.f, 0.f);
      if (row && a.lse) a.lse[(static_cast<int64_t>(first) + row0 + r) * a.H + h] = (m + log2f(l)) * kLn2;
    }
  }
  __syncthreads();
  // ---- latent sums of the records, relative to M
  const int cols = J.a_pitch - 4, per = cols / 4;
  for (int i = tid; i < kRows * per; i += kJoinThreads) {
    const int r = i / per, c = (i - r * per) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < nr && c < a.r_v) {
      const float m = srow[r].x;
      const float* rec = recs + r * stride;
#pragma unroll 2
      for (int k = 0; k < nrec; ++k, rec += next) {
        const float f = exp2f(__ldcg(rec) - m);
        const float4 y = __ldcg(reinterpret_cast<const float4*>(rec + kTreeHead + c));
        x.x = fmaf(f, y.x, x.x); x.y = fmaf(f, y.y, x.y); x.z = fmaf(f, y.z, x.z); x.w = fmaf(f, y.w, x.w);
      }
    }
    *reinterpret_cast<float4*>(sa + r * J.a_pitch + c) = x;
  }
  __syncthreads();

  // ---- A W^T + P V: this warp's 16 nodes, 128 / kSplit dimensions
  float acc[kTiles][4];
#pragma unroll
  for (int t = 0; t < kTiles; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
  const int e0 = part * (kHeadDim / kSplit);
  const __nv_bfloat16* W = static_cast<const __nv_bfloat16*>(a.w_up_v) + (static_cast<int64_t>(h) * kHeadDim + e0 + g) * a.r_v;
  for (int c = 0; c < cols && nrec > 0; c += 32) {
    uint4 x[kTiles], y[2][3];
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
      x[t] = c + 8 * q < a.r_v ? __ldg(reinterpret_cast<const uint4*>(W + static_cast<int64_t>(8 * t) * a.r_v + c + 8 * q)) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < 2; ++r) {                     // rows g and g + 8
      const float* from = sa + (g + 8 * r) * J.a_pitch + c + 8 * q;
      const float4 u = *reinterpret_cast<const float4*>(from), v = *reinterpret_cast<const float4*>(from + 4);
      split_bf16(u.x, u.y, y[r][0].x, y[r][1].x, y[r][2].x);
      split_bf16(u.z, u.w, y[r][0].y, y[r][1].y, y[r][2].y);
      split_bf16(v.x, v.y, y[r][0].z, y[r][1].z, y[r][2].z);
      split_bf16(v.z, v.w, y[r][0].w, y[r][1].w, y[r][2].w);
    }
#pragma unroll
    for (int e = 0; e < 3; ++e)
#pragma unroll
      for (int t = 0; t < kTiles; ++t) mma_k32(acc[t], y[0][e], y[1][e], x[t]);
  }
  for (int k = 0; k < nk16; k += 16) {
    uint32_t x[4][3];                                 // (all parts of the weights: rows g and g + 8, keys 2 q and 2 q + 8)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 u = *reinterpret_cast<const float2*>(ss + (g + 8 * (e & 1)) * J.s_pitch + k + 2 * q + 8 * (e >> 1));
      split_bf16(u.x, u.y, x[e][0], x[e][1], x[e][2]);
    }
#pragma unroll
    for (int t = 0; t < kTiles; t += 2) {
      uint32_t b0, b1, b2, b3;
      asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                   : "=r"(b0), "=r"(b1), "=r"(b2), "=r"(b3)
                   : "r"(smem_u32(sv + (k + (lane & 15)) * (kHeadDim + 8) + e0 + 8 * t + 8 * (lane >> 4)))
                   : "memory");
#pragma unroll
      for (int e = 0; e < 3; ++e) {
        mma16816(acc[t], x[0][e], x[1][e], x[2][e], x[3][e], b0, b1);
        mma16816(acc[t + 1], x[0][e], x[1][e], x[2][e], x[3][e], b2, b3);
      }
    }
  }
  if (odd) {
    for (int j = 0; j < nk; ++j) {
      const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v) + (first + j) * a.v_stride + h * kHeadDim + e0;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = g + 8 * r;
        if (row >= nr || !(__ldcg(reinterpret_cast<const uint32_t*>(a.paths + static_cast<int64_t>(b) * a.max_nodes + row0 + row) + (j >> 5)) >> (j & 31) & 1)) continue;
        const float w = ss[row * J.s_pitch + j];
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float y = __bfloat162float(v[8 * t + 2 * q + k]);
            if (!isfinite(y)) acc[t][2 * r + k] = fmaf(w, y, acc[t][2 * r + k]);
          }
      }
    }
  }
  // ---- means, division, one rounding
  const float4 r0 = srow[g], r1 = srow[g + 8];
  const int n0 = g, n1 = g + 8;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + ((static_cast<int64_t>(first) + row0) * a.H + h) * kHeadDim;
  const float* mu = a.mu_v + h * a.mu_hstride;
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    const int e = e0 + 8 * t + 2 * q;
    float2 m = make_float2(0.f, 0.f);
    if (nrec > 0) m = __ldg(reinterpret_cast<const float2*>(mu + e));
    if (n0 < nr)
      *reinterpret_cast<__nv_bfloat162*>(out + static_cast<int64_t>(n0) * a.H * kHeadDim + e) =
          __floats2bfloat162_rn(fmaf(r0.y, m.x, acc[t][0]) * r0.z, fmaf(r0.y, m.y, acc[t][1]) * r0.z);
    if (n1 < nr)
      *reinterpret_cast<__nv_bfloat162*>(out + static_cast<int64_t>(n1) * a.H * kHeadDim + e) =
          __floats2bfloat162_rn(fmaf(r1.y, m.x, acc[t][2]) * r1.z, fmaf(r1.y, m.y, acc[t][3]) * r1.z);
  }
}

}  // namespace

bool make_tree_plan(int r_k, int r_v, int rows, TreePlan* p) {
  *p = TreePlan{};
  p->kplan = make_chunk_plan(r_k, kTile);
  p->vplan = make_chunk_plan_32(r_v, kTile);
  p->blocks = (r_v + 127) / 128;
  auto al = [](int x) { return (x + 1023) / 1024 * 1024; };
  p->k_stage = al(p->kplan.bytes);
  p->v_stage = al(p->vplan.bytes);
  // weights in two parts (two buffers of them for up to 32 nodes); queries (two parts), W, bias, ones
  const int weights = kTile * rows * 2 * 2 * (rows <= 32 ? 2 : 1), refs = rows <= 32 ? 15 * rows * 4 : 12 * rows * 4 + kTile * 4;
  const int fixed = rows * 512 + al(p->kplan.bytes) + weights + 4096 + 512 + refs + 1024 + 256 + 768 + 1024;
  auto fits = [&](int sk, int sv) { return fixed + sk * p->k_stage + sv * p->v_stage <= kSmemLimit; };
  if (!fits(1, 1)) return false;
  p->SK = p->SV = 1;
  while (true) {
    if (p->SK <= p->SV && p->SK < kMaxStages && fits(p->SK + 1, p->SV)) { ++p->SK; continue; }
    if (p->SV < kMaxStages && fits(p->SK, p->SV + 1)) { ++p->SV; continue; }
    if (p->SK < kMaxStages && fits(p->SK + 1, p->SV)) { ++p->SK; continue; }
    break;
  }
  // (the V ring first: the last stage's products may read up to 128 columns, 32 KB, past it)
  int off = 0;
  p->v_ring = off; off += p->SV * p->v_stage;
  p->k_ring = off; off += p->SK * p->k_stage;
  p->w = off;      off += al(p->kplan.bytes);
  p->q = off;      off += rows * 512;
  p->p = off;      off += weights;
  p->mu = off;     off += 4096;
  p->ones = off;   off += 512;
  p->refs = off;   off += refs;
  p->base = off;   off += 1024;
  p->chunks = off; off += 256;
  p->misc = off;   off += 768;
  p->bytes = off + 1024;
  return true;
}

template <int kPage>
static cudaError_t launch_tiles(const TreeArgs& a, const TreeMaps& maps, cudaStream_t s) {
  auto kern = a.rows == 16 ? tree_tile_kernel<kPage, 16> : a.rows == 32 ? tree_tile_kernel<kPage, 32> : tree_tile_kernel<kPage, 64>;
  // (the most any shape takes, at every call)
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(a.grid), dim3(kTreeThreads), a.plan.bytes, s, a, maps);
}

cudaError_t launch_tree_tensor(const TreeArgs& a, const TreeMaps& maps, cudaStream_t s) {
  const cudaError_t e = launch_pdl(tree_prepare_kernel, dim3(a.B * a.H * a.groups + a.B + (a.B * a.H + kPrepWarps - 1) / kPrepWarps + a.H + 1), dim3(kPrepThreads), 0, s, a);
  if (e != cudaSuccess) return e;
  const cudaError_t t = !a.block_table              ? launch_tiles<0>(a, maps, s)
                        : a.page_size % kTile == 0 ? launch_tiles<1>(a, maps, s)
                        : a.piece >= 8             ? launch_tiles<2>(a, maps, s)
                                                   : launch_tiles<3>(a, maps, s);
  if (t != cudaSuccess) return t;
  // (the most any shape takes, at every call)
  const cudaError_t c = cudaFuncSetAttribute(tree_join_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             join_plan(kTreeMaxNodes, kMaxRankPerHead, kMaxRankPerHead).bytes);
  if (c != cudaSuccess) return c;
  return launch_pdl(tree_join_kernel, dim3(a.B * a.H, (a.max_nodes + kJoinRows - 1) / kJoinRows), dim3(kJoinThreads),
                    join_plan(a.max_nodes, a.r_k, a.r_v).bytes, s, a);
}

}  // namespace lla
