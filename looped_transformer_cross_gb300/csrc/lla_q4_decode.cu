// lla_q4_decode.cu — latent decode attention over the 4-bit paged cache on the tensor
// cores (bf16 storage; lla_q4.cu holds the fp32 kernel and the entry point).
//
// Score of Eq. (3) with RoPE after reconstruction, regrouped per frequency pair f as in
// lla_decode.cu: with the folded query Z_f = sc (q'_i0 W_i0 + q'_i1 W_i1) and
// Z_64+f = sc (q'_i1 W_i0 - q'_i0 W_i1), U = c_j Z^T + bias,
//     s_j = sum_f cos(j th_f) U_f + sin(j th_f) U_64+f         (log2 units).
// A 4-bit row is 144 bytes at (96, 160), 3.6 times less than in bf16, so at HBM speed an SM has about
// 6 cycles per token-head: the contractions run on the tensor cores, and a code
// costs about one ALU instruction on its way there.
//   K  Each thread of the K warpgroup owns one token: codes become f16 pairs (two magic
//      operations), are scaled by the group scale relative to the token's largest (a power of two,
//      multiplied back in the epilogue, so latents of any size stay in f16 range) and go
//      straight to TMEM as the A operand of U = c Z^T (M = 128 tokens, N = 128, K = r_k + 16:
//      one more step carries the bias, f16 high and low parts against that power).
//   s  Two epilogue warpgroups share a head-tile, 32 frequencies each.  A thread keeps its
//      row's cos / sin in registers and turns them by one tile's angle (table row 128) from tile to
//      tile: rows read from L2 (64 KB a tile) would be more traffic than the latents.  Partial
//      scores meet in shared memory, and the groups take turns at the softmax.
//   V  sum_j p_j c_v,j is a warp-level MMA: A = the codes themselves, as f16
//      subnormals (code * 2^-24 and code * 2^-20: masking is the whole conversion), B = one
//      column per scale group holding p_j scale_j,g, so that a group's scale is applied to a
//      weight and never to a code; a row of ones gives the sum that takes the codes' offset of 8 back.  Every
//      code is finite, so rows behind the last token only need weight 0.
//
// Work: positions (sequence, head group, 128-token tile) in that order, cut into
// equal contiguous ranges, one per CTA.  A run is a CTA's part of one (sequence, head
// group); the query operand of its nh heads is built in shared memory at its start, and
// one record {m, l, acc} per head is written at its end.  Warps: 0 producer (bulk
// copies of page pieces into the ring), 1 MMA issuer, 4-7 K, 8-15 epilogue, 16-19 V.
#include <algorithm>
#include <cmath>

#include "lla_q4.h"

namespace lla {

namespace {

constexpr int kQ4TileThreads = 640;
constexpr int kWorkers = 512;                    // K, epilogue and V warpgroups
constexpr int kQ4MaxNS = 16;
constexpr int kWStride = 136;                    // halves between the groups of a weight tile
constexpr int kWBytes = 8 * kWStride * 2;
constexpr int kStageTail = kWBytes + 64;         // weights, then the four references
constexpr int kTrigRow = 20;                     // words of a staged row of 16 table values
constexpr int kTrigBytes = 8 * 32 * kTrigRow * 4;
constexpr int kUCol = 0;                         // TMEM: two U buffers of 128 columns
constexpr int kACol = 256;                       // then the A operand buffers
constexpr float kQ4Scale = 0.08838834764831845f * 1.4426950408889634f;   // log2(e) / sqrt(128)
constexpr int kSeedTiles = 512;                  // tiles between reads of the table (a power of two)
constexpr float kRaise = 8.f;                    // lazy maximum: raised when passed by 2^8
constexpr int kNoRef = -(1 << 28);
// named barriers: 1 workers + MMA warp, 2 workers, 3.. one per (quadrant, parity) of the epilogue
enum { kBarRun = 1, kBarWork = 2, kBarPair = 3 };

struct alignas(16) Q4Misc {
  uint64_t full[kQ4MaxNS], empty[kQ4MaxNS], wfull[kQ4MaxNS];
  uint64_t afull[2], aempty[2], ufull[2], uempty[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
  int start_b, start_hg, start_t, count;
  int scan[kQ4TileThreads];
  float2 ml[2][8];                               // run end: (m, l) per head and epilogue warp
  int vref[4];                                   // run end: reference of each V warp
  float qs[2][2][64];                            // rotated query, sc q'_i0 and sc q'_i1, per head
  float tile_cos[64], tile_sin[64], tile_nsin[64];   // table row 128 (and - sin): one tile's angles
  float part[2][128];                            // half scores of a head-tile, by parity
};

struct Slot {
  int i;
  uint32_t phase;
  __device__ __forceinline__ void next(int n) {
    if (++i == n) { i = 0; phase ^= 1u; }
  }
};

// A run of positions of one (sequence, head group).
struct Run {
  int b, hg, t0, n, L;   // tiles t0 .. t0 + n - 1
};

__device__ __forceinline__ int tile_len(const Q4DecodeArgs& a, int b) {
  const int L = __ldg(a.seq_lens + b);
  return L < 0 ? 0 : (L > a.L_max ? static_cast<int>(a.L_max) : L);
}
__device__ __forceinline__ int tiles_of(int L) { return (L + kTile - 1) / kTile; }

// The CTA's runs in order: every role walks the same list.
struct RunWalker {
  int b, hg, t, left;
  __device__ __forceinline__ bool next(const Q4DecodeArgs& a, int ngroups, Run& r) {
    if (left <= 0) return false;
    int L = tile_len(a, b);
    while (t >= tiles_of(L)) {           // the next non-empty unit
      t = 0;
      if (++hg == ngroups || L == 0) { hg = 0; ++b; L = tile_len(a, b); }
      if (L == 0) continue;
      break;
    }
    r.b = b;
    r.hg = hg;
    r.t0 = t;
    r.L = L;
    r.n = min(left, tiles_of(L) - t);
    left -= r.n;
    t += r.n;
    return true;
  }
};

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float sum2(uint64_t v) {
  float lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
  return lo + hi;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }
__device__ __forceinline__ uint32_t h2_bits(__half2 v) { return *reinterpret_cast<uint32_t*>(&v); }
__device__ __forceinline__ __half2 bits_h2(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }
__device__ __forceinline__ void pair_arrive(int id) { asm volatile("bar.arrive %0, 64;" ::"r"(id) : "memory"); }

// D[16 x 8] += A[16 x 16] B[16 x 8], f16 operands, fp32 accumulator (one warp).
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Exponent of the power of two that a token's K codes are scaled against, from the bits of
// its largest scale.  Not below -14: 2^14 is the largest that multiplies the bias in f16, and
// latents that small against it no longer move a score.
__device__ __forceinline__ int k_exponent(uint32_t top) { return min(max(static_cast<int>(top >> 7) - 127, -14), 126); }
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127
__device__ __forceinline__ uint32_t scale_bits(const uint8_t* p) { return *reinterpret_cast<const uint16_t*>(p); }

// Register shares of the warpgroups: 56 + 72 + 2 x 120 + 112 = 480 = 5 x 96, what the
// block is launched with (640 threads of 96).
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// The eight f16 pairs of a 4-code-pair word: columns (2i, 2i + 1) as code - 8, exact, times `s`.
// 0x6400 is 1024 in f16, whose unit in the last place is 1.
__device__ __forceinline__ void k_word(uint32_t w, __half2 s, uint32_t (&o)[4]) {
  const __half2 off = __half2half2(__ushort_as_half(0x6408));   // 1032
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = h2_bits(__hmul2(__hsub2(bits_h2(((w >> (4 * i)) & 0x000F000Fu) | 0x64006400u), off), s));
}

// RV32 = ceil(r_v / 32): V columns in chunks of 64 (four MMAs of 16 rows) and at most
// one of 32 (two).  Columns beyond r_v read the bytes behind the codes, and their rows
// of the accumulator are never read.
template <int RV32>
__global__ void __launch_bounds__(kQ4TileThreads, 1) q4_tile_kernel(const __grid_constant__ Q4DecodeArgs a) {
  constexpr int F = RV32 / 2, HF = RV32 & 1, NM = 4 * F + 2 * HF;
  extern __shared__ uint8_t smem_raw[];
  // swizzle atoms need 1024-byte alignment in the shared window itself
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const Q4Plan& P = a.plan;
  const uint32_t sbase = smem_u32(sm);
  Q4Misc* misc = reinterpret_cast<Q4Misc*>(sm + P.misc);
  volatile int* abort = &misc->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nh = P.nh, ngroups = P.ngroups, NS = P.NS, NA = P.NA, rk = a.r_k, rv = a.r_v, rb = a.row_bytes;
  const int scale_at = q4_scale_offset(rk, rv), gk = q4_groups(rk);

  // ---------------------------------------------------------- work range
  RunWalker start{0, 0, 0, 0};
  {
    const int per_thr = (a.B + kQ4TileThreads - 1) / kQ4TileThreads;
    const int b0 = min(a.B, tid * per_thr), b1 = min(a.B, b0 + per_thr);
    long long local = 0;
    for (int b = b0; b < b1; ++b) {
      const int L0 = __ldg(a.seq_lens + b), qp = __ldg(a.q_pos + b);
      if (blockIdx.x == 0 && (L0 < 0 || L0 > a.L_max || qp < 0 || qp >= a.rope_len)) record_status(a.status, LLA_ERR_DEVICE_ARG);
      local += tiles_of(tile_len(a, b));
    }
    misc->scan[tid] = static_cast<int>(local);
    if (tid == 0) { misc->abort = 0; misc->count = 0; }
    __syncthreads();
    if (warp == 0) {
      constexpr int kPer = kQ4TileThreads / 32;
      int s = 0;
      for (int i = 0; i < kPer; ++i) s += misc->scan[lane * kPer + i];
      int incl = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += n;
      }
      int excl = incl - s;
      for (int i = 0; i < kPer; ++i) {
        const int v = misc->scan[lane * kPer + i];
        misc->scan[lane * kPer + i] = excl;
        excl += v;
      }
      if (lane == 31) misc->start_t = incl;   // total tiles, read below
    }
    __syncthreads();
    const long long total = static_cast<long long>(misc->start_t) * ngroups;
    const long long per = max(1LL, (total + a.grid - 1) / a.grid);
    const long long f0 = static_cast<long long>(blockIdx.x) * per, f1 = min(total, f0 + per);
    long long p0 = static_cast<long long>(misc->scan[tid]) * ngroups;
    __syncthreads();
    for (int b = b0; b < b1; ++b) {
      const long long nb = static_cast<long long>(tiles_of(tile_len(a, b)));
      if (nb > 0 && f0 < f1 && p0 <= f0 && f0 < p0 + nb * ngroups) {
        misc->start_b = b;
        misc->start_hg = static_cast<int>((f0 - p0) / nb);
        misc->start_t = static_cast<int>((f0 - p0) % nb);
        misc->count = static_cast<int>(f1 - f0);
      }
      p0 += nb * ngroups;
    }
    __syncthreads();
    start = RunWalker{misc->start_b, misc->start_hg, misc->start_t, misc->count};
  }
  if (start.left == 0) return;

  // ---------------------------------------------------------- set-up
  auto bar = [&](const uint64_t& m) { return smem_u32(&m); };
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(bar(misc->full[s]), 1);
      mbar_init(bar(misc->empty[s]), 4 + 4 / nh);   // K warps, the head's V warps
      mbar_init(bar(misc->wfull[s]), 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(misc->afull[i]), 4);
      mbar_init(bar(misc->aempty[i]), 1);
      mbar_init(bar(misc->ufull[i]), 1);
      mbar_init(bar(misc->uempty[i]), 8);
    }
    mbar_init(bar(misc->mma_done), 1);
    fence_mbar_init();
  }
  if (tid >= 64 && tid < 128 && a.rope_len > kTile) {   // (at most 128 positions: one tile, no step)
    const int f = tid - 64;
    misc->tile_cos[f] = __ldg(a.rope_cos + kTile * 64 + f);
    misc->tile_sin[f] = __ldg(a.rope_sin + kTile * 64 + f);
    misc->tile_nsin[f] = -misc->tile_sin[f];
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc(smem_u32(&misc->tmem_base), 512);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the combine waits for this grid
  const uint32_t tmem = misc->tmem_base;
  const int acols = rk / 2 + 8;                  // TMEM columns of an A operand
  RunWalker walk = start;
  Run run{0, 0, 0, 0, 0};
  bool ok = true;
  // every role keeps its place in the loops when a wait has expired: the named barriers
  // below count on it
  auto wait = [&](const uint64_t& m, uint32_t parity) {
    if (ok) ok = warp_wait(bar(m), parity, abort, a.status);
  };
  auto arrive = [&](const uint64_t& m) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(m));
  };

  // Builds the run's query operands: Z rows of its heads in the K-major chunk layout, and
  // the bias chunk {high, low, 0...}.  All workers; the previous run has ended.
  auto build = [&](int wtid) {
    const int nhg = min(nh, a.H - run.hg * nh);
    int qp = __ldg(a.q_pos + run.b);
    qp = qp < 0 ? 0 : (qp >= a.rope_len ? static_cast<int>(a.rope_len - 1) : qp);
    float amax = 0.f;
    for (int i = wtid; i < nhg * 64; i += kWorkers) {
      const int hi = i >> 6, f = i & 63, h = run.hg * nh + hi;
      const int i0 = a.rope_style == 0 ? f : 2 * f, i1 = a.rope_style == 0 ? f + 64 : 2 * f + 1;
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (static_cast<int64_t>(run.b) * a.H + h) * kHeadDim;
      const float c = __ldg(a.rope_cos + static_cast<int64_t>(qp) * 64 + f);
      const float s = __ldg(a.rope_sin + static_cast<int64_t>(qp) * 64 + f);
      const float x0 = __bfloat162float(q[i0]), x1 = __bfloat162float(q[i1]);
      const float q0 = (x0 * c - x1 * s) * kQ4Scale, q1 = (x0 * s + x1 * c) * kQ4Scale;
      misc->qs[hi][0][f] = q0;
      misc->qs[hi][1][f] = q1;
      const float m0 = __ldg(a.mu_k + h * a.mu_hstride + i0), m1 = __ldg(a.mu_k + h * a.mu_hstride + i1);
      const float bias[2] = {q0 * m0 + q1 * m1, q1 * m0 - q0 * m1};
      uint8_t* img = sm + P.z + hi * P.z_stride + P.z_bias;
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        const float hi16 = __half2float(__float2half_rn(bias[part]));
        amax = fmaxf(amax, fabsf(bias[part]));
        const uint32_t row = (64 * part + f) * 32;
        *reinterpret_cast<uint4*>(img + swizzle_offset(row, 32)) =
            make_uint4(h2_bits(__floats2half2_rn(hi16, bias[part] - hi16)), 0, 0, 0);
        *reinterpret_cast<uint4*>(img + swizzle_offset(row + 16, 32)) = make_uint4(0, 0, 0, 0);
      }
    }
    named_bar_sync(kBarWork, kWorkers);
    const int k8 = rk / 8;
    for (int i = wtid; i < nhg * 64 * k8; i += kWorkers) {
      const int hf = i / k8, k = (i - hf * k8) * 8, hi = hf >> 6, f = hf & 63, h = run.hg * nh + hi;
      const int i0 = a.rope_style == 0 ? f : 2 * f, i1 = a.rope_style == 0 ? f + 64 : 2 * f + 1;
      const __nv_bfloat16* W = static_cast<const __nv_bfloat16*>(a.w_up_k) + static_cast<int64_t>(h) * kHeadDim * rk + k;
      float w0[8], w1[8], zc[8], zs[8];
      unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(W + static_cast<int64_t>(i0) * rk)), w0);
      unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(W + static_cast<int64_t>(i1) * rk)), w1);
      const float q0 = misc->qs[hi][0][f], q1 = misc->qs[hi][1][f];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        zc[e] = q0 * w0[e] + q1 * w1[e];
        zs[e] = q1 * w0[e] - q0 * w1[e];
        amax = fmaxf(amax, fmaxf(fabsf(zc[e]), fabsf(zs[e])));
      }
      // chunk of column k: 64-wide chunks first, then one of 32, then one of 16
      const int c64 = rk / 64 * 64;
      int width = 64, at = k / 64 * 16384, col = k & 63;
      if (k >= c64) {
        const int rest = rk - c64;
        at = c64 / 64 * 16384;
        col = k - c64;
        width = 32;
        if (rest < 32 || col >= 32) {
          width = 16;
          if (rest >= 32) { at += 8192; col -= 32; }
        }
      }
      uint8_t* img = sm + P.z + hi * P.z_stride + at;
      const int row_b = 2 * width;
      *reinterpret_cast<uint4*>(img + swizzle_offset(f * row_b + 2 * col, row_b)) =
          make_uint4(h2_bits(__floats2half2_rn(zc[0], zc[1])), h2_bits(__floats2half2_rn(zc[2], zc[3])),
                     h2_bits(__floats2half2_rn(zc[4], zc[5])), h2_bits(__floats2half2_rn(zc[6], zc[7])));
      *reinterpret_cast<uint4*>(img + swizzle_offset((64 + f) * row_b + 2 * col, row_b)) =
          make_uint4(h2_bits(__floats2half2_rn(zs[0], zs[1])), h2_bits(__floats2half2_rn(zs[2], zs[3])),
                     h2_bits(__floats2half2_rn(zs[4], zs[5])), h2_bits(__floats2half2_rn(zs[6], zs[7])));
    }
    if (amax > 65504.f) record_status(a.status, LLA_ERR_RANGE);   // NaN queries stay NaN
    fence_proxy_async_smem();
    named_bar_sync(kBarRun, kWorkers + 32);
  };

  if (warp < 4) {
    regs_dec<56>();
    if (warp == 0) {
      // ======================================================== producer
      // Per head-tile: the page pieces that its rows lie in, lane i copying piece i.
      Slot st{0, 0u};
      int issued = 0;
      while (walk.next(a, ngroups, run)) {
        const int nhg = min(nh, a.H - run.hg * nh);
        for (int t = run.t0; t < run.t0 + run.n && ok; ++t) {
          const int y0 = t * kTile, y1 = min(y0 + kTile, run.L), pg = a.page_size;
          const int lp0 = y0 / pg, np = (y1 - 1) / pg - lp0 + 1;
          const int32_t* table = a.block_table + static_cast<int64_t>(run.b) * a.max_pages + lp0;
          for (int hi = 0; hi < nhg && ok; ++hi) {
            wait(misc->empty[st.i], st.phase ^ 1u);
            if (!ok) break;
            const uint32_t fb = bar(misc->full[st.i]), dst = sbase + P.ring + st.i * P.stage;
            if (lane == 0) mbar_arrive_expect_tx(fb, (y1 - y0) * rb);
            __syncwarp();
            for (int i = lane; i < np; i += 32) {
              const int p0 = (lp0 + i) * pg, t0 = max(y0, p0), t1 = i + 1 < np ? p0 + pg : y1;
              int page = __ldg(table + i);
              if (page < 0 || page >= a.num_pages) {
                record_status(a.status, LLA_ERR_DEVICE_ARG);
                page = 0;
              }
              const int64_t r0 = static_cast<int64_t>(page * a.H + run.hg * nh + hi) * pg + (t0 - p0);
              bulk_load(dst + (t0 - y0) * rb, a.rows + r0 * rb, (t1 - t0) * rb, fb);
            }
            __syncwarp();
            ++issued;
            st.next(NS);
          }
        }
      }
      // let every copy land before the CTA can exit
      // (st is the next stage: the oldest of the last NS copies, or not yet used)
      if (lane == 0)
        for (int i = min(issued, NS); i > 0; --i) {
          if (issued < NS && i == issued) st = Slot{0, 0u};
          const uint32_t phase = issued < NS ? 0u : st.phase ^ 1u;
          const uint64_t t0 = global_timer_ns();
          while (!mbar_try_wait(bar(misc->full[st.i]), phase) && global_timer_ns() - t0 < kWaitLimitNs) {}
          st.next(NS);
        }
    } else if (warp == 1) {
      // ======================================================== MMA issuer
      // U = A Z^T per head-tile; the whole warp runs the loop, one elected lane issues
      const uint32_t idesc = umma_idesc_f16(128, 128);
      const int n64 = rk / 64, r32 = (rk & 63) >= 32, r16 = (rk & 31) >= 16;
      Slot as{0, 0u};
      uint32_t n = 0;
      while (walk.next(a, ngroups, run)) {
        const int nhg = min(nh, a.H - run.hg * nh);
        named_bar_sync(kBarRun, kWorkers + 32);   // operands built
        for (int t = 0; t < run.n; ++t)
          for (int hi = 0; hi < nhg; ++hi, ++n) {
            wait(misc->afull[as.i], as.phase);
            wait(misc->uempty[n & 1], ((n >> 1) & 1) ^ 1u);
            if (ok) {
              tc_fence_after();
              const uint32_t d = tmem + kUCol + (n & 1) * 128;
              uint32_t ac = tmem + kACol + as.i * acols;
              uint32_t z = sbase + P.z + hi * P.z_stride;
              uint32_t acc = 0;
              for (int c = 0; c < n64; ++c, z += 16384) {
                const uint64_t bd = umma_desc(z, 16, 1024, kSw128);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk, ac += 8) {
                  umma_bf16_ts_warp(d, ac, bd + 2 * kk, idesc, acc);
                  acc = 1;
                }
              }
              if (r32) {
                const uint64_t bd = umma_desc(z, 16, 512, kSw64);
                umma_bf16_ts_warp(d, ac, bd, idesc, acc);
                umma_bf16_ts_warp(d, ac + 8, bd + 2, idesc, 1);
                acc = 1;
                ac += 16;
                z += 8192;
              }
              if (r16) {
                umma_bf16_ts_warp(d, ac, umma_desc(z, 16, 256, kSw32), idesc, acc);
                ac += 8;
                z += 4096;
              }
              umma_bf16_ts_warp(d, ac, umma_desc(z, 16, 256, kSw32), idesc, 1);   // the bias step
              umma_commit_warp(bar(misc->ufull[n & 1]));
              umma_commit_warp(bar(misc->aempty[as.i]));
            }
            as.next(NA);
          }
        named_bar_sync(kBarRun, kWorkers + 32);   // run ended
      }
      // this warp's MMAs complete before TMEM is released
      umma_commit_warp(bar(misc->mma_done));
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(bar(misc->mma_done), 0) && global_timer_ns() - t0 < kWaitLimitNs) {}
    }
  } else if (warp < 8) {
    regs_dec<72>();
    // ======================================================== K: codes to the A operand
    const int q = warp & 3, row = 32 * q + lane, wtid = tid - 128;
    const uint32_t lane_base = static_cast<uint32_t>(32 * q) << 16;
    Slot st{0, 0u}, as{0, 0u};
    while (walk.next(a, ngroups, run)) {
      const int nhg = min(nh, a.H - run.hg * nh);
      build(wtid);
      for (int t = 0; t < run.n; ++t)
        for (int hi = 0; hi < nhg; ++hi) {
          wait(misc->full[st.i], st.phase);
          wait(misc->aempty[as.i], as.phase ^ 1u);
          tc_fence_after();
          const uint8_t* r = sm + P.ring + st.i * P.stage + row * rb;
          const uint32_t at = tmem + lane_base + kACol + as.i * acols;
          // the token's power of two: that of its largest group scale
          uint32_t top = 0;
          for (int g = 0; g < gk; ++g) top = max(top, scale_bits(r + scale_at + 2 * g) & 0x7FFFu);
          const float down = pow2(-k_exponent(top));
          int c = 0;
          for (; c + 32 <= rk; c += 32) {
            const float s = __uint_as_float(scale_bits(r + scale_at + c / 16) << 16);
            const __half2 s2 = __float2half2_rn(s * down);
            uint32_t o[16], u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              k_word(*reinterpret_cast<const uint32_t*>(r + c / 2 + 4 * i), s2, u);
#pragma unroll
              for (int j = 0; j < 4; ++j) o[4 * i + j] = u[j];
            }
            tmem_st_x16(at + c / 2, o);
          }
          uint32_t o[8], u[4];
          if (c < rk) {
            const float s = __uint_as_float(scale_bits(r + scale_at + c / 16) << 16);
            const __half2 s2 = __float2half2_rn(s * down);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              k_word(*reinterpret_cast<const uint32_t*>(r + c / 2 + 4 * i), s2, u);
#pragma unroll
              for (int j = 0; j < 4; ++j) o[4 * i + j] = u[j];
            }
            tmem_st_x8(at + c / 2, o);
          }
          // the bias step: the power of two against the bias rows' high and low parts
          o[0] = h2_bits(__float2half2_rn(down));
#pragma unroll
          for (int i = 1; i < 8; ++i) o[i] = 0;
          tmem_st_x8(at + rk / 2, o);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(misc->afull[as.i]));
            mbar_arrive(bar(misc->empty[st.i]));
          }
          st.next(NS);
          as.next(NA);
        }
      named_bar_sync(kBarRun, kWorkers + 32);
    }
  } else if (warp < 16) {
    regs_inc<120>();
    // ======================================================== epilogue: scores and weights
    const int grp = (warp - 8) >> 2, q = warp & 3, row = 32 * q + lane, wtid = tid - 128;
    const uint32_t lane_base = static_cast<uint32_t>(32 * q) << 16;
    float* stage = reinterpret_cast<float*>(sm + P.trig) + (warp - 8) * 32 * kTrigRow;
    Slot st{0, 0u};
    uint32_t n = 0;
    uint64_t tc[16], ts[16];   // cos and sin of the own row, pairs of frequencies 32 grp + (2i, 2i + 1)
    // rows of tile t from the table, through shared memory (a thread's own row straight from
    // global memory would touch 32 lines per load)
    auto seed = [&](int t) {
#pragma unroll
      for (int p = 0; p < 4; ++p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          int64_t j = static_cast<int64_t>(t) * kTile + 32 * q + 8 * i + (lane >> 2);
          j = j < a.rope_len ? j : a.rope_len - 1;    // behind the sequence's end: masked
          *reinterpret_cast<float4*>(stage + (8 * i + (lane >> 2)) * kTrigRow + 4 * (lane & 3)) = __ldg(
              reinterpret_cast<const float4*>((p < 2 ? a.rope_cos : a.rope_sin) + j * 64 + 32 * grp + 16 * (p & 1) + 4 * (lane & 3)));
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 v = *reinterpret_cast<const float4*>(stage + lane * kTrigRow + 4 * i);
          (p < 2 ? tc : ts)[8 * (p & 1) + 2 * i] = pack2(v.x, v.y);
          (p < 2 ? tc : ts)[8 * (p & 1) + 2 * i + 1] = pack2(v.z, v.w);
        }
        __syncwarp();
      }
    };
    // one tile further: by the angle sum with row 128
    auto step = [&]() {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const ulonglong2 C = *reinterpret_cast<const ulonglong2*>(&misc->tile_cos[32 * grp + 4 * i]);
        const ulonglong2 S = *reinterpret_cast<const ulonglong2*>(&misc->tile_sin[32 * grp + 4 * i]);
        const ulonglong2 N = *reinterpret_cast<const ulonglong2*>(&misc->tile_nsin[32 * grp + 4 * i]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint64_t c = tc[2 * i + e], s = ts[2 * i + e], c1 = e ? C.y : C.x, s1 = e ? S.y : S.x, n1 = e ? N.y : N.x;
          tc[2 * i + e] = fma2(c, c1, mul2(s, n1));
          ts[2 * i + e] = fma2(c, s1, mul2(s, c1));
        }
      }
    };
    while (walk.next(a, ngroups, run)) {
      const int nhg = min(nh, a.H - run.hg * nh);
      build(wtid);
      float m0 = -INFINITY, l0 = 0.f, m1 = -INFINITY, l1 = 0.f;
      for (int t = 0; t < run.n; ++t) {
        // each step adds about an fp32 rounding: seeded again before they add up
        if ((t & (kSeedTiles - 1)) == 0) seed(run.t0 + t);
        else step();
        const bool valid = row < run.L - (run.t0 + t) * kTile;
        // this group's half of a head-tile's scores
        auto half_score = [&]() -> float {
          const uint32_t par = n & 1;
          wait(misc->ufull[par], (n >> 1) & 1);
          tc_fence_after();
          uint64_t s2 = 0, s3 = 0;
          // 16 cosine and 16 sine columns at a time: the table rows hold half of the registers
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float u0[16], u1[16];
            const uint32_t u = tmem + lane_base + kUCol + par * 128 + 32 * grp + 16 * c;
            tmem_ld_x16(u, u0);
            tmem_ld_x16(u + 64, u1);
            tmem_wait_ld();
            if (c == 1) {
              tc_fence_before();
              arrive(misc->uempty[par]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              s2 = fma2(tc[8 * c + i], pack2(u0[2 * i], u0[2 * i + 1]), s2);
              s3 = fma2(ts[8 * c + i], pack2(u1[2 * i], u1[2 * i + 1]), s3);
            }
          }
          return sum2(s2) + sum2(s3);
        };
        // hand the half over, or take the other group's and finish the head-tile
        auto finish = [&](float half, float& m, float& l) {
          const uint32_t par = n & 1;
          const int id = kBarPair + 2 * q + static_cast<int>(par);
          if (grp != static_cast<int>(par)) {
            misc->part[par][row] = half;
            pair_arrive(id);
          } else {
            wait(misc->full[st.i], st.phase);   // the rows' scales (complete long since)
            const uint8_t* r = sm + P.ring + st.i * P.stage + row * rb + scale_at;
            uint32_t ktop = 0, vtop = 0;
            for (int g = 0; g < gk; ++g) ktop = max(ktop, scale_bits(r + 2 * g) & 0x7FFFu);
            uint32_t vs[RV32];
#pragma unroll
            for (int g = 0; g < RV32; ++g) {
              vs[g] = scale_bits(r + 2 * (gk + g));
              vtop = max(vtop, vs[g] & 0x7FFFu);
            }
            // 2^E: above every V scale of the warp's tokens
            const int E = min(static_cast<int>(__reduce_max_sync(0xffffffffu, valid ? vtop >> 7 : 0u)) - 126, 126);
            const float up = pow2(k_exponent(ktop)), ie = pow2(-E);
            named_bar_sync(id, 64);
            const float s = valid ? (half + misc->part[par][row]) * up : -INFINITY;
            // ---- softmax of the warp's 32 tokens: integer reference, raised lazily
            const float mt = warp_max_redux(s);
            if (mt > m + kRaise) {
              const float mn = ceilf(mt);
              l *= exp2f(m - mn);
              m = mn;
            }
            const float p = s == -INFINITY ? 0.f : exp2f(s - m);
            l += p;
            // ---- weights p * scale of each V group, relative to 2^(m + E)
            uint8_t* tail = sm + P.ring + st.i * P.stage + kTile * rb;
            __half* w = reinterpret_cast<__half*>(tail) + row;
#pragma unroll
            for (int g = 0; g < RV32; ++g)
              w[g * kWStride] = __float2half_rn(valid ? p * (__uint_as_float(vs[g] << 16) * ie) : 0.f);
            if (lane == 0) reinterpret_cast<int*>(tail + kWBytes)[q] = m == -INFINITY ? kNoRef : static_cast<int>(m) + E;
            arrive(misc->wfull[st.i]);
          }
          st.next(NS);
          ++n;
        };
        if (nhg == 2) finish(half_score(), m0, l0);
        finish(half_score(), m1, l1);
      }
      // ---- run end: (m, l) of each head
      l0 = warp_sum(l0);
      l1 = warp_sum(l1);
      if (lane == 0) {
        misc->ml[0][warp - 8] = make_float2(m0, l0);
        misc->ml[nhg - 1][warp - 8] = make_float2(m1, l1);
      }
      named_bar_sync(kBarRun, kWorkers + 32);
    }
  } else {
    regs_inc<112>();
    // ======================================================== V: sum_j p_j c_v,j
    const int v = warp - 16, gid = lane >> 2, tig = lane & 3, wtid = tid - 128;
    const int mine = nh == 2 ? v >> 1 : 0;                        // head of the group
    const int tg0 = nh == 2 ? 2 * (v & 1) : v, ntg = nh == 2 ? 2 : 1;   // its 32-token groups
    float* accs = reinterpret_cast<float*>(sm + P.acc);            // [4][RV32 * 32]
    const uint32_t half_sel = (gid & 1) ? 0x7632u : 0x5410u;
    Slot st{0, 0u};
    while (walk.next(a, ngroups, run)) {
      const int nhg = min(nh, a.H - run.hg * nh);
      build(wtid);
      float d[NM][4], one[4];
#pragma unroll
      for (int i = 0; i < NM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) d[i][j] = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) one[j] = 0.f;
      int ref = kNoRef;
      for (int t = 0; t < run.n; ++t)
        for (int hi = 0; hi < nhg; ++hi, st.next(NS)) {
          if (hi != mine) continue;
          wait(misc->wfull[st.i], st.phase);
          wait(misc->full[st.i], st.phase);
          const uint8_t* rows = sm + P.ring + st.i * P.stage;
          const uint8_t* tail = rows + kTile * rb;
#pragma unroll 1
          for (int g = tg0; g < tg0 + ntg; ++g) {
            const int r = reinterpret_cast<const int*>(tail + kWBytes)[g];
            if (r > ref) {
              const float f = exp2f(static_cast<float>(ref) - static_cast<float>(r));
#pragma unroll
              for (int i = 0; i < NM; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) d[i][j] *= f;
#pragma unroll
              for (int j = 0; j < 4; ++j) one[j] *= f;
              ref = r;
            }
            const __half2 f2 = __float2half2_rn(exp2f(static_cast<float>(r) - static_cast<float>(ref)));
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
              const int t0 = 32 * g + 16 * ks + 2 * tig;
              const __half* w = reinterpret_cast<const __half*>(tail) + gid * kWStride + t0;
              const uint32_t b0 = h2_bits(__hmul2(*reinterpret_cast<const __half2*>(w), f2));
              const uint32_t b1 = h2_bits(__hmul2(*reinterpret_cast<const __half2*>(w + 8), f2));
              mma16816(one, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, b0, b1);
              const uint8_t* p0 = rows + t0 * rb + rk / 2;
              // code word `at` of tokens t0, t0 + 1 (k of the low half) and t0 + 8, t0 + 9
              auto words = [&](int at, uint32_t sel, uint32_t& x, uint32_t& y) {
                const uint8_t* c = p0 + 4 * at;
                x = prmt(*reinterpret_cast<const uint32_t*>(c), *reinterpret_cast<const uint32_t*>(c + rb), sel);
                y = prmt(*reinterpret_cast<const uint32_t*>(c + 8 * rb), *reinterpret_cast<const uint32_t*>(c + 9 * rb), sel);
              };
              // a pair of half-words holds four columns: two MMAs of 8 + 8 rows
              auto two = [&](float (&d0)[4], float (&d1)[4], uint32_t x, uint32_t y) {
                mma16816(d0, x & 0x000F000Fu, x & 0x00F000F0u, y & 0x000F000Fu, y & 0x00F000F0u, b0, b1);
                x >>= 8;
                y >>= 8;
                mma16816(d1, x & 0x000F000Fu, x & 0x00F000F0u, y & 0x000F000Fu, y & 0x00F000F0u, b0, b1);
              };
#pragma unroll
              for (int c = 0; c < F; ++c) {
                const uint8_t* cp = p0 + 4 * (8 * c + gid);
                const uint32_t w0 = *reinterpret_cast<const uint32_t*>(cp), w1 = *reinterpret_cast<const uint32_t*>(cp + rb);
                const uint32_t w8 = *reinterpret_cast<const uint32_t*>(cp + 8 * rb), w9 = *reinterpret_cast<const uint32_t*>(cp + 9 * rb);
                two(d[4 * c], d[4 * c + 1], prmt(w0, w1, 0x5410), prmt(w8, w9, 0x5410));
                two(d[4 * c + 2], d[4 * c + 3], prmt(w0, w1, 0x7632), prmt(w8, w9, 0x7632));
              }
              if constexpr (HF) {
                uint32_t x, y;
                words(8 * F + (gid >> 1), half_sel, x, y);
                two(d[4 * F], d[4 * F + 1], x, y);
              }
            }
          }
          arrive(misc->empty[st.i]);
        }
      // ---- run end: the thread whose accumulator columns are a chunk's groups holds its
      // sums; column of (chunk, word gid, MMA i, row half): see `two`
      float* acc = accs + v * RV32 * 32;
#pragma unroll
      for (int c = 0; c < F; ++c) {
        if (tig != c) continue;
        const int jj = gid >> 2;
        const float o8 = 8.f * (jj ? one[1] : one[0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int col = 64 * c + 8 * gid + 4 * (i & 1) + (i >> 1);   // low half: even columns, high half: odd
          acc[col] = (jj ? d[4 * c + i][1] : d[4 * c + i][0]) * 16777216.f - o8;
          acc[col + 2] = (jj ? d[4 * c + i][3] : d[4 * c + i][2]) * 1048576.f - o8;
        }
      }
      if constexpr (HF) {
        if (tig == F) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int col = 64 * F + 8 * (gid >> 1) + 4 * i + (gid & 1);
            acc[col] = d[4 * F + i][0] * 16777216.f - 8.f * one[0];
            acc[col + 2] = d[4 * F + i][2] * 1048576.f - 8.f * one[0];
          }
        }
      }
      if (lane == 0) misc->vref[v] = ref;
      named_bar_sync(kBarRun, kWorkers + 32);
      // ---- one record per head: {m, l, -, -, acc[r_v]}
      const int u = run.b * ngroups + run.hg, vt = tid - (kQ4TileThreads - 128);
      for (int hi = 0; hi < nhg; ++hi) {
        float M = -INFINITY, ls = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) M = fmaxf(M, misc->ml[hi][i].x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 x = misc->ml[hi][i];
          ls = fmaf(x.y, M == -INFINITY ? 1.f : exp2f(x.x - M), ls);   // no maximum: every score was NaN
        }
        float* rec = a.records + ((static_cast<int64_t>(u) + blockIdx.x) * nh + hi) * (rv + kRecordHead);
        for (int k = vt; k < rv; k += 128) {
          float s = 0.f;
          for (int i = 0; i < 4 / nh; ++i) {
            const int vv = hi * (4 / nh) + i;
            s = fmaf(accs[vv * RV32 * 32 + k], exp2f(static_cast<float>(misc->vref[vv]) - M), s);
          }
          rec[kRecordHead + k] = s;
        }
        if (vt == 0) { rec[0] = M; rec[1] = ls; }
      }
      // which CTAs hold records of this unit
      if (vt == 0 && run.t0 == 0) a.ranges[2 * u] = blockIdx.x;
      if (vt == 0 && run.t0 + run.n == tiles_of(run.L)) a.ranges[2 * u + 1] = blockIdx.x;
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

// Merge the records of each (sequence, head) by log-sum-exp, apply W_up,v once (Appendix J
// "Absorbed attention") and normalise.  Block = (head, a.combine_units sequences).
constexpr int kCombineThreads = 128;
constexpr int kMaxCombineUnits = 8;
__global__ void __launch_bounds__(kCombineThreads) q4_combine_kernel(const __grid_constant__ Q4DecodeArgs a) {
  __shared__ float acc[kMaxCombineUnits][kMaxRankPerHead], inv[kMaxCombineUnits];
  const int h = blockIdx.x % a.H, b0 = static_cast<int>(blockIdx.x / a.H) * a.combine_units, tid = threadIdx.x;
  const int rv = a.r_v, nh = a.plan.nh, nu = min(a.combine_units, a.B - b0);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int i = 0; i < nu; ++i) {
    const int b = b0 + i, u = b * a.plan.ngroups + h / nh;
    const int L = tile_len(a, b);
    float v0 = 0.f, v1 = 0.f, l = 1.f, m = -INFINITY;
    if (L > 0) {
      const int c0 = a.ranges[2 * u], c1 = a.ranges[2 * u + 1];
      const int64_t stride = static_cast<int64_t>(nh) * (rv + kRecordHead);
      const float* rec = a.records + (static_cast<int64_t>(u) + c0) * stride + (h % nh) * (rv + kRecordHead);
      for (int c = 0; c <= c1 - c0; ++c) m = fmaxf(m, rec[c * stride]);
      l = 0.f;
      for (int c = 0; c <= c1 - c0; ++c) {
        const float* r = rec + c * stride;
        const float w = m == -INFINITY ? 1.f : exp2f(r[0] - m);
        l = fmaf(r[1], w, l);
        if (tid < rv) v0 = fmaf(r[kRecordHead + tid], w, v0);
        if (tid + 128 < rv) v1 = fmaf(r[kRecordHead + tid + 128], w, v1);
      }
    }
    if (tid < rv) acc[i][tid] = v0;
    if (tid + 128 < rv) acc[i][tid + 128] = v1;
    if (tid == 0) {
      inv[i] = 1.f / l;
      if (a.lse) a.lse[static_cast<int64_t>(b) * a.H + h] = L > 0 ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
  }
  __syncthreads();
  const __nv_bfloat16* W = static_cast<const __nv_bfloat16*>(a.w_up_v) + (static_cast<int64_t>(h) * kHeadDim + tid) * rv;
  float o[kMaxCombineUnits];
#pragma unroll
  for (int i = 0; i < kMaxCombineUnits; ++i) o[i] = 0.f;
  for (int k = 0; k < rv; k += 8) {
    float w8[8];
    unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(W + k)), w8);
#pragma unroll
    for (int i = 0; i < kMaxCombineUnits; ++i) {
      if (i >= nu) break;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[i] = fmaf(acc[i][k + e], w8[e], o[i]);
    }
  }
  const float mu = __ldg(a.mu_v + h * a.mu_hstride + tid);
#pragma unroll
  for (int i = 0; i < kMaxCombineUnits; ++i) {
    if (i >= nu) break;
    const float y = tile_len(a, b0 + i) > 0 ? fmaf(o[i], inv[i], mu) : 0.f;
    static_cast<__nv_bfloat16*>(a.out)[(static_cast<int64_t>(b0 + i) * a.H + h) * kHeadDim + tid] = __float2bfloat16_rn(y);
  }
}

template <int RV32>
cudaError_t launch_tile(const Q4DecodeArgs& a, cudaStream_t s) {
  cudaError_t e = allow_smem(q4_tile_kernel<RV32>, a.plan.bytes);
  if (e != cudaSuccess) return e;
  q4_tile_kernel<RV32><<<a.grid, kQ4TileThreads, a.plan.bytes, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

bool make_q4_plan(int H, int r_k, int r_v, Q4Plan* p) {
  const int rb = q4_row_bytes(r_k, r_v), rv32 = (r_v + 31) / 32;
  auto al = [](int x, int a) { return (x + a - 1) / a * a; };
  for (int nh = H >= 2 ? 2 : 1; nh >= 1; --nh) {
    *p = Q4Plan{};
    p->nh = nh;
    p->ngroups = (H + nh - 1) / nh;
    p->z_bias = make_chunk_plan(r_k, kTile).bytes;
    p->z_stride = p->z_bias + 4096;
    p->NA = 2 * (r_k / 2 + 8) <= 512 - kACol ? 2 : 1;
    p->stage = al(kTile * rb + kStageTail, 128);
    int off = 0;
    p->z = off; off += nh * p->z_stride;
    p->trig = off; off += kTrigBytes;
    p->acc = off; off += 4 * rv32 * 32 * 4;
    p->misc = off; off += al(static_cast<int>(sizeof(Q4Misc)), 128);
    p->ring = off;
    p->NS = std::min((kSmemLimit - 1024 - off) / p->stage, kQ4MaxNS);
    p->bytes = off + p->NS * p->stage + 1024;
    // a head-tile stays in the ring while K, scores and V take their turns: two heads
    // per group (they share a position's table rows) only with room for copies ahead
    if (p->NS >= (nh == 2 ? 4 : 2)) return true;
  }
  return false;
}

cudaError_t launch_q4_tile(const Q4DecodeArgs& a, cudaStream_t s) {
  cudaError_t e;
  switch ((a.r_v + 31) / 32) {
    case 1: e = launch_tile<1>(a, s); break;
    case 2: e = launch_tile<2>(a, s); break;
    case 3: e = launch_tile<3>(a, s); break;
    case 4: e = launch_tile<4>(a, s); break;
    case 5: e = launch_tile<5>(a, s); break;
    case 6: e = launch_tile<6>(a, s); break;
    case 7: e = launch_tile<7>(a, s); break;
    default: e = launch_tile<8>(a, s); break;
  }
  if (e != cudaSuccess) return e;
  const int blocks = a.H * ((a.B + a.combine_units - 1) / a.combine_units);
  return launch_pdl(q4_combine_kernel, dim3(blocks), dim3(kCombineThreads), 0, s, a);
}

}  // namespace lla
