// lla_q4_decode.cu — latent decode attention over the 4-bit paged cache on the tensor
// cores (bf16 storage; lla_q4.cu holds the fp32 kernel and the entry point).
//
// Score of Eq. (3) with RoPE after reconstruction, regrouped as in lla_decode_small.cu: with the
// query folded into W_up,k,t (Z_n over 128 rotary coordinates) and the position's rotary row
// R_j = (cos(j th_0..63), sin(j th_0..63)),
//     s_j = sum_n c_j,n G_j,n + bias,   G_j = R_j Z^T        (log2 units),
// so G of a 128-token tile is one MMA chain (M = 128 tokens, N = r_k + 16 or 32, K = 128), and the codes
// never enter it: a token's c_n = (code - 8) scale meets G in one thread's registers.
// A 4-bit row is 144 bytes at (96, 160), 3.6 times less than in bf16: at HBM speed an SM has about
// 6 cycles per token-head, and what bounds the kernel is the work per code and the chain of scores,
// softmax and weights in the epilogue warps; the choices below are for few instructions per code.
// 32 x 4096 tokens of 16 heads at (96, 160) take 109 us (43 for the bytes), 128 x 2048..4096 at
// (16, 32) 150 (31).
//   G  A = the rotary rows, f16, one 32 KB tile per position for all of its heads.  They are
//      rounded once per call from the fp32 table into tiles in the layout that the MMA reads, so that a
//      bulk copy brings a tile: an fp32 table read here would be more L2 traffic than
//      the latents, and rows turned in registers from tile to tile took a fifth of all
//      instructions.  B = a head's Z rows (f16), two bias rows (f16 high and low part) and two rows
//      -8 sum Z per scale group of 32, which take the codes' offset back (high and low part as well: up to 256
//      times a Z of its own, a single f16 would be off by more than all of the Z).  A last group of 16 has
//      none: its codes lose their offset in f16 (so r_k = 240 stays at one MMA chain: 161 us at 32 x 4096
//      of 15 heads and r_v = 112, with rows for it and two chains 236).  All heads of a group
//      share one chain.  Both operands are formed by q4_prepare_kernel: formed here
//      at the start of each run they stopped every role for 7 us.
//   s  One token per thread, two warpgroups alternate head-tiles.  Codes are masked into f16
//      subnormals (code * 2^-24, or * 2^-20 from the next nibble), converted, and summed per
//      scale group in fp32; the group's scale multiplies the sum.
//   V  sum_j p_j c_v,j is a warp-level MMA: A = the codes themselves, as f16 subnormals (masking is
//      the whole conversion), B = one column per scale group holding p_j scale_j,g, so that a
//      scale is applied to a weight and never to a code; a row of ones gives the sum that takes the offset of 8
//      back.  Every code is finite, so rows behind the last token only need weight 0.
//
// Work: positions (sequence, head group, 128-token tile) in that order, cut into
// equal contiguous ranges, one per CTA.  A run is a CTA's part of one (sequence, head
// group).  Roles meet only at mbarriers, at run ends too: each epilogue and V warp writes its own
// part of the run's records, which the combine merges.  Warps: 0 copies rows (bulk copies of page
// pieces), 1 copies query operands and issues MMAs, 2 copies rotary tiles, 3 gives them back, 4-11 epilogue, 12-19 V.
#include <algorithm>
#include <cmath>
#include <cstddef>
#include <type_traits>

#include "lla_q4.h"

namespace lla {

namespace {

constexpr int kQ4TileThreads = 640;
constexpr int kQ4MaxNS = 16;
constexpr int kMaxG = 16;                        // positions whose G is in TMEM
constexpr int kMaxNh = 8;                        // heads of a group
constexpr int kRowChunk = 16384;                 // half a rotary tile: a K-major chunk of 128 rows x 128 bytes
constexpr int kRowTile = 2 * kRowChunk;
constexpr int kMinNR = 3, kMaxNR = 8;             // chunks of rotary tiles in shared memory
constexpr int kState = 36;                        // floats of a (warp, head)'s state
constexpr int kWStride = 136;                    // halves between the groups of a weight tile
constexpr int kWExp = 2 * kTile;                 // bytes into it: behind the first group's weights, four exponents
constexpr float kQ4Scale = 0.08838834764831845f * 1.4426950408889634f;   // log2(e) / sqrt(128)
constexpr float kRaise = 8.f;                    // lazy maximum: raised when passed by 2^8
constexpr float kBelow = 64.f;                   // V weights count down to 2^-64 of the largest
// a record per (unit, CTA) and head: (m, l) of each epilogue warp, the reference (m, E) of each V warp, their sums
constexpr int kRecMl = 0, kRecRef = 16, kRecAcc = 32;

struct alignas(16) Q4Misc {
  uint64_t full[kQ4MaxNS], empty[kQ4MaxNS], wfull[kQ4MaxNS];
  uint64_t rfull[kMaxNR], rempty[kMaxNR], gfull[kMaxG], gempty[kMaxG];
  uint64_t zfull, zdone;                         // query operands: copied; no longer read
  uint32_t tmem_base;
  int abort;
  int start_b, start_hg, start_t, count;
};

// Position of a ring with its barriers' phase.  A wait tells a phase from the one before it only, so no
// warp may leave out phases of a barrier that it waits on.  Every ring that several groups take
// turns at therefore has a multiple of their number of barriers, which gives each barrier one
// waiting group: the head-tiles of the two epilogue groups (NS even; with one head PB too), the heads of
// the V warps (NS a multiple of nh, and so is H).
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

// Shared-memory accesses by 32-bit address (the loops below are bound by instruction issue).
__device__ __forceinline__ uint32_t lds32(uint32_t p) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(p));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t p) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(p));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t p) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(p));
  return v;
}
__device__ __forceinline__ void sts32(uint32_t p, uint32_t v) { asm volatile("st.shared.u32 [%0], %1;" ::"r"(p), "r"(v) : "memory"); }
__device__ __forceinline__ void sts16(uint32_t p, __half v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(p), "h"(__half_as_ushort(v)) : "memory");
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }
__device__ __forceinline__ uint32_t h2_bits(__half2 v) { return *reinterpret_cast<uint32_t*>(&v); }
__device__ __forceinline__ __half2 bits_h2(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }
// D[16 x 8] += A[16 x 16] B[16 x 8], f16 operands, fp32 accumulator (one warp).
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127

// Warp-collective bounded wait for a barrier phase: every lane tests it, so each makes its own
// acquire; the clock and the abort flag are looked at now and then only, because a
// waiting warp's instructions are taken from the warps that work.
__device__ __forceinline__ bool q4_wait(uint32_t bar, uint32_t parity, volatile int* abort, uint32_t* status) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (__all_sync(0xffffffffu, mbar_try_wait_sleep(bar, parity, 20000))) return true;
    const bool give_up = *abort != 0 || global_timer_ns() - t0 > kWaitLimitNs;
    if (__any_sync(0xffffffffu, give_up)) {
      record_status(status, LLA_ERR_TIMEOUT);
      *abort = 1;
      return false;
    }
  }
}

// Register shares of the warpgroups: 64 + 2 x 96 + 2 x 112 = 480 = 5 x 96, what the
// block is launched with (640 threads of 96); up to 192 V columns 72 + 2 x 96 + 2 x 104 (at 160 the
// producers spill with 64: 32 x 4096 takes 112 us, else 109).
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

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
  const int nh = P.nh, ngroups = P.ngroups, NS = P.NS, PG = P.PG, PB = P.PB, NR = P.NR, N = P.N, gstep = P.gstep, rk = a.r_k, rv = a.r_v, rb = a.row_bytes;
  const int scale_at = q4_scale_offset(rk, rv), gk = q4_groups(rk);

  // ---------------------------------------------------------- work range
  int* scan = reinterpret_cast<int*>(sm + P.ring);   // (before any copy)
  RunWalker start{0, 0, 0, 0};
  {
    const int per_thr = (a.B + kQ4TileThreads - 1) / kQ4TileThreads;
    const int b0 = min(a.B, tid * per_thr), b1 = min(a.B, b0 + per_thr);
    long long local = 0;
    for (int b = b0; b < b1; ++b) {
      const int L0 = __ldg(a.seq_lens + b);
      if (blockIdx.x == 0 && (L0 < 0 || L0 > a.L_max)) record_status(a.status, LLA_ERR_DEVICE_ARG);
      local += tiles_of(tile_len(a, b));
    }
    scan[tid] = static_cast<int>(local);
    if (tid == 0) { misc->abort = 0; misc->count = 0; }
    __syncthreads();
    if (warp == 0) {
      constexpr int kPer = kQ4TileThreads / 32;
      int s = 0;
      for (int i = 0; i < kPer; ++i) s += scan[lane * kPer + i];
      int incl = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += n;
      }
      int excl = incl - s;
      for (int i = 0; i < kPer; ++i) {
        const int v = scan[lane * kPer + i];
        scan[lane * kPer + i] = excl;
        excl += v;
      }
      if (lane == 31) misc->start_t = incl;   // total tiles, read below
    }
    __syncthreads();
    const long long total = static_cast<long long>(misc->start_t) * ngroups;
    const long long per = max(1LL, (total + a.grid - 1) / a.grid);
    const long long f0 = static_cast<long long>(blockIdx.x) * per, f1 = min(total, f0 + per);
    long long p0 = static_cast<long long>(scan[tid]) * ngroups;
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
      mbar_init(bar(misc->empty[s]), 8 / nh);       // the head's V warps, the last to read it
      mbar_init(bar(misc->wfull[s]), 4);
    }
    for (int i = 0; i < NR; ++i) {
      mbar_init(bar(misc->rfull[i]), 1);
      mbar_init(bar(misc->rempty[i]), 1);
    }
    for (int i = 0; i < PB; ++i) {
      mbar_init(bar(misc->gfull[i]), 1);
      mbar_init(bar(misc->gempty[i]), 4 * nh);
    }
    mbar_init(bar(misc->zfull), 1);
    mbar_init(bar(misc->zdone), 1);
    fence_mbar_init();
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
  RunWalker walk = start;
  Run run{0, 0, 0, 0, 0};
  bool ok = true;
  auto wait = [&](const uint64_t& m, uint32_t parity) {
    if (ok) ok = q4_wait(bar(m), parity, abort, a.status);
  };
  auto arrive = [&](const uint64_t& m) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(m));
  };

  // record of head hi of the run in this CTA
  auto record = [&](int hi) {
    return a.records + ((static_cast<int64_t>(run.b) * ngroups + run.hg + blockIdx.x) * nh + hi) * a.rec_stride;
  };
  // Waits (bounded) for the last `count` copies of a ring of n slots to land: none may be in
  // flight when the CTA exits.  (`at`, the next slot, holds the oldest of the last n, or none yet.)
  auto land = [&](uint64_t* full, Slot at, int n, int count) {
    for (int i = min(count, n); i > 0; --i) {
      if (count < n && i == count) at = Slot{0, 0u};
      const uint32_t phase = count < n ? 0u : at.phase ^ 1u;
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(bar(full[at.i]), phase) && global_timer_ns() - t0 < kWaitLimitNs) {}
      at.next(n);
    }
  };
  if (warp < 4) {
    regs_dec<RV32 <= 6 ? 72 : 64>();
    if (warp == 0) {
      // ======================================================== producer of rows
      // Per head-tile the page pieces that its rows lie in, lane i copying piece i.  A position's page ids are
      // requested one position ahead: read when needed, their latency would pace the ring.
      struct Pos {
        int b, hg, y0, y1, lp0, np, page;
      };
      Slot st{0, 0u};
      int issued = 0, left = 0, t = 0;
      const int pg = a.page_size;
      const int64_t head_bytes = static_cast<int64_t>(pg) * rb;
      auto next = [&](Pos& x) -> bool {
        if (left == 0) {
          if (!walk.next(a, ngroups, run)) return false;
          left = run.n;
          t = run.t0;
        }
        x.b = run.b;
        x.hg = run.hg;
        x.y0 = t * kTile;
        x.y1 = min(x.y0 + kTile, run.L);
        x.lp0 = x.y0 / pg;
        x.np = (x.y1 - 1) / pg - x.lp0 + 1;
        if (lane < x.np) x.page = __ldg(a.block_table + static_cast<int64_t>(x.b) * a.max_pages + x.lp0 + lane);
        --left;
        ++t;
        return true;
      };
      // piece i of a position: bytes, offset in the stage, address of the first head's rows
      struct Piece {
        uint32_t bytes, to;
        const uint8_t* from;
      };
      auto piece = [&](const Pos& x, int i, int page) -> Piece {
        const int p0 = (x.lp0 + i) * pg, t0 = max(x.y0, p0), t1 = i + 1 < x.np ? p0 + pg : x.y1;
        if (page < 0 || page >= a.num_pages) {
          record_status(a.status, LLA_ERR_DEVICE_ARG);
          page = 0;
        }
        return Piece{static_cast<uint32_t>((t1 - t0) * rb), static_cast<uint32_t>((t0 - x.y0) * rb),
                     a.rows + (static_cast<int64_t>(page) * a.H + x.hg * nh) * head_bytes + static_cast<int64_t>(t0 - p0) * rb};
      };
      Pos x{}, y{};
      bool more = next(y);
      while (more && ok) {
        x = y;
        more = next(y);
        Piece mine{};
        if (lane < x.np) mine = piece(x, lane, x.page);
        for (int hi = 0; hi < nh && ok; ++hi) {
          wait(misc->empty[st.i], st.phase ^ 1u);
          if (!ok) break;
          const uint32_t fb = bar(misc->full[st.i]), dst = sbase + P.ring + st.i * P.stage;
          if (lane == 0) mbar_arrive_expect_tx(fb, (x.y1 - x.y0) * rb);
          __syncwarp();
          if (lane < x.np) bulk_load(dst + mine.to, mine.from + hi * head_bytes, mine.bytes, fb);
          for (int i = lane + 32; i < x.np; i += 32) {   // pages of fewer than four tokens
            const Piece z = piece(x, i, __ldg(a.block_table + static_cast<int64_t>(x.b) * a.max_pages + x.lp0 + i));
            bulk_load(dst + z.to, z.from + hi * head_bytes, z.bytes, fb);
          }
          __syncwarp();
          ++issued;
          st.next(NS);
        }
      }
      if (lane == 0) land(misc->full, st, NS, issued);
    } else if (warp == 2) {
      // ======================================================== producer of rotary tiles
      Slot rs{0, 0u};
      int issued = 0;
      asm volatile("griddepcontrol.wait;" ::: "memory");   // they are written
      while (walk.next(a, ngroups, run))
        for (int c = 2 * run.t0; c < 2 * (run.t0 + run.n) && ok; ++c) {
          wait(misc->rempty[rs.i], rs.phase ^ 1u);
          if (!ok) break;
          if (lane == 0) {
            const uint32_t fb = bar(misc->rfull[rs.i]);
            mbar_arrive_expect_tx(fb, kRowChunk);
            bulk_load(sbase + P.rows + rs.i * kRowChunk, a.row_tiles + static_cast<int64_t>(c) * kRowChunk, kRowChunk, fb);
          }
          __syncwarp();
          ++issued;
          rs.next(NR);
        }
      if (lane == 0) land(misc->rfull, rs, NR, issued);
    } else if (warp == 3) {
      // ======================================================== rotary chunks of finished MMAs
      // (gfull cannot come round twice unseen: NR <= 2 PB + 1 chunks, and position t + PB needs one of t's)
      Slot rs{0, 0u}, gp{0, 0u};
      while (walk.next(a, ngroups, run))
        for (int t = 0; t < run.n; ++t) {
          wait(misc->gfull[gp.i], gp.phase);
          gp.next(PB);
          for (int c = 0; c < 2; ++c) {
            if (ok && lane == 0) mbar_arrive(bar(misc->rempty[rs.i]));
            rs.next(NR);
          }
        }
    } else if (warp == 1) {
      // ======================================================== MMA issuer
      // G = R Z^T; the whole warp runs the loop, one elected lane issues.  With A in shared memory a
      // step takes about as long for 256 columns as for 128, so the heads of a group share one chain
      // (r_k = 256: two chains).  Commits took this warp 570 cycles each, more than
      // issuing the eight MMAs, so there is one per position: of all heads' buffers and, passed on by
      // warp 3, of the rotary chunks.  (One per head and chunk bound the kernel: 122 us at 32 x 4096, one per
      // position 106.)
      // A run's query operands come by two bulk copies once the last run's MMAs are done; the epilogue
      // still has up to PG positions of that run to go.
      Slot rs{0, 0u}, gp{0, 0u};
      uint32_t runs = 0;
      asm volatile("griddepcontrol.wait;" ::: "memory");   // the operands are written
      while (walk.next(a, ngroups, run)) {
        if (runs > 0) {
          if (ok) umma_commit_warp(bar(misc->zdone));
          wait(misc->zdone, (runs - 1) & 1);
        }
        if (ok && lane == 0) {
          const uint32_t bytes = nh * N * 128;
          const uint8_t* src = a.zimg + (static_cast<int64_t>(run.b) * ngroups + run.hg) * 2 * P.z_chunk;
          mbar_arrive_expect_tx(bar(misc->zfull), 2 * bytes);
          bulk_load(sbase + P.z, src, bytes, bar(misc->zfull));
          bulk_load(sbase + P.z + P.z_chunk, src + P.z_chunk, bytes, bar(misc->zfull));
        }
        __syncwarp();
        wait(misc->zfull, runs & 1);
        if (ok) ++runs;
        for (int t = 0; t < run.n; ++t) {
          // the position's buffers (PG = 1: two barriers take turns at one), then its chunks: cosines, sines
          if (PG > 1) wait(misc->gempty[gp.i], gp.phase ^ 1u);
          else wait(misc->gempty[gp.i ^ 1], gp.phase ^ static_cast<uint32_t>(gp.i ^ 1));
          uint64_t ad[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            wait(misc->rfull[rs.i], rs.phase);
            ad[c] = umma_desc(sbase + P.rows + rs.i * kRowChunk, 16, 1024, kSw128);
            rs.next(NR);
          }
          tc_fence_after();
          if (ok) {
            for (int r0 = 0; r0 < nh * N; r0 += 256) {
              const uint32_t idesc = umma_idesc_f16(128, min(nh * N - r0, 256));
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const uint64_t bd = umma_desc(sbase + P.z + c * P.z_chunk + r0 * 128, 16, 1024, kSw128);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  umma_bf16_warp(tmem + gp.i * gstep + r0, ad[c] + 2 * kk, bd + 2 * kk, idesc, c + kk > 0 ? 1u : 0u);
              }
            }
            umma_commit_warp(bar(misc->gfull[gp.i]));
          }
          gp.next(PB);
        }
      }
      // this warp's copies and MMAs complete before shared memory and TMEM are released
      if (!ok && lane == 0) {
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(bar(misc->zfull), runs & 1) && global_timer_ns() - t0 < kWaitLimitNs) {}
      }
      umma_commit_warp(bar(misc->zdone));
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(bar(misc->zdone), (runs + 1) & 1) && global_timer_ns() - t0 < kWaitLimitNs) {}
    }
  } else if (warp < 12) {
    // ======================================================== epilogue: scores, weights
    const int grp = (warp - 4) >> 2, q = warp & 3, row = 32 * q + lane;
    const uint32_t lane_base = static_cast<uint32_t>(32 * q) << 16;
    Slot st{0, 0u}, gp{0, 0u};
    uint32_t n = 0;         // head-tiles so far: group n & 1 takes the n-th
    // per head each thread's own sum, the warp's reference, and the units of its query operands
    float* state = reinterpret_cast<float*>(sm + P.state) + (warp - 4) * nh * kState;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the units are written
    while (walk.next(a, ngroups, run)) {
      for (int hi = 0; hi < nh; ++hi) {
        state[hi * kState + lane] = 0.f;
        if (lane == 0) state[hi * kState + 32] = -INFINITY;
        if (lane == 0)
          *reinterpret_cast<float2*>(state + hi * kState + 34) =
              __ldcg(a.z_unit + static_cast<int64_t>(run.b) * a.H + run.hg * nh + hi);
      }
      __syncwarp();
#pragma unroll 1
      for (int t = 0; t < run.n; ++t) {
        const bool valid = row < run.L - (run.t0 + t) * kTile;
#pragma unroll 1
        for (int hi = 0; hi < nh; ++hi, ++n, st.next(NS)) {
          if (grp != static_cast<int>(n & 1)) continue;
          const uint32_t base = sbase + P.ring + st.i * P.stage, tail = base + kTile * rb, r = base + row * rb;
          wait(misc->full[st.i], st.phase);
          wait(misc->gfull[gp.i], gp.phase);
          tc_fence_after();
          const uint32_t gcol = tmem + lane_base + gp.i * gstep + hi * N;
          float bias[2], s = 0.f;
          tmem_ld_x2(gcol + rk, bias);
          // ---- V scales
          uint32_t vtop = 0, vs[RV32];
#pragma unroll
          for (int g = 0; g < RV32; ++g) {
            vs[g] = 0;
            if (valid) vs[g] = lds16(r + scale_at + 2 * (gk + g));   // (a row that holds no token may hold anything)
            vtop = max(vtop, vs[g] & 0x7FFFu);
          }
          // ---- per scale group its codes against G: 32 columns, or 16 in a last group
          auto sum8 = [&](uint32_t w, const float* G, float& lo, float& hi, auto centred) {   // columns of one code word
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              __half2 x = bits_h2(w & 0x000F000Fu), y = bits_h2(w & 0x00F000F0u);
              if constexpr (centred.value) {   // (code + 8) - 8, exact
                x = __hsub2(x, bits_h2(0x00080008u));
                y = __hsub2(y, bits_h2(0x00800080u));
              }
              const float2 c = __half22float2(x), d = __half22float2(y);
              w >>= 8;
              lo = fmaf(c.x, G[4 * j], lo);
              lo = fmaf(c.y, G[4 * j + 1], lo);
              hi = fmaf(d.x, G[4 * j + 2], hi);
              hi = fmaf(d.y, G[4 * j + 3], hi);
            }
          };
          auto scaled = [&](uint32_t sc, float lo, float hi, float off) {
            s = fmaf(__uint_as_float(sc << 16), fmaf(lo, 16777216.f, fmaf(hi, 1048576.f, off)), s);
          };
          const int whole = rk / kQ4Group;
#pragma unroll 1
          for (int g = 0; g < whole; ++g) {
            float G[32], off[2];
            tmem_ld_x32(gcol + 32 * g, G);
            tmem_ld_x2(gcol + rk + 2 + 2 * g, off);
            const uint4 w = lds128(r + 16 * g);
            const uint32_t sc = lds16(r + scale_at + 2 * g);
            tmem_wait_ld();
            float lo[2] = {0.f, 0.f}, hi2[2] = {0.f, 0.f};
            sum8(w.x, G, lo[0], hi2[0], std::false_type{});
            sum8(w.y, G + 8, lo[1], hi2[1], std::false_type{});
            sum8(w.z, G + 16, lo[0], hi2[0], std::false_type{});
            sum8(w.w, G + 24, lo[1], hi2[1], std::false_type{});
            scaled(sc, lo[0] + lo[1], hi2[0] + hi2[1], off[0] + off[1]);
          }
          if (whole < gk) {
            float G[16];
            tmem_ld_x16(gcol + 32 * whole, G);
            const uint2 w = lds64(r + 16 * whole);
            const uint32_t sc = lds16(r + scale_at + 2 * whole);
            tmem_wait_ld();
            float lo[2] = {0.f, 0.f}, hi2[2] = {0.f, 0.f};
            sum8(w.x, G, lo[0], hi2[0], std::true_type{});
            sum8(w.y, G + 8, lo[1], hi2[1], std::true_type{});
            scaled(sc, lo[0] + lo[1], hi2[0] + hi2[1], 0.f);
          }
          tc_fence_before();
          arrive(misc->gempty[gp.i]);
          const float2 unit = *reinterpret_cast<const float2*>(state + hi * kState + 34);
          s = valid ? fmaf(s, unit.x, (bias[0] + bias[1]) * unit.y) : -INFINITY;
          // ---- softmax of the warp's 32 tokens: integer reference, raised lazily
          const float mt = warp_max_redux(s);
          float m = state[hi * kState + 32], l = state[hi * kState + lane];
          if (mt > m + kRaise) {
            const float mn = ceilf(mt);
            l *= exp2f(m - mn);
            m = mn;
            __syncwarp();
            if (lane == 0) state[hi * kState + 32] = m;
          }
          const float p = s == -INFINITY ? 0.f : exp2f(s - m);
          state[hi * kState + lane] = l + p;
          // ---- weights p * scale of each V group, relative to 2^(m + E): the largest of the warp's comes to
          // 2^7 .. 2^15, so f16 keeps all its digits down to 2^21 below it.  m + E is a multiple of 8 less 7,
          // which makes it the same for most tiles, whichever warp they come from.
          const float p9 = p * 0.001953125f;   // (2^-9: p is at most 2^8, the products stay finite)
          const uint32_t wtop = __reduce_max_sync(0xffffffffu, __float_as_uint(p9 * __uint_as_float(vtop << 16)) & 0x7FFFFFFFu);
          const int m8 = __float2int_rz(m) & 7;   // (m past 2^31 saturates: any fixed value serves)
          const int E = max(((static_cast<int>(wtop >> 23) - 118 + m8) & ~7) - m8 - 7, -118);
          const uint32_t out = tail + 2 * row;
          const float ie = pow2(9 - E);
#pragma unroll
          for (int g = 0; g < RV32; ++g) sts16(out + 2 * g * kWStride, __float2half_rn(p9 * __uint_as_float(vs[g] << 16) * ie));
          // (two numbers: from 2^24 on m + E would lose E; m of -inf: no token with a weight)
          if (lane == 0) {
            sts32(tail + P.w_bytes + 4 * q, __float_as_uint(wtop != 0 ? m : -INFINITY));
            sts32(tail + kWExp + 4 * q, __float_as_uint(static_cast<float>(E)));
          }
          arrive(misc->wfull[st.i]);
        }
        gp.next(PB);
      }
      // ---- run end: (m, l) of this warp's tokens
      for (int hi = 0; hi < nh; ++hi) {
        const float l = warp_sum(state[hi * kState + lane]);
        if (lane == 0) *reinterpret_cast<float2*>(record(hi) + kRecMl + 2 * (warp - 4)) = make_float2(state[hi * kState + 32], l);
      }
      __syncwarp();
    }
  } else {
    regs_inc<RV32 <= 6 ? 104 : 112>();
    // ======================================================== V: sum_j p_j c_v,j
    const int v = warp - 12, gid = lane >> 2, tig = lane & 3;
    // a head has 8 / nh warps, each with 16 nh of a tile's tokens
    const int per = 8 / nh, mine = v / per, ks_first = v % per * nh;
    const uint32_t half_sel = (gid & 1) ? 0x7632u : 0x5410u;
    Slot st{0, 0u};
    while (walk.next(a, ngroups, run)) {
      float d[NM][4], one[4];
#pragma unroll
      for (int i = 0; i < NM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) d[i][j] = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) one[j] = 0.f;
      float ref_m = -INFINITY, ref_e = 0.f, below = 0.f;   // the sums are relative to 2^(ref_m + ref_e); the highest reference is 2^below above
      for (int t = 0; t < run.n; ++t)
        for (int hi = 0; hi < nh; ++hi, st.next(NS)) {
          if (hi != mine) continue;
          wait(misc->wfull[st.i], st.phase);
          const uint32_t rows = sbase + P.ring + st.i * P.stage, tail = rows + kTile * rb;
#pragma unroll 1
          for (int g = ks_first >> 1; 2 * g < ks_first + nh; ++g) {
            // The reference of these 32 tokens' weights.  The sums follow it up and down: f16 has no room for
            // weights relative to another one, and the tokens that it leaves out may be thousands (a
            // sink's followers).  fp32 sums of weights up to 2^15 hold the 2^64 above the reference
            // that this may need; what lies further below the highest one is less than their last bit.
            const float r_m = __uint_as_float(lds32(tail + P.w_bytes + 4 * g)), r_e = __uint_as_float(lds32(tail + kWExp + 4 * g));
            if (r_m == -INFINITY) continue;   // no token has a weight (scores that are NaN: so is the sum of the weights)
            const float gap = (ref_m - r_m) + (ref_e - r_e);
            if (gap != 0.f) {
              if (below + gap > kBelow) continue;
              const float f = gap < -126.f ? 0.f : pow2(static_cast<int>(gap));
#pragma unroll
              for (int i = 0; i < NM; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) d[i][j] *= f;
#pragma unroll
              for (int j = 0; j < 4; ++j) one[j] *= f;
              ref_m = r_m;
              ref_e = r_e;
              below = fmaxf(below + gap, 0.f);
            }
            const int ks_end = min(2 * g + 2, ks_first + nh);
#pragma unroll 1
            for (int ks = max(2 * g, ks_first); ks < ks_end; ++ks) {
              // tokens t0, t0 + 1 (k of the low half of B) and t0 + 8, t0 + 9
              // (columns without a scale group repeat the last one's weights: never read from D)
              const int t0 = 16 * ks + 2 * tig;
              const uint32_t w = tail + 2 * (min(gid, RV32 - 1) * kWStride + t0), p0 = rows + t0 * rb + rk / 2;
              const uint32_t b0 = lds32(w), b1 = lds32(w + 16);
              const uint32_t p1 = p0 + rb, p8 = p0 + 8 * rb, p9 = p1 + 8 * rb;
              mma16816(one, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, b0, b1);
              // a pair of half-words holds four columns: two MMAs of 8 + 8 rows
              auto two = [&](float (&d0)[4], float (&d1)[4], uint32_t x, uint32_t y) {
                mma16816(d0, x & 0x000F000Fu, x & 0x00F000F0u, y & 0x000F000Fu, y & 0x00F000F0u, b0, b1);
                x >>= 8;
                y >>= 8;
                mma16816(d1, x & 0x000F000Fu, x & 0x00F000F0u, y & 0x000F000Fu, y & 0x00F000F0u, b0, b1);
              };
#pragma unroll
              for (int c = 0; c < F; ++c) {
                const uint32_t o = 4 * gid + 32 * c;
                const uint32_t w0 = lds32(p0 + o), w1 = lds32(p1 + o), w8 = lds32(p8 + o), w9 = lds32(p9 + o);
                two(d[4 * c], d[4 * c + 1], prmt(w0, w1, 0x5410), prmt(w8, w9, 0x5410));
                two(d[4 * c + 2], d[4 * c + 3], prmt(w0, w1, 0x7632), prmt(w8, w9, 0x7632));
              }
              if constexpr (HF) {
                const uint32_t o = 4 * (gid >> 1) + 32 * F;
                two(d[4 * F], d[4 * F + 1], prmt(lds32(p0 + o), lds32(p1 + o), half_sel),
                    prmt(lds32(p8 + o), lds32(p9 + o), half_sel));
              }
            }
          }
          arrive(misc->empty[st.i]);
        }
      // ---- run end: the thread whose accumulator columns are a chunk's groups holds its
      // sums; column of (chunk, word gid, MMA i, row half): see `two`
      float* rec = record(mine);
      float* acc = rec + kRecAcc + v % per * rv;
      if (lane == 0) *reinterpret_cast<float2*>(rec + kRecRef + 2 * (v % per)) = make_float2(ref_m, ref_e);
      auto put = [&](int col, float x) {
        if (col < rv) acc[col] = x;
      };
#pragma unroll
      for (int c = 0; c < F; ++c) {
        if (tig != c) continue;
        const int jj = gid >> 2;
        const float o8 = 8.f * (jj ? one[1] : one[0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int col = 64 * c + 8 * gid + 4 * (i & 1) + (i >> 1);   // low half: even columns, high half: odd
          put(col, (jj ? d[4 * c + i][1] : d[4 * c + i][0]) * 16777216.f - o8);
          put(col + 2, (jj ? d[4 * c + i][3] : d[4 * c + i][2]) * 1048576.f - o8);
        }
      }
      if constexpr (HF) {
        if (tig == F) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int col = 64 * F + 8 * (gid >> 1) + 4 * i + (gid & 1);
            put(col, d[4 * F + i][0] * 16777216.f - 8.f * one[0]);
            put(col + 2, d[4 * F + i][2] * 1048576.f - 8.f * one[0]);
          }
        }
      }
      // which CTAs hold records of this unit
      const int u = run.b * ngroups + run.hg;
      if (v == 0 && lane == 0 && run.t0 == 0) a.ranges[2 * u] = blockIdx.x;
      if (v == 0 && lane == 0 && run.t0 + run.n == tiles_of(run.L)) a.ranges[2 * u + 1] = blockIdx.x;
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

// The operands of the decode grid's MMAs, in the layouts that they are read in.
// Blocks below a.z_blocks: the query operands of one head and up to kQ4PrepSeqs sequences.  Per (sequence,
// head group) two K-major chunks (cosine, then sine coordinates) of nh N rows of 128 bytes,
// 128-byte swizzle; a head's N rows are its r_k rows Z_n, bias high and low, -8 sum Z high and low of each
// scale group of 32, zeros.  With q' = RoPE(q, q_pos) and the frequency pair (i0, i1) of f:
//     Z_n,f = sc (q'_i0 W_i0,n + q'_i1 W_i1,n),  Z_n,64+f = sc (q'_i1 W_i0,n - q'_i0 W_i1,n),
// the bias rows the same over mu; either times a power of two that brings the largest (for Z a
// bound of it) to 2^7, because f16 has no range to spare for queries and weights of any size.  The
// inverses, the units, are multiplied back into the score.  A warp holds the weights of 32 columns and 32 frequencies in
// registers and serves the block's sequences with them.
// The other blocks: the f16 rotary rows of every position below the longest length, as
// tiles of 128 positions (chunk 0 cosines, chunk 1 sines); 512 bytes read and 256 written
// per position.  The decode grid's set-up overlaps this kernel.
constexpr int kPrepThreads = 256;

constexpr int kRowsPart = 16;        // positions of a block: short contexts want many blocks
__global__ void __launch_bounds__(kPrepThreads) q4_prepare_kernel(const __grid_constant__ Q4DecodeArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (static_cast<int>(blockIdx.x) >= a.z_blocks) {
    __shared__ int longest[kPrepThreads / 32];
    int L = 0;
    for (int b = tid; b < a.B; b += kPrepThreads) L = max(L, tile_len(a, b));
    L = __reduce_max_sync(0xffffffffu, L);
    if (lane == 0) longest[warp] = L;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPrepThreads / 32; ++i) L = max(L, longest[i]);
    const int64_t end = static_cast<int64_t>(tiles_of(L)) * kTile;
    const int row0 = tid >> 4, c = tid & 15;   // 16 positions x 16 pieces of 8 coordinates
    const int64_t step = static_cast<int64_t>(gridDim.x - a.z_blocks) * kRowsPart;
    for (int64_t p = static_cast<int64_t>(blockIdx.x - a.z_blocks) * kRowsPart + row0; p < end; p += step) {
      const int64_t j = p < a.rope_len ? p : a.rope_len - 1;   // behind the sequence's end: masked
      const int row = static_cast<int>(p & (kTile - 1));
      const float4* src = reinterpret_cast<const float4*>((c < 8 ? a.rope_cos : a.rope_sin) + j * 64 + 8 * (c & 7));
      const float4 x = __ldg(src), y = __ldg(src + 1);
      *reinterpret_cast<uint4*>(a.row_tiles + p / kTile * kRowTile + (c >> 3) * kRowChunk +
                                swizzle_offset(row * 128 + 16 * (c & 7), 128)) =
          make_uint4(h2_bits(__floats2half2_rn(x.x, x.y)), h2_bits(__floats2half2_rn(x.z, x.w)),
                     h2_bits(__floats2half2_rn(y.x, y.y)), h2_bits(__floats2half2_rn(y.z, y.w)));
    }
    return;
  }
  static_assert(kPrepThreads == 64 * kQ4PrepSeqs, "a thread per sequence and frequency");
  __shared__ float qs[kQ4PrepSeqs][2][64];   // sc q'_i0 and sc q'_i1
  __shared__ uint32_t tops[3][kPrepThreads / 32];   // bits of the largest |q'|, |bias|, |W| of each warp
  const int h = blockIdx.x % a.H, b0 = blockIdx.x / a.H * kQ4PrepSeqs, seqs = min(kQ4PrepSeqs, a.B - b0);
  const Q4Plan& P = a.plan;
  const int N = P.N, rk = a.r_k, gk = q4_groups(rk), nh = P.nh, hi = h % nh;
  auto i0_of = [&](int f) { return a.rope_style == 0 ? f : 2 * f; };
  auto i1_of = [&](int f) { return a.rope_style == 0 ? f + 64 : 2 * f + 1; };
  // rows of (sequence s of the block, this head): 8-byte aligned coordinates of a row
  auto at = [&](int s, int row, int coord) {
    return a.zimg + (static_cast<int64_t>(b0 + s) * P.ngroups + h / nh) * 2 * P.z_chunk + (coord >> 6) * P.z_chunk +
           swizzle_offset((hi * N + row) * 128 + 2 * (coord & 63), 128);
  };
  __half2 top = __half2half2(__ushort_as_half(0));   // largest magnitude written (infinite: out of range)
  const int ms = tid >> 6, mf = tid & 63;    // the thread's sequence and frequency
  float bias[2] = {0.f, 0.f};
  {
    uint32_t w_top = 0;
    const uint4* W = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.w_up_k) + static_cast<int64_t>(h) * kHeadDim * rk);
#pragma unroll 4
    for (int i = tid; i < kHeadDim * rk / 8; i += kPrepThreads) {
      const uint4 x = __ldg(W + i);
      w_top = __vmaxu2(w_top, __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
    }
    float q0 = 0.f, q1 = 0.f;
    if (ms < seqs) {
      const int b = b0 + ms;
      int qp = __ldg(a.q_pos + b);
      if (qp < 0 || qp >= a.rope_len) {
        if (mf == 0) record_status(a.status, LLA_ERR_DEVICE_ARG);
        qp = qp < 0 ? 0 : static_cast<int>(a.rope_len - 1);
      }
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (static_cast<int64_t>(b) * a.H + h) * kHeadDim;
      const float c = __ldg(a.rope_cos + static_cast<int64_t>(qp) * 64 + mf);
      const float sn = __ldg(a.rope_sin + static_cast<int64_t>(qp) * 64 + mf);
      const float x0 = __bfloat162float(q[i0_of(mf)]), x1 = __bfloat162float(q[i1_of(mf)]);
      q0 = (x0 * c - x1 * sn) * kQ4Scale;
      q1 = (x0 * sn + x1 * c) * kQ4Scale;
      const float m0 = __ldg(a.mu_k + h * a.mu_hstride + i0_of(mf)), m1 = __ldg(a.mu_k + h * a.mu_hstride + i1_of(mf));
      bias[0] = q0 * m0 + q1 * m1;
      bias[1] = q1 * m0 - q0 * m1;
    }
    qs[ms][0][mf] = q0;
    qs[ms][1][mf] = q1;
    auto bits = [](float x) { return __float_as_uint(x) & 0x7FFFFFFFu; };   // (NaN sorts above infinity)
    w_top = __reduce_max_sync(0xffffffffu, max(w_top << 16, w_top & 0xFFFF0000u));
    const uint32_t q_top = __reduce_max_sync(0xffffffffu, max(bits(q0), bits(q1)));
    const uint32_t b_top = __reduce_max_sync(0xffffffffu, max(bits(bias[0]), bits(bias[1])));
    if (lane == 0) {
      tops[0][warp] = q_top;
      tops[1][warp] = b_top;
      tops[2][warp] = w_top;
    }
  }
  __syncthreads();
  uint32_t w_top = 0;
#pragma unroll
  for (int i = 0; i < kPrepThreads / 32; ++i) w_top = max(w_top, tops[2][i]);
  // the exponent that brings a value of these bits to 2^7 at most; 0 if not finite: nor is the result
  auto lift = [](uint32_t bits) {
    return bits >= 0x7F800000u ? 0 : max(-100, min(100, 133 - static_cast<int>(bits >> 23)));
  };
  auto z_lift = [&](int s) {   // of sequence s: |Z| <= 2 max|q'| max|W|
    return lift(__float_as_uint(2.f * __uint_as_float(max(tops[0][2 * s], tops[0][2 * s + 1])) * __uint_as_float(w_top)));
  };
  if (ms < seqs) {
    const int e = lift(max(tops[1][2 * ms], tops[1][2 * ms + 1]));
    if (mf == 0) a.z_unit[static_cast<int64_t>(b0 + ms) * a.H + h] = make_float2(pow2(-z_lift(ms)), pow2(-e));
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const float x = bias[part] * pow2(e);
      const __half high = __float2half_rn(x);
      top = __hmax2(top, __habs2(__half2half2(high)));
      *reinterpret_cast<__half*>(at(ms, rk, 64 * part + mf)) = high;
      *reinterpret_cast<__half*>(at(ms, rk + 1, 64 * part + mf)) = __float2half_rn(x - __half2float(high));
      for (int row = rk + 2 + 2 * (rk / kQ4Group); row < N; ++row) *reinterpret_cast<__half*>(at(ms, row, 64 * part + mf)) = __ushort_as_half(0);
    }
  }
  // item = (scale group, half of the frequencies); lane = (8 columns, 4 frequencies).  The (item,
  // sequence) pairs are dealt out evenly, a warp's in a row so that its weights serve several
  const int pairs = 2 * gk * seqs, share = (pairs + kPrepThreads / 32 - 1) / (kPrepThreads / 32);
  const int last = min(pairs, (warp + 1) * share);
  for (int pair = warp * share, s; pair < last;) {
    const int it = pair / seqs, g = it >> 1, n = 32 * g + 8 * (lane >> 3), f0 = 32 * (it & 1) + 4 * (lane & 7);
    const bool live = n < rk;
    uint4 w0[4], w1[4];
    const __nv_bfloat16* W = static_cast<const __nv_bfloat16*>(a.w_up_k) + static_cast<int64_t>(h) * kHeadDim * rk + n;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w0[e] = w1[e] = make_uint4(0, 0, 0, 0);
      if (live) w0[e] = __ldg(reinterpret_cast<const uint4*>(W + static_cast<int64_t>(i0_of(f0 + e)) * rk));
      if (live) w1[e] = __ldg(reinterpret_cast<const uint4*>(W + static_cast<int64_t>(i1_of(f0 + e)) * rk));
    }
    for (s = pair - it * seqs; s < seqs && pair < last; ++s, ++pair) {
      float q0[4], q1[4], sum_c[4] = {0.f, 0.f, 0.f, 0.f}, sum_s[4] = {0.f, 0.f, 0.f, 0.f};
      uint8_t* z0 = at(s, n, 0);
      const float up = pow2(z_lift(s));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        q0[e] = qs[s][0][f0 + e] * up;
        q1[e] = qs[s][1][f0 + e] * up;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float zc[4], zs[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t x0 = (&w0[e].x)[j >> 1], x1 = (&w1[e].x)[j >> 1];
          const float u = __uint_as_float(j & 1 ? x0 & 0xFFFF0000u : x0 << 16);
          const float v = __uint_as_float(j & 1 ? x1 & 0xFFFF0000u : x1 << 16);
          zc[e] = fmaf(q0[e], u, q1[e] * v);
          zs[e] = fmaf(q1[e], u, -q0[e] * v);
        }
        const __half2 c0 = __floats2half2_rn(zc[0], zc[1]), c1 = __floats2half2_rn(zc[2], zc[3]);
        const __half2 s0 = __floats2half2_rn(zs[0], zs[1]), s1 = __floats2half2_rn(zs[2], zs[3]);
        top = __hmax2(__hmax2(top, __habs2(c0)), __hmax2(__habs2(c1), __hmax2(__habs2(s0), __habs2(s1))));
        // (the sums of what the MMA reads: of the rounded values)
        const float2 cf0 = __half22float2(c0), cf1 = __half22float2(c1), sf0 = __half22float2(s0), sf1 = __half22float2(s1);
        sum_c[0] += cf0.x; sum_c[1] += cf0.y; sum_c[2] += cf1.x; sum_c[3] += cf1.y;
        sum_s[0] += sf0.x; sum_s[1] += sf0.y; sum_s[2] += sf1.x; sum_s[3] += sf1.y;
        if (live) {   // (row n + j, n a multiple of 8: j alone makes the swizzle)
          uint8_t* z = z0 + ((2 * f0) ^ (j << 4)) + 128 * j;
          *reinterpret_cast<uint2*>(z) = make_uint2(h2_bits(c0), h2_bits(c1));
          *reinterpret_cast<uint2*>(z + P.z_chunk) = make_uint2(h2_bits(s0), h2_bits(s1));
        }
      }
      // the codes' offset: -8 sum Z over the scale group's columns (groups of 32)
      if (32 * g + 32 > rk) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sum_c[e] += __shfl_xor_sync(0xffffffffu, sum_c[e], 8);
        sum_s[e] += __shfl_xor_sync(0xffffffffu, sum_s[e], 8);
        sum_c[e] = -8.f * (sum_c[e] + __shfl_xor_sync(0xffffffffu, sum_c[e], 16));
        sum_s[e] = -8.f * (sum_s[e] + __shfl_xor_sync(0xffffffffu, sum_s[e], 16));
      }
      if (lane < 8) {
        // (high and low part; row rk + 2 + 2 g and the next)
        auto put = [&](int coord, const float (&sum)[4]) {
          const __half2 h0 = __floats2half2_rn(sum[0], sum[1]), h1 = __floats2half2_rn(sum[2], sum[3]);
          const float2 r0 = __half22float2(h0), r1 = __half22float2(h1);
          top = __hmax2(top, __hmax2(__habs2(h0), __habs2(h1)));
          *reinterpret_cast<uint2*>(at(s, rk + 2 + 2 * g, coord)) = make_uint2(h2_bits(h0), h2_bits(h1));
          *reinterpret_cast<uint2*>(at(s, rk + 3 + 2 * g, coord)) =
              make_uint2(h2_bits(__floats2half2_rn(sum[0] - r0.x, sum[1] - r0.y)),
                         h2_bits(__floats2half2_rn(sum[2] - r1.x, sum[3] - r1.y)));
        };
        put(f0, sum_c);
        put(64 + f0, sum_s);
      }
    }
  }
  if (__hisinf(__low2half(top)) || __hisinf(__high2half(top))) record_status(a.status, LLA_ERR_RANGE);   // (NaN queries stay NaN)
}

// Merge the records of each (sequence, head) by log-sum-exp, apply W_up,v once (Appendix J
// "Absorbed attention") and normalise.  Block = (head, a.combine_units sequences), a warp
// merging a sequence at a time, then two threads per output, each with half of its row of
// W_up,v in registers: requested before the wait for the decode grid, they serve every sequence.
constexpr int kCombineThreads = 256;
template <int RV32>
__global__ void __launch_bounds__(kCombineThreads) q4_combine_kernel(const __grid_constant__ Q4DecodeArgs a) {
  constexpr int kRegs = 2 * RV32;   // 16-byte loads of half a row, rounded up
  __shared__ float acc[kQ4CombineUnits][RV32 * 32], inv[kQ4CombineUnits];
  const int h = blockIdx.x % a.H, b0 = static_cast<int>(blockIdx.x / a.H) * a.combine_units, tid = threadIdx.x;
  const int rv = a.r_v, nh = a.plan.nh, nu = min(a.combine_units, a.B - b0), warp = tid >> 5, lane = tid & 31;
  const int e = tid >> 1, half = tid & 1;   // output, and which 8-column pieces of its row: half, half + 2, ..
  uint4 w[kRegs];
  const uint4* W = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.w_up_v) +
                                                  (static_cast<int64_t>(h) * kHeadDim + e) * rv);
#pragma unroll
  for (int i = 0; i < kRegs; ++i) w[i] = 8 * (2 * i + half) < rv ? __ldg(W + 2 * i + half) : make_uint4(0, 0, 0, 0);
  const float mu = __ldg(a.mu_v + h * a.mu_hstride + e);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int i = warp; i < nu; i += kCombineThreads / 32) {
    const int b = b0 + i, u = b * a.plan.ngroups + h / nh;
    float v[RV32], l = 1.f, m = -INFINITY;
#pragma unroll
    for (int k = 0; k < RV32; ++k) v[k] = 0.f;
    if (tile_len(a, b) > 0) {
      const int2 c = *reinterpret_cast<const int2*>(a.ranges + 2 * u);
      const int64_t stride = static_cast<int64_t>(nh) * a.rec_stride;
      const float* rec = a.records + (static_cast<int64_t>(u) + c.x) * stride + (h % nh) * a.rec_stride;
      const int n = c.y - c.x + 1, per = 8 / nh;
      // references and sums: 8 epilogue warps per record, four records a step
      for (int j = lane >> 3; j < n; j += 4) m = fmaxf(m, rec[j * stride + kRecMl + 2 * (lane & 7)]);
      m = warp_max(m);
      l = 0.f;
      for (int j = lane >> 3; j < n; j += 4) {
        const float2 x = *reinterpret_cast<const float2*>(rec + j * stride + kRecMl + 2 * (lane & 7));
        l = fmaf(x.y, m == -INFINITY ? 1.f : exp2f(x.x - m), l);   // (no maximum: every score was NaN)
      }
      l = warp_sum(l);
      for (int j = 0; j < n; ++j)
        for (int p = 0; p < per; ++p) {
          const float* r = rec + j * stride;
          const float2 ref = *reinterpret_cast<const float2*>(r + kRecRef + 2 * p);
          // (2^E alone may leave fp32's range: half of it each)
          const float e2 = floorf(0.5f * ref.y), f = exp2f((ref.x - m) + e2), f2 = exp2f(ref.y - e2);
#pragma unroll
          for (int k = 0; k < RV32; ++k)
            if (32 * k + lane < rv) v[k] = fmaf(r[kRecAcc + p * rv + 32 * k + lane] * f, f2, v[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < RV32; ++k) acc[i][32 * k + lane] = v[k];
    if (lane == 0) {
      inv[i] = 1.f / l;
      if (a.lse) a.lse[static_cast<int64_t>(b) * a.H + h] = m == -INFINITY && l == 1.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
  }
  __syncthreads();
  for (int i = 0; i < nu; ++i) {
    float o = 0.f;
#pragma unroll
    for (int k = 0; k < kRegs; ++k) {
      const int c = 8 * (2 * k + half);
      if (c >= rv) break;
      float w8[8];
      unpack_bf16x8(w[k], w8);
#pragma unroll
      for (int j = 0; j < 8; ++j) o = fmaf(acc[i][c + j], w8[j], o);
    }
    o += __shfl_xor_sync(0xffffffffu, o, 1);
    const int b = b0 + i;
    if (half == 0)
      static_cast<__nv_bfloat16*>(a.out)[(static_cast<int64_t>(b) * a.H + h) * kHeadDim + e] =
          __float2bfloat16_rn(tile_len(a, b) > 0 ? fmaf(o, inv[i], mu) : 0.f);
  }
}

template <int RV32>
cudaError_t launch_tile(const Q4DecodeArgs& a, cudaStream_t s) {
  cudaError_t e = allow_smem(q4_tile_kernel<RV32>, kSmemLimit);
  if (e != cudaSuccess) return e;
  q4_prepare_kernel<<<a.z_blocks + a.rows_grid, kPrepThreads, 0, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // programmatic dependents: each grid's set-up overlaps the one before
  if ((e = launch_pdl(q4_tile_kernel<RV32>, dim3(a.grid), dim3(kQ4TileThreads), a.plan.bytes, s, a)) != cudaSuccess) return e;
  const int blocks = a.H * ((a.B + a.combine_units - 1) / a.combine_units);
  return launch_pdl(q4_combine_kernel<RV32>, dim3(blocks), dim3(kCombineThreads), 0, s, a);
}

}  // namespace

bool make_q4_plan(int H, int r_k, int r_v, Q4Plan* p) {
  const int rb = q4_row_bytes(r_k, r_v), rv32 = (r_v + 31) / 32;
  auto al = [](int x, int a) { return (x + a - 1) / a * a; };
  // Heads of a group: they share a position's rotary tile and MMA chain, which takes as long for
  // one head as for all.  Only as many as divide the heads and fit a chain; a head-tile stays in the ring while scores and V take
  // their turns, so groups of several heads need room for copies ahead.  What the head-tiles leave
  // goes to rotary chunks: with few heads a position is over before the next tile has come.
  for (int nh = kMaxNh; nh >= 1; nh /= 2) {
    const int N = r_k + al(2 + 2 * (r_k / kQ4Group), 16);
    if (H % nh || (nh > 1 && nh * N > 256)) continue;
    *p = Q4Plan{};
    p->nh = nh;
    p->ngroups = H / nh;
    p->N = N;
    p->PG = std::min(kMaxG, 512 / p->N / nh);
    if (nh == 1 && p->PG > 1) p->PG -= p->PG % 2;
    p->PB = nh == 1 ? std::max(2, p->PG) : p->PG;
    p->gstep = p->PG > 1 ? nh * p->N : 0;
    p->z_chunk = nh * p->N * 128;
    p->w_bytes = rv32 * kWStride * 2;
    p->stage = kTile * rb + p->w_bytes + 16;
    const int state = al(8 * nh * kState * 4, 16), misc = al(static_cast<int>(sizeof(Q4Misc)), 16);
    p->z = 0;
    p->rows = al(2 * p->z_chunk, 1024);
    const int room = kSmemLimit - 1024 - p->rows - state - misc;
    p->NS = std::min((room - kMinNR * kRowChunk) / p->stage, kQ4MaxNS);
    p->NS -= p->NS % std::max(2, nh);
    p->NR = std::min((room - p->NS * p->stage) / kRowChunk, std::min(kMaxNR, 2 * p->PB + 1));
    p->state = p->rows + p->NR * kRowChunk;
    p->misc = p->state + state;
    p->ring = p->misc + misc;
    p->bytes = p->ring + p->NS * p->stage + 1024;
    if (p->NS >= (nh == 1 ? 2 : std::max(4, nh))) return true;
  }
  return false;
}

cudaError_t launch_q4_tile(const Q4DecodeArgs& a, cudaStream_t s) {
  switch ((a.r_v + 31) / 32) {
    case 1: return launch_tile<1>(a, s);
    case 2: return launch_tile<2>(a, s);
    case 3: return launch_tile<3>(a, s);
    case 4: return launch_tile<4>(a, s);
    case 5: return launch_tile<5>(a, s);
    case 6: return launch_tile<6>(a, s);
    case 7: return launch_tile<7>(a, s);
    default: return launch_tile<8>(a, s);
  }
}

}  // namespace lla
