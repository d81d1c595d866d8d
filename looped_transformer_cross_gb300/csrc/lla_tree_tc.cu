// lla_tree_tc.cu — lla_tree_attn over bf16 latents on the tensor cores: the cached tokens'
// part of every node's softmax, one record (m, l, latent sum) per (unit, CTA, node).
//
// A unit is one (sequence, head); the flat list of its 128-token tiles over all units is cut into
// equal contiguous ranges, one persistent CTA per SM.  Per tile, three matrix products:
//   U = C_k W^T + mu          128 tokens x 128 dimensions, tcgen05, latents by TMA
//   S = Q^ K^^T               queries x 128 tokens; Q^ (rotated, scaled to log2 units) comes from
//                             tree_prepare_kernel, K^ is U rotated by the epilogue below
//   D += P C_v                queries x r_v, P from TMEM, V latents as the MN-major operand
// so a key is reconstructed and rotated once for all nodes of its sequence, and V never is.
// The rows of S are nodes: a softmax row is one thread's own, with no exchange between lanes.
// S always has 128 rows; with at most 64 (32) nodes they are two (four) copies of the queries,
// and each copy's warps take every second (fourth) stretch of tokens, leaving zeros in P elsewhere, so
// that all four softmax warps have work and the copies' sums are merged like any other records.
//
// Roles: warp 0 copies K and V tiles, warp 1 issues U and S, warp 2 issues D, warp 3 copies each
// unit's W and Q^; warps 4..11 rotate (two per TMEM lane quadrant, 32 frequencies each, one token
// per lane), warps 12..15 do the softmax.  cos/sin of a token's angle are the angle sum of the tile's
// base row (shared memory) and the lane's own row (registers).
#include <algorithm>
#include <cmath>

#include "lla_tree.h"

namespace lla {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kInvSqrtD = 0.08838834764831845f;   // 1/sqrt(128)
constexpr float kRescaleLog2 = 8.f;                 // the reference moves when the maximum passes it by 2^8
constexpr int kPrepThreads = 256;
constexpr int kRotWarps = 8;
constexpr int kSoftWarp0 = 4 + kRotWarps;
constexpr int kTreeThreads = 32 * (kSoftWarp0 + 4);
constexpr int kUCol = 0, kSCol = 128;               // TMEM columns

struct alignas(16) TreeMisc {
  uint64_t kfull[kMaxStages], kempty[kMaxStages], vfull[kMaxStages], vempty[kMaxStages];
  uint64_t bfull[kMaxStages + 1];                   // a tile's base row of the RoPE table
  uint64_t wfull, wfree, qfull, qfree;              // the unit's W and bias; its queries
  uint64_t ufull, ufree;                            // U computed; read by the rotating warps
  uint64_t rfull;                                   // rotated keys in shared memory
  uint64_t sfull;                                   // S computed (and the rotated keys read)
  uint64_t pfull, vdone;                            // P written (and S read); D += P C_v done
  uint64_t done[2];
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(TreeMisc) <= 512, "misc region");

struct Walk {
  int b, h, t, nb, L;
};

// Tiles of sequence b: none without nodes.
__device__ __forceinline__ void walk_load(Walk& w, const TreeArgs& a) {
  int first;
  const int n = tree_nodes(a, w.b, first, false);
  w.L = tree_cached(a, w.b, false);
  w.nb = n > 0 ? (w.L + kTile - 1) / kTile : 0;
}

__device__ __forceinline__ void walk_next(Walk& w, const TreeArgs& a) {
  if (++w.t < w.nb) return;
  w.t = 0;
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
// The two lanes rounded to bf16, the lower one in the low half.
__device__ __forceinline__ uint32_t pack2(uint64_t x) {
  float lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
  return pack_bf16(lo, hi);
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

__device__ __forceinline__ int page_at(const TreeArgs& a, int b, int lp) {
  const int pg = __ldg(a.block_table + static_cast<int64_t>(b) * a.max_pages + lp);
  return min(max(pg, 0), static_cast<int>(a.num_pages) - 1);
}

// One latent tile (chunk plan cp, map of chunk c from map_of) into dst, completing on fb: a box per
// chunk, or with pages of 8..64 tokens a box per chunk and page that holds tokens (lane i issues page
// i; the whole warp calls it).
template <int kPage, typename MapOf>
__device__ __forceinline__ void load_tile(const TreeArgs& a, const Walk& w, uint32_t dst, uint32_t fb, const ChunkPlan& cp, MapOf map_of) {
  const int lane = threadIdx.x & 31;
  if constexpr (kPage != 2) {
    if (lane == 0) {
      mbar_arrive_expect_tx(fb, cp.bytes);
      int y = w.t * kTile, z = w.b * a.H + w.h;
      if constexpr (kPage == 1) {
        const int lp = y / a.page_size;
        z = page_at(a, w.b, lp) * a.H + w.h;
        y -= lp * a.page_size;
      }
      for (int c = 0; c < cp.n; ++c) tma_load_3d(dst + cp.off[c], map_of(c), fb, cp.start[c], y, z);
    }
  } else {
    const int pg = a.page_size;
    const int np = (min(kTile, w.L - w.t * kTile) + pg - 1) / pg;
    if (lane == 0) mbar_arrive_expect_tx(fb, static_cast<uint32_t>(cp.bytes / kTile * pg * np));
    __syncwarp();
    const int lp0 = w.t * (kTile / pg);
    if (lane < np) {
      const int z = page_at(a, w.b, lp0 + lane) * a.H + w.h;
      for (int c = 0; c < cp.n; ++c) tma_load_3d(dst + cp.off[c] + lane * pg * cp.width[c] * 2, map_of(c), fb, cp.start[c], 0, z);
    }
  }
}

// ---------------------------------------------------------------- preparation

// Blocks 0 .. units-1: the unit's query operand, RoPE(q, pos) log2(e)/sqrt(d) in bf16, as the
// shared-memory image (two chunks of 64 columns, 128-byte rows, swizzled); dimensions in the order
// first members of the pairs, then second members, as U's.  Blocks units .. units+H-1: mu of a head
// as an operand that ones multiply, in three bf16 parts (24 bits).  The last block: tiles per
// sequence, and every CTA's first tile.
__global__ void __launch_bounds__(kPrepThreads) tree_prepare_kernel(const __grid_constant__ TreeArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  const int units = a.B * a.H;
  if (blockIdx.x < units) {
    const int b = blockIdx.x / a.H, h = blockIdx.x - b * a.H;
    int first;
    const int n = tree_nodes(a, b, first, false);
    const int L = tree_cached(a, b, false);
    if (n == 0 || L == 0) return;
    if (a.block_table && h == 0) {
      const int used = (L + a.page_size - 1) / a.page_size;
      for (int lp = tid; lp < used; lp += kPrepThreads) {
        const int pg = __ldg(a.block_table + static_cast<int64_t>(b) * a.max_pages + lp);
        if (pg < 0 || pg >= a.num_pages) record_status(a.status, LLA_ERR_DEVICE_ARG);
      }
    }
    uint8_t* img = a.qimg + static_cast<int64_t>(blockIdx.x) * a.rows * 256;
    for (int i = tid; i < a.rows * 8; i += kPrepThreads) {
      const int r = i >> 3, f0 = (i & 7) * 8;
      uint32_t y0[4] = {0, 0, 0, 0}, y1[4] = {0, 0, 0, 0};
      if (r < n) {
        const __nv_bfloat16* qv = static_cast<const __nv_bfloat16*>(a.q) + (first + r) * a.q_stride + h * kHeadDim;
        float x0[8], x1[8];
        if (a.rope_style == 0) {
          unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(qv + f0)), x0);
          unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(qv + 64 + f0)), x1);
        } else {
          float lo[8], hi[8];
          unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(qv + 2 * f0)), lo);
          unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(qv + 2 * f0 + 8)), hi);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x0[k] = lo[2 * k]; x1[k] = lo[2 * k + 1];
            x0[4 + k] = hi[2 * k]; x1[4 + k] = hi[2 * k + 1];
          }
        }
        int p = __ldg(a.pos + first + r);
        p = p < 0 ? 0 : (p >= a.rope_len ? static_cast<int>(a.rope_len - 1) : p);
        const float* c = a.rope_cos + static_cast<int64_t>(p) * 64 + f0;
        const float* s = a.rope_sin + static_cast<int64_t>(p) * 64 + f0;
        const float sc = kLog2e * kInvSqrtD;
        float z0[8], z1[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float cc = __ldg(c + k), ss = __ldg(s + k);
          z0[k] = (x0[k] * cc - x1[k] * ss) * sc;
          z1[k] = (x0[k] * ss + x1[k] * cc) * sc;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          y0[k] = pack_bf16(z0[2 * k], z0[2 * k + 1]);
          y1[k] = pack_bf16(z1[2 * k], z1[2 * k + 1]);
        }
      }
      const uint32_t o = swizzle_offset(r * 128 + f0 * 2, 128);
      *reinterpret_cast<uint4*>(img + o) = make_uint4(y0[0], y0[1], y0[2], y0[3]);
      *reinterpret_cast<uint4*>(img + a.rows * 128 + o) = make_uint4(y1[0], y1[1], y1[2], y1[3]);
    }
    return;
  }
  if (blockIdx.x < units + a.H) {
    const int h = blockIdx.x - units;
    if (tid < kHeadDim) {
      const int src = tid < 64 ? (a.rope_style == 0 ? tid : 2 * tid) : (a.rope_style == 0 ? tid : 2 * (tid - 64) + 1);
      const float mu = __ldg(a.mu_k + h * a.mu_hstride + src);
      const float hi = __bfloat162float(__float2bfloat16_rn(mu));
      const float mid = __bfloat162float(__float2bfloat16_rn(mu - hi));
      uint8_t* ab = a.bias + h * 4096;
      *reinterpret_cast<uint4*>(ab + swizzle_offset(tid * 32, 32)) = make_uint4(pack_bf16(hi, mid), pack_bf16(mu - hi - mid, 0.f), 0, 0);
      *reinterpret_cast<uint4*>(ab + swizzle_offset(tid * 32 + 16, 32)) = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  // ---- the plan: prefix of the sequences' tiles, then each CTA's first (sequence, head, tile)
  constexpr int kHeld = 2048;
  __shared__ int tot[kPrepThreads];
  __shared__ int starts[kHeld];
  const int per = (a.B + kPrepThreads - 1) / kPrepThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  auto tiles = [&](int b) {
    Walk w;
    w.b = b;
    walk_load(w, a);
    return w.nb;
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
      const int nb = tiles(lo);
      s = make_int4(lo, static_cast<int>(rem / nb), static_cast<int>(rem % nb), static_cast<int>(min(share, total - f0)));
    }
    a.cta_start[c] = s;
  }
}

// ---------------------------------------------------------------- the cached tokens

// kPage: 0 dense, 1 pages of a multiple of 128 tokens, 2 pages of 8..64 tokens.  kCopies: copies of
// the queries in S's rows (4: at most 32 nodes, 2: 64, 1: 128).
template <int kPage, int kCopies>
__global__ void __launch_bounds__(kTreeThreads, 1)
tree_tile_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ TreeMaps maps) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const TreePlan& P = a.plan;
  const uint32_t sbase = smem_u32(sm);
  TreeMisc* misc = reinterpret_cast<TreeMisc*>(sm + P.misc);
  volatile int* abort = &misc->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto bar = [&](const uint64_t& m) { return smem_u32(&m); };

  if (tid == 0) {
    misc->abort = 0;
    for (int s = 0; s <= kMaxStages; ++s) mbar_init(bar(misc->bfull[s]), 1);
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(bar(misc->kfull[s]), 1); mbar_init(bar(misc->kempty[s]), 1);
      mbar_init(bar(misc->vfull[s]), 1); mbar_init(bar(misc->vempty[s]), 1);
    }
    mbar_init(bar(misc->wfull), 1); mbar_init(bar(misc->wfree), 1);
    mbar_init(bar(misc->qfull), 1); mbar_init(bar(misc->qfree), 1);
    mbar_init(bar(misc->ufull), 1); mbar_init(bar(misc->ufree), kRotWarps);
    mbar_init(bar(misc->rfull), kRotWarps);
    mbar_init(bar(misc->sfull), 1);
    mbar_init(bar(misc->pfull), 4); mbar_init(bar(misc->vdone), 1);
    mbar_init(bar(misc->done[0]), 1); mbar_init(bar(misc->done[1]), 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc(smem_u32(&misc->tmem_base), 512);
  }
  if (warp >= kSoftWarp0) {
    // ones that meet the three parts of mu
    const int r = tid - 32 * kSoftWarp0;
    *reinterpret_cast<uint4*>(sm + P.ones + swizzle_offset(r * 32, 32)) = make_uint4(0x3F803F80u, 0x00003F80u, 0, 0);
    *reinterpret_cast<uint4*>(sm + P.ones + swizzle_offset(r * 32 + 16, 32)) = make_uint4(0, 0, 0, 0);
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
  w.t = first_tile.z;
  if (count > 0) walk_load(w, a);
  auto agree = [](bool r) { return __all_sync(0xffffffffu, r); };

  if (warp == 0) {
    // ======================================================== K and V tiles
    // (V tile i - 1 after K tile i: it is needed only once tile i - 1 has weights.)  Tile i's base row
    // goes to slot i mod SK + 1: K tile i + SK + 1 is requested once U(i + 1) is computed, for which
    // every rotating warp has read the base row of tile i.
    Walk wv = w;
    Ring kr, vr, br;
    int issued_k = 0, issued_v = 0;
    for (int i = 0; i <= count && count > 0; ++i) {
      if (i < count) {
        if (!warp_wait(bar(misc->kempty[kr.slot]), kr.phase ^ 1u, abort, a.status)) break;
        const uint32_t kb = bar(misc->kfull[kr.slot]);
        load_tile<kPage>(a, w, sbase + P.k_ring + kr.slot * P.k_stage, kb, P.kplan,
                         [&](int c) { return &maps.k[chunk_map_index(P.kplan.width[c])]; });
        if (lane == 0) {
          const uint32_t bb = bar(misc->bfull[br.slot]), dst = sbase + P.base + br.slot * 512;
          mbar_arrive_expect_tx(bb, 512);
          bulk_load(dst, a.rope_cos + static_cast<int64_t>(w.t) * kTile * 64, 256, bb);
          bulk_load(dst + 256, a.rope_sin + static_cast<int64_t>(w.t) * kTile * 64, 256, bb);
        }
        issued_k = i + 1;
        kr.next(P.SK);
        br.next(P.SK + 1);
        walk_next(w, a);
      }
      if (i > 0) {
        if (!warp_wait(bar(misc->vempty[vr.slot]), vr.phase ^ 1u, abort, a.status)) break;
        load_tile<kPage>(a, wv, sbase + P.v_ring + vr.slot * P.v_stage, bar(misc->vfull[vr.slot]), P.vplan,
                         [&](int) { return &maps.v; });
        issued_v = i;
        vr.next(P.SV);
        walk_next(wv, a);
      }
    }
    // every copy lands before the CTA can exit
    auto drain = [&](uint64_t* full, int n, int issued) {
      for (int i = max(0, issued - n); i < issued; ++i) {
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(bar(full[i % n]), (i / n) & 1) && global_timer_ns() - t0 < kWaitLimitNs) {}
      }
    };
    if (lane == 0) {
      drain(misc->kfull, P.SK, issued_k);
      drain(misc->vfull, P.SV, issued_v);
      drain(misc->bfull, P.SK + 1, issued_k);
    }
  } else if (warp == 3) {
    // ======================================================== a unit's weights and queries
    if (lane == 0) {
      int unit = 0, issued_w = 0, issued_q = 0;
      for (int i = 0; i < count; ++unit) {
        const int left = min(w.nb - w.t, count - i);
        if (unit > 0 && !mbar_wait(bar(misc->wfree), (unit - 1) & 1, abort, a.status)) break;
        const uint32_t wf = bar(misc->wfull);
        mbar_arrive_expect_tx(wf, P.kplan.bytes + 4096);
        for (int c = 0; c < P.kplan.n; ++c)
          tma_load_4d(sbase + P.w + P.kplan.off[c], &maps.w[chunk_map_index(P.kplan.width[c])], wf, P.kplan.start[c], 0, 0, w.h);
        bulk_load(sbase + P.mu, a.bias + static_cast<int64_t>(w.h) * 4096, 4096, wf);
        issued_w = unit + 1;
        if (unit > 0 && !mbar_wait(bar(misc->qfree), (unit - 1) & 1, abort, a.status)) break;
        const uint32_t qf = bar(misc->qfull);
        mbar_arrive_expect_tx(qf, 32768);
        const uint8_t* img = a.qimg + static_cast<int64_t>(w.b * a.H + w.h) * (32768 / kCopies);
        constexpr uint32_t part = 16384 / kCopies;       // a copy's rows of one chunk
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int c = 0; c < kCopies; ++c) bulk_load(sbase + P.q + k * 16384 + c * part, img + k * part, part, qf);
        issued_q = unit + 1;
        i += left;
        w.t += left - 1;
        walk_next(w, a);
      }
      auto drain = [&](const uint64_t& full, int issued) {
        const uint64_t t0 = global_timer_ns();
        while (issued > 0 && !mbar_try_wait(bar(full), (issued - 1) & 1) && global_timer_ns() - t0 < kWaitLimitNs) {}
      };
      drain(misc->wfull, issued_w);
      drain(misc->qfull, issued_q);
    }
  } else if (warp == 1) {
    // ======================================================== U(i + 1), then S(i)
    const uint32_t idesc = umma_idesc_bf16(128, 128, false, false);
    const uint64_t d_ones = umma_desc(sbase + P.ones, 16, 256, kSw32), d_mu = umma_desc(sbase + P.mu, 16, 256, kSw32);
    const uint64_t d_q = umma_desc(sbase + P.q, 16, 1024, kSw128), d_r = umma_desc(sbase + P.rot, 16, 1024, kSw128);
    Walk ws = w;
    Ring kr;
    int unit_u = -1, unit_s = -1;
    bool ok = true;
    for (int i = 0; i <= count && count > 0 && ok; ++i) {
      if (i < count) {
        if (i == 0 || w.t == 0) {
          ++unit_u;
          if (!(ok = agree(mbar_wait(bar(misc->wfull), unit_u & 1, abort, a.status)))) break;
        }
        if (!(ok = agree(mbar_wait(bar(misc->kfull[kr.slot]), kr.phase, abort, a.status)))) break;
        if (i > 0 && !(ok = agree(mbar_wait(bar(misc->ufree), (i - 1) & 1, abort, a.status)))) break;
        tc_fence_after();
        const uint32_t ka = sbase + P.k_ring + kr.slot * P.k_stage;
        uint32_t acc = 0;
        for (int c = 0; c < P.kplan.n; ++c) {
          const int rb = P.kplan.width[c] * 2;
          const uint32_t lay = sw_mode_for_row_bytes(rb);
          const uint64_t a0 = umma_desc(ka + P.kplan.off[c], 16, 8 * rb, lay);
          const uint64_t b0 = umma_desc(sbase + P.w + P.kplan.off[c], 16, 8 * rb, lay);
          for (int k = 0; k < P.kplan.width[c] / 16; ++k) {
            umma_bf16_warp(tmem + kUCol, a0 + 2 * k, b0 + 2 * k, idesc, acc);
            acc = 1;
          }
        }
        umma_bf16_warp(tmem + kUCol, d_ones, d_mu, idesc, 1);
        umma_commit_warp(bar(misc->kempty[kr.slot]));
        umma_commit_warp(bar(misc->ufull));
        if (w.t == w.nb - 1) umma_commit_warp(bar(misc->wfree));
        kr.next(P.SK);
        walk_next(w, a);
      }
      if (i > 0) {
        const int j = i - 1;
        if (j == 0 || ws.t == 0) {
          ++unit_s;
          if (!(ok = agree(mbar_wait(bar(misc->qfull), unit_s & 1, abort, a.status)))) break;
        }
        if (!(ok = agree(mbar_wait(bar(misc->rfull), j & 1, abort, a.status)))) break;
        // S(j - 1) read; where P lies in S's columns, also P(j - 1)
        if (j > 0 && !(ok = agree(mbar_wait(P.p_col == kSCol ? bar(misc->vdone) : bar(misc->pfull), (j - 1) & 1, abort, a.status)))) break;
        tc_fence_after();
#pragma unroll 1
        for (int k = 0; k < 8; ++k)
          umma_bf16_warp(tmem + kSCol, d_q + (k >> 2) * 1024 + (k & 3) * 2, d_r + (k >> 2) * 1024 + (k & 3) * 2, idesc, k > 0);
        umma_commit_warp(bar(misc->sfull));
        if (ws.t == ws.nb - 1) umma_commit_warp(bar(misc->qfree));
        walk_next(ws, a);
      }
    }
    // this warp's products complete before TMEM is released
    umma_commit_warp(bar(misc->done[0]));
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar(misc->done[0]), 0) && global_timer_ns() - t0 < kWaitLimitNs) {}
  } else if (warp == 2) {
    // ======================================================== D += P C_v
    const uint32_t idesc = umma_idesc_bf16(128, a.r_v, false, true);
    const uint64_t d_v = umma_desc(sbase + P.v_ring, kTile * 64, 512, kSw64);
    const uint32_t vst = static_cast<uint32_t>(P.v_stage) >> 4;
    Ring vr;
    for (int j = 0; j < count; ++j, vr.next(P.SV)) {
      if (!agree(mbar_wait(bar(misc->vfull[vr.slot]), vr.phase, abort, a.status))) break;
      if (!agree(mbar_wait(bar(misc->pfull), j & 1, abort, a.status))) break;
      // rows past the sequence's end: whole steps of 16 tokens are left out, the rest of a partial step
      // is zeroed (it may hold anything; its weights are 0 and 0 * x stays 0)
      const int valid = min(kTile, w.L - w.t * kTile);
      const int steps = (valid + 15) / 16;
      if (valid < steps * 16) {
        uint8_t* vs = sm + P.v_ring + vr.slot * P.v_stage;
        const int per = (steps * 16 - valid) * 4;
        for (int x = lane; x < P.vplan.n * per; x += 32) {
          const int c = x / per, r = valid + (x - c * per) / 4, g = x & 3;
          *reinterpret_cast<uint4*>(vs + P.vplan.off[c] + swizzle_offset(r * 64 + g * 16, 64)) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      tc_fence_after();
      const uint64_t b0 = d_v + vr.slot * vst;
      const uint32_t fresh = j == 0 || w.t == 0;      // a unit's first product starts the sum
      for (int k = 0; k < steps; ++k)
        umma_bf16_ts_warp(tmem + P.d_col, tmem + P.p_col + 8 * k, b0 + 64 * k, idesc, k > 0 || !fresh);
      umma_commit_warp(bar(misc->vempty[vr.slot]));
      umma_commit_warp(bar(misc->vdone));
      walk_next(w, a);
    }
    umma_commit_warp(bar(misc->done[1]));
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar(misc->done[1]), 0) && global_timer_ns() - t0 < kWaitLimitNs) {}
  } else if (warp < kSoftWarp0) {
    // ======================================================== rotation: U -> K^ in shared memory
    const int quad = warp & 3, row = 32 * quad + lane, f0 = 32 * ((warp - 4) >> 2);
    const uint32_t t_u = tmem + (static_cast<uint32_t>(32 * quad) << 16) + kUCol + f0;
    uint64_t cl[16], sl[16];                          // the lane's own row of the table, by twos
#pragma unroll
    for (int f = 0; f < 16; f += 2) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(a.rope_cos + row * 64 + f0 + 2 * f));
      const float4 s = __ldg(reinterpret_cast<const float4*>(a.rope_sin + row * 64 + f0 + 2 * f));
      cl[f] = pair2(c.x, c.y); cl[f + 1] = pair2(c.z, c.w);
      sl[f] = pair2(s.x, s.y); sl[f + 1] = pair2(s.z, s.w);
    }
    const uint64_t minus = pair2(-1.f, -1.f);
    uint8_t* rot = sm + P.rot;
    Ring br;
    for (int i = 0; i < count; ++i, br.next(P.SK + 1)) {
      // the tile's base row: cos, then sin
      const float* base = reinterpret_cast<const float*>(sm + P.base + br.slot * 512) + f0;
      if (!warp_wait(bar(misc->bfull[br.slot]), br.phase, abort, a.status)) break;
      if (!warp_wait(bar(misc->ufull), i & 1, abort, a.status)) break;
      // K^(i - 1) has been read
      if (i > 0 && !warp_wait(bar(misc->sfull), (i - 1) & 1, abort, a.status)) break;
      tc_fence_after();
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        float u0[16], u1[16];
        tmem_ld_x16(t_u + 16 * g, u0);
        tmem_ld_x16(t_u + 64 + 16 * g, u1);
        tmem_wait_ld();
        uint32_t y0[8], y1[8];
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          const float4 c4 = *reinterpret_cast<const float4*>(base + 16 * g + 2 * k);
          const float4 s4 = *reinterpret_cast<const float4*>(base + 64 + 16 * g + 2 * k);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint64_t cb = e == 0 ? pair2(c4.x, c4.y) : pair2(c4.z, c4.w), sb = e == 0 ? pair2(s4.x, s4.y) : pair2(s4.z, s4.w);
            const int f = 8 * g + k + e;
            const uint64_t c = fma2(mul2(sb, sl[f]), minus, mul2(cb, cl[f])), sn = fma2(sb, cl[f], mul2(cb, sl[f]));
            const uint64_t x0 = pair2(u0[2 * (k + e)], u0[2 * (k + e) + 1]), x1 = pair2(u1[2 * (k + e)], u1[2 * (k + e) + 1]);
            y0[k + e] = pack2(fma2(mul2(x1, sn), minus, mul2(x0, c)));
            y1[k + e] = pack2(fma2(x0, sn, mul2(x1, c)));
          }
        }
        if (g == 1) {                                 // U and the base row have been read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(misc->ufree));
        }
        const uint32_t o = row * 128 + (f0 + 16 * g) * 2;
        *reinterpret_cast<uint4*>(rot + swizzle_offset(o, 128)) = make_uint4(y0[0], y0[1], y0[2], y0[3]);
        *reinterpret_cast<uint4*>(rot + swizzle_offset(o + 16, 128)) = make_uint4(y0[4], y0[5], y0[6], y0[7]);
        *reinterpret_cast<uint4*>(rot + 16384 + swizzle_offset(o, 128)) = make_uint4(y1[0], y1[1], y1[2], y1[3]);
        *reinterpret_cast<uint4*>(rot + 16384 + swizzle_offset(o + 16, 128)) = make_uint4(y1[4], y1[5], y1[6], y1[7]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(misc->rfull));
    }
  } else {
    // ======================================================== softmax: S -> P, records
    constexpr int kRows = kTile / kCopies, kCols = kTile / kCopies;   // a copy's rows; its tokens of a tile
    const int quad = warp & 3, row = 32 * quad + lane;
    const int copy = row / kRows, node = row - copy * kRows;
    const int tok0 = copy * kCols;                    // (uniform in a warp)
    const uint32_t lane_base = static_cast<uint32_t>(32 * quad) << 16;
    const uint32_t t_s = tmem + lane_base + kSCol + tok0, t_p = tmem + lane_base + P.p_col, t_d = tmem + lane_base + P.d_col;
    const bool overlay = P.p_col == kSCol;
    const uint32_t zeros[8] = {};
    if (kCopies > 1 && !overlay) {                    // the other copies' tokens stay zero
      for (int c = 0; c < 64; c += 8) tmem_st_x8(t_p + c, zeros);
      tmem_wait_st();
    }
    float m_ref = -INFINITY, l = 0.f;
    bool ok = true;
    int cur_b = w.b, cur_h = w.h;
    // the finished unit's rows (its last product was tile `last`)
    auto finish = [&](int last) -> bool {
      if (!warp_wait(bar(misc->vdone), last & 1, abort, a.status)) return false;
      tc_fence_after();
      int first;
      const int n = tree_nodes(a, cur_b, first, false);
      const int64_t slot = static_cast<int64_t>(cur_b) * a.H + cur_h + blockIdx.x;
      float* rec = a.records + ((slot * kCopies + copy) * a.max_nodes + node) * (a.r_v + kRecordHead);
      if (node < n) *reinterpret_cast<float4*>(rec) = make_float4(m_ref, l, 0.f, 0.f);
      for (int c = 0; c < a.r_v; c += 16) {
        float v[16];
        tmem_ld_x16(t_d + c, v);
        tmem_wait_ld();
        if (node < n) {
#pragma unroll
          for (int k = 0; k < 16; k += 4) *reinterpret_cast<float4*>(rec + kRecordHead + c + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
        }
      }
      tc_fence_before();
      return true;
    };
    for (int i = 0; i < count; ++i) {
      if (i > 0 && w.t == 0) {
        if (!(ok = finish(i - 1))) break;
        cur_b = w.b; cur_h = w.h;
        m_ref = -INFINITY; l = 0.f;
      }
      if (!(ok = warp_wait(bar(misc->sfull), i & 1, abort, a.status))) break;
      tc_fence_after();
      const int valid = w.L - w.t * kTile - tok0;     // of this copy's tokens
      // (16 columns at a time, in loops: the code of all roles has to stay in the instruction caches)
      float m_tile = -INFINITY;
#pragma unroll 1
      for (int c = 0; c < kCols; c += 16) {
        float s[16];
        tmem_ld_x16(t_s + c, s);
        tmem_wait_ld();
        if (c + 16 > valid) {
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (c + k >= valid) s[k] = -INFINITY;
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) m_tile = fmaxf(m_tile, s[k]);
      }
      const bool move = m_tile > m_ref + kRescaleLog2 || (m_ref == -INFINITY && m_tile > -INFINITY);
      // P and (where it is rescaled) D are at rest once the product of tile i - 1 is done
      if (i > 0 && !(ok = warp_wait(bar(misc->vdone), (i - 1) & 1, abort, a.status))) break;
      tc_fence_after();
      if (__any_sync(0xffffffffu, move && m_ref != -INFINITY)) {
        const float alpha = move ? exp2f(m_ref - m_tile) : 1.f;   // (0 from a reference of -inf)
        for (int c = 0; c < a.r_v; c += 16) {
          float v[16];
          tmem_ld_x16(t_d + c, v);
          tmem_wait_ld();
          uint32_t x[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(v[k] * alpha);
          tmem_st_x16(t_d + c, x);
        }
        l *= alpha;
      }
      if (move) m_ref = m_tile;
      const float ref = m_ref == -INFINITY ? 0.f : m_ref;   // (nothing above -inf yet: weights of 0)
      // weights, in bf16 as the product takes them; l adds up what was rounded.  Where P lies over S, the
      // weights of 16 columns go to 8 that lie before or among them and have been read.
      float l0 = 0.f, l1 = 0.f;
#pragma unroll 1
      for (int c = 0; c < kCols; c += 16) {
        float s[16];
        tmem_ld_x16(t_s + c, s);
        tmem_wait_ld();
        if (c + 16 > valid) {
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (c + k >= valid) s[k] = -INFINITY;
        }
        uint32_t x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          x[k] = pack_bf16(exp2_fast(s[2 * k] - ref), exp2_fast(s[2 * k + 1] - ref));
          l0 += __uint_as_float(x[k] << 16);
          l1 += __uint_as_float(x[k] & 0xFFFF0000u);
        }
        tmem_st_x8(t_p + (tok0 + c) / 2, x);
      }
      l += l0 + l1;
      if (kCopies > 1 && overlay) {                   // S of the other copies' tokens makes way for zeros
#pragma unroll 1
        for (int c = 0; c < 64; c += 8)
          if (c < tok0 / 2 || c >= (tok0 + kCols) / 2) tmem_st_x8(t_p + c, zeros);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(misc->pfull));
      walk_next(w, a);
    }
    if (ok && count > 0) finish(count - 1);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

bool make_tree_plan(int r_k, int r_v, TreePlan* p) {
  *p = TreePlan{};
  p->kplan = make_chunk_plan(r_k, kTile);
  p->vplan = make_chunk_plan_32(r_v, kTile);
  auto al = [](int x) { return (x + 1023) / 1024 * 1024; };
  p->k_stage = al(p->kplan.bytes);
  p->v_stage = al(p->vplan.bytes);
  // W, two 4 KB bias operands, queries, rotated keys, base rows, barriers, alignment
  const int fixed = al(p->kplan.bytes) + 8192 + 32768 + 32768 + 512 + 1024;
  auto fits = [&](int sk, int sv) { return fixed + (sk + 1) * 512 + sk * p->k_stage + sv * p->v_stage <= kSmemLimit; };
  if (!fits(1, 1)) return false;
  p->SK = p->SV = 1;
  while (true) {
    if (p->SK <= p->SV && p->SK < kMaxStages && fits(p->SK + 1, p->SV)) { ++p->SK; continue; }
    if (p->SV < kMaxStages && fits(p->SK, p->SV + 1)) { ++p->SV; continue; }
    if (p->SK < kMaxStages && fits(p->SK + 1, p->SV)) { ++p->SK; continue; }
    break;
  }
  int off = 0;
  p->v_ring = off; off += p->SV * p->v_stage;
  p->k_ring = off; off += p->SK * p->k_stage;
  p->w = off;      off += al(p->kplan.bytes);
  p->q = off;      off += 32768;
  p->rot = off;    off += 32768;
  p->ones = off;   off += 4096;
  p->mu = off;     off += 4096;
  p->base = off;   off += (p->SK + 1) * 512;
  p->misc = off;   off += 512;
  p->bytes = off + 1024;
  // TMEM: U 0..127, S 128..255, then P (64 columns) and D; P shares S's columns where D needs the room
  p->p_col = r_v <= 192 ? 256 : kSCol;
  p->d_col = r_v <= 192 ? 320 : 256;
  return true;
}

template <int kPage>
static cudaError_t launch_tiles(const TreeArgs& a, const TreeMaps& maps, cudaStream_t s) {
  auto kern = a.copies == 4 ? tree_tile_kernel<kPage, 4> : a.copies == 2 ? tree_tile_kernel<kPage, 2> : tree_tile_kernel<kPage, 1>;
  // (the most any shape takes, at every call)
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(a.grid), dim3(kTreeThreads), a.plan.bytes, s, a, maps);
}

cudaError_t launch_tree_tensor(const TreeArgs& a, const TreeMaps& maps, cudaStream_t s) {
  const cudaError_t e = launch_pdl(tree_prepare_kernel, dim3(a.B * a.H + a.H + 1), dim3(kPrepThreads), 0, s, a);
  if (e != cudaSuccess) return e;
  if (!a.block_table) return launch_tiles<0>(a, maps, s);
  return a.page_size % kTile == 0 ? launch_tiles<1>(a, maps, s) : launch_tiles<2>(a, maps, s);
}

}  // namespace lla
