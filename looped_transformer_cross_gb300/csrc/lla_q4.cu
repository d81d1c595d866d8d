// lla_q4.cu — the 4-bit paged latent cache: latents rounded into rows (lla_q4_store), rows
// read back (lla_q4_load), and the plain decode attention over them (fp32 storage).
//
// Latents are centred by construction (Eq. (2) subtracts mu), so codes are symmetric: per
// 32 columns s = bf16(max|c| / 7) and code = round(c / s), half to even, which both
// divide in fp32.  bf16 scales keep the whole exponent range of a bf16 latent; their
// 8-bit mantissa only moves the grid (a scale rounded down puts max|c| / s at no more
// than 7.03, which still rounds to 7).
#include <algorithm>
#include <cmath>

#include "lla_q4.h"

namespace lla {

namespace {

constexpr int kQ4Threads = 256;

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(p)), v);
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint4 w;
  __nv_bfloat162 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  w.x = *reinterpret_cast<uint32_t*>(&h[0]); w.y = *reinterpret_cast<uint32_t*>(&h[1]);
  w.z = *reinterpret_cast<uint32_t*>(&h[2]); w.w = *reinterpret_cast<uint32_t*>(&h[3]);
  *reinterpret_cast<uint4*>(p) = w;
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

struct Q4CopyArgs {
  int H, r_k, r_v, row_bytes, page_size;
  int64_t num_slots;                 // num_pages * page_size
  uint32_t n_items;                  // token-heads * 4 (groups of K + groups of V)
  uint32_t tok0;
  const int64_t* slots;
  void* k;                           // [N][H][r_k] storage dtype
  void* v;
  uint8_t* rows;
  uint32_t* status;
};

// Row of (slot, head); -1 for a slot that holds no token (negative) or lies outside.
__device__ __forceinline__ int64_t q4_row(const Q4CopyArgs& a, int64_t slot, int h, bool report) {
  if (slot < 0) return -1;
  if (slot >= a.num_slots) {
    if (report) record_status(a.status, LLA_ERR_DEVICE_ARG);
    return -1;
  }
  const int64_t page = slot / a.page_size;
  return (page * a.H + h) * a.page_size + (slot - page * a.page_size);
}

// Four neighbouring threads hold one group of 32 columns, eight columns each (the last
// group may have 16: two of the four idle).  Both directions are HBM-bound: the
// store reads 2 (r_k + r_v) bytes (bf16) and writes a row per token-head.
struct Q4Item {
  int sub, col, r, code_at, scale_at;
  bool k_axis, active;
  uint32_t n, h;
};
__device__ __forceinline__ Q4Item q4_item(const Q4CopyArgs& a, uint32_t i) {
  Q4Item it;
  const uint32_t gk = q4_groups(a.r_k), ng = gk + q4_groups(a.r_v);
  const uint32_t g_all = i >> 2, th = g_all / ng, g = g_all - th * ng;
  it.sub = i & 3;
  it.n = th / a.H;
  it.h = th - it.n * a.H;
  it.k_axis = g < gk;
  it.r = it.k_axis ? a.r_k : a.r_v;
  it.col = (it.k_axis ? g : g - gk) * kQ4Group + 8 * it.sub;
  it.active = it.col < it.r;
  it.code_at = (it.k_axis ? 0 : a.r_k / 2) + it.col / 2;
  it.scale_at = q4_scale_offset(a.r_k, a.r_v) + 2 * g;
  return it;
}

template <typename T>
__global__ void __launch_bounds__(kQ4Threads) q4_store_kernel(const __grid_constant__ Q4CopyArgs a) {
  const uint32_t i = blockIdx.x * kQ4Threads + threadIdx.x;
  // whole warps: every lane takes part in the shuffles below
  const bool live = i < a.n_items;
  const Q4Item it = q4_item(a, live ? i : a.n_items - 1);
  const int64_t n = static_cast<int64_t>(a.tok0) + it.n;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const T* src = static_cast<const T*>(it.k_axis ? a.k : a.v) + (n * a.H + it.h) * it.r + it.col;
  if (live && it.active) load8(src, v);
  const int64_t row = live ? q4_row(a, __ldg(a.slots + n), it.h, true) : -1;
  // max |c| over the group, on the bits of |c|: NaN sorts above infinity, so either shows
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  if (row < 0) return;
  uint8_t* dst = a.rows + row * a.row_bytes;
  const bool finite = top < 0x7f800000u;
  // a group with a value that is not finite stores a NaN scale: all of it reads as NaN
  const __nv_bfloat16 s16 =
      finite ? __float2bfloat16_rn(__fdiv_rn(__uint_as_float(top), 7.f)) : __ushort_as_bfloat16(0x7fc0);
  const float s = __bfloat162float(s16);
  const bool some = finite && s > 0.f;
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int code = some ? min(max(__float2int_rn(__fdiv_rn(v[e], s)), -7), 7) : 0;
    w |= static_cast<uint32_t>(code + 8) << (4 * (e >> 1) + 16 * (e & 1));
  }
  if (it.active) *reinterpret_cast<uint32_t*>(dst + it.code_at) = w;
  if (it.sub == 0) *reinterpret_cast<__nv_bfloat16*>(dst + it.scale_at) = s16;
  // the row's padding, by the last group's threads: rows are fully defined
  if (!it.k_axis && it.scale_at + 2 == q4_scale_offset(a.r_k, a.r_v) + 2 * (q4_groups(a.r_k) + q4_groups(a.r_v)))
    for (int p = it.scale_at + 2 + 2 * it.sub; p < a.row_bytes; p += 8) *reinterpret_cast<uint16_t*>(dst + p) = 0;
}

// Eight values of a code word.
__device__ __forceinline__ void q4_unpack8(uint32_t w, float s, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    v[e] = static_cast<float>(static_cast<int>((w >> (4 * (e >> 1) + 16 * (e & 1))) & 15u) - 8) * s;
}

template <typename T>
__global__ void __launch_bounds__(kQ4Threads) q4_load_kernel(const __grid_constant__ Q4CopyArgs a) {
  const uint32_t i = blockIdx.x * kQ4Threads + threadIdx.x;
  if (i >= a.n_items) return;
  const Q4Item it = q4_item(a, i);
  if (!it.active) return;
  const int64_t n = static_cast<int64_t>(a.tok0) + it.n;
  const int64_t row = q4_row(a, __ldg(a.slots + n), it.h, true);
  if (row < 0) return;
  const uint8_t* src = a.rows + row * a.row_bytes;
  const float s = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(src + it.scale_at));
  float v[8];
  q4_unpack8(*reinterpret_cast<const uint32_t*>(src + it.code_at), s, v);
  store8(static_cast<T*>(it.k_axis ? a.k : a.v) + (n * a.H + it.h) * it.r + it.col, v);
}

// ----------------------------------------------------------------- fp32 decode

// Decode attention over 4-bit rows for fp32 storage, in fp32 arithmetic: one block
// per (sequence, head, split of whole 128-token tiles), one token per thread.  The
// score is Eq. (3) with RoPE after reconstruction, regrouped per frequency pair as in
// lla_paged_generic.cu, with the folded query in fp32; one online softmax over the
// split's tiles, the value path absorbed; a record per split, merged by the combine.
constexpr int kPlainThreads = 128;
constexpr float kPlainScale = 0.08838834764831845f * 1.4426950408889634f;   // log2(e) / sqrt(128)

__device__ __forceinline__ int q4_len(const Q4DecodeArgs& a, int b) {
  const int L = __ldg(a.seq_lens + b);
  return L < 0 ? 0 : (L > a.L_max ? static_cast<int>(a.L_max) : L);
}

__global__ void __launch_bounds__(kPlainThreads) q4_f32_kernel(const __grid_constant__ Q4DecodeArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float bc[64], bs[64], qr[kHeadDim], pw[kPlainThreads], red[4];
  const int rk = a.r_k, rv = a.r_v, rb = a.row_bytes;
  float* zc = reinterpret_cast<float*>(smem);                        // [rk][64] cosine part
  float* zs = zc + rk * 64;                                          // [rk][64] sine part
  uint8_t* tile = smem + static_cast<size_t>(rk) * 512;              // [128][rb + 16]
  const int ts = rb + 16;
  const int64_t id = blockIdx.x;
  const int64_t u = id / a.splits;
  const int sp = static_cast<int>(id - u * a.splits);
  const int b = static_cast<int>(u / a.H), h = static_cast<int>(u - static_cast<int64_t>(b) * a.H);
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int L0 = __ldg(a.seq_lens + b);
  if (sp == 0 && (L0 < 0 || L0 > a.L_max) && tid == 0) record_status(a.status, LLA_ERR_DEVICE_ARG);
  const int L = q4_len(a, b);
  const int64_t j_lo = sp * a.chunk, j_hi = min(static_cast<int64_t>(L), j_lo + a.chunk);
  if (j_lo >= j_hi) return;
  int qp = __ldg(a.q_pos + b);
  if (qp < 0 || qp >= a.rope_len) {
    if (tid == 0) record_status(a.status, LLA_ERR_DEVICE_ARG);
    qp = qp < 0 ? 0 : static_cast<int>(a.rope_len - 1);
  }
  auto pair_of = [&](int f, int& i0, int& i1) {
    i0 = a.rope_style == 0 ? f : 2 * f;
    i1 = a.rope_style == 0 ? f + 64 : 2 * f + 1;
  };
  const float* q = static_cast<const float*>(a.q) + u * kHeadDim;
  const float* mk = a.mu_k + h * a.mu_hstride;
  if (tid < 64) {
    int i0, i1;
    pair_of(tid, i0, i1);
    const float c = __ldg(a.rope_cos + static_cast<int64_t>(qp) * 64 + tid);
    const float s = __ldg(a.rope_sin + static_cast<int64_t>(qp) * 64 + tid);
    const float x0 = __ldg(q + i0), x1 = __ldg(q + i1);
    const float q0 = (x0 * c - x1 * s) * kPlainScale, q1 = (x0 * s + x1 * c) * kPlainScale;
    qr[i0] = q0;
    qr[i1] = q1;
    bc[tid] = q0 * mk[i0] + q1 * mk[i1];
    bs[tid] = q1 * mk[i0] - q0 * mk[i1];
  }
  __syncthreads();
  const float* W = static_cast<const float*>(a.w_up_k) + static_cast<int64_t>(h) * kHeadDim * rk;
  for (int i = tid; i < 64 * rk; i += kPlainThreads) {
    const int f = i / rk, k = i - f * rk;
    int i0, i1;
    pair_of(f, i0, i1);
    const float w0 = __ldg(W + static_cast<int64_t>(i0) * rk + k), w1 = __ldg(W + static_cast<int64_t>(i1) * rk + k);
    zc[k * 64 + f] = qr[i0] * w0 + qr[i1] * w1;
    zs[k * 64 + f] = qr[i1] * w0 - qr[i0] * w1;
  }
  float acc[2] = {0.f, 0.f};
  float m_run = -INFINITY, l_run = 0.f;
  __syncthreads();
  for (int64_t j0 = j_lo; j0 < j_hi; j0 += kPlainThreads) {
    const int64_t j = j0 + tid;
    const bool valid = j < j_hi;
    const int nt = static_cast<int>(min(static_cast<int64_t>(kPlainThreads), j_hi - j0));
    uint8_t* mine = tile + static_cast<size_t>(tid) * ts;
    float s = -INFINITY;
    if (valid) {
      const int64_t row = latent_row(a.block_table, a.page_size, a.max_pages, a.num_pages, a.L_max, a.H, b, h, j, a.status);
      const uint4* src = reinterpret_cast<const uint4*>(a.rows + row * rb);
      for (int i = 0; i < rb / 16; ++i) reinterpret_cast<uint4*>(mine)[i] = __ldg(src + i);
      float A[64];
      const float* cr = a.rope_cos + j * 64;
      const float* sr = a.rope_sin + j * 64;
      s = 0.f;
      // the cosine part, then the sine part: 64 running sums each
#pragma unroll 1
      for (int part = 0; part < 2; ++part) {
        const float* z = part == 0 ? zc : zs;
        const float* bias = part == 0 ? bc : bs;
#pragma unroll
        for (int f = 0; f < 64; ++f) A[f] = bias[f];
#pragma unroll 1
        for (int k0 = 0; k0 < rk; k0 += 8) {
          float c8[8];
          const float sc = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(
              mine + q4_scale_offset(rk, rv) + 2 * (k0 / kQ4Group)));
          q4_unpack8(*reinterpret_cast<const uint32_t*>(mine + k0 / 2), sc, c8);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4* zr = reinterpret_cast<const float4*>(z + (k0 + e) * 64);
#pragma unroll
            for (int g = 0; g < 16; ++g) {
              const float4 z4 = zr[g];
              A[4 * g] = fmaf(c8[e], z4.x, A[4 * g]);
              A[4 * g + 1] = fmaf(c8[e], z4.y, A[4 * g + 1]);
              A[4 * g + 2] = fmaf(c8[e], z4.z, A[4 * g + 2]);
              A[4 * g + 3] = fmaf(c8[e], z4.w, A[4 * g + 3]);
            }
          }
        }
        const float* t = part == 0 ? cr : sr;
#pragma unroll
        for (int f = 0; f < 64; f += 4) {
          const float4 t4 = __ldg(reinterpret_cast<const float4*>(t + f));
          s = fmaf(t4.x, A[f], fmaf(t4.y, A[f + 1], fmaf(t4.z, A[f + 2], fmaf(t4.w, A[f + 3], s))));
        }
      }
    }
    // ---- online softmax over the tile (log2 units)
    float mt = warp_max(s);
    if (lane == 0) red[wid] = mt;
    __syncthreads();
    const float m_new = fmaxf(m_run, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float scale = m_new == -INFINITY ? 1.f : exp2f(m_run - m_new);   // the first tile: 0
    const float p = valid ? (m_new == -INFINITY ? s - s : exp2f(s - m_new)) : 0.f;   // all NaN: stays NaN
    pw[tid] = p;
    __syncthreads();   // pw and the tile's rows are complete; red is free again
    const float ps = warp_sum(p);
    if (lane == 0) red[wid] = ps;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int k = tid + half * kPlainThreads;
      if (k >= rv) break;
      const int at = rk / 2 + 4 * (k / 8) , bit = 4 * ((k & 7) >> 1) + 16 * (k & 1);
      const int sat = q4_scale_offset(rk, rv) + 2 * (q4_groups(rk) + k / kQ4Group);
      float v = 0.f;
      for (int i = 0; i < nt; ++i) {
        const uint8_t* r = tile + static_cast<size_t>(i) * ts;
        const float c = static_cast<float>(static_cast<int>((*reinterpret_cast<const uint32_t*>(r + at) >> bit) & 15u) - 8);
        v = fmaf(pw[i], c * __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(r + sat)), v);
      }
      acc[half] = fmaf(acc[half], scale, v);
    }
    __syncthreads();   // sums complete; the rows are free for the next tile
    l_run = l_run * scale + (red[0] + red[1] + red[2] + red[3]);
    m_run = m_new;
    __syncthreads();   // everyone has read red
  }
  float* rec = a.records + id * (rv + kRecordHead);
  if (tid == 0) {
    rec[0] = m_run;
    rec[1] = l_run;
  }
  for (int half = 0; half < 2; ++half)
    if (tid + half * kPlainThreads < rv) rec[kRecordHead + tid + half * kPlainThreads] = acc[half];
}

// Merge a (sequence, head)'s split records by log-sum-exp, apply W_up,v once (Appendix J
// "Absorbed attention") and normalise.  Block = (head, sequence), one output per thread.
__global__ void __launch_bounds__(kPlainThreads) q4_f32_combine_kernel(const __grid_constant__ Q4DecodeArgs a) {
  __shared__ float acc[kMaxRankPerHead];
  const int64_t u = blockIdx.x;
  const int b = static_cast<int>(u / a.H), h = static_cast<int>(u - static_cast<int64_t>(b) * a.H), tid = threadIdx.x;
  const int L = q4_len(a, b), rv = a.r_v;
  float* out = static_cast<float*>(a.out) + u * kHeadDim;
  if (L == 0) {
    out[tid] = 0.f;
    if (tid == 0 && a.lse) a.lse[u] = -INFINITY;
    return;
  }
  const int n = static_cast<int>((L + a.chunk - 1) / a.chunk);
  const float* rec = a.records + u * a.splits * (rv + kRecordHead);
  float m = -INFINITY;
  for (int i = 0; i < n; ++i) m = fmaxf(m, rec[static_cast<int64_t>(i) * (rv + kRecordHead)]);
  float l = 0.f, v[2] = {0.f, 0.f};
  for (int i = 0; i < n; ++i) {
    const float* r = rec + static_cast<int64_t>(i) * (rv + kRecordHead);
    const float w = m == -INFINITY ? 1.f : exp2f(r[0] - m);   // no maximum: every score was NaN, and so is l
    l = fmaf(r[1], w, l);
    for (int half = 0; half < 2; ++half)
      if (tid + half * kPlainThreads < rv) v[half] = fmaf(r[kRecordHead + tid + half * kPlainThreads], w, v[half]);
  }
  for (int half = 0; half < 2; ++half)
    if (tid + half * kPlainThreads < rv) acc[tid + half * kPlainThreads] = v[half];
  __syncthreads();
  const float* W = static_cast<const float*>(a.w_up_v) + (static_cast<int64_t>(h) * kHeadDim + tid) * rv;
  float o = 0.f;
  for (int k = 0; k < rv; k += 8) {
    float w8[8];
    load8(W + k, w8);
#pragma unroll
    for (int e = 0; e < 8; ++e) o = fmaf(acc[k + e], w8[e], o);
  }
  out[tid] = o / l + a.mu_v[h * a.mu_hstride + tid];
  if (tid == 0 && a.lse) a.lse[u] = (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

cudaError_t launch_q4_f32(const Q4DecodeArgs& a, cudaStream_t s) {
  const size_t smem = static_cast<size_t>(a.r_k) * 512 + static_cast<size_t>(kPlainThreads) * (a.row_bytes + 16);
  cudaError_t e = allow_smem(q4_f32_kernel, smem);
  if (e != cudaSuccess) return e;
  const int64_t units = static_cast<int64_t>(a.B) * a.H;
  q4_f32_kernel<<<static_cast<unsigned>(units * a.splits), kPlainThreads, smem, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  q4_f32_combine_kernel<<<static_cast<unsigned>(units), kPlainThreads, 0, s>>>(a);
  return cudaGetLastError();
}

int64_t q4_plain_chunk(int B, int H, int64_t L_max, int sms) {
  const int64_t tiles = (L_max + kTile - 1) / kTile, units = static_cast<int64_t>(B) * H;
  const int64_t want = std::max<int64_t>(1, (2 * static_cast<int64_t>(sms) + units - 1) / units);
  return (tiles + std::min(want, tiles) - 1) / std::min(want, tiles) * kTile;
}


}  // namespace lla

using namespace lla;

namespace {

// Host checks of a 4-bit pool description; LLA_OK also for B == 0.
lla_status q4_pool_checks(const lla_dims* dims, const lla_q4_cache* c) {
  if (!c || c->B < 0 || c->page_size < 1 || c->num_pages < 1) return LLA_ERR_INVALID_ARG;
  if (dims->variant != LLA_PER_HEAD) return LLA_ERR_UNSUPPORTED;
  if (c->num_pages * static_cast<int64_t>(dims->H) >= (int64_t(1) << 31) ||
      c->num_pages * static_cast<int64_t>(c->page_size) >= (int64_t(1) << 40))
    return LLA_ERR_UNSUPPORTED;
  return LLA_OK;
}

bool at16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

lla_status q4_copy(const lla_dims* dims, void* k, void* v, int N, const int64_t* slots, const lla_q4_cache* cache,
                   void* workspace, size_t ws_bytes, void* stream, bool store) {
  lla_status st = checked_dims(dims);
  if (st != LLA_OK) return st;
  if ((st = q4_pool_checks(dims, cache)) != LLA_OK) return st;
  if (N < 0) return LLA_ERR_INVALID_ARG;
  if (N == 0) return LLA_OK;
  if (!at16(k) || !at16(v) || !at16(cache->rows) || !at16(workspace) || !slots ||
      (reinterpret_cast<uintptr_t>(slots) & 7u) || ws_bytes < 256)
    return LLA_ERR_INVALID_ARG;
  Q4CopyArgs a{};
  a.H = dims->H;
  a.r_k = dims->r_k;
  a.r_v = dims->r_v;
  a.row_bytes = q4_row_bytes(dims->r_k, dims->r_v);
  a.page_size = cache->page_size;
  a.num_slots = cache->num_pages * cache->page_size;
  a.slots = slots;
  a.k = k;
  a.v = v;
  a.rows = static_cast<uint8_t*>(cache->rows);
  a.status = static_cast<uint32_t*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // launches of at most 2^30 items keep the item arithmetic in 32 bits
  const int64_t per_tok = static_cast<int64_t>(dims->H) * 4 * (q4_groups(dims->r_k) + q4_groups(dims->r_v));
  if (per_tok > (int64_t(1) << 30)) return LLA_ERR_UNSUPPORTED;
  const int64_t chunk = (int64_t(1) << 30) / per_tok;
  for (int64_t t = 0; t < N; t += chunk) {
    const int64_t n = std::min<int64_t>(chunk, N - t);
    a.tok0 = static_cast<uint32_t>(t);
    a.n_items = static_cast<uint32_t>(n * per_tok);
    const unsigned blocks = (a.n_items + kQ4Threads - 1) / kQ4Threads;
    if (store) {
      if (dims->dtype == LLA_BF16) q4_store_kernel<__nv_bfloat16><<<blocks, kQ4Threads, 0, s>>>(a);
      else q4_store_kernel<float><<<blocks, kQ4Threads, 0, s>>>(a);
    } else {
      if (dims->dtype == LLA_BF16) q4_load_kernel<__nv_bfloat16><<<blocks, kQ4Threads, 0, s>>>(a);
      else q4_load_kernel<float><<<blocks, kQ4Threads, 0, s>>>(a);
    }
    if (cudaGetLastError() != cudaSuccess) return LLA_ERR_CUDA;
  }
  return LLA_OK;
}

// Workspace of a decode call: status word; tensor-core kernel: the CTA range of every
// (sequence, head group), a record per head of every (unit, CTA) of a run (at most
// units + grid of them), the f16 rotary tiles of L_max positions; fp32 kernel: a record per split.
struct Q4Ws {
  size_t ranges, records, row_tiles, total;
  int grid;
};
Q4Ws q4_ws(const lla_dims* d, int B, int64_t L_max, int sms) {
  Q4Ws w{};
  const int64_t tiles = std::max<int64_t>(1, (L_max + kTile - 1) / kTile);
  const size_t rec = static_cast<size_t>(d->r_v + kRecordHead) * 4;
  w.ranges = 256;
  if (d->dtype == LLA_BF16) {
    Q4Plan p;
    make_q4_plan(d->H, d->r_k, d->r_v, &p);
    const int64_t units = static_cast<int64_t>(B) * p.ngroups;
    w.grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min(sms, kMaxGrid), units * tiles)));
    w.records = (256 + static_cast<size_t>(units) * 8 + 255) / 256 * 256;
    w.row_tiles = (w.records + (static_cast<size_t>(units) + w.grid) * p.nh * rec + 255) / 256 * 256;
    w.total = w.row_tiles + static_cast<size_t>(tiles) * kTile * 256;
    return w;
  }
  const int64_t chunk = q4_plain_chunk(std::max(B, 1), d->H, std::max<int64_t>(L_max, 1), sms) / kTile;
  w.records = 256;
  w.total = 256 + static_cast<size_t>(B) * d->H * ((tiles + chunk - 1) / chunk) * rec;
  return w;
}

}  // namespace

extern "C" {

size_t lla_q4_row_bytes(const lla_dims* dims) {
  if (checked_dims(dims) != LLA_OK || dims->variant != LLA_PER_HEAD) return 0;
  return static_cast<size_t>(q4_row_bytes(dims->r_k, dims->r_v));
}

size_t lla_q4_workspace_size(const lla_dims* dims, int B, int64_t L_max) {
  if (checked_dims(dims) != LLA_OK || dims->variant != LLA_PER_HEAD || B < 0 || L_max < 0) return 0;
  return q4_ws(dims, B, L_max, device_sm_count()).total;
}

lla_status lla_q4_store(const lla_dims* dims, const void* c_k, const void* c_v, int N, const int64_t* slots,
                        const lla_q4_cache* cache, void* workspace, size_t ws_bytes, void* stream) {
  return q4_copy(dims, const_cast<void*>(c_k), const_cast<void*>(c_v), N, slots, cache, workspace, ws_bytes, stream, true);
}

lla_status lla_q4_load(const lla_dims* dims, const int64_t* slots, int N, const lla_q4_cache* cache, void* c_k,
                       void* c_v, void* workspace, size_t ws_bytes, void* stream) {
  return q4_copy(dims, c_k, c_v, N, slots, cache, workspace, ws_bytes, stream, false);
}

lla_status lla_decode_attn_q4(const lla_dims* dims, int loop_t, const void* q, const lla_q4_cache* cache,
                              const int32_t* seq_lens, const int32_t* q_pos, const void* w_up_k, const void* w_up_v,
                              const float* mu_k, const float* mu_v, const float* rope_cos, const float* rope_sin,
                              int64_t rope_len, void* out, float* lse, void* workspace, size_t ws_bytes,
                              void* stream) {
  lla_status st = checked_dims(dims);
  if (st != LLA_OK) return st;
  if ((st = q4_pool_checks(dims, cache)) != LLA_OK) return st;
  if (loop_t < 0 || loop_t >= dims->T || cache->max_pages < 1) return LLA_ERR_INVALID_ARG;
  const int64_t L_max = static_cast<int64_t>(cache->max_pages) * cache->page_size;
  if (L_max > (int64_t(1) << 30) || static_cast<int64_t>(cache->B) * cache->max_pages >= (int64_t(1) << 31) ||
      static_cast<int64_t>(cache->B) * dims->H > (int64_t(1) << 24) ||
      static_cast<int64_t>(cache->B) * ((L_max + kTile - 1) / kTile) >= (int64_t(1) << 31))
    return LLA_ERR_UNSUPPORTED;
  if (cache->B == 0) return LLA_OK;
  if (rope_len < L_max || rope_len < kTile) return LLA_ERR_INVALID_ARG;
  const void* ptrs[] = {q, cache->rows, seq_lens, q_pos, w_up_k, w_up_v, mu_k, mu_v, rope_cos, rope_sin, out, workspace};
  for (const void* p : ptrs)
    if (!at16(p)) return LLA_ERR_INVALID_ARG;
  if (!cache->block_table || (reinterpret_cast<uintptr_t>(cache->block_table) & 3u) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u))
    return LLA_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return LLA_ERR_CUDA;
  const Q4Ws w = q4_ws(dims, cache->B, L_max, sms);
  if (ws_bytes < w.total) return LLA_ERR_INVALID_ARG;
  const size_t es = dims->dtype == LLA_BF16 ? 2 : 4;
  const size_t wk = static_cast<size_t>(dims->H) * kHeadDim * dims->r_k * es;
  const size_t wv = static_cast<size_t>(dims->H) * kHeadDim * dims->r_v * es;
  Q4DecodeArgs a{};
  a.B = cache->B;
  a.H = dims->H;
  a.r_k = dims->r_k;
  a.r_v = dims->r_v;
  a.rope_style = dims->rope_style;
  a.row_bytes = q4_row_bytes(dims->r_k, dims->r_v);
  a.L_max = L_max;
  a.rope_len = rope_len;
  a.mu_hstride = static_cast<int64_t>(dims->T) * kHeadDim;
  a.q = q;
  a.rows = static_cast<const uint8_t*>(cache->rows);
  a.block_table = cache->block_table;
  a.page_size = cache->page_size;
  a.max_pages = cache->max_pages;
  a.num_pages = cache->num_pages;
  a.seq_lens = seq_lens;
  a.q_pos = q_pos;
  a.w_up_k = static_cast<const uint8_t*>(w_up_k) + loop_t * wk;
  a.w_up_v = static_cast<const uint8_t*>(w_up_v) + loop_t * wv;
  a.mu_k = mu_k + static_cast<size_t>(loop_t) * kHeadDim;
  a.mu_v = mu_v + static_cast<size_t>(loop_t) * kHeadDim;
  a.rope_cos = rope_cos;
  a.rope_sin = rope_sin;
  a.out = out;
  a.lse = lse;
  a.status = static_cast<uint32_t*>(workspace);
  a.records = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + w.records);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dims->dtype == LLA_BF16) {
    if (!make_q4_plan(a.H, a.r_k, a.r_v, &a.plan)) return LLA_ERR_UNSUPPORTED;
    a.ranges = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + w.ranges);
    a.grid = w.grid;
    a.row_tiles = static_cast<uint8_t*>(workspace) + w.row_tiles;
    a.rows_grid = static_cast<int>(std::min<int64_t>((L_max + kTile - 1) / kTile, 4 * sms));
    // sequences per combine block: W_up,v is read once for them; about four blocks per SM
    a.combine_units = static_cast<int>(std::min<int64_t>(8, std::max<int64_t>(1, static_cast<int64_t>(a.B) * a.H / (4 * sms))));
    return launch_q4_tile(a, s) == cudaSuccess ? LLA_OK : LLA_ERR_CUDA;
  }
  a.chunk = q4_plain_chunk(a.B, a.H, L_max, sms);
  a.splits = static_cast<int>((L_max + a.chunk - 1) / a.chunk);
  return launch_q4_f32(a, s) == cudaSuccess ? LLA_OK : LLA_ERR_CUDA;
}

}  // extern "C"
